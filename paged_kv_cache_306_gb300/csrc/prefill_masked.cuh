// prefill_masked.cuh -- chunked prefill with capped, biased or masked scores, on tcgen05.
//
// What is computed: see pa_prefill_masked in pa.h.  The row at position p sees the keys t with
//     max(0, p - window + 1) <= t <= max(p, prefix - 1),
// with scores z_t = cap tanh(x_t / cap) - slope |p - t| of x_t = scale q.k_t.
//
// The kernel is built as prefill_ws.cuh's, whose header describes it: units of four 128-row tiles
// taken by clusters of two CTAs, K and V multicast into both, a pair of tiles per CTA in
// ping-pong between the tensor cores and the softmax warps.  What differs:
//
//   * Keys.  A unit takes the chunks of 128 keys from the one its first row's window starts in to the last one
//     that any of its rows sees.  Within them each row hides what it does not see; half a chunk that no row of a
//     warp sees leaves P = 0 without a score looked at.  V of keys below the unit's first one reads as
//     zero, as V past the sequence does (P is 0 there, but 0 * NaN would poison O).  A row's first chunks may
//     be hidden whole: its maximum is -inf until one is not, and every term 0.
//   * The cap.  cap - 2 cap / (1 + e^(2x)) costs two operations of the special-function unit (16 a clock and SM)
//     beside the softmax's own one: 452 us for 16 chunks of 512 tokens behind 3584 (28 heads of 128 dims, fp16), which
//     take 283 us uncapped; and it is off by a share of the cap, whatever the score.  So: the tanh keeps the scores'
//     order, the row's maximum is the raw scores' one, and the cap becomes an odd polynomial in the raw score within the
//     exponentials' loop, its multiply-adds (128 a clock and SM) beside the exponentials: 4 terms where all scores of
//     the warp's half chunk lie within cap / 2 (358 us), 6 within cap (397 us), the exponential form past it (with a
//     large cap for the scores that need it alone: cap_any, cap_small).  The coefficients serve any cap (set_tanh): 358 us
//     at caps of 500 and 10^6 too.  (Polynomials over all scores first, then the softmax: 403 us for the 4 terms; so now
//     only where a mask cuts the half, or with a bias, after which the maximum is another one: 361 us biased, 488 us
//     capped and biased.)
//   * Two threads to a row, one for each half of a chunk's keys, which exchange their maxima; each reads
//     its scores twice, for the maximum and for P, and keeps 32 in registers at a time.  A row's softmax is a
//     step of the chain S, softmax, P V, S; halved, 16 chunks of 512 tokens with capped scores in a window of 1024 take
//     179 us for 192, whole prompts in bf16 675 for 779.  (The first half of P handed over before the second is
//     done, so that its P V may start, cost more than it gave: 207 us.)
//   * Registers.  640 threads have 96 each; the softmax's four warpgroups take 8 of each thread of the fifth
//     (setmaxnreg), which copies, issues the MMAs and assigns.
//   * Units are assigned in rounds (assign_units) and their figures handed over in the ring (unit_view).
//   * Q is loaded and the output stored four threads to a row (load_q, store_rows).
//   * The MMA warp waits for the next chunk's K before it issues a chunk's P V, so that nothing stands between
//     a tile's P V and its next S (a wait takes 100 to 200 clocks even when what it waits for is there): 177.1 us for
//     179.6 in fp16.  In bf16, whose P V is twice as long, the K is waited for behind it: 677 us for 686.
#pragma once

#include "prefill_ws.cuh"

namespace pa {
namespace wsm {

using namespace ws;

// the kinds of kernels: any sum of these
constexpr int kCapped = 1, kBiased = 2;

// Warps 0..7 are tile A's softmax, 8..15 tile B's, four for each half of a chunk's keys; then the copies,
// the MMAs, the unit ring and one without work.
constexpr int kHalf = kKeys / 2, kStep = 32, kTileThreads = 256;  // (scores are taken kStep at a time)
constexpr int kSoftmaxWarps = 16, kCopyWarp = 16, kSchedWarp = 18, kIdleWarp = 19;
constexpr int kThreads = 20 * 32;  // (the warps' numbers of prefill_ws.cuh's header are 16 to 18 here)
constexpr int kUnitReaders = kSoftmaxWarps + 2;
// registers per thread of the softmax warps and the others, out of the launch's 640 x 96
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64, kLaunchRegs = 96;
static_assert(kSoftmaxWarps * 32 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "what the launch has");

// the smallest of three (a NaN operand is ignored, as by fminf)
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The largest (smallest) of N scores, as a tree of three-input maxima in 8 chains
template <int N>
__device__ __forceinline__ float largest(const float (&sv)[N]) {
  static_assert(N % 16 == 0, "8 chains, two keys a step");
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = fmaxf(sv[i], sv[8 + i]);
#pragma unroll
  for (int j = 16; j < N; j += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = max3(t[i], sv[j + i], sv[j + 8 + i]);
  return fmaxf(max3(t[0], t[1], t[2]), max3(max3(t[3], t[4], t[5]), t[6], t[7]));
}
template <int N>
__device__ __forceinline__ float smallest(const float (&sv)[N]) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = fminf(sv[i], sv[8 + i]);
#pragma unroll
  for (int j = 16; j < N; j += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = min3(t[i], sv[j + i], sv[j + 8 + i]);
  return fminf(min3(t[0], t[1], t[2]), min3(min3(t[3], t[4], t[5]), t[6], t[7]));
}

// 1 / x by the hardware's approximate reciprocal (1 / inf = 0)
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// cap tanh(v / cap) of a score v, both in log2 units, inv = 1 / cap.  Past cap / 2 cap - 2 cap / (1 + e^(2 v / cap)), off
// by 2^-22 of the cap; a score below it may be small against that, so it goes through tanh_ratio.
__device__ __forceinline__ float cap_any(float v, float cap, float inv) {
  const float t = v * inv, far = fmaf(-2.f * cap, rcp(1.f + ex2(t * (2.f * kLog2e))), cap);
  return fabsf(t) <= 0.5f ? v * tanh_ratio(t * t) : far;
}

// Up to this cap (in log2 units; 88 in the scores' own) its second form alone is within 2^-15 of every score, less
// than a weight's rounding, and serves the small scores beside the large ones too: 621 us where cap_any takes 919 (16
// chunks of 512 tokens behind 3584, 28 heads, scores of twice the cap).
constexpr float kSmallCap = 128.f;
// It, of a raw score s; e brings that to 2 log2(e) v / cap.
__device__ __forceinline__ float cap_small(float s, float e, float cap, float top) {
  return fmaf(-2.f * cap, rcp(1.f + ex2(s * e)), top);
}

// The odd polynomial c[0] s + c[1] s^3 + .. of a pair (each coefficient twice in a pair), plus d.
template <int N>
__device__ __forceinline__ uint64_t odd_poly(uint64_t x, const uint64_t (&c)[N], uint64_t d) {
  const uint64_t u = mul2(x, x);
  uint64_t t = fma2(u, c[N - 1], c[N - 2]);
#pragma unroll
  for (int k = N - 3; k >= 0; --k) t = fma2(t, u, c[k]);
  return fma2(x, t, d);
}

// Half a row of out, which a warp's threads hold (N elements each, as N / 2 words), to rows `at` of D elements
// (below 0: nowhere).  Four threads exchange their pieces of 16 bytes first, so that they store 64 bytes of one row
// side by side, then of the next.  (Each thread on its own row made 32 requests of every store: 4096 a unit, behind
// which the MMA warp's look-ups of its next unit waited ~5000 clocks.)
template <typename T, int N, int D>
__device__ __forceinline__ void store_rows(uint32_t (&w)[N / 2], T* out, long long at) {
  const int q = threadIdx.x & 3;
#pragma unroll
  for (int g = 0; g < N / 32; ++g) {  // four pieces: piece i of lane j of the four becomes piece j of lane i
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        if (a & m) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t &x = w[16 * g + 4 * a + i], &y = w[16 * g + 4 * (a | m) + i];
          const uint32_t got = __shfl_xor_sync(0xffffffffu, (q & m) ? x : y, m);
          if (q & m) x = got;
          else y = got;
        }
      }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const long long row = __shfl_sync(0xffffffffu, at, (threadIdx.x & 28) + a);
    if (row < 0) continue;
#pragma unroll
    for (int g = 0; g < N / 32; ++g)
      reinterpret_cast<uint4*>(out + row * D)[4 * g + q] =
          make_uint4(w[16 * g + 4 * a], w[16 * g + 4 * a + 1], w[16 * g + 4 * a + 2], w[16 * g + 4 * a + 3]);
  }
}

// Unit selection's figures of each sequence, in shared memory (5 kMaxSeqsPerLaunch ints): tokens
// before the chunk, the chunk's n G query rows, its tiles (the plain kernel's three, see
// units_reading), the prefix within the sequence, and the chunk's first query row.  One warp fills it once per CTA
// and checks the lengths; returns the most chunks any unit would read without a window or prefix.
__device__ __forceinline__ int build_table(const PrefillMaskedParams& p, int* tab) {
  const int lane = threadIdx.x & 31, G = p.group, S = p.num_seqs;
  bool bad = false;
  int longest = 0;
  for (int s = lane; s < S; s += 32) {
    const int L = __ldg(p.seq_lens + s), a = __ldg(p.query_start_loc + s), b = __ldg(p.query_start_loc + s + 1);
    const int n = b - a;
    int ctx = 0, rows = 0, nt = 0, prefix = 0;
    if (L < 1 || L > p.max_seq_len || a < 0 || b > p.num_query_tokens || n < 0 || n > L) {
      bad = true;
    } else {
      ctx = L - n;
      rows = n * G;
      nt = (rows + kRows - 1) / kRows;
      if (nt && p.prefix_lens) prefix = max(0, min(L, __ldg(p.prefix_lens + s)));
    }
    tab[s] = ctx;
    tab[kMaxSeqsPerLaunch + s] = rows;
    tab[2 * kMaxSeqsPerLaunch + s] = nt;
    tab[3 * kMaxSeqsPerLaunch + s] = prefix;
    tab[4 * kMaxSeqsPerLaunch + s] = a;
    if (nt) longest = max(longest, (ctx + (rows - 1) / G) / kKeys + 1);
  }
  if (bad && blockIdx.x == 0) set_error(p.err, kErrSeqLen);
  longest = __reduce_max_sync(0xffffffffu, longest);
  __syncwarp();
  return longest;
}

// The keys that unit `ui` of a sequence takes (its n G query rows `rows`, the first at
// position ctx), from the first one its first row's window reaches (lo) to the last one any
// of its rows sees (hi): its own position's, or the prefix's.
__device__ __forceinline__ void masked_keys(int window, int prefix, int ctx, int rows, int G, int ui, int& lo, int& hi) {
  const int row_hi = min(rows, (kUnitTiles * ui + kUnitTiles) * kRows);
  hi = max(ctx + (row_hi - 1) / G, prefix - 1);
  lo = window > 0 ? max(0, ctx + (kUnitTiles * ui * kRows) / G - (window - 1)) : 0;
}

// The assignment of units to clusters: longest first, to the clusters with the
// least work so far, as the plain kernel's; every warp that calls it replays the same sequence, and mine(sequence,
// kv head, unit) is called for the units of cluster `cid` until it returns false.
//   * A prefix makes all units of its sequence read at least its chunks; a window bounds what any
//     unit reads (with prefixes, what any sequence's rows see), so that all units that would read that much or more
//     come first, together (there is no walk over a long context's chunks).
//   * The units that read as many chunks, of 32 sequences and all kv heads, are given out in rounds: every
//     cluster whose work is below the least one's plus a unit's gets one (the least loaded ones, where the units do
//     not suffice), which is what giving them one by one to the least loaded comes to.  One by one, a unit took
//     ~390 clocks to give, 30,000 for a cluster's next one -- three times as long as the cluster worked on it with
//     short windows or short prompts.
// Loads are kept small by lowering all of them together: a unit's work is at most 2^24 + 4.
template <typename Mine>
__device__ __forceinline__ void assign_units(const PrefillMaskedParams& p, const int* tab, int longest, int cid,
                                              int ncl, Mine mine) {
  const int lane = threadIdx.x & 31, G = p.group, S = p.num_seqs, Hkv = p.num_kv_heads;
  int load[kLoadsPerLane];  // work of cluster lane + 32 i
#pragma unroll
  for (int i = 0; i < kLoadsPerLane; ++i) load[i] = lane + 32 * i < ncl ? 0 : INT_MAX;
  int top = longest;
  if (p.prefix_lens) {
    int seen = 1;
    for (int s = lane; s < S; s += 32) {
      const int prefix = tab[3 * kMaxSeqsPerLaunch + s], rows = tab[kMaxSeqsPerLaunch + s], ctx = tab[s];
      top = max(top, prefix / kKeys + (prefix % kKeys != 0));
      const int lo = p.window > 0 ? max(0, ctx - (p.window - 1)) : 0;
      if (rows) seen = max(seen, max(ctx + (rows - 1) / G, prefix - 1) / kKeys - lo / kKeys + 1);
    }
    top = min(__reduce_max_sync(0xffffffffu, top), __reduce_max_sync(0xffffffffu, seen));
  } else if (p.window > 0) {  // what a unit's rows and the window before them span
    top = static_cast<int>(min((long long)top, ((long long)p.window + (kUnitTiles * kRows - 1) / G) / kKeys + 2));
  }
  auto reading = [&](int s, int x) {  // units of sequence s, per kv head, that would read >= x chunks without a window
    const int prefix = tab[3 * kMaxSeqsPerLaunch + s];
    if (x <= prefix / kKeys + (prefix % kKeys != 0)) return (tab[2 * kMaxSeqsPerLaunch + s] + kUnitTiles - 1) / kUnitTiles;
    return units_reading(tab, G, s, x);
  };
  for (int x = top; x >= 1; --x) {
    for (int s0 = 0; s0 < S; s0 += 32) {
      // lane i: the units of sequence s0 + i that read x chunks (at the top, x or more): how many per kv head, the
      // first, and the work of the middle one
      const int s = s0 + lane;
      int e = 0, first = 0, work = 0;
      if (s < S) {
        const int a = reading(s, x), b = x == top ? 0 : reading(s, x + 1);
        e = a - b;
        first = (tab[2 * kMaxSeqsPerLaunch + s] + kUnitTiles - 1) / kUnitTiles - a;
        if (e > 0) {
          int lo, hi;
          masked_keys(p.window, tab[3 * kMaxSeqsPerLaunch + s], tab[s], tab[kMaxSeqsPerLaunch + s], G, first + e / 2, lo, hi);
          work = hi / kKeys - lo / kKeys + 1 + kUnitCost;
        }
      }
      if (!__any_sync(0xffffffffu, e > 0)) continue;
      int upto = e * Hkv;  // units of the sequences up to this lane's
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const int n = __shfl_sync(0xffffffffu, upto, 31);
      // the work of one: the most (all are x but for windows, which leave units of the top differ by a chunk, and for
      // windows with prefixes)
      const int w = __reduce_max_sync(0xffffffffu, work);
      for (int done = 0; done < n;) {
        int least = load[0];
#pragma unroll
        for (int i = 1; i < kLoadsPerLane; ++i) least = min(least, load[i]);
        least = __reduce_min_sync(0xffffffffu, least);
        const int low = least >= 1 << 29 ? least : 0;
        auto below = [&](int t) {  // clusters with less work than t
          int k = 0;
#pragma unroll
          for (int i = 0; i < kLoadsPerLane; ++i) k += __popc(__ballot_sync(0xffffffffu, load[i] < t));
          return k;
        };
        // this turn's: those below `t`, then, where the units do not suffice for all below least + w, of those
        // at `t` the first ones
        int t = least + w, all = below(t), ties = 0;
        if (all > n - done) {
          for (int a = least; t - a > 1;) {
            const int mid = a + (t - a) / 2;
            if (below(mid) <= n - done) a = mid;
            else t = mid;
          }
          all = below(--t);
          ties = 1;
        }
        int before = 0, tied = all;
#pragma unroll
        for (int i = 0; i < kLoadsPerLane; ++i) {
          const unsigned who = __ballot_sync(0xffffffffu, load[i] < t);
          const unsigned tie = __ballot_sync(0xffffffffu, ties && load[i] == t);
          auto rank = [&](int l) {  // of cluster l + 32 i among this turn's; INT_MAX / 2: not one of them
            const unsigned less = (1u << l) - 1;
            return who >> l & 1 ? before + __popc(who & less) : tie >> l & 1 ? tied + __popc(tie & less) : INT_MAX / 2;
          };
          const int u = cid / 32 == i ? done + rank(cid % 32) : INT_MAX;
          if (done + rank(lane) < n) load[i] += w;
          if (load[i] != INT_MAX) load[i] -= low;
          if (u < n) {  // the u-th unit is this cluster's
            const int src = __ffs(__ballot_sync(0xffffffffu, upto > u)) - 1;
            const int ee = __shfl_sync(0xffffffffu, e, src), ff = __shfl_sync(0xffffffffu, first, src);
            const int v = u - (__shfl_sync(0xffffffffu, upto, src) - ee * Hkv);
            if (!mine(s0 + src, v / ee, ff + v % ee)) return;
          }
          before += __popc(who);
          tied += __popc(tie);
        }
        done += min(tied, n - done);
      }
    }
  }
}

template <typename T, int D, int BS>
struct Shape {  // the plain kernel's, but for the ring and the table
  static constexpr int kTile = D * BS * 2;                 // one block's K (or V) tile
  static constexpr int kBlocks = kKeys / BS;               // blocks per chunk
  static constexpr int kQTile = kRows * D * 2;             // one tile's Q, core-matrix layout
  static constexpr int kKBytes = kKeys * D * 2;            // a chunk's K as [D/8][128][8]
  static constexpr int kVBytes = kKeys * D * 2;            // a chunk's V: kBlocks swizzled tiles [D][bs]
  static constexpr int kOffK = 2 * kQTile;                 // K ring
  static constexpr int kOffV = kOffK + kKStages * kKBytes; // V ring
  static constexpr int kOffBar = kOffV + kVStages * kVBytes;
  // fullk[K], fullv[V], kfree[K], vfree[V], per tile 5 (sfull, pfull, pvdone, qfull,
  // ofree), ufull[U], uempty[U], pair[8], never
  static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 2 * 5 + 2 * kUnitSlots + 8 + 1;
  static constexpr int kOffMisc = kOffBar + (kNumBars * 8 + 15) / 16 * 16;  // TMEM address, abort flag
  static constexpr int kOffUnits = kOffMisc + 16;                           // [kUnitSlots][kUnitInts]: the unit ring
  static constexpr int kUnitInts = 9;                                       // a slot: see unit_view
  static constexpr int kOffTab = kOffUnits + kUnitSlots * kUnitInts * 4;    // unit selection's table
  static constexpr int kOffMax = kOffTab + 5 * kMaxSeqsPerLaunch * 4;       // [2 turns][2 tiles][2 halves][128 rows]
  static constexpr int kEnd = kOffMax + 2 * 2 * 2 * kRows * 4;
  // more than half an SM's shared memory, so one CTA per SM: it takes all of TMEM
  static constexpr int kSmem = kEnd > 116 * 1024 ? kEnd : 116 * 1024;
  static constexpr int kTmemCols = 512;  // tile X at 256 X: S/P 0..127, O 128..128+D
};

// The figures of one unit that every role needs: the same in every role, and in both
// CTAs of the cluster except for the pair, which is this CTA's.  Keys are counted from
// the sequence's start; chunk c of the unit holds the kKeys keys from (c0 + c) kKeys on, and
// no block below key lo's is looked up or read.
struct UnitView {
  int s, kvh, L, tok0, pair_lo, pair_hi, ntiles, ctx, nblk, nchunks, c0, lo, prefix;
};
// `slot`: the ring's words of the unit: s, kvh, unit, the sequence's length, its first query row and its new tokens,
// the unit's keys lo and hi, and the prefix.  (No reader of the ring looks anything up: each look-up of the lengths in
// memory kept the softmax from a unit's last chunk, and the MMAs from the next unit's first one, for ~3000 clocks.)
template <int BS>
__device__ __forceinline__ UnitView unit_view(int G, const volatile int* slot, uint32_t crank) {
  UnitView v;
  v.s = slot[0];  // (below 0: no more units, and the other words are not used)
  v.kvh = slot[1];
  const int unit = slot[2], n = slot[5], rows = n * G, hi = slot[7];
  v.L = slot[3];
  v.tok0 = slot[4];
  v.lo = slot[6];
  v.prefix = slot[8];
  // this CTA's pair: tiles kUnitTiles unit + 2 crank and the next (either may be past the rows)
  v.pair_lo = (kUnitTiles * unit + 2 * static_cast<int>(crank)) * kRows;
  v.pair_hi = min(rows, v.pair_lo + 2 * kRows);
  v.ntiles = v.pair_lo >= rows ? 0 : (v.pair_lo + kRows < rows ? 2 : 1);  // tiles with rows: A, then B
  v.ctx = v.L - n;
  // keys: what the unit's rows see (the same in both CTAs: they share every chunk)
  v.c0 = v.lo / kKeys;
  v.nblk = hi / BS + 1;
  v.nchunks = hi / kKeys + 1 - v.c0;
  return v;
}

// kKind: kCapped, kBiased, both or neither.  A kernel each, so that none holds registers for
// what it does not do.
template <typename T, int D, int BS, int kKind>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_masked_kernel(const PrefillMaskedParams p, const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v) {
  constexpr bool kCap = (kKind & kCapped) != 0, kBias = (kKind & kBiased) != 0;
  using Sh = Shape<T, D, BS>;
  static_assert(Sh::kSmem > 114 * 1024, "two CTAs on one SM would contend for TMEM");
  static_assert(Sh::kSmem <= 227 * 1024, "shared memory per CTA");
  static_assert(kKeys % BS == 0, "a chunk is whole blocks");
  // P in one 16-bit part for fp16 (11 significant bits, the operands' own precision); for
  // bf16 a high and a low part (~16 bits), since one bf16 part (8 bits) would add
  // errors as large as the output's own rounding
  constexpr int kParts = std::is_same<T, __half>::value ? 1 : 2;
  constexpr bool kEarlyK = kParts == 1;  // when the MMA warp waits for the next chunk's K
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kOffBar);
  uint64_t* fullk = bars;                   // [kKStages] K buffer landed (TMA bytes)
  uint64_t* fullv = fullk + kKStages;       // [kVStages] V buffer landed (TMA bytes)
  uint64_t* kfree = fullv + kVStages;       // [kKStages] both CTAs' S read the K buffer (a commit from each)
  uint64_t* vfree = kfree + kKStages;       // [kVStages] both CTAs' P V read the V buffer (a commit from each)
  uint64_t* tbars = vfree + kVStages;       // per tile X at 5 X: sfull, pfull, pvdone, qfull, ofree
  uint64_t* ufull = tbars + 10;             // [kUnitSlots] the scheduler wrote the slot
  uint64_t* uempty = ufull + kUnitSlots;    // [kUnitSlots] every reader took the slot
  uint64_t* pair = uempty + kUnitSlots;     // [8] the two warps that hold a row's halves: tile X, quarter i at 4 X + i
  uint64_t* never = pair + 8;               // nothing completes it: the timeout-path test waits on it
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + Sh::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);  // a thread gave up
  volatile int* s_unit = reinterpret_cast<volatile int*>(smem + Sh::kOffUnits);  // [kUnitSlots][kUnitInts]
  int* tab = reinterpret_cast<int*>(smem + Sh::kOffTab);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // S(c) in TMEM (commit); P(c) in TMEM, O rescaled, V tail zeroed (256 arrivals); the
  // unit's last P V done (commit); the next unit's Q in shared memory (256 arrivals);
  // the unit's O read out of TMEM (256 arrivals)
  auto sfull = [&](int X) { return tbars + 5 * X; };
  auto pfull = [&](int X) { return tbars + 5 * X + 1; };
  auto pvdone = [&](int X) { return tbars + 5 * X + 2; };
  auto qfull = [&](int X) { return tbars + 5 * X + 3; };
  auto ofree = [&](int X) { return tbars + 5 * X + 4; };

  griddep_launch_dependents();
  griddep_wait();
  const uint32_t crank = cluster_rank();
  if (tid == 0) {
    *s_abort = 0;
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&fullk[i], 1);
      mbar_init(&kfree[i], kCluster);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&fullv[i], 1);
      mbar_init(&vfree[i], kCluster);
    }
    for (int X = 0; X < 2; ++X) {
      mbar_init(sfull(X), 1);
      mbar_init(pfull(X), kTileThreads);
      mbar_init(pvdone(X), 1);
      mbar_init(qfull(X), kTileThreads);
      mbar_init(ofree(X), kTileThreads);
    }
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(&ufull[i], 1);
      mbar_init(&uempty[i], kUnitReaders);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&pair[i], 2);
    mbar_init(never, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)),
                 "r"(Sh::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  cluster_sync_all();  // both CTAs' mbarriers are initialised before either copies into the other
  const uint32_t tmem = *s_tmem;
  const int G = p.group;
  int issued_k = 0, issued_v = 0;  // chunks (of all units) whose K (V) copies the copy warp issued
  auto wait = [&](uint64_t* bar, int parity) { return wait_or_abort(bar, parity, s_abort, p.err); };
  // the k-th unit of the ring (the slot's ufull phase k / kUnitSlots); every reader
  // takes it once and frees it with one arrival per warp
  auto take_unit = [&](int k, UnitView& v) -> bool {
    const int slot = k % kUnitSlots;
    if (!__all_sync(0xffffffffu, wait(&ufull[slot], (k / kUnitSlots) & 1))) return false;
    v = unit_view<BS>(p.group, s_unit + Sh::kUnitInts * slot, crank);  // v.s < 0: no more units
    __syncwarp();
    if (lane == 0) mbar_arrive(&uempty[slot]);
    return true;
  };

  if (warp < kSoftmaxWarps) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp < kSoftmaxWarps) {
    // ================= softmax: tile X, row r, half hf of the keys of each chunk of each unit =================
    const int X = warp >> 3, hf = (warp >> 2) & 1, r = tid & (kRows - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + 256 * X + lane_base;
    const uint32_t t_h = t_s + hf * kHalf, t_o = t_s + kKeys;  // this half's scores; the tile's O
    const float sl2 = kCap || kBias ? 1.f : p.scale_log2;  // modify() leaves scores in log2 units
    // kCap, kBias: the row's scores of the keys at positions dist .. dist + kStep - 1 relative to its
    // own, capped and biased, in log2 units
    auto modify = [&](float(&sv)[kStep], int dist, float slope) {
      if constexpr (kCap) {
        const float size = fmaxf(largest(sv), -smallest(sv));
        if (!__any_sync(0xffffffffu, size > p.tanh_near_to)) {
          const uint64_t zero = f2pack(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < kStep; j += 2) {
            const float2 v = f2unpack(odd_poly(f2pack(sv[j], sv[j + 1]), p.tanh_near, zero));
            sv[j] = v.x;
            sv[j + 1] = v.y;
          }
        } else if (__any_sync(0xffffffffu, size > p.tanh_wide_to)) {
          if (p.cap_log2 <= kSmallCap) {
#pragma unroll
            for (int j = 0; j < kStep; ++j) sv[j] = cap_small(sv[j], p.tanh_exp, p.cap_log2, p.cap_log2);
          } else {
#pragma unroll
            for (int j = 0; j < kStep; ++j) sv[j] = cap_any(sv[j] * p.scale_log2, p.cap_log2, p.cap_inv);
          }
        } else {
          const uint64_t zero = f2pack(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < kStep; j += 2) {
            const float2 v = f2unpack(odd_poly(f2pack(sv[j], sv[j + 1]), p.tanh_wide, zero));
            sv[j] = v.x;
            sv[j + 1] = v.y;
          }
        }
      }
      if constexpr (kBias) {
        const float d0 = static_cast<float>(dist), in = kCap ? 1.f : p.scale_log2;
        if (p.prefix_lens) {  // keys on both sides of the row's position
#pragma unroll
          for (int j = 0; j < kStep; ++j) sv[j] = fmaf(-slope, fabsf(d0 + j), sv[j] * in);
        } else {              // keys up to it: the distance is -(d0 + j)
          const uint64_t in2 = f2pack(in, in), slope2 = f2pack(slope, slope), base2 = f2pack(slope * d0, slope * d0);
#pragma unroll
          for (int j = 0; j < kStep; j += 2) {
            const uint64_t bias = fma2(slope2, f2pack(static_cast<float>(j), static_cast<float>(j + 1)), base2);
            const float2 v = f2unpack(fma2(f2pack(sv[j], sv[j + 1]), in2, bias));
            sv[j] = v.x;
            sv[j + 1] = v.y;
          }
        }
      }
    };
    // the warp's rows of Q_X for unit v into shared memory: every 16-byte piece in flight at
    // once, zeros for a padding row (completed and handed over by q_landed).  Four threads read 64 bytes of
    // one row side by side, as store_rows writes them (and for the same reason: a thread on each row, the
    // copies took ~4500 clocks to issue); eight rows of a piece are 128 bytes of shared memory.
    auto load_q = [&](const UnitView& v) {
      const int row = v.pair_lo + X * kRows + r;
      const long long at = row < v.pair_hi ? (long long)(v.tok0 + row / G) * p.num_heads + (long long)v.kvh * G + row % G : -1;
      const uint32_t sq = smem_addr(smem + X * Sh::kQTile) + (warp & 3) * (4 * (D / 8) * 128) + (lane >> 2) * 16 + (lane & 3) * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // rows 8 i .. 8 i + 7 of the warp's
        const long long from = __shfl_sync(0xffffffffu, at, 8 * i + (lane >> 2));
        const T* q = static_cast<const T*>(p.q) + (from < 0 ? 0 : from) * D + (lane & 3) * 8;
        const uint32_t nbytes = from < 0 ? 0u : 16u;
#pragma unroll
        for (int c = hf * (D / 16); c < (hf + 1) * (D / 16); c += 4)  // (its half's warps take half of a row)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sq + i * (D / 8) * 128 + c * 128),
                       "l"(q + 8 * c), "r"(nbytes)
                       : "memory");
      }
    };
    auto key0 = [](const UnitView& v, int c) { return (v.c0 + c) * kKeys; };  // a chunk's first key
    // this thread's number for the thread with the row's other half, and that one's for it; ok as for every wait
    int turn = 0;
    float* s_max = reinterpret_cast<float*>(smem + Sh::kOffMax);
    auto exchange = [&](float mine, float& other) -> bool {
      float* at = s_max + ((turn & 1) * 2 + X) * 2 * kRows + r;
      at[hf * kRows] = mine;
      __syncwarp();
      uint64_t* bar = pair + 4 * X + (warp & 3);
      if (lane == 0) mbar_arrive(bar);
      if (!__all_sync(0xffffffffu, wait(bar, turn & 1))) return false;
      other = at[(hf ^ 1) * kRows];
      ++turn;  // (two turns' numbers: a warp writes over one only after both have met again)
      return true;
    };
    auto q_landed = [&]() {  // the Q copies done, visible to the MMAs, handed over
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(qfull(X));
    };
    int cx = 0, ux = 0;  // chunks and units this tile had rows in: the phases of its barriers
    int g = 0;           // chunks of all units before this one: the K/V ring positions
    UnitView U{};
    bool ok = take_unit(0, U);
    if (ok && U.s >= 0) {
      if (U.ntiles > X) {
        load_q(U);
        q_landed();
      }
    }
    for (int k = 0; ok && U.s >= 0; ++k) {
      UnitView N{};  // the next unit, taken once this one's last chunk is handed over
      N.s = -1;
      auto next = [&]() {
        if (!(ok = take_unit(k + 1, N))) return;
        if (N.s >= 0 && N.ntiles > X) load_q(N);  // Q_X is free: the last S_X of this unit is done
      };
      if (U.ntiles > X) {
        const int row = U.pair_lo + X * kRows + r;
        const bool valid = row < U.pair_hi;
        const int pos = valid ? U.ctx + row / G : U.ctx + (U.pair_hi - 1) / G;  // a padding row behaves as a real one
        // first key whose V must read as zero (the blocks' end as an unsigned number: it may be 2^31)
        const int kz = static_cast<int>(min(static_cast<unsigned>(U.L), static_cast<unsigned>(U.nblk) * BS));
        // keys from `from` to `last` are visible to the row
        const int last = max(pos, U.prefix - 1);
        int from = 0;
        float slope = 0.f;
        if (p.window > 0) from = max(0, pos - (p.window - 1));  // (from - k0c below would not fit an int otherwise)
        if constexpr (kBias) slope = slope_log2(__ldg(p.slopes + U.kvh * G + (valid ? row % G : 0)));
        float m = -INFINITY, l = 0.f;
        for (int c = 0; c < U.nchunks; ++c, ++cx) {
          // tcgen05.ld / st are warp-collective (.sync.aligned): every branch around them
          // is taken by the whole warp, so each wait's outcome is agreed across the warp
          if (!(ok = __all_sync(0xffffffffu, wait(sfull(X), cx & 1)))) break;
          fence_after();
          const int k0c = key0(U, c) + hf * kHalf;       // the half's first key
          const int lim = last - k0c, lo = from - k0c;  // of the half, keys lo .. lim are visible to the row
          const bool seen = __any_sync(0xffffffffu, lo < kHalf && lim >= 0);  // by any of the warp's rows
          int form = 0;
          float mx = -INFINITY;
          if (seen) {
            auto hide = [&]() {  // the scores changed and hidden, in TMEM, and their maximum
              mx = -INFINITY;
#pragma unroll 1
              for (int k0 = 0; k0 < kHalf; k0 += kStep) {
                float sv[kStep];
                ld32(t_h + k0, sv);
                if constexpr (kCap || kBias) modify(sv, k0c + k0 - pos, slope);
                if (lo > k0) {
#pragma unroll
                  for (int j = 0; j < kStep; ++j)
                    if (j < lo - k0) sv[j] = -INFINITY;
                }
                if (lim - k0 < kStep - 1) {  // the diagonal chunk (or past it): hide the later keys
#pragma unroll
                  for (int j = 0; j < kStep; ++j)
                    if (j > lim - k0) sv[j] = -INFINITY;
                }
                mx = fmaxf(mx, largest(sv) * sl2);
                st32(t_h + k0, sv);
              }
            };
            // Capped without a bias, where the warp's rows see the half whole: the tanh keeps the order of the
            // scores, so the row's maximum is that of the raw ones, and the cap is taken within the exponentials'
            // loop below, by the form that the scores' size allows (so that its multiply-adds run beside the
            // exponentials).  Elsewhere, and where no form serves all of the scores, they are changed first.
            const bool whole = !kBias && !__any_sync(0xffffffffu, lo > 0 || lim < kHalf - 1);
            float sv[kHalf];
            if constexpr (kCap) {
              bool change = !whole;
              if (whole) {
                ld64(t_h, sv);
                mx = largest(sv);  // (scale > 0 keeps the order)
                const float size = fmaxf(mx, -smallest(sv));
                const bool past = __any_sync(0xffffffffu, size > p.tanh_wide_to);
                change = past && p.cap_log2 > kSmallCap;
                form = change ? 0 : past ? 3 : __any_sync(0xffffffffu, size > p.tanh_near_to) ? 2 : 1;
                mx = cap_any(mx * p.scale_log2, p.cap_log2, p.cap_inv);
              }
              if (change) hide();
            } else if (whole) {
              ld64(t_h, sv);
              mx = largest(sv) * sl2;  // (scale > 0 keeps the order)
            } else {
              hide();
            }
          }
          {
            float other;
            if (!(ok = exchange(mx, other))) break;
            mx = fmaxf(mx, other);
          }
          float corr = 1.f;
          const bool move = mx > m + 8.f;
          if (move) {
            corr = m == -INFINITY ? 1.f : exp2f(m - mx);  // (l and O are still zero)
            m = mx;
            l *= corr;
          }
          // P over the row's S columns, 16 keys at a time: the 16 columns of keys 16 k ..
          // 16 k + 15 become 8 columns of high parts (then, for bf16, 8 of low parts)
          if (seen) {
            // P = 2^(scale * s - m) (s = -inf gives 0): the scaling of a pair of scores and
            // the row sums in paired fp32 operations
            // (a row whose window starts in a later chunk has seen no score yet: P is 0)
            const float mref = m == -INFINITY ? 0.f : m;
            const uint64_t sl2x2 = f2pack(sl2, sl2), negm2 = f2pack(-mref, -mref);
            uint64_t ps2[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
            auto store_p = [&](auto exponent) {
#pragma unroll
              for (int k0 = 0; k0 < kHalf; k0 += kStep) {
                float sv[kStep];
                ld32(t_h + k0, sv);
#pragma unroll
                for (int k2 = 0; k2 < kStep; k2 += 16) {
                  uint32_t blk[8 * kParts];
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const float2 y = f2unpack(exponent(f2pack(sv[k2 + 2 * j], sv[k2 + 2 * j + 1])));
                    const float x0 = ex2(y.x), x1 = ex2(y.y);
                    ps2[j & 1] = add2(ps2[j & 1], f2pack(x0, x1));
                    blk[j] = pack2<T>(x0, x1);
                    if constexpr (kParts == 2) {
                      const float2 back = unpack2<T>(blk[j]);
                      blk[8 + j] = pack2<T>(x0 - back.x, x1 - back.y);
                    }
                  }
                  if constexpr (kParts == 2) st16(t_h + k0 + k2, blk);
                  else st8(t_h + k0 + k2, blk);
                }
              }
            };
            if constexpr (kCap && !kBias) {
              if (form == 1) {
                store_p([&](uint64_t x) { return odd_poly(x, p.tanh_near, negm2); });
              } else if (form == 2) {
                store_p([&](uint64_t x) { return odd_poly(x, p.tanh_wide, negm2); });
              } else if (form == 3) {
                const float e = p.tanh_exp, cap = p.cap_log2, top = p.cap_log2 - mref;
                store_p([&](uint64_t x) {
                  const float2 v = f2unpack(x);
                  return f2pack(cap_small(v.x, e, cap, top), cap_small(v.y, e, cap, top));
                });
              }
            }
            if (form == 0) store_p([&](uint64_t x) { return fma2(x, sl2x2, negm2); });
            const float2 s0 = f2unpack(ps2[0]), s1 = f2unpack(ps2[1]);
            l += (s0.x + s0.y) + (s1.x + s1.y);
          } else {
            const uint32_t zero[16] = {};
#pragma unroll
            for (int k2 = 0; k2 < kHalf / 16; ++k2) st16(t_h + 16 * k2, zero);
          }
          wait_st();
          // O holds P V up to chunk c - 1, finished (S(c) was issued after it): rescale half of the
          // row's columns if the maximum moved (the whole warp takes the branch when one of its rows
          // needs it; the others scale by 1)
          const bool rescale = c > 0 && move && corr != 1.f;
          if (__any_sync(0xffffffffu, rescale)) {
            const float f = rescale ? corr : 1.f;
#pragma unroll
            for (int c0 = hf * (D / 2); c0 < (hf + 1) * (D / 2); c0 += 32) {
              float o[32];
              ld32(t_o + c0, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= f;
              st32(t_o + c0, o);
            }
          }
          // the first chunk: V of keys below the unit's first one reads as zero too (blocks
          // before it are not copied)
          if (X == 0 && c == 0 && U.lo > key0(U, c)) {
            const int gc = g + c;
            if (!(ok = __all_sync(0xffffffffu, wait(&fullv[gc % kVStages], (gc / kVStages) & 1)))) break;
            unsigned char* vbase = smem + Sh::kOffV + (gc % kVStages) * Sh::kVBytes;
            constexpr int kRow = 2 * BS, kUnits = kRow / 16;
            const int k1 = U.lo - key0(U, c);  // keys 0 .. k1 - 1 of the chunk (k1 < kKeys)
            for (int i = tid; i < (k1 + 7) / 8 * D; i += kTileThreads) {
              const int g8 = i / D, d = i % D;  // as below
              const int a = d * kRow + ((8 * g8) % BS) * 2;
              unsigned char* ptr = vbase + ((8 * g8) / BS) * Sh::kTile + (a ^ (((a >> 7) & (kUnits - 1)) << 4));
              if (8 * g8 + 8 <= k1) {
                *reinterpret_cast<uint4*>(ptr) = make_uint4(0, 0, 0, 0);
              } else {
                for (int kk = 0; 8 * g8 + kk < k1; ++kk) *reinterpret_cast<T*>(ptr + 2 * kk) = DType<T>::from_f32(0.f);
              }
            }
            fence_proxy_async_smem();
          }
          // the last chunk: V of keys past the sequence (or past the blocks loaded) reads as
          // zero; tile A's threads clear it before either tile's P V of the chunk is issued
          if (X == 0 && c == U.nchunks - 1 && kz - key0(U, c) < kKeys) {
            const int gc = g + c;
            if (!(ok = __all_sync(0xffffffffu, wait(&fullv[gc % kVStages], (gc / kVStages) & 1)))) break;
            // block b's tile [D][bs]: dim d's keys 8 g .. 8 g + 7 are the 16 bytes at d * 2 bs + 16 g
            // within the row, moved by the swizzle (16-byte unit bits xor'ed with bits 7 and up)
            unsigned char* vbase = smem + Sh::kOffV + (gc % kVStages) * Sh::kVBytes;
            constexpr int kRow = 2 * BS, kUnits = kRow / 16;
            const int k0 = kz - key0(U, c);  // first key to clear (0 <= k0 < kKeys)
            const int g0 = k0 / 8;          // the 8-key group holding it
            for (int i = tid; i < (kKeys / 8 - g0) * D; i += kTileThreads) {
              const int g8 = g0 + i / D, d = i % D;  // keys 8 g8 .. 8 g8 + 7 of dim d
              const int a = d * kRow + ((8 * g8) % BS) * 2;
              unsigned char* ptr = vbase + ((8 * g8) / BS) * Sh::kTile + (a ^ (((a >> 7) & (kUnits - 1)) << 4));
              if (8 * g8 >= k0) {
                *reinterpret_cast<uint4*>(ptr) = make_uint4(0, 0, 0, 0);
              } else {
                for (int kk = k0 - 8 * g8; kk < 8; ++kk) *reinterpret_cast<T*>(ptr + 2 * kk) = DType<T>::from_f32(0.f);
              }
            }
            fence_proxy_async_smem();
          }
          fence_before();
          mbar_arrive(pfull(X));
        }
        if (!ok) break;
        next();
        if (!ok) break;
        // the unit's output: O / l, read out of TMEM (then the columns are free for the
        // next unit's P V), rounded to T, stored as the row's D contiguous elements
        if (!(ok = __all_sync(0xffffffffu, wait(pvdone(X), ux & 1)))) break;
        fence_after();
        {
          float other;
          if (!(ok = exchange(l, other))) break;
          l = hf ? other + l : l + other;  // (the same sum in both)
        }
        const float inv = 1.f / l;
        const uint64_t inv2 = f2pack(inv, inv);
        uint32_t o16[D / 4];
#pragma unroll
        for (int c0 = 0; c0 < D / 2; c0 += 32) {  // half of the row's columns
          float o[32];
          ld32(t_o + hf * (D / 2) + c0, o);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 v = f2unpack(mul2(f2pack(o[j], o[j + 1]), inv2));
            o16[(c0 + j) / 2] = pack2<T>(v.x, v.y);
          }
        }
        fence_before();
        mbar_arrive(ofree(X));
        if (N.s >= 0 && N.ntiles > X) q_landed();  // the next unit's first S_X may go
        store_rows<T, D / 2, D>(o16, static_cast<T*>(p.out) + hf * (D / 2),
                         valid ? (long long)(U.tok0 + row / G) * p.num_heads + (long long)U.kvh * G + row % G : -1);
        ++ux;
      } else {  // no rows of this tile in the unit: only the next unit's Q
        next();
        if (!ok) break;
        if (N.s >= 0 && N.ntiles > X) q_landed();
      }
      g += U.nchunks;
      U = N;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no Q copy lands after the CTA exits
  } else if (warp == kCopyWarp) {
    // ================= copies (warp 16): K gathers, then V boxes, chunk after chunk of each unit =================
    // This CTA issues its half of each chunk's copies, each into both CTAs of the
    // cluster: lane i the gather4 load crank * kGathers / 2 + i of K (8-dim slice dc,
    // keys 64 h .. 64 h + 63), lane b the V box of the chunk's block b when b % 2 is
    // its rank.  Each CTA's full barriers expect the whole chunk.  Buffer positions run
    // on over the units (g counts the chunks of all units so far).
    constexpr int kGathers = (D / 8) * (kKeys / 64), kMine = kGathers / kCluster;
    static_assert(kGathers <= 32 && Sh::kBlocks <= 32 && kGathers % kCluster == 0, "one copy per lane");
    const int gi = static_cast<int>(crank) * kMine + lane;  // this lane's gather (lanes < kMine)
    const int dc = gi / (kKeys / 64), h = gi % (kKeys / 64);
    bool ok = true;
    int g = 0;
    for (int k = 0; ok; ++k) {
      UnitView U{};
      if (!(ok = take_unit(k, U)) || U.s < 0) break;
      const int32_t* bt = p.block_tables + (long long)U.s * p.max_blocks_per_seq;
      auto phys_of = [&](int c) {  // lane b: the physical block of the chunk's block b (-1 past the keys)
        const int gb = (U.c0 + c) * Sh::kBlocks + lane;
        return lane < Sh::kBlocks && gb < U.nblk && gb >= U.lo / BS ? __ldg(bt + gb) : -1;
      };
      int ph = phys_of(0);  // the next chunk's table entries land while a chunk is in flight
      for (int c = 0; c < U.nchunks; ++c) {
        const int gc = g + c, kb = gc % kKStages, vb = gc % kVStages;
        const int gb0 = (U.c0 + c) * Sh::kBlocks;
        const bool live = lane < Sh::kBlocks && gb0 + lane < U.nblk && gb0 + lane >= U.lo / BS;
        const bool bad = ph < 0 || ph >= p.num_blocks;
        if (live && bad) set_error(p.err, kErrBlockId);
        // the first block of a chunk that holds keys: block 0, or the one a window starts in
        const int ph0 = __shfl_sync(0xffffffffu, bad ? 0 : ph, max(0, U.lo / BS - gb0));
        // a block past (or before) the keys: any rows do (S there is masked; its V is not copied)
        const long long tl = (long long)(live ? (bad ? 0 : ph) : ph0) * p.num_kv_heads + U.kvh;
        const int nlive = __popc(__ballot_sync(0xffffffffu, live));
        int rw[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // the rows (16 keys each) of this lane's 64 keys
          const int key = 64 * h + 16 * q;
          const long long tb = __shfl_sync(0xffffffffu, tl, key / BS);
          rw[q] = static_cast<int>((tb * (D / 8) + dc) * (BS / 16) + (key % BS) / 16);
        }
        if (gc >= kKStages &&  // both CTAs' S read the buffer (in both CTAs)
            !(ok = __all_sync(0xffffffffu, wait(&kfree[kb], ((gc - kKStages) / kKStages) & 1))))
          break;
        if (lane == 0) mbar_arrive_expect_tx(&fullk[kb], Sh::kKBytes);
        __syncwarp();
        if (lane < kMine)  // lands as [64 keys][8 dims] in the slice's rows, in both CTAs
          tma_gather4_mc(smem + Sh::kOffK + kb * Sh::kKBytes + dc * (kKeys * 16) + h * (64 * 16), &tmap_k, rw,
                         &fullk[kb], kClusterMask);
        issued_k = gc + 1;
        if (gc >= kVStages &&  // both CTAs' P V read the buffer (in both CTAs)
            !(ok = __all_sync(0xffffffffu, wait(&vfree[vb], ((gc - kVStages) / kVStages) & 1))))
          break;
        if (lane == 0) mbar_arrive_expect_tx(&fullv[vb], nlive * Sh::kTile);
        __syncwarp();
        if (live && lane % kCluster == static_cast<int>(crank))  // the (block, kv head) tile [D][bs], swizzled;
          tma_2d_mc(smem + Sh::kOffV + vb * Sh::kVBytes + lane * Sh::kTile, &tmap_v, 0,  // V past the keys is zeroed
                    static_cast<int>(tl * D), &fullv[vb], kClusterMask);                // by the softmax threads
        issued_v = gc + 1;
        ph = phys_of(c + 1);
      }
      g += U.nchunks;
    }
  } else if (warp == kIdleWarp) {
    // =============== nothing (warp 19) ===============
  } else if (warp == kSchedWarp) {
    // ================= the unit ring (warp 18): this cluster's units =================
    // Every cluster replays the same assignment of all units of the launch (assign_units);
    // this cluster's enter the ring in that order.  Both CTAs of a cluster write
    // the same sequence; a unit with x < 0 ends it.
    const int longest = build_table(p, tab);
    const int cid = blockIdx.x / kCluster, ncl = gridDim.x / kCluster;  // ncl <= 32 kLoadsPerLane
    int k = 0;
    bool ok = true;
    auto push = [&](int s, int kvh, int ui) {  // the next unit of this cluster into the ring
      const int slot = k % kUnitSlots;
      if (k >= kUnitSlots && !__all_sync(0xffffffffu, wait(&uempty[slot], ((k - kUnitSlots) / kUnitSlots) & 1))) {
        ok = false;
        return;
      }
      if (lane == 0) {
        volatile int* at = s_unit + Sh::kUnitInts * slot;
        at[0] = s;
        at[1] = kvh;
        at[2] = ui;
        if (s >= 0) {
          const int ctx = tab[s], rows = tab[kMaxSeqsPerLaunch + s], n = rows / G;
          int lo, hi;
          masked_keys(p.window, tab[3 * kMaxSeqsPerLaunch + s], ctx, rows, G, ui, lo, hi);
          at[3] = ctx + n;
          at[4] = tab[4 * kMaxSeqsPerLaunch + s];
          at[5] = n;
          at[6] = lo;
          at[7] = hi;
          at[8] = tab[3 * kMaxSeqsPerLaunch + s];
        }
        mbar_arrive(&ufull[slot]);  // release: the slot's words before the phase completes
      }
      __syncwarp();
      ++k;
    };
    assign_units(p, tab, longest, cid, ncl, [&](int s, int kvh, int ui) {
      push(s, kvh, ui);
      return ok;
    });
    if (ok) push(-1, 0, 0);
  } else {
    // ================= MMAs (warp 17): per unit S_X(0), then per chunk P V_A(c), S_A(c + 1), P V_B(c), S_B(c + 1) =================
    // The whole warp runs the loop and the waits (so the loop state and the descriptors
    // stay warp-uniform); one elected lane issues the MMAs and the commits.  A CTA
    // without rows in a unit (the unit's second pair missing) still frees each buffer
    // for its partner: it commits to the free barriers of both CTAs with no MMA before.
    constexpr uint32_t kIdS = idesc<T>(kRows, kKeys), kIdO = idesc<T>(kRows, D);
    const bool leader = elect_one();
    // descriptors of the first Q tile, K buffer and V buffer; a step moves the address
    // field (bits 0..13, 16-byte units), which stays below 2^14 for any shared address
    const uint64_t dq0 = sdesc(smem_addr(smem), 128, (D / 8) * 128);
    const uint64_t dk0 = sdesc(smem_addr(smem + Sh::kOffK), kKeys * 16, 128);
    // V: one [D][bs] tile per block, rows of 2 bs bytes with the matching swizzle; the keys
    // 16 kk .. 16 kk + 15 are block 16 kk / bs, at byte 2 (16 kk % bs) of its rows
    const uint64_t dv0 = sdesc_swizzled(smem_addr(smem + Sh::kOffV), 8 * BS * 2, BS == 16 ? 6u : 4u);
    auto wait_all = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
    uint64_t* last_bar = nullptr;  // the last barrier a commit was issued to, and its phase
    int last_par = 0;
    auto commit_to = [&](uint64_t* bar, int parity, bool both = false) {  // both: the free barriers of both CTAs
      if (leader) {
        if (both) commit_mc(bar, kClusterMask);
        else commit(bar);
      }
      __syncwarp();
      last_bar = bar;
      last_par = parity;
    };
    int cx[2] = {0, 0}, ux[2] = {0, 0};  // per tile: chunks (S, P V) and units it had rows in
    auto issue_s = [&](int Xm, int gc) {  // S_X = Q_X K(gc)^T into X's S columns
      if (leader) {
        const uint64_t da = dq0 + Xm * (Sh::kQTile >> 4), db = dk0 + (gc % kKStages) * (Sh::kKBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma(tmem + 256 * Xm, da + ks * 16, db + ks * (2 * kKeys), kIdS, ks > 0);
      }
      commit_to(sfull(Xm), cx[Xm] & 1);
    };
    auto issue_pv = [&](int Xm, int gc, bool first) {  // O_X (+)= P_X V(gc): high parts, then low parts
      if (leader) {
        const uint64_t db = dv0 + (gc % kVStages) * (Sh::kVBytes >> 4);
        const uint32_t tb = tmem + 256 * Xm;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)  // keys 16 kk ..: high parts in 8 columns, low in the next 8
            mma_ts(tb + kKeys, tb + 16 * kk + 8 * part,
                   db + (((16 * kk) / BS) * Sh::kTile + ((16 * kk) % BS) * 2) / 16, kIdO, !first || part > 0 || kk > 0);
        }
      }
    };
    // the timeout-path test: the first wait runs out on `never` (no MMA issued yet);
    // the producer then drains its copies with the normal limit
    bool ok = __all_sync(0xffffffffu, !p.test_wait_ns || wait_or_abort(never, 0, s_abort, p.err, p.test_wait_ns));
    int g = 0;  // chunks of all units so far
    UnitView N{};  // the next unit, taken during a unit's last chunk
    if (ok) ok = take_unit(0, N);
    for (int k = 0; ok; ++k) {
      if (N.s < 0) break;
      const UnitView U = N;
      const int nt = U.ntiles, nc = U.nchunks;
      // S of the unit's first chunk, for each tile as soon as its Q has landed (the
      // previous unit's P V run ahead of it on the tensor cores)
      if (!(ok = wait_all(&fullk[g % kKStages], (g / kKStages) & 1))) break;
      for (int Xm = 0; Xm < nt && ok; ++Xm) {
        if (!(ok = wait_all(qfull(Xm), ux[Xm] & 1))) break;
        fence_after();
        issue_s(Xm, g);
      }
      if (!ok) break;
      commit_to(&kfree[g % kKStages], (g / kKStages) & 1, true);
      for (int c = 0; c < nc && ok; ++c) {
        const int gc = g + c, vb = gc % kVStages, g1 = gc + 1;
        if (c == nc - 1 && !(ok = take_unit(k + 1, N))) break;
        if (!(ok = wait_all(&fullv[vb], (gc / kVStages) & 1))) break;
        if (kEarlyK && c + 1 < nc && nt > 0 && !(ok = wait_all(&fullk[g1 % kKStages], (g1 / kKStages) & 1))) break;
        for (int Xm = 0; Xm < nt && ok; ++Xm) {
          if (!(ok = wait_all(pfull(Xm), cx[Xm] & 1))) break;  // the softmax wrote P_X(c)
          // the first P V of a unit overwrites O_X: the previous unit's O_X is read out
          if (c == 0 && ux[Xm] > 0 && !(ok = wait_all(ofree(Xm), (ux[Xm] - 1) & 1))) break;
          fence_after();
          issue_pv(Xm, gc, c == 0);
          if (Xm == nt - 1) commit_to(&vfree[vb], (gc / kVStages) & 1, true);
          if (c == nc - 1) commit_to(pvdone(Xm), ux[Xm] & 1);  // O_X is complete
          ++cx[Xm];
          if (c + 1 < nc) {
            if (!kEarlyK && Xm == 0 && !(ok = wait_all(&fullk[g1 % kKStages], (g1 / kKStages) & 1))) break;
            // S_X(c + 1) overwrites the columns P V_X(c) reads, issued right behind it: MMAs
            // of one thread run in issue order, so no wait is needed between the two
            fence_after();
            issue_s(Xm, g1);
            if (Xm == nt - 1) commit_to(&kfree[g1 % kKStages], (g1 / kKStages) & 1, true);
          }
        }
        if (nt == 0 && ok) {  // no rows: free the buffers for the partner as they land
          commit_to(&vfree[vb], (gc / kVStages) & 1, true);
          if (c + 1 < nc) {
            if (!(ok = wait_all(&fullk[g1 % kKStages], (g1 / kKStages) & 1))) break;
            commit_to(&kfree[g1 % kKStages], (g1 / kKStages) & 1, true);
          }
        }
      }
      for (int Xm = 0; Xm < nt; ++Xm) ++ux[Xm];
      g += nc;
    }
    // The partner's last commits arrive on this CTA's free barriers: wait (bounded) for
    // their final phases, so nothing lands in this CTA's shared memory after it exits.
    if (ok) {
      for (int c = max(0, g - kKStages); c < g; ++c)
        mbar_wait_bounded(&kfree[c % kKStages], (c / kKStages) & 1, kWaitNs / 8);
      for (int c = max(0, g - kVStages); c < g; ++c)
        mbar_wait_bounded(&vfree[c % kVStages], (c / kVStages) & 1, kWaitNs / 8);
    }
    // MMAs committed but maybe not finished: a commit tracks every earlier MMA of the
    // issuing thread, so the last commit's barrier covers them all
    if (!ok && last_bar != nullptr) mbar_wait_bounded(last_bar, last_par, kWaitNs / 8);
  }

  fence_before();
  __syncthreads();
  // After an abort no consumer waits for the copies still landing: the copy warp waits
  // (bounded) for the last chunks it issued, so nothing lands after the CTA exits.
  if (*s_abort && warp == kCopyWarp && lane == 0) {
    for (int c = issued_k - kKStages; c < issued_k; ++c)
      if (c >= 0) mbar_wait_bounded(&fullk[c % kKStages], (c / kKStages) & 1, kWaitNs / 8);
    for (int c = issued_v - kVStages; c < issued_v; ++c)
      if (c >= 0) mbar_wait_bounded(&fullv[c % kVStages], (c / kVStages) & 1, kWaitNs / 8);
  }
  // Neither CTA of the cluster leaves while the other may still copy into it or
  // commit to its barriers (every wait above is bounded, so both arrive here).
  __syncthreads();
  cluster_sync_all();
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kTmemCols));
  }
}

}  // namespace wsm
}  // namespace pa
