// fp4_decode.cu -- decode attention over FP4 pools (see fp4.cuh).
//
// What is computed: for a sequence s and the query heads that share a kv head,
//     out = s_v sum_t p_t (code sf)_t / sum_t p_t,  p_t = 2^(hs q . (code sf)_t - m),
// with hs = scale s_k log2 e and a running maximum m (one pass over the tokens).
// With m = hs m': pieces of a sequence done apart are merged with M' = max m'_i and factors
// 2^(hs (m'_i - M')): like a weight's exponent, the difference first, so that scores of any size
// leave the largest however the work is cut (hs m' itself may be past fp32's largest number).
//
// How it maps to the GPU.
//   * Work: a segment is (sequence, head unit), cut into chunks of 32 tokens.  All
//     chunks of the launch are laid end to end; the grid is at most one CTA per SM and
//     every warp of it takes one equal run of chunks, crossing segments; where segments are
//     short, the CTAs' shares are rounded to whole segments (the rule and why: at kExtraRounds'
//     use; 30 sequences of 300-500 tokens, 32/8 heads, 10.3 -> 7.8 us).  12 warps (up to
//     168 registers each): 16 of 128 registers measured 3-7% slower, 10 and 13 12%.
//   * Copies: each warp has its own ring of stages in shared memory, filled by asynchronous
//     16-byte copies (cp.async) of its own lanes: a chunk is one or two blocks of K and of V,
//     each a contiguous tile.  No other warp takes part, so a warp waits on nobody.
//     (Bulk copies with an mbarrier a stage cost more instructions and latency to issue than
//     these nine copies a lane: four contexts of 32K-128K tokens 80 against 75 us.  Loads
//     straight into registers left too little in flight: 98 us.)  Two stages a warp; three
//     measured 1-3% slower.
//   * Math: m16n8k16 tensor-core tiles with fp16 operands: S^T = K Q^T, O^T += V^T P^T,
//     tokens and dims on the 16-row side, query heads on the 8-column side.  A code is
//     widened by one conversion per two codes and one multiplication by its group's scale
//     per two codes, both exact (code * sf has 6 significant bits).  The tile's byte order
//     gives each lane whole 32-bit words of codes: K as it lies; V with the nibbles of two
//     tokens interleaved by four bit operations per two words, because an operand register
//     holds two tokens of one dim.  About 530 instructions a chunk of 128 dims and 8 heads,
//     260 of them on the half-rate ALU: the math of a chunk takes an SM about as long as its
//     4608 bytes take from DRAM, so both bound the kernel at once.
//   * Merging: a warp that did a whole segment writes its output.  Pieces cut at a warp's
//     ends go to shared memory and the CTA merges them once at its end.  A segment cut at
//     CTAs' ends is merged by the CTA that holds its last piece: every other CTA of it
//     publishes its piece in the workspace with a tag of this call, and the last one waits
//     for the tags, merges, and clears them.  It waits for CTAs of lower index only, which
//     are dispatched before it and publish before they wait themselves; the wait is bounded.
//     A tag is 64 random bits a launch, so the workspace needs no initialisation, and
//     cleared when used, so a call replayed from a graph never meets an older one's.
//
// Measured on a GB300 (fp16, 128 dims, 16-token blocks unless said; floor: the bytes at the
// measured copy rate): 64 sequences of 512-4096 tokens, 28/4 heads, 23.4 us (floor 12.6);
// 16 x 2048 tokens, 32/32 heads, 32.5 us (22.3); 4 x 32K-131K tokens, 32/8 heads, bf16,
// 71.7 us (60.5); one sequence of 100 tokens 3.1 us, what its launch, three dependent loads
// and one chunk take.  About 5 us of the larger calls are the schedule (1.2), the first
// copies (1), and the merging of pieces with the waits for the slowest warp and CTA (3).
#include <math.h>

#include <type_traits>

#include "fp4.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kChunk = 32;            // tokens
constexpr float kNoScore = -1e30f;    // below every score (|score| < 2^35)
// Weights are taken 2^7 times as large (it cancels in the normalised sum) and may grow by another
// 2^8 before the reference moves: up to 2^15, inside fp16, while a weight of 2^-21 of the largest
// score's still has all 11 bits, and one below 2^-32 of it vanishes.
constexpr float kRaise = 7.f, kSlack = 8.f;

// NT: 8-column tiles of query heads (a unit has up to 8 NT heads).
template <int D, int NT>
struct Fp4Shape {
  static constexpr int kWarps = NT == 1 || D == 64 ? 12 : 8;
  static constexpr int kRows = 8 * NT;
  static constexpr int kStage = 2 * kChunk * (D / 2 + D / 16);
  static constexpr int kStages = D == 64 ? 4 : NT == 1 ? 2 : 4;
  static constexpr int kPiece = kRows * D * 4;                  // an unnormalised partial output
  static constexpr int kFirst = kWarps * kStages * kStage;      // [warps]: the piece a warp starts with
  static constexpr int kMl = kFirst + kWarps * kPiece;          // [2 warps][rows]: (m', l)
  static constexpr int kRun = kMl + 2 * kWarps * kRows * 8;     // [warps + 1][rows]: a run's (M', W), by its first warp
  static constexpr int kFactor = kRun + (kWarps + 1) * kRows * 8; // [2 warps][rows]: a piece's hs, then its weight in its run
  static constexpr int kHs = kFactor + 2 * kWarps * kRows * 4;  // [rows]: hs of the run that warp 0 does not begin
  static constexpr int kSeg = kHs + kRows * 4;                  // [2 warps] int2: (sequence or -1, unit and kBegins)
  static constexpr int kLen = kSeg + 2 * kWarps * 8;            // [seqs]
  static constexpr int kPre = kLen + kMaxSeqsPerLaunch * 4;     // [seqs + 1], then the scan's warp sums and maxima
  static constexpr int kBytes = kPre + (kMaxSeqsPerLaunch + 1 + 2 * kWarps + 3) * 4;
  static_assert(kStages >= 2 && kPiece <= kStages * kStage, "a warp's last piece takes its ring's place");
  static_assert(kStage % 128 == 0 && kMl % 16 == 0, "alignment");
  static_assert(kWarps <= 31 && kBytes <= 227 * 1024, "a bit per warp; shared memory per CTA");
};

// n tokens in pieces of `size`, for any int n >= 0.
__host__ __device__ constexpr int pieces_of(int n, int size) { return static_cast<int>((static_cast<unsigned>(n) + size - 1) / size); }

constexpr uint64_t kFp4WaitNs = 1000000000ull;  // 1 s, then PA_DEVERR_TIMEOUT
constexpr int kMergeBatch = 8;                  // pieces of other CTAs loaded at once
constexpr int kExtraRounds = 2;                 // chunks of a warp that are worth not cutting segments at CTAs' ends
constexpr int kBegins = 1 << 30;  // beside a unit's number: the piece holds its segment's first chunk

__device__ __forceinline__ float ex2(float x) {  // |relative error| < 2^-22, 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const unsigned char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the last N groups of this lane's copies have landed
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The value in memory at this moment, whatever an earlier load of this kernel saw.
__device__ __forceinline__ int ld_now(const int32_t* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ uint64_t ld_acquire(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.acquire.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint64_t* p, uint64_t v) {
  asm volatile("st.release.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}

// One half of a pair, twice.
__device__ __forceinline__ uint32_t low2(uint32_t a) {
  const __half2 r = __low2half2(*reinterpret_cast<const __half2*>(&a));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t high2(uint32_t a) {
  const __half2 r = __high2half2(*reinterpret_cast<const __half2*>(&a));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// d += a b, and d = a b (the first product of a sum, with no zeroing of d before it).
__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// One warp's running softmax of a unit's query heads.
template <typename T, int D, int BS, int NT>
struct Fp4Math {
  static constexpr int KS = D / 16;  // k-steps of S^T, and 16-row tiles of O^T
  static constexpr int KW = D / 32;  // words of codes a lane holds of a K row
  static constexpr int VW = D / 64;  // and of a V row
  static constexpr int TILE = fp4::tile_bytes(D, BS);

  uint32_t qb[KS][NT][2];
  float acc[KS][NT][4];
  float lacc[NT][4];  // the weights' sums of heads 8n + 2 t4 + {0, 1} (twice): a product with ones
  // of those heads: the reference m of the exponents, the score above which m moves, hs
  float m_[NT][2], lim_[NT][2], hs_[NT][2];
  int g, t4;
  int k_at, ks_at, v_at[2], vs_at;  // this lane's places in a sub-tile (fp4::code_at and its scales')

  __device__ __forceinline__ void init(int lane) {
    g = lane >> 2;
    t4 = lane & 3;
    const int row = ((g >> 1) ^ ((g & 1) ? 3 : 0)) + 4 * (g & 1);  // of token tok; of tok + 2: 8 rows on
    k_at = row * (D / 2) + ((t4 * (D / 8)) ^ (D == 128 ? ((row >> 1) & 1) << 5 : 0));
    ks_at = BS * (D / 2) + g * (D / 8) + t4 * (D / 32);
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {  // of tokens 4 t4 + {0, 2} and {1, 3}; i: 4 i rows on
      const int r = t4 ^ (odd ? 3 : 0);
      v_at[odd] = r * (D / 2) + (D == 128 ? (8 * g) ^ (((r >> 1) & 1) << 5) : 4 * g);
    }
    vs_at = BS * (D / 2) + (D == 128 ? g : g >> 1) * 16 + 4 * t4;
  }

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[k][n][0] = acc[k][n][1] = acc[k][n][2] = acc[k][n][3] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      lacc[n][0] = lacc[n][1] = lacc[n][2] = lacc[n][3] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) m_[n][c] = lim_[n][c] = kNoScore;  // the first chunk sets them
    }
  }

  // Q^T fragments: lane (g, t4) holds dims D/4 t4 .. of head 8n + g, four per k-step, as
  // the K words hold them.
  __device__ __forceinline__ void load_q(const T* q, int nh) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = 8 * n + g;
#pragma unroll
      for (int k = 0; k < KS / 2; ++k) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (h < nh) w = *reinterpret_cast<const uint4*>(q + h * D + t4 * (D / 4) + 8 * k);
        qb[2 * k][n][0] = w.x;
        qb[2 * k][n][1] = w.y;
        qb[2 * k + 1][n][0] = w.z;
        qb[2 * k + 1][n][1] = w.w;
      }
    }
  }

  // scale_log2 may be negative: its sign goes into q, so that the largest score is the
  // largest exponent.  bf16 heads become fp16 with a power of two taken from the head's
  // largest |q|, put back by hs_.  An element down to 2^-30 of the largest keeps its 8 bits; a
  // smaller one lands among fp16's subnormals and is off by at most 2^-25, 2^-38 of the largest.
  __device__ __forceinline__ void scale_q(float scale_log2) {
    const float mag = fabsf(scale_log2);
    if (scale_log2 < 0.f) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          qb[k][n][0] ^= 0x80008000u;
          qb[k][n][1] ^= 0x80008000u;
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      hs_[n][0] = hs_[n][1] = mag;
      if constexpr (!std::is_same<T, __half>::value) {
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 v = unpack2<T>(qb[k][n][i]);
            mx = fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 2^e with mx 2^e in [2^13, 2^14): the exponent field of mx names it
        int e = mx > 0.f ? 13 - (static_cast<int>(__float_as_uint(mx) >> 23) - 127) : 0;
        e = min(max(e, -120), 120);
        const float up = __uint_as_float((127 + e) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 v = unpack2<T>(qb[k][n][i]);
            qb[k][n][i] = pack2<__half>(v.x * up, v.y * up);
          }
        const float down = fminf(mag * __uint_as_float((127 - e) << 23), 0x1p127f);  // (inf * 0 would be NaN)
        hs_[n][0] = __shfl_sync(0xffffffffu, down, 8 * t4);  // heads 2 t4 and 2 t4 + 1
        hs_[n][1] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
      }
    }
  }

  // A chunk's bytes as this lane needs them.
  struct Raw {
    uint32_t lo[2][KW], hi[2][KW], ks[2];  // K codes of tokens tok and tok + 2 of each sub-tile, their scales
    uint32_t x[2][4][VW], vs[2];           // V codes of tokens 4 t4 + i, dims 16 g .. (D 128) or 8 g .. (D 64)
  };

  static constexpr int kSub = BS == 16 ? TILE : 16 * (D / 2);        // codes of the chunk's second 16 tokens
  static constexpr int kSubScale = BS == 16 ? TILE : 16 * (D / 16);  // and their scales

  __device__ __forceinline__ void fetch_k(const unsigned char* kc, Raw& f) const {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const unsigned char *at = kc + mt * kSub + k_at, *sc = kc + mt * kSubScale + ks_at;
      if constexpr (D == 128) {
        const uint4 a = *reinterpret_cast<const uint4*>(at), b = *reinterpret_cast<const uint4*>(at + 4 * D);
        f.lo[mt][0] = a.x, f.lo[mt][1] = a.y, f.lo[mt][2] = a.z, f.lo[mt][KW - 1] = a.w;
        f.hi[mt][0] = b.x, f.hi[mt][1] = b.y, f.hi[mt][2] = b.z, f.hi[mt][KW - 1] = b.w;
        f.ks[mt] = *reinterpret_cast<const uint32_t*>(sc);
      } else {
        const uint2 a = *reinterpret_cast<const uint2*>(at), b = *reinterpret_cast<const uint2*>(at + 4 * D);
        f.lo[mt][0] = a.x, f.lo[mt][KW - 1] = a.y;
        f.hi[mt][0] = b.x, f.hi[mt][KW - 1] = b.y;
        f.ks[mt] = *reinterpret_cast<const uint16_t*>(sc);
      }
    }
  }

  __device__ __forceinline__ void fetch_v(const unsigned char* vc, Raw& f) const {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned char* at = vc + mt * kSub + v_at[i & 1] + i * 2 * D;
        if constexpr (D == 128) {
          const uint2 w = *reinterpret_cast<const uint2*>(at);
          f.x[mt][i][0] = w.x, f.x[mt][i][VW - 1] = w.y;
        } else {
          f.x[mt][i][0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
      f.vs[mt] = *reinterpret_cast<const uint32_t*>(vc + mt * kSubScale + vs_at);
    }
  }

  // S^T of a chunk.
  __device__ __forceinline__ void scores(const Raw& f, float (&sc)[2][NT][4]) const {
    uint32_t sf[2][4];  // the two rows' groups' scales, each twice
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      if constexpr (D == 128) {
        const uint32_t s0 = fp4::e4m3x2_to_f16x2(f.ks[mt]), s1 = fp4::e4m3x2_to_f16x2(f.ks[mt] >> 16);
        sf[mt][0] = low2(s0), sf[mt][1] = high2(s0), sf[mt][2] = low2(s1), sf[mt][3] = high2(s1);
      } else {
        const uint32_t s = fp4::e4m3x2_to_f16x2(f.ks[mt]);
        sf[mt][0] = sf[mt][1] = low2(s), sf[mt][2] = sf[mt][3] = high2(s);
      }
    }
#pragma unroll
    for (int w = 0; w < KW; ++w)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {  // the sub-tiles' chains of MMAs in turn
        uint32_t a[4], b[4];
        fp4::e2m1x8_to_f16x2(f.lo[mt][w], a);
        fp4::e2m1x8_to_f16x2(f.hi[mt][w], b);
        const uint32_t fa = sf[mt][D == 128 ? w / 2 : 0], fb = sf[mt][2 + (D == 128 ? w / 2 : 0)];
        const uint32_t a0[4] = {fp4::hmul2(a[0], fa), fp4::hmul2(b[0], fb), fp4::hmul2(a[1], fa), fp4::hmul2(b[1], fb)};
        const uint32_t a1[4] = {fp4::hmul2(a[2], fa), fp4::hmul2(b[2], fb), fp4::hmul2(a[3], fa), fp4::hmul2(b[3], fb)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (w == 0) mma_first(sc[mt][n], a0, qb[0][n][0], qb[0][n][1]);
          else mma_add(sc[mt][n], a0, qb[2 * w][n][0], qb[2 * w][n][1]);
          mma_add(sc[mt][n], a1, qb[2 * w + 1][n][0], qb[2 * w + 1][n][1]);
        }
      }
  }

  __device__ __forceinline__ static void mask(float (&sc)[2][NT][4], int tok, int rem, float with) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (16 * mt + tok + (c >> 1) * 2 >= rem) sc[mt][n][c] = with;
  }

  // The scores of a chunk become weights, in fp16 as the operand P^T; `rem` valid tokens (more than 31: all).
  __device__ __forceinline__ void weigh(float (&sc)[2][NT][4], uint32_t (&pb)[2][NT][2], int rem) {
    const int tok = 4 * (g >> 1) + (g & 1);  // rows g and g + 8 of S^T are tokens tok and tok + 2 of a sub-tile
    const bool part = rem < kChunk;  // the sequence's last chunk: what lies past its end may be anything
    if (part) mask(sc, tok, rem, kNoScore);
    // The exponents' reference m is the largest score of some earlier chunk.  It moves only when a
    // score is more than kSlack above it (in log2 units): until then the chunk needs no reduction over
    // lanes and no rescaling.
    float top[NT][2];
    bool moves = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[n][c] = fmaxf(fmaxf(sc[0][n][c], sc[0][n][c + 2]), fmaxf(sc[1][n][c], sc[1][n][c + 2]));
        moves |= top[n][c] > lim_[n][c];
      }
    if (__any_sync(0xffffffffu, moves)) move(top);
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // the difference first: exact where it counts, and never above kSlack whatever the scores' size
          sc[mt][n][c] = ex2(fmaf(sc[mt][n][c] - m_[n][c & 1], hs_[n][c & 1], kRaise));
        }
    if (part) mask(sc, tok, rem, 0.f);
    // rounded to fp16 (11 bits, as the operands are fp16); their sums are of what was rounded
    const uint32_t ones[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          pb[mt][n][r] = movmatrix_trans(pack2<__half>(sc[mt][n][2 * r], sc[mt][n][2 * r + 1]));
        mma_add(lacc[n], ones, pb[mt][n][0], pb[mt][n][1]);
      }
  }

  // O^T += V^T P^T.
  __device__ __forceinline__ void add(Raw& f, const uint32_t (&pb)[2][NT][2], int rem) {
    if (rem < kChunk) {  // a scale past the sequence's end may be NaN, and 0 * NaN would stay
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int ok = rem - 16 * mt - 4 * t4;
        f.vs[mt] = ok >= 4 ? f.vs[mt] : ok <= 0 ? 0u : f.vs[mt] & ((1u << (8 * ok)) - 1u);
      }
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t w = f.vs[mt];
      const uint32_t f01 = fp4::e4m3x2_to_f16x2(w), f23 = fp4::e4m3x2_to_f16x2(w >> 16);
#pragma unroll
      for (int v = 0; v < VW; ++v) {
        constexpr uint32_t kLow = 0x0f0f0f0fu;
        uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd dims, token pairs
        fp4::e2m1x8_to_f16x2((f.x[mt][0][v] & kLow) | ((f.x[mt][1][v] << 4) & ~kLow), e01);
        fp4::e2m1x8_to_f16x2(((f.x[mt][0][v] >> 4) & kLow) | (f.x[mt][1][v] & ~kLow), o01);
        fp4::e2m1x8_to_f16x2((f.x[mt][2][v] & kLow) | ((f.x[mt][3][v] << 4) & ~kLow), e23);
        fp4::e2m1x8_to_f16x2(((f.x[mt][2][v] >> 4) & kLow) | (f.x[mt][3][v] & ~kLow), o23);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t a[4] = {fp4::hmul2(e01[b], f01), fp4::hmul2(o01[b], f01), fp4::hmul2(e23[b], f23),
                                 fp4::hmul2(o23[b], f23)};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_add(acc[4 * v + b][n], a, pb[mt][n][0], pb[mt][n][1]);
        }
      }
    }
  }

  // Move the reference to the largest score so far and bring what is summed to it.
  __device__ __forceinline__ void move(const float (&top)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = fmaxf(top[n][c], m_[n][c]);
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        f[c] = ex2((m_[n][c] - v) * hs_[n][c]);  // (at first m is kNoScore, and there is nothing to bring)
        m_[n][c] = v;
        lim_[n][c] = __fadd_rd(v, __fdividef(kSlack, hs_[n][c]));  // (hs 0: infinity)
        lacc[n][c] *= f[c];
        lacc[n][c + 2] *= f[c];
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[k][n][c] *= f[c & 1];
    }
  }

  // Lane (g, t4) holds dims D/8 g .. of heads 8n + 2 t4 + {0, 1}.
  __device__ __forceinline__ void store_out(T* out, int nh, float oscale) const {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = 8 * n + 2 * t4 + c;
        if (h >= nh) continue;
        const float f = oscale / lacc[n][c];
#pragma unroll
        for (int k = 0; k < KS; k += 4) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pack2<T>(acc[k + i][n][c] * f, acc[k + i][n][c + 2] * f);
          *reinterpret_cast<uint4*>(out + h * D + g * (D / 8) + 2 * k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
  }

  // A piece in shared memory: vectors of 4 dims, [head parts (n, c)][vectors of D/8 dims][lane ^ vector],
  // so that neither the lanes that write nor those that read a head's row meet in a bank.
  __device__ __forceinline__ void store_piece(float4* o, float2* ml, float* hs) const {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int k = 0; k < KS; k += 2)
          o[((2 * n + c) * (KS / 2) + k / 2) * 32 + ((4 * g + t4) ^ (k / 2))] =
              make_float4(acc[k][n][c], acc[k][n][c + 2], acc[k + 1][n][c], acc[k + 1][n][c + 2]);
        if (g == 0) {
          ml[8 * n + 2 * t4 + c] = make_float2(m_[n][c], lacc[n][c]);
          hs[8 * n + 2 * t4 + c] = hs_[n][c];
        }
      }
  }
  // Dims 4 i .. 4 i + 3 of head r of a piece.
  __device__ __forceinline__ static const float4* piece_at(const float4* o, int r, int i) {
    const int v = i % (KS / 2), gg = i / (KS / 2);
    return o + ((2 * (r >> 3) + (r & 1)) * (KS / 2) + v) * 32 + ((4 * gg + ((r >> 1) & 3)) ^ v);
  }
};

// Head unit u: its kv head, first query head and number of them.  Past 16 heads a kv head's heads are
// units of 16 and a rest, each of which reads and widens all of K and V for itself, with 16 columns: a rest of
// one head costs nearly what 16 do (16 sequences of 2048 tokens, 4 kv heads of 128 dims: 8 heads each 11.0 us, 9 to
// 16 12.8, 17 17.7, 32 18.4, 33 22.3; of 64 dims 9.5, 10.5 to 11.1, 13.9, 14.3, 16.6).
__device__ __forceinline__ void unit_heads(const Fp4DecodeParams& p, int u, int& kvh, int& h0, int& nh) {
  if (p.group <= 16) {
    kvh = u;
    h0 = u * p.group;
    nh = p.group;
    return;
  }
  const int per = (p.group + 15) >> 4;
  kvh = u / per;
  h0 = kvh * p.group + (u - kvh * per) * 16;
  nh = min(16, kvh * p.group + p.group - h0);
}

// Warps of each CTA that share `total` chunks.
template <int WARPS>
__device__ __forceinline__ int active_warps(int total) {
  const int grid = static_cast<int>(gridDim.x);
  return total >= grid * WARPS ? WARPS : (total + grid - 1) / grid;
}

template <typename T, int D, int BS, int NT>
__global__ void __launch_bounds__(Fp4Shape<D, NT>::kWarps * 32, 1) decode_fp4_kernel(const Fp4DecodeParams p) {
  using Sh = Fp4Shape<D, NT>;
  using Math = Fp4Math<T, D, BS, NT>;
  constexpr int WARPS = Sh::kWarps, STAGES = Sh::kStages, TILE = Math::TILE, NB = kChunk / BS;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* ring = smem + warp * STAGES * Sh::kStage;
  // entry e: a warp's first piece has a place of its own, its last one takes its ring's
  auto piece = [&](int e) {
    return reinterpret_cast<float4*>(e & 1 ? smem + (e >> 1) * STAGES * Sh::kStage
                                           : smem + Sh::kFirst + (e >> 1) * Sh::kPiece);
  };
  float2* s_ml = reinterpret_cast<float2*>(smem + Sh::kMl);
  float2* s_run = reinterpret_cast<float2*>(smem + Sh::kRun);
  float* s_factor = reinterpret_cast<float*>(smem + Sh::kFactor);
  float* s_hs = reinterpret_cast<float*>(smem + Sh::kHs);
  int2* s_seg = reinterpret_cast<int2*>(smem + Sh::kSeg);
  int* s_len = reinterpret_cast<int*>(smem + Sh::kLen);
  int* s_pre = reinterpret_cast<int*>(smem + Sh::kPre);
  int *s_sum = s_pre + kMaxSeqsPerLaunch + 1, *s_most = s_sum + WARPS;

  if (lane < 2) s_seg[2 * warp + lane] = make_int2(-1, 0);  // no piece
  griddep_launch_dependents();

  // The schedule: lengths (0 when outside [1, max_seq_len]), the prefix sum of their chunks,
  // this warp's run of chunks and its first 32 chunks' tiles.  It is made before the wait on
  // the previous kernel, from what seq_lens and block_tables hold then, and kept only if both
  // read the same after it (they seldom change at the last moment); nothing is written or
  // reported before that.  On a busy stream this hides some 3000 cycles.
  const int S = p.num_seqs, U = p.units;
  constexpr int PER = (kMaxSeqsPerLaunch + WARPS * 32 - 1) / (WARPS * 32);
  int lens[PER];  // of sequences tid * PER + k
#pragma unroll
  for (int k = 0; k < PER; ++k) lens[k] = tid * PER + k < S ? ld_now(p.seq_lens + tid * PER + k) : 0;
  int start = 0, len = 0, s = 0, u = 0, j = 0;  // the run; its first chunk is chunk j of unit u of sequence s
  int gs = 0, gu = 0, gj = 0;                   // the first position of the next 32 to look up
  int cur[NB], nxt[NB];                         // lane i: the tiles of position i of 32 (-1: none)
  bool bad = false;                             // some length is outside the contract

  // Lane i finds position i of the next 32: where its blocks' numbers are (`have` of them), and their kv head.
  auto find = [&](int positions, const int32_t*& row, int& have, int& head) {
    int ls = gs, lu = gu, lj = gj + lane;
    have = head = 0;
    row = p.block_tables;
    if (lane < positions) {
      for (int c = s_pre[ls + 1] - s_pre[ls]; lj >= c;) {
        lj -= c;
        if (++lu < U) continue;
        lu = 0;
        do {
          ++ls;
          c = s_pre[ls + 1] - s_pre[ls];
        } while (c == 0);
      }
      int h, c;
      unit_heads(p, lu, head, h, c);
      have = min(pieces_of(s_len[ls], BS) - lj * NB, NB);
      row += (long long)ls * p.max_blocks_per_seq + lj * NB;
    }
    // the next group, if there is one, starts right after lane 31 (a chunk index past its unit is brought in
    // range there)
    gs = __shfl_sync(0xffffffffu, ls, 31);
    gu = __shfl_sync(0xffffffffu, lu, 31);
    gj = __shfl_sync(0xffffffffu, lj, 31) + 1;
  };
  auto read_blocks = [&](const int32_t* row, int have, int (&id)[NB]) {
#pragma unroll
    for (int b = 0; b < NB; ++b) id[b] = b < have ? ld_now(row + b) : 0;
  };
  // Blocks to tiles (-1: none); block 0 for one outside the pool.  Whether there was one.
  auto to_tiles = [&](const int (&id)[NB], int have, int head, int (&tile)[NB]) {
    bool out = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const bool wrong = id[b] < 0 || id[b] >= p.num_blocks;
      out |= b < have && wrong;
      tile[b] = b < have ? (wrong ? 0 : id[b]) * p.num_kv_heads + head : -1;
    }
    return out;
  };
  // Chunk k, its tiles in lane k % 32, into its stage: K, then V, 16 bytes a lane at a time.  (The second
  // tile of a chunk that ends in its first block is not read; the first is copied again.)
  auto copy_chunk = [&](int k) {
    const unsigned char* from[2 * NB];  // tile i, less the pieces before it: piece x of the chunk is at from[i] + 16 x
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      int t = __shfl_sync(0xffffffffu, cur[b], k & 31);
      if (b > 0 && t < 0) t = __shfl_sync(0xffffffffu, cur[0], k & 31);
      from[b] = static_cast<const unsigned char*>(p.k_cache) + (long long)t * TILE + (16 * lane - b * TILE);
      from[NB + b] = static_cast<const unsigned char*>(p.v_cache) + (long long)t * TILE + (16 * lane - (NB + b) * TILE);
    }
    constexpr int kPer = TILE / 16, kAll = 2 * NB * kPer;  // 16-byte pieces of a tile, of a chunk
    const uint32_t to = smem_addr(ring) + (k % STAGES) * Sh::kStage + 16 * lane;
#pragma unroll
    for (int x = 0; x < kAll; x += 32) {
      const int i0 = x / kPer, i1 = (x + 31 < kAll ? x + 31 : kAll - 1) / kPer;  // at most two tiles
      const unsigned char* src = from[i0];
      if (i1 != i0 && x + lane >= i1 * kPer) src = from[i1];
      if (x + 32 <= kAll || x + lane < kAll) copy16(to + 16 * x, src + 16 * x);
    }
  };
  Math math;
  math.init(lane);
  int L = 0, n = 0, h0 = 0, nh = 0, kvh = 0;  // the current segment
  auto fetch_q = [&]() {
    L = s_len[s];
    n = pieces_of(L, kChunk);
    unit_heads(p, u, kvh, h0, nh);
    math.load_q(static_cast<const T*>(p.q) + ((long long)s * p.num_heads + h0) * D, nh);
  };

  bool bad_id = false;
  for (bool waited = false;; waited = true) {
    int count[PER], sum = 0, most = 0;
    bad = false;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = tid * PER + k;
      const bool out = lens[k] < 1 || lens[k] > p.max_seq_len;
      const int L = out ? 0 : lens[k];
      bad |= out && i < S;
      if (i < S) s_len[i] = L;
      count[k] = pieces_of(L, kChunk);
      sum += count[k];
      most = max(most, count[k]);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_sum[warp] = incl, s_most[warp] = most;
    bad = __syncthreads_or(bad);
    int before = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0);
    most = __reduce_max_sync(0xffffffffu, lane < WARPS ? s_most[lane] : 0);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = tid * PER + k;
      if (i <= S) s_pre[i] = before;
      before += count[k];
    }
    if (tid == WARPS * 32 - 1) s_pre[S] = before;
    __syncthreads();

    // The sequence of a chunk: the last one whose prefix is at most the chunk, found by the warp together
    // in 32-way steps (empty sequences have their successor's prefix).
    auto sequence_of = [&](int chunk) {
      int s = 0;
      for (int step = S > 32 ? (S + 31) / 32 : 1;; step = 1) {
        const int i = s + lane * step;
        s += (31 - __clz(__ballot_sync(0xffffffffu, i < S && s_pre[min(i, S)] * U <= chunk))) * step;
        if (step == 1) return s;
      }
    };
    // A share of the launch's chunks (fewer than 2^31).
    const int total = s_pre[S] * U, grid = static_cast<int>(gridDim.x);
    start = len = 0;
    const int per_cta = total / grid, rest = total - per_cta * grid;
    // Where segments are short, a CTA's chunks start where a segment does: no segment is cut at CTAs' ends, which
    // saves the wait for another CTA (about 2 us) and costs longer runs in some CTAs: at most `most` chunks more,
    // whole segments where segments are alike.  It is done where that makes the longest run of a warp at most two
    // chunks longer, and one in the second case (a chunk takes a warp about 1 us).  Measured with and without:
    // 64 sequences of 50-120 tokens, 32/8 heads, 6.4 and 8.8 us; 100 of 200-300 11.1 and 13.5; 210 of 497-774, 64/8
    // heads, 35.0 and 36.7; one of 1000, 8/8 heads, three chunks a warp against one, would be 7.1 against 5.9.
    const int share = per_cta + (rest > 0);
    auto rounds = [](int chunks) { return (chunks + WARPS - 1) / WARPS; };
    if (rounds(share + most) <= rounds(share) + kExtraRounds &&
        rounds(share <= most ? most : (share + most - 1) / most * most) < rounds(share) + kExtraRounds) {
      auto bound = [&](int cta) {
        const int chunk = cta * per_cta + min(cta, rest);
        if (chunk >= total) return total;
        const int s = sequence_of(chunk);
        const unsigned c = s_pre[s + 1] - s_pre[s], in = chunk - s_pre[s] * U;
        return chunk - static_cast<int>(in % c);
      };
      const int from = bound(blockIdx.x), chunks = bound(blockIdx.x + 1) - from;
      if (chunks <= WARPS) {
        start = from + warp;
        len = warp < chunks;
      } else {
        start = from + warp * chunks / WARPS;
        len = from + (warp + 1) * chunks / WARPS - start;
      }
    } else {
      // Equal shares.  With fewer chunks than the grid has warps, every CTA puts an equal number of its warps
      // to work, with one chunk each.
      const int active = active_warps<WARPS>(total);
      const int workers = min(total, grid * active);
      const int me = blockIdx.x * active + warp;
      if (warp < active && me < workers) {  // me * total / workers, the odd chunks spread over the grid
        const int each = total / workers, more = total - each * workers;  // (more < workers <= 16 * SMs)
        start = me * each + me * more / workers;
        len = (me + 1) * each + (me + 1) * more / workers - start;
      }
    }
    int id[NB], have = 0, head = 0;
    const int32_t* row = p.block_tables;
    if (len > 0) {
      s = sequence_of(start);
      const unsigned c = s_pre[s + 1] - s_pre[s], r = start - s_pre[s] * U;
      u = r / c;
      j = r - u * c;
      gs = s, gu = u, gj = j;
      find(len, row, have, head);
    }
    read_blocks(row, have, id);
    int now_len[PER], now_id[NB] = {};
    if (!waited) {  // what has to read the same
      griddep_wait();
#pragma unroll
      for (int k = 0; k < PER; ++k) now_len[k] = tid * PER + k < S ? ld_now(p.seq_lens + tid * PER + k) : 0;
      read_blocks(row, have, now_id);
    }
    // the first chunks and the query rows are asked for in the meantime (every tile lies in the pool)
    bad_id = to_tiles(id, have, head, cur);
    if (len > 0) fetch_q();
#pragma unroll 1
    for (int k = 0; k < STAGES; ++k) {  // a group of copies per chunk, empty past the end
      if (k < len) copy_chunk(k);
      copies_close();
    }
    if (waited) break;
    bool again = false;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      again |= now_len[k] != lens[k];
      lens[k] = now_len[k];
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) again |= now_id[b] != id[b];
    if (!__syncthreads_or(again)) break;
    copies_wait<0>();
    __syncwarp();
  }
  if (bad_id) set_error(p.err, kErrBlockId);

  if (bad && blockIdx.x == 0) {
    if (tid == 0) set_error(p.err, kErrSeqLen);
    for (int i = 0; i < S; ++i) {
      if (s_len[i] != 0) continue;
      uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (long long)i * p.num_heads * D);
      for (int x = tid; x < p.num_heads * D / 8; x += WARPS * 32) out[x] = make_uint4(0, 0, 0, 0);
    }
  }

  if (len > 0) {
    int group = 0;
    auto look_up_next = [&](int positions) {
      int id[NB], have, head;
      const int32_t* row;
      find(positions, row, have, head);
      read_blocks(row, have, id);
      if (to_tiles(id, have, head, nxt)) set_error(p.err, kErrBlockId);
    };
    if (len > 32) look_up_next(len - 32);
    auto issue = [&](int k) {
      if ((k >> 5) != group) {
#pragma unroll
        for (int b = 0; b < NB; ++b) cur[b] = nxt[b];
        if (32 * (++group + 1) < len) look_up_next(len - 32 * (group + 1));
      }
      copy_chunk(k);
    };
    math.reset();
    math.scale_q(p.scale_log2);
    int j0 = j;  // where the current piece starts
    for (int k = 0; k < len; ++k) {
      copies_wait<STAGES - 1>();
      __syncwarp();
      const unsigned char* stage = ring + (k % STAGES) * Sh::kStage;
      const int rem = L - j * kChunk;
      typename Math::Raw raw;
      float sc[2][NT][4];
      uint32_t pb[2][NT][2];
      math.fetch_k(stage, raw);
      math.scores(raw, sc);
      math.fetch_v(stage + NB * TILE, raw);
      __syncwarp();
      if (k + STAGES < len) issue(k + STAGES);  // the chunk is in registers: refill its stage
      copies_close();
      math.weigh(sc, pb, rem);
      math.add(raw, pb, rem);
      ++j;
      const bool ends = j == n, last = k + 1 == len;
      if (!ends && !last) continue;
      if (j0 == 0 && ends) {
        math.store_out(static_cast<T*>(p.out) + ((long long)s * p.num_heads + h0) * D, nh, p.out_scale);
      } else {
        // a piece that ends its segment but did not begin it can only be this warp's first (entry
        // 2 warp), the other kind only its last (entry 2 warp + 1)
        const int e = 2 * warp + (ends ? 0 : 1);
        math.store_piece(piece(e), s_ml + e * Sh::kRows, s_factor + e * Sh::kRows);
        if (lane == 0) s_seg[e] = make_int2(s, u | (j0 == 0 ? kBegins : 0));
      }
      if (last) break;
      if (ends && ++u == U) {
        u = 0;
        do {
          ++s;
        } while (s_pre[s + 1] == s_pre[s]);
      }
      j = j0 = 0;
      fetch_q();
      math.reset();
      math.scale_q(p.scale_log2);
    }
  }
  __syncthreads();

  // The CTA's pieces: a run of them is one segment's, one per warp, warps w0 .. w1.  A run starts
  // with a last piece that begins its segment, or with warp 0; it stops at the first warp after
  // that has a first piece (which ends the segment), or with the CTA's last working warp.
  const int2 first = lane < WARPS ? s_seg[2 * lane] : make_int2(-1, 0);
  const int2 final = lane < WARPS ? s_seg[2 * lane + 1] : make_int2(-1, 0);
  const uint32_t firsts = __ballot_sync(0xffffffffu, first.x >= 0), finals = __ballot_sync(0xffffffffu, final.x >= 0);
  const uint32_t begin = __ballot_sync(0xffffffffu, final.x >= 0 && (final.y & kBegins));
  // the last warp of a run whose piece of warp w does not end it, and whether the run ends its segment
  auto run_end = [&](int w, bool& ends) {
    const uint32_t stops = firsts & ~((2u << w) - 1u);
    ends = stops != 0;
    return ends ? __ffs(stops) - 1 : 31 - __clz(finals);
  };
  // Every (piece, head)'s factor in its run, and the run's (M', W) beside its first piece.  (hs is the same in
  // every piece of a head's segment.)
  for (int i = tid; i < 2 * WARPS * Sh::kRows; i += WARPS * 32) {
    const int e = i / Sh::kRows, r = i % Sh::kRows, w = e >> 1;
    if (!(((e & 1 ? finals : firsts) >> w) & 1u)) continue;
    const uint32_t before = begin & ((1u << (w + (e & 1))) - 1u);  // a first piece's run began in an earlier warp
    const int w0 = before ? 31 - __clz(before) : 0;
    bool ends = true;
    const int w1 = e & 1 ? run_end(w, ends) : w;
    auto ml = [&](int x) { return s_ml[(2 * x + (ends && x == w1 ? 0 : 1)) * Sh::kRows + r]; };
    const float hs = s_factor[i];
    float M = kNoScore, W = 0.f;
#pragma unroll 4
    for (int x = w0; x <= w1; ++x) M = fmaxf(M, ml(x).x);
    if (w == w0) {
#pragma unroll 4
      for (int x = w0; x <= w1; ++x) W = fmaf(ex2((ml(x).x - M) * hs), ml(x).y, W);
      s_run[(e & 1 ? w : WARPS) * Sh::kRows + r] = make_float2(M, W);  // (a first piece alone: warp 0's)
      if (!before) s_hs[r] = hs;
    }
    s_factor[i] = ex2((s_ml[i].x - M) * hs);
  }
  __syncthreads();
  // A warp takes a head of a run, a lane D/32 dims.
  constexpr int C = D / 32, kRingBytes = STAGES * Sh::kStage;
  using Vec = std::conditional_t<C == 4, float4, float2>;
  bool publish = false;                // this CTA's last run goes on in the next CTA
  int tail_s = -1, tail_u = 0;         // the segment of an earlier CTA that ends in this one
  int task = warp;
  // bit 0 of `heads` below: the run that warp 0 starts without beginning a segment; bit w + 1: one that warp w begins
  for (uint32_t heads = begin << 1 | (firsts & 1u) | (finals & ~begin & 1u); heads; heads &= heads - 1) {
    const int hd = __ffs(heads) - 1, w0 = hd ? hd - 1 : 0;
    const bool alone = hd == 0 && (firsts & 1u);  // warp 0's first piece ends a segment that an earlier CTA began
    const bool begins = hd != 0;
    bool ends = true;
    const int w1 = alone ? 0 : run_end(w0, ends);
    const int2 seg = s_seg[alone ? 0 : 2 * w0 + 1];
    const int s = seg.x, u = seg.y & ~kBegins;
    if (!ends) publish = true;
    else if (!begins) tail_s = s, tail_u = u;
    int kvh, h0, nh;
    unit_heads(p, u, kvh, h0, nh);
    for (; task < nh; task += WARPS) {
      const int r = task;
      // the same place in every piece: in the warps' rings, and at a run's end perhaps in a first piece
      const unsigned char* at = reinterpret_cast<const unsigned char*>(Math::piece_at(
                                    reinterpret_cast<const float4*>(smem), r, lane * C / 4)) + lane * C % 4 * 4;
      const int rings = w1 + (ends ? 0 : 1);
      float O[C] = {};
      auto add = [&](const unsigned char* from, float f) {
        const Vec v = *reinterpret_cast<const Vec*>(from);
        const float* vf = reinterpret_cast<const float*>(&v);
#pragma unroll
        for (int c = 0; c < C; ++c) O[c] = fmaf(f, vf[c], O[c]);
      };
#pragma unroll 4
      for (int w = w0; w < rings; ++w) add(at + w * kRingBytes, s_factor[(2 * w + 1) * Sh::kRows + r]);
      if (ends) add(at + Sh::kFirst + w1 * Sh::kPiece, s_factor[2 * w1 * Sh::kRows + r]);
      const float2 sum = s_run[(alone ? WARPS : w0) * Sh::kRows + r];
      if (begins && ends) {
        const float il = p.out_scale / sum.y;
        T* out = static_cast<T*>(p.out) + ((long long)s * p.num_heads + h0 + r) * D + lane * C;
#pragma unroll
        for (int c = 0; c < C; c += 2) *reinterpret_cast<uint32_t*>(out + c) = pack2<T>(O[c] * il, O[c + 1] * il);
      } else {
        const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
        Vec v;
        float* vf = reinterpret_cast<float*>(&v);
#pragma unroll
        for (int c = 0; c < C; ++c) vf[c] = O[c];
        *reinterpret_cast<Vec*>(p.part_o + (slot * 16 + r) * D + lane * C) = v;
        if (lane == 0) p.part_ml[slot * 16 + r] = sum;
      }
    }
    task -= nh;
  }
  if (!publish && tail_s < 0) return;  // (the same for all threads of the CTA)
  __syncthreads();
  // The barrier orders the CTA's pieces before this thread's release, which covers what it has observed so:
  // no fence of its own (with one: 2 to 7% on calls of 6 to 10 us).
  if (publish && tid == (WARPS - 1) * 32) {  // (not the warp that waits below)
    st_release(p.part_tag + blockIdx.x, p.tag);
  }
  if (tail_s < 0) return;

  // The segment's pieces: its first in CTA head (slot 2 head + 1), the others in slots 2 (head + i),
  // the last of them this CTA's own.
  const int total = s_pre[S] * U, active = active_warps<WARPS>(total);
  const int workers = min(total, static_cast<int>(gridDim.x) * active);
  const int share = total / workers, more = total - share * workers;
  const int at = s_pre[tail_s] * U + tail_u * (s_pre[tail_s + 1] - s_pre[tail_s]);  // its first chunk
  int head = blockIdx.x;
  for (;;) {  // the last CTA before this one whose first chunk is not past it
    const int w = max(head - 1 - lane, 0) * active;
    const uint32_t from = __ballot_sync(0xffffffffu, w * share + w * more / workers <= at);
    if (from) {
      head -= __ffs(from);
      break;
    }
    head -= 32;
  }
  const int pieces = static_cast<int>(blockIdx.x) - head + 1;
  if (warp == 0) {
    const uint64_t t0 = global_timer_ns(), limit = p.test_wait_ns ? p.test_wait_ns : kFp4WaitNs;
    const uint64_t want = p.test_wait_ns ? ~p.tag : p.tag;  // (the test's wait: for what nobody publishes)
    for (int c = head + lane; c < static_cast<int>(blockIdx.x); c += 32)
      for (unsigned tries = 1; ld_acquire(p.part_tag + c) != want; ++tries)
        if (tries % 16 == 0 && global_timer_ns() - t0 > limit) {
          set_error(p.err, kErrTimeout);
          break;
        }
  }
  __syncthreads();
  unit_heads(p, tail_u, kvh, h0, nh);
  auto slot = [&](int i) { return i == 0 ? 2 * head + 1 : 2 * (head + i); };
  for (int r = warp; r < nh; r += WARPS) {  // a warp per query head, 32 pieces at a time
    const float hs = s_hs[r];
    float M = kNoScore, W = 0.f, O[C] = {};
    for (int i0 = 0; i0 < pieces; i0 += 32) {
      const int cnt = min(32, pieces - i0);
      float2 ml = make_float2(kNoScore, 0.f);
      if (lane < cnt) ml = __ldcg(p.part_ml + slot(i0 + lane) * 16 + r);
      Vec o[kMergeBatch];
      auto load = [&](int i1) {
#pragma unroll
        for (int i = 0; i < kMergeBatch; ++i)
          if (i1 + i < cnt)
            o[i] = __ldcg(reinterpret_cast<const Vec*>(p.part_o + (slot(i0 + i1 + i) * 16 + r) * D + lane * C));
      };
      load(0);
      float top = fmaxf(ml.x, M);
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float keep = ex2((M - top) * hs), f = ex2((ml.x - top) * hs);
      float w = f * ml.y;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) w += __shfl_xor_sync(0xffffffffu, w, x);
      M = top;
      W = W * keep + w;
#pragma unroll
      for (int c = 0; c < C; ++c) O[c] *= keep;
      for (int i1 = 0; i1 < cnt; i1 += kMergeBatch) {
        if (i1 > 0) load(i1);
#pragma unroll
        for (int i = 0; i < kMergeBatch; ++i) {
          const float fi = __shfl_sync(0xffffffffu, f, (i1 + i) & 31);
          if (i1 + i < cnt) {
            const float* v = reinterpret_cast<const float*>(&o[i]);
#pragma unroll
            for (int c = 0; c < C; ++c) O[c] = fmaf(fi, v[c], O[c]);
          }
        }
      }
    }
    const float il = p.out_scale / W;
    T* out = static_cast<T*>(p.out) + ((long long)tail_s * p.num_heads + h0 + r) * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; c += 2) *reinterpret_cast<uint32_t*>(out + c) = pack2<T>(O[c] * il, O[c + 1] * il);
  }
  for (int c = head + tid; c < static_cast<int>(blockIdx.x); c += WARPS * 32) p.part_tag[c] = 0;
}

template <typename T, int D, int BS, int NT>
cudaError_t launch_t(const Fp4DecodeParams& p, int grid, cudaStream_t stream, int* launches) {
  using Sh = Fp4Shape<D, NT>;
  static unsigned done = 0;  // bit d: the attribute is set on device d
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !((__atomic_load_n(&done, __ATOMIC_ACQUIRE) >> dev) & 1u)) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&decode_fp4_kernel<T, D, BS, NT>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 32) __atomic_fetch_or(&done, 1u << dev, __ATOMIC_RELEASE);
  }
  e = launch_pdl(decode_fp4_kernel<T, D, BS, NT>, dim3(grid), dim3(Sh::kWarps * 32), Sh::kBytes, stream, p);
  if (e != cudaSuccess) return e;
  *launches = 1;
  return cudaSuccess;
}

template <typename T, int D, int BS>
cudaError_t launch_nt(const Fp4DecodeParams& p, int grid, cudaStream_t stream, int* launches) {
  return p.group <= 8 ? launch_t<T, D, BS, 1>(p, grid, stream, launches)
                      : launch_t<T, D, BS, 2>(p, grid, stream, launches);
}

template <typename T>
cudaError_t launch_shape(int head_size, int block_size, const Fp4DecodeParams& p, int grid, cudaStream_t stream,
                         int* launches) {
  if (head_size == 64)
    return block_size == 16 ? launch_nt<T, 64, 16>(p, grid, stream, launches)
                            : launch_nt<T, 64, 32>(p, grid, stream, launches);
  return block_size == 16 ? launch_nt<T, 128, 16>(p, grid, stream, launches)
                          : launch_nt<T, 128, 32>(p, grid, stream, launches);
}

}  // namespace

// CTAs of a launch, from the most chunks it can have.  A CTA gets about four chunks, one for
// each of its SM's schedulers -- whole segments where they are short, since a segment cut at
// CTAs' ends costs a wait for the other CTA -- and where that cuts segments into more than 32
// pieces, rather as many chunks as it has warps.
int fp4_decode_grid(int sms, int num_seqs, int num_heads, int num_kv_heads, int head_size, int max_seq_len) {
  const long long each = pieces_of(max_seq_len, kChunk);
  const long long segs = (long long)num_seqs * fp4_decode_units(num_heads, num_kv_heads), chunks = segs * each;
  const bool one = num_heads / num_kv_heads <= 8;
  const int warps = head_size == 64 ? (one ? Fp4Shape<64, 1>::kWarps : Fp4Shape<64, 2>::kWarps)
                                    : (one ? Fp4Shape<128, 1>::kWarps : Fp4Shape<128, 2>::kWarps);
  const long long per_cta = each <= 8 ? (each + 3) / each * each : 4;
  long long want = (chunks + per_cta - 1) / per_cta;
  const long long few = (chunks + warps - 1) / warps;
  if (want > 32 * segs) want = few > 32 * segs ? few : 32 * segs;
  return static_cast<int>(want < sms ? (want > 0 ? want : 1) : sms);
}

cudaError_t launch_decode_fp4(bool q_is_bf16, int head_size, int block_size, const Fp4DecodeParams& p, int grid,
                              cudaStream_t stream, int* launches) {
  *launches = 0;
  return q_is_bf16 ? launch_shape<__nv_bfloat16>(head_size, block_size, p, grid, stream, launches)
                   : launch_shape<__half>(head_size, block_size, p, grid, stream, launches);
}

}  // namespace pa
