// rope.cu -- rotary positions on rows of q and k, alone and with the write into the paged pool.
//
// What is computed.  A token at position p turns pair i of each head's first rotary_dim
// dims by the angle p f_i and scales it by A:
//     x' = A (x cos(p f_i) - y sin(p f_i)),   y' = A (x sin(p f_i) + y cos(p f_i))
// with the pair (x, y) at dims (i, i + rotary_dim / 2) or (2 i, 2 i + 1); the dims past
// rotary_dim are copied.  fp32 arithmetic, one rounding at the end (an FP8 code straight
// from the fp32 value).
//
// The angle.  Positions are whole numbers, so the angle is taken in turns and fixed
// point: with F_i = f_i / 2 pi as a 64-bit fraction of a turn, p F_i mod 2^64 is the
// product's low word -- the reduction to one turn costs nothing and is exact for every
// position, and the error is that of F_i alone, which is rounded once: |p| 2^-65 turns, whatever f_i.
// What is left after the nearest quarter turn lies within 1/8 turn, so as fp32 it is off by at most
// 2^-28 turns, and sincospif finishes it.  (fp64 per token and pair would be bound by this GPU's fp64
// rate; f_i / 2 pi is computed in fp64 once per CTA.)
//
// Work.  A unit is two 16-byte pieces of a row: the two halves' pieces of the same pairs,
// or two neighbouring ones.  A CTA takes a tile of up to 16 tokens and some of their rows (q heads, then k heads,
// then v heads), puts the cosines and sines of its tokens into shared memory, and a thread keeps one unit and one
// token for all rows of a kind, with that unit's cosines and sines in registers.  It reads both pieces of a unit before it writes
// either, so q may be rotated in place.  For q a warp reads and writes whole rows; for k and v it runs over
// 16 tokens with the pieces of a pair of units innermost: rows are read in whole 32-byte sectors, and
// consecutive slots of a block are written in whole sectors too, for K (16 bytes a token) and V (one element a
// token) alike.
//
// What bounds it: memory.  16384 tokens of 32 + 8 heads of 128 dims in bf16, 64 of them turned (336 MB): 53.8 us,
// 6.2 TB/s, 93% of a copy's rate.  8192 tokens of 28 + 4 + 4 heads in fp16 into the pools (151 MB): 28 us, 5.4 TB/s;
// what lies between is V, two bytes to each place.  fp32 rows: 16381 tokens of 32 + 8 heads (671 MB) 125.5 us, 5.3 TB/s;
// 8192 of 28 + 4 + 4 into the pools (302 MB) 50 us, 6.0 TB/s.  FP8 pools: 1537 tokens of 32 + 8 + 8 heads (35 MB) 8.6 us
// from L2, 11.1 from memory: V is 16 stores of a byte a unit.  One token: 2.2 us in a graph, latency: the launch, the
// frequencies, a row.
#include <stdint.h>

#include <numeric>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTile = 16;  // tokens per CTA at most
constexpr int kRopeBatch = 2;  // units per thread in flight
constexpr int kRopeValueRows = 4;               // rows of q that a row of v counts as (see launch_rope)
constexpr int kRopeBusy = 7, kRopeMost = 9;     // units a thread

// f / 2 pi as a 64-bit fraction of a turn (whole turns drop out), to nearest.  The quotient is kept as an
// unevaluated sum hi + lo: 1 / 2 pi to twice the precision of a double.
__device__ __forceinline__ uint64_t turns_of(double f) {
  constexpr double kInv2Pi = 0x1.45f306dc9c883p-3;     // 1 / 2 pi, the nearest double
  constexpr double kInv2PiLo = -0x1.6b01ec5417056p-57;  // 1 / 2 pi - kInv2Pi
  const double hi = f * kInv2Pi;
  const double lo = fma(f, kInv2Pi, -hi) + f * kInv2PiLo;
  const double frac = hi - floor(hi);  // [0, 1]; 1 only by rounding, and then it wraps to 0
  const double scaled = frac >= 1.0 ? 0.0 : frac * 0x1p64, whole = floor(scaled);
  // (what hi has below 2^-64, as small frequencies do, is rounded together with lo)
  return __double2ull_rz(whole) + static_cast<uint64_t>(__double2ll_rn(lo * 0x1p64 + (scaled - whole)));
}

// cos and sin of `turns` 2^-64 of a turn
__device__ __forceinline__ float2 cos_sin(uint64_t turns) {
  const uint64_t up = turns + (1ull << 61);  // the nearest quarter turn is the two highest bits
  const int quarter = static_cast<int>(up >> 62);
  const int64_t rest = static_cast<int64_t>((up & ((1ull << 62) - 1))) - (1ll << 61);  // within 1/8 turn
  float s, c;
  sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
  const float c1 = (quarter & 1) ? s : c, s1 = (quarter & 1) ? c : s;  // a quarter turn: (-s, c)
  return make_float2((quarter == 1 || quarter == 2) ? -c1 : c1, (quarter == 2 || quarter == 3) ? -s1 : s1);
}

// X consecutive elements of T (16 bytes) to and from fp32.
template <typename T, int X>
__device__ __forceinline__ void widen(const uint4& raw, float (&v)[X]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(raw.x);
    v[1] = __uint_as_float(raw.y);
    v[2] = __uint_as_float(raw.z);
    v[3] = __uint_as_float(raw.w);
  } else {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
template <typename T, int X>
__device__ __forceinline__ uint4 narrow(const float (&v)[X]) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

// x / scale, correctly rounded where an E4M3 code can tell: the product with the rounded
// reciprocal, corrected once by its remainder (P. Markstein's division by a rounded reciprocal; exact for the
// quotients in [2^-12, 1024) and scales in [2^-64, 2^64]).  Other quotients keep the product: smaller ones
// become zero (of their sign) in any case, larger ones, infinities and NaN saturate as they do.  inv == 0: a scale
// outside that range, divided.
__device__ __forceinline__ float quotient(float x, float scale, float inv) {
  if (inv == 0.f) return __fdiv_rn(x, scale);
  const float q = x * inv;
  const float c = fmaf(fmaf(-q, scale, x), inv, q);
  constexpr uint32_t kLo = 0x39800000u, kHi = 0x44800000u;  // the bits of 2^-12 and 1024
  return (__float_as_uint(q) & 0x7fffffffu) - kLo < kHi - kLo ? c : q;
}

// X elements as E4M3 codes of x / scale, to nearest even and at most 448 in size, as the write
// path stores them (the first X bytes).
template <int X>
__device__ __forceinline__ uint2 e4m3_codes8(const float (&v)[X], float scale, float inv) {
  static_assert(X == 8 || X == 4, "a 16-byte piece");
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < X; i += 2) {
    const float2 q = make_float2(quotient(v[i], scale, inv), quotient(v[i + 1], scale, inv));
    w[i / 4] |= (__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) & 0xffffu) << (16 * ((i / 2) & 1));
  }
  return make_uint2(w[0], w[1]);
}

// T: the rows' type.  TC: the pool's type; void: the turned keys go to rows (key_out) instead,
// and there are no values.
template <typename T, typename TC, int D, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  constexpr bool kPool = !std::is_void<TC>::value;
  constexpr int E = sizeof(T), X = 16 / E, U = D / (2 * X);  // units per row
  __shared__ uint64_t s_turn[D / 2];
  // (a row's length is 4 past a multiple of 32 floats, so that the threads of four tokens read other banks)
  __shared__ __align__(16) float s_cos[kRopeTile][D / 2 + 4], s_sin[kRopeTile][D / 2 + 4];
  __shared__ long long s_pos[kRopeTile], s_blk[kRopeTile];
  __shared__ int s_off[kRopeTile];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, tile = 1 << p.log2_tile, H = p.num_heads, Hkv = p.num_kv_heads;
  const long long t0 = (long long)blockIdx.x << p.log2_tile;
  const int ntok = static_cast<int>(min((long long)tile, p.num_tokens - t0));
  const int r2 = p.rotary_dim / 2;
  // a token's rows: q heads, k heads, v heads; of each kind this CTA's
  const int row0 = blockIdx.y * p.rows_per, row1 = row0 + p.rows_per;
  const int v0 = (max(row0 - H - Hkv, 0) + p.value_rows - 1) / p.value_rows;
  const int v1 = kPool ? min(Hkv, (max(row1 - H - Hkv, 0) + p.value_rows - 1) / p.value_rows) : 0;

  if (tid < r2) s_turn[tid] = turns_of(__ldg(p.inv_freq + tid));
  if (tid >= kRopeThreads - kRopeTile) {
    const int j = tid - (kRopeThreads - kRopeTile);
    if (j < ntok) {
      s_pos[j] = __ldg(p.positions + t0 + j);
      if constexpr (kPool) {
        const long long slot = __ldg(p.slot_mapping + t0 + j);
        long long blk = -1;
        int off = 0;
        if (slot >= p.num_blocks * p.block_size) {
          if (blockIdx.y == 0) set_error(p.err, kErrSlot);
        } else if (slot >= 0) {  // (negative: a padding token)
          blk = slot / p.block_size;
          off = static_cast<int>(slot - blk * p.block_size);
        }
        s_blk[j] = blk;
        s_off[j] = off;
      }
    }
  }
  __syncthreads();
  if (row0 < H + Hkv)  // (rows of v are not turned)
    for (int i = tid; i < ntok * r2; i += kRopeThreads) {
      const int j = i / r2, c = i - j * r2;
      const float2 cs = cos_sin(static_cast<uint64_t>(s_pos[j]) * s_turn[c]);
      s_cos[j][c] = cs.x * p.amplitude;
      s_sin[j][c] = cs.y * p.amplitude;
    }
  __syncthreads();

  // A thread keeps its unit u and its token j for all rows of a kind, so that the cosines and sines of
  // both stay in registers; `per` rows are under way in the CTA at once.
  constexpr int kLog2U = U == 4 ? 2 : U == 8 ? 3 : 4;
  static_assert(1 << kLog2U == U, "units per row");
  const int spot = tid & ((tile << kLog2U) - 1), per = kRopeThreads >> (p.log2_tile + kLog2U);
  const int mine = tid >> (p.log2_tile + kLog2U);
  struct Spot {
    int u, j, d0, d1;  // the unit, the token, and the first dims of the unit's pieces
    bool turned;
    float c[X], s[X];
  };
  auto settle = [&](int u, int j, bool turn) {
    Spot w;
    w.u = u;
    w.j = j;
    w.turned = turn && u < p.rotary_dim / (2 * X);
    w.d0 = !kPairs && w.turned ? u * X : 2 * u * X;
    w.d1 = !kPairs && w.turned ? w.d0 + r2 : w.d0 + X;
    if (w.turned) {  // pair indices u X .. u X + X - 1 in both layouts
#pragma unroll
      for (int e = 0; e < X; e += 4) {
        const float4 c = *reinterpret_cast<const float4*>(&s_cos[j][u * X + e]);
        const float4 v = *reinterpret_cast<const float4*>(&s_sin[j][u * X + e]);
        w.c[e] = c.x, w.c[e + 1] = c.y, w.c[e + 2] = c.z, w.c[e + 3] = c.w;
        w.s[e] = v.x, w.s[e + 1] = v.y, w.s[e + 2] = v.z, w.s[e + 3] = v.w;
      }
    }
    return w;
  };
  auto turn = [&](const Spot& w, uint4& ra, uint4& rb, float(&a)[X], float(&b)[X]) {
    widen<T>(ra, a);
    widen<T>(rb, b);
    if (!w.turned) return;
#pragma unroll
    for (int e = 0; e < X; ++e) {
      float& x = kPairs ? (e < X / 2 ? a[2 * e % X] : b[2 * e % X]) : a[e];
      float& y = kPairs ? (e < X / 2 ? a[(2 * e + 1) % X] : b[(2 * e + 1) % X]) : b[e];
      const float x0 = x, y0 = y;
      x = fmaf(x0, w.c[e], -(y0 * w.s[e]));
      y = fmaf(x0, w.s[e], y0 * w.c[e]);
    }
    ra = narrow<T>(a);
    rb = narrow<T>(b);
  };
  // rows first .. last - 1 of a kind, from src (the token's row 0 of the kind) to put(row, pieces): kRopeBatch
  // rows' loads are on their way together
  auto walk = [&](const Spot& w, const T* src, int first, int last, auto put) {
    for (int row = first + mine; row < last; row += kRopeBatch * per) {
      uint4 ra[kRopeBatch], rb[kRopeBatch];
#pragma unroll
      for (int b = 0; b < kRopeBatch; ++b)
        if (row + b * per < last) {
          ra[b] = *reinterpret_cast<const uint4*>(src + (row + b * per) * D + w.d0);
          rb[b] = *reinterpret_cast<const uint4*>(src + (row + b * per) * D + w.d1);
        }
#pragma unroll
      for (int b = 0; b < kRopeBatch; ++b)
        if (row + b * per < last) {
          float x[X], y[X];
          turn(w, ra[b], rb[b], x, y);
          put(row + b * per, ra[b], rb[b], x, y);
        }
    }
  };

  // q (and k as rows): a row's units side by side
  auto to_rows = [&](const void* src, long long stride, void* dst, int heads, int first, int last) {
    const Spot w = settle(spot & (U - 1), spot >> kLog2U, true);
    if (w.j >= ntok) return;
    const long long t = t0 + w.j;
    T* out = static_cast<T*>(dst) + t * heads * D;
    walk(w, static_cast<const T*>(src) + t * stride, first, last,
         [&](int row, const uint4& ra, const uint4& rb, const float(&)[X], const float(&)[X]) {
           *reinterpret_cast<uint4*>(out + row * D + w.d0) = ra;
           *reinterpret_cast<uint4*>(out + row * D + w.d1) = rb;
         });
  };
  if (row0 < H) to_rows(p.q, p.q_stride, p.q_out, H, row0, min(row1, H));
  if constexpr (!kPool) {
    if (row1 > H) to_rows(p.key, p.key_stride, p.key_out, Hkv, max(row0, H) - H, min(row1 - H, Hkv));
  } else {
    constexpr int EC = sizeof(TC), XC = 16 / EC;
    const int bs = p.block_size;
    // k and v: two units, the tokens, the other units
    const int pr = spot >> (p.log2_tile + 1), k = spot & ((2 << p.log2_tile) - 1);
    if (row1 > H && row0 < H + Hkv) {
      const Spot w = settle(2 * pr + (k & 1), k >> 1, true);
      const long long t = t0 + w.j, blk = w.j < ntok ? s_blk[w.j] : -1;
      if (blk >= 0) {  // (a padding token's key goes nowhere)
        const int off = s_off[w.j];
        unsigned char* kc = static_cast<unsigned char*>(p.k_cache);
        walk(w, static_cast<const T*>(p.key) + t * p.key_stride, max(row0, H) - H, min(row1, H + Hkv) - H,
             [&](int h, const uint4& ra, const uint4& rb, const float(&x)[X], const float(&y)[X]) {
               // 16-byte group g of the row -> k_cache[blk, h, g, off, :]
               const long long base = (blk * Hkv + h) * (D / XC);
               if constexpr (EC == 1) {
                 auto put = [&](int d, const float(&v)[X]) {
                   unsigned char* at = kc + ((base + d / XC) * bs + off) * 16 + d % XC;
                   const uint2 codes = e4m3_codes8(v, p.k_scale, p.k_inv);
                   if constexpr (X == 8) *reinterpret_cast<uint2*>(at) = codes;
                   else *reinterpret_cast<uint32_t*>(at) = codes.x;
                 };
                 put(w.d0, x);
                 put(w.d1, y);
               } else {
                 *reinterpret_cast<uint4*>(kc + ((base + w.d0 / XC) * bs + off) * 16) = ra;
                 *reinterpret_cast<uint4*>(kc + ((base + w.d1 / XC) * bs + off) * 16) = rb;
               }
             });
      }
    }
    if (v1 > v0) {
      const Spot w = settle(2 * pr + (k & 1), k >> 1, false);
      const long long t = t0 + w.j, blk = w.j < ntok ? s_blk[w.j] : -1;
      if (blk >= 0) {
        const int off = s_off[w.j];
        walk(w, static_cast<const T*>(p.value) + t * p.value_stride, v0, v1,
             [&](int h, const uint4& ra, const uint4& rb, const float(&x)[X], const float(&y)[X]) {
               // element d -> v_cache[blk, h, d, off]
               const long long base = (blk * Hkv + h) * D;
               if constexpr (EC == 1) {
                 unsigned char* vc = static_cast<unsigned char*>(p.v_cache);
                 auto put = [&](int d, const float(&v)[X]) {
                   const uint2 codes = e4m3_codes8(v, p.v_scale, p.v_inv);
#pragma unroll
                   for (int e = 0; e < X; ++e)
                     vc[(base + d + e) * bs + off] =
                         static_cast<unsigned char>((e < 4 ? codes.x : codes.y) >> (8 * (e & 3)));
                 };
                 put(w.d0, x);
                 put(w.d1, y);
               } else {
                 using W = std::conditional_t<E == 4, uint32_t, uint16_t>;
                 W* vc = static_cast<W*>(p.v_cache);
                 const W *ea = reinterpret_cast<const W*>(&ra), *eb = reinterpret_cast<const W*>(&rb);
#pragma unroll
                 for (int e = 0; e < X; ++e) {
                   vc[(base + w.d0 + e) * bs + off] = ea[e];
                   vc[(base + w.d1 + e) * bs + off] = eb[e];
                 }
               }
             });
      }
    }
  }
}

template <typename T, typename TC, int D>
cudaError_t launch_rope_d(const RopeParams& p, bool pairs, dim3 grid, cudaStream_t stream) {
  return pairs ? launch_pdl(rope_kernel<T, TC, D, true>, grid, dim3(kRopeThreads), 0, stream, p)
               : launch_pdl(rope_kernel<T, TC, D, false>, grid, dim3(kRopeThreads), 0, stream, p);
}
template <typename T, typename TC>
cudaError_t launch_rope_t(const RopeParams& p, int head_size, bool pairs, dim3 grid, cudaStream_t stream) {
  return head_size == 64 ? launch_rope_d<T, TC, 64>(p, pairs, grid, stream)
                         : launch_rope_d<T, TC, 128>(p, pairs, grid, stream);
}
template <typename T>
cudaError_t launch_rope_rows(const RopeParams& p, int head_size, bool pairs, int cache_dtype, dim3 grid,
                             cudaStream_t stream) {
  if (cache_dtype < 0) return launch_rope_t<T, void>(p, head_size, pairs, grid, stream);
  if (cache_dtype == 3) return launch_rope_t<T, __nv_fp8_e4m3>(p, head_size, pairs, grid, stream);
  return launch_rope_t<T, T>(p, head_size, pairs, grid, stream);
}

}  // namespace

cudaError_t launch_rope(int dtype, int cache_dtype, int head_size, bool pairs, RopeParams p, int sms,
                        cudaStream_t stream, int* launches) {
  *launches = 0;
  if (p.num_tokens == 0) return cudaSuccess;
  p.value_rows = kRopeValueRows;
  const int rows = p.num_heads + (cache_dtype >= 0 ? 1 + p.value_rows : 1) * p.num_kv_heads;
  const int units = head_size * (dtype == 0 ? 4 : 2) / 32;  // per row
  auto inverse = [](float scale) { return scale >= 0x1p-64f && scale <= 0x1p64f ? 1.f / scale : 0.f; };
  p.k_inv = inverse(p.k_scale);
  p.v_inv = inverse(p.v_scale);
  // The split.  A CTA takes tile x per rows; what it costs beside them (the turns of its frequencies, its tokens'
  // cosines) takes 1.5 us, so the launch is two CTAs an SM, or four (one wave still) where two would have more than
  // kRopeBusy units a thread each.  In a CTA about as many tokens as rows: fewer tokens compute the same cosines in
  // more CTAs, more leave the tile's rows to few.  A row of v, whose elements go to places of their own, costs as
  // much as several of q: counted as one, the CTAs with v ran alone at the end of a decode step (64/8 heads of 128
  // dims fp16, 128 tokens: 10.3 us for 4.9; 32/8 heads into FP8 pools 7.0 for 4.8); counted as 8, long prompts slow
  // down (16/16 heads bf16, 20000 tokens: 95 us for 85).  At least a unit a thread and 4 CTAs an SM whatever the work:
  // 28/4 heads fp16, 1 token 3.3 us for 2.5, 256 tokens 6.2 for 5.0, 1024 7.2 for 5.7, 4096 17.6 for 15.8 (in a
  // graph, inputs in L2; 16/16 heads bf16 8.6 for 4.5 at 400 tokens, but 7.7 for 10.3 at 1024).
  const long long all = p.num_tokens * rows * units;
  const long long target = (all > 2ll * sms * kRopeBusy * kRopeThreads ? 4ll : 2ll) * sms;
  const long long share = (p.num_tokens * rows + target - 1) / target;  // rows of tokens a CTA
  int tile = 1;
  while (tile < kRopeTile && tile < p.num_tokens && 16ll * tile * tile <= 9 * share) tile *= 2;
  p.log2_tile = 0;
  while (1 << p.log2_tile < tile) ++p.log2_tile;
  const long long tiles = (p.num_tokens + tile - 1) / tile;
  const long long most = target / tiles > 1 ? target / tiles : 1;  // CTAs a tile
  int per = static_cast<int>(most >= rows ? 1 : (rows + most - 1) / most);
  // (CTAs of many more units with v among them leave SMs idle at the end: 64/8 heads, 8192 tokens 57.6 us for 61.4;
  // without v the cosines are better computed once: 32 + 8 heads, 16381 tokens 53.8 us for 56.5)
  if (cache_dtype >= 0 && per * tile * units > kRopeMost * kRopeThreads)
    per = kRopeMost * kRopeThreads / (tile * units);
  // Small launches: rows of one kind where the heads allow it, since a CTA walks over its q, k and v rows one after
  // the other (a token of 16/16 heads 2.4 us for 4.8 with all three); large ones keep even shares.
  const int common = std::gcd(p.num_heads, p.num_kv_heads);
  if (target == 2ll * sms && per <= common)
    while (common % per) ++per;
  const int parts = (rows + per - 1) / per;
  p.rows_per = (rows + parts - 1) / parts;  // (equal shares)
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(parts));
  const cudaError_t e = dtype == 0   ? launch_rope_rows<float>(p, head_size, pairs, cache_dtype, grid, stream)
                        : dtype == 1 ? launch_rope_rows<__half>(p, head_size, pairs, cache_dtype, grid, stream)
                                     : launch_rope_rows<__nv_bfloat16>(p, head_size, pairs, cache_dtype, grid, stream);
  if (e == cudaSuccess) *launches = 1;
  return e;
}

}  // namespace pa
