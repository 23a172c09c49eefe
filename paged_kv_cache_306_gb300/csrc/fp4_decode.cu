// fp4_decode.cu -- decode attention over FP4 pools (see fp4.cuh).
//
// What is computed: for a sequence s and the query heads that share a kv head,
//     out = s_v sum_t p_t (code sf)_t / sum_t p_t,  p_t = 2^(hs q . (code sf)_t - m),
// with hs = scale s_k log2 e and a running maximum m (one pass over the tokens).
// Pieces of a sequence done apart are merged with M = max m_i, weights 2^(m_i - M).
//
// How it maps to the GPU.
//   * Work: a segment is (sequence, head unit), cut into chunks of 32 tokens.  All
//     chunks of the launch are laid end to end; the grid is at most one CTA per SM and
//     every warp of it takes one equal run of chunks, crossing segments.
//   * Copies: each warp has its own ring of stages; a chunk is one or two blocks of K and
//     of V, each a contiguous tile, brought in by bulk copies that signal an mbarrier.
//   * Math: m16n8k16 tensor-core tiles with fp16 operands: S^T = K Q^T, O^T += V^T P^T,
//     tokens and dims on the 16-row side, query heads on the 8-column side.  A code is
//     widened by one conversion per two codes and one multiplication by its group's scale
//     per two codes, both exact (code * sf has 6 significant bits).  The tile's byte order
//     gives each lane whole 32-bit words of codes: K as it lies; V with the nibbles of two
//     tokens interleaved by four bit operations per two words, because an operand register
//     holds two tokens of one dim.
//   * Merging: a warp that did a whole segment writes its output.  Pieces cut at a warp's
//     ends go to shared memory and the CTA merges them once at its end; only pieces cut
//     at a CTA's ends (at most two a CTA) go through the workspace to a second kernel.
//     Every slot the second kernel reads was written by this launch, so a call replayed
//     from a graph never meets an older launch's pieces.
#include <math.h>

#include <type_traits>

#include "fp4.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kChunk = 32;                       // tokens of a stage
constexpr uint64_t kFp4WaitNs = 1000000000ull;   // 1 s, then PA_DEVERR_TIMEOUT
constexpr float kNoScore = -1e30f;               // below every score (|score| < 2^33)

// NT: 8-column tiles of query heads (a unit has up to 8 NT heads).
template <int D, int NT>
struct Fp4Shape {
  static constexpr int kWarps = NT == 1 ? 16 : 8;
  static constexpr int kRows = 8 * NT;
  static constexpr int kStage = 2 * kChunk * (D / 2 + D / 16);
  static constexpr int kStages = 147456 / (kWarps * kStage);  // 144 KiB of copies in flight
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kPiece = kRows * D * 4;                // an unnormalised partial output
  static constexpr int kFirst = kRing;                        // [warps]: the piece a warp starts with
  static constexpr int kMl = kFirst + kWarps * kPiece;        // [2 warps][rows]: (m, l)
  static constexpr int kBars = kMl + 2 * kWarps * kRows * 8;  // [warps][stages], and one nothing completes
  static constexpr int kSeg = kBars + (kWarps * kStages + 2) * 8;  // [2 warps] int2: (segment, flags)
  static constexpr int kLen = kSeg + 2 * kWarps * 8;          // [seqs]
  static constexpr int kPre = kLen + kMaxSeqsPerLaunch * 4;   // [seqs + 1], then the scan's warp sums
  static constexpr int kBytes = kPre + (kMaxSeqsPerLaunch + 1 + kWarps + 3) * 4;
  static_assert(kStages >= 2 && kPiece <= kStages * kStage, "a warp's last piece takes its ring's place");
  static_assert(kRing % 128 == 0 && kPiece % 16 == 0 && kMl % 16 == 0 && kBars % 8 == 0 && kSeg % 8 == 0, "alignment");
  static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
};

constexpr int kBegins = 1, kEnds = 2;  // a piece holds its segment's first / last chunk

__device__ __forceinline__ float ex2(float x) {  // |relative error| < 2^-22, 0 below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t sel) { return __byte_perm(a, 0, sel); }

// One warp's running softmax of a unit's query heads.
template <typename T, int D, int BS, int NT>
struct Fp4Math {
  static constexpr int KS = D / 16;  // k-steps of S^T, and 16-row tiles of O^T
  static constexpr int KW = D / 32;  // words of codes a lane holds of a K row
  static constexpr int VW = D / 64;  // and of a V row
  static constexpr int TILE = fp4::tile_bytes(D, BS);
  static constexpr int kSub = BS == 16 ? TILE : 16 * (D / 2);        // codes of the chunk's second 16 tokens
  static constexpr int kSubScale = BS == 16 ? TILE : 16 * (D / 16);  // and their scales

  uint32_t qb[KS][NT][2];
  float acc[KS][NT][4];
  float m_[NT][2], l_[NT][2], hs_[NT][2];
  int g, t4;

  __device__ __forceinline__ void init(int lane) {
    g = lane >> 2;
    t4 = lane & 3;
  }

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[k][n][0] = acc[k][n][1] = acc[k][n][2] = acc[k][n][3] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m_[n][c] = kNoScore;
        l_[n][c] = 0.f;
      }
  }

  // Q^T fragments: lane (g, t4) holds dims D/4 t4 .. of head 8n + g, four per k-step, as
  // the K words hold them.  scale_log2 may be negative: its sign goes into q, so that the
  // largest score is the largest exponent.  bf16 heads become fp16 with a power of two
  // taken from the head's largest |q| (every element keeps its 8 bits), put back by hs_.
  __device__ __forceinline__ void load_q(const T* q, int nh, float scale_log2) {
    const uint32_t flip = scale_log2 < 0.f ? 0x80008000u : 0u;
    const float mag = fabsf(scale_log2);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = 8 * n + g;
#pragma unroll
      for (int k = 0; k < KS / 2; ++k) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (h < nh) w = *reinterpret_cast<const uint4*>(q + h * D + t4 * (D / 4) + 8 * k);
        qb[2 * k][n][0] = w.x ^ flip;
        qb[2 * k][n][1] = w.y ^ flip;
        qb[2 * k + 1][n][0] = w.z ^ flip;
        qb[2 * k + 1][n][1] = w.w ^ flip;
      }
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
        const float down = mag * __uint_as_float((127 - e) << 23);
        hs_[n][0] = __shfl_sync(0xffffffffu, down, 8 * t4);  // heads 2 t4 and 2 t4 + 1
        hs_[n][1] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
      }
    }
  }

  // One chunk: `rem` valid tokens (more than 31: all).  kc, vc: the stage's K and V tiles.
  __device__ __forceinline__ void chunk(const unsigned char* kc, const unsigned char* vc, int rem) {
    float sc[2][NT][4];
    // rows g and g + 8 of S^T are tokens tok and tok + 2 of a sub-tile
    const int tok = 4 * (g >> 1) + (g & 1);
    const int krow = ((g >> 1) ^ ((g & 1) ? 3 : 0)) + 4 * (g & 1);  // fp4::code_at's row of tok; tok + 2: 8 rows on
    const int kat = krow * (D / 2) + ((t4 * (D / 8)) ^ (D == 128 ? ((krow >> 1) & 1) << 5 : 0));
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t lo[KW], hi[KW], f[4];  // codes of the two rows; their groups' scales (pairs equal)
      const unsigned char* base = kc + mt * kSub + kat;
      const unsigned char* sbase = kc + BS * (D / 2) + mt * kSubScale;
      if constexpr (D == 128) {
        const uint4 a = *reinterpret_cast<const uint4*>(base), b = *reinterpret_cast<const uint4*>(base + 4 * D);
        lo[0] = a.x, lo[1] = a.y, lo[2] = a.z, lo[3] = a.w;
        hi[0] = b.x, hi[1] = b.y, hi[2] = b.z, hi[3] = b.w;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(sbase + g * 16 + t4 * 4);
        const uint32_t s0 = fp4::e4m3x2_to_f16x2(w), s1 = fp4::e4m3x2_to_f16x2(w >> 16);
        f[0] = prmt(s0, 0x1010), f[1] = prmt(s0, 0x3232), f[2] = prmt(s1, 0x1010), f[3] = prmt(s1, 0x3232);
      } else {
        const uint2 a = *reinterpret_cast<const uint2*>(base), b = *reinterpret_cast<const uint2*>(base + 4 * D);
        lo[0] = a.x, lo[1] = a.y;
        hi[0] = b.x, hi[1] = b.y;
        const uint32_t s = fp4::e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sbase + g * 8 + t4 * 2));
        f[0] = f[1] = prmt(s, 0x1010), f[2] = f[3] = prmt(s, 0x3232);
      }
      float so[NT][4];  // the odd k-steps' sums: two chains of MMAs instead of one
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[mt][n][c] = so[n][c] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        uint32_t a[4], b[4];
        fp4::e2m1x8_to_f16x2(lo[w], a);
        fp4::e2m1x8_to_f16x2(hi[w], b);
        const uint32_t fa = f[D == 128 ? w / 2 : 0], fb = f[2 + (D == 128 ? w / 2 : 0)];
        const uint32_t a0[4] = {fp4::hmul2(a[0], fa), fp4::hmul2(b[0], fb), fp4::hmul2(a[1], fa), fp4::hmul2(b[1], fb)};
        const uint32_t a1[4] = {fp4::hmul2(a[2], fa), fp4::hmul2(b[2], fb), fp4::hmul2(a[3], fa), fp4::hmul2(b[3], fb)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_16816<__half>(sc[mt][n], a0, qb[2 * w][n][0], qb[2 * w][n][1]);
          mma_16816<__half>(so[n], a1, qb[2 * w + 1][n][0], qb[2 * w + 1][n][1]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[mt][n][c] += so[n][c];
    }
    const bool part = rem < kChunk;  // the sequence's last chunk: what lies past its end may be anything
    if (part) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (16 * mt + tok + (c >> 1) * 2 >= rem) sc[mt][n][c] = kNoScore;
    }
    // running maximum (over the eight lanes of a head) and weights
    bool moved = false;
    float corr[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = fmaxf(fmaxf(sc[0][n][c], sc[0][n][c + 2]), fmaxf(sc[1][n][c], sc[1][n][c + 2]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        const float mn = fmaxf(m_[n][c], v), off = -mn * hs_[n][c];
        corr[n][c] = ex2((m_[n][c] - mn) * hs_[n][c]);
        moved |= mn != m_[n][c];
        m_[n][c] = mn;
        float sum = 0.f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float p = ex2(fmaf(sc[mt][n][c + 2 * r], hs_[n][c], off));
            if (part && 16 * mt + tok + 2 * r >= rem) p = 0.f;
            sc[mt][n][c + 2 * r] = p;
            sum += p;
          }
        l_[n][c] = l_[n][c] * corr[n][c] + sum;
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[k][n][0] *= corr[n][0];
          acc[k][n][1] *= corr[n][1];
          acc[k][n][2] *= corr[n][0];
          acc[k][n][3] *= corr[n][1];
        }
    }
    // O^T += V^T P^T: the weights rounded to fp16 (11 bits, as the operands are fp16)
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          pb[n][r] = movmatrix_trans(pack2<__half>(sc[mt][n][2 * r], sc[mt][n][2 * r + 1]));
      uint32_t x[4][VW];  // codes of tokens 4 t4 + i, dims 16 g .. (D 128) or 8 g .. (D 64)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = (t4 ^ ((i & 1) ? 3 : 0)) + 4 * i;
        const unsigned char* at = vc + mt * kSub + row * (D / 2);
        if constexpr (D == 128) {
          const uint2 w = *reinterpret_cast<const uint2*>(at + ((8 * g) ^ (((row >> 1) & 1) << 5)));
          x[i][0] = w.x, x[i][VW - 1] = w.y;
        } else {
          x[i][0] = *reinterpret_cast<const uint32_t*>(at + 4 * g);
        }
      }
      uint32_t w = *reinterpret_cast<const uint32_t*>(vc + BS * (D / 2) + mt * kSubScale +
                                                      (D == 128 ? g : g >> 1) * 16 + 4 * t4);
      if (part) {  // a scale past the end may be NaN, and 0 * NaN would stay
        const int ok = rem - 16 * mt - 4 * t4;
        w = ok >= 4 ? w : ok <= 0 ? 0u : w & ((1u << (8 * ok)) - 1u);
      }
      const uint32_t f01 = fp4::e4m3x2_to_f16x2(w), f23 = fp4::e4m3x2_to_f16x2(w >> 16);
#pragma unroll
      for (int v = 0; v < VW; ++v) {
        constexpr uint32_t kLow = 0x0f0f0f0fu;
        uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd dims, token pairs
        fp4::e2m1x8_to_f16x2((x[0][v] & kLow) | ((x[1][v] << 4) & ~kLow), e01);
        fp4::e2m1x8_to_f16x2(((x[0][v] >> 4) & kLow) | (x[1][v] & ~kLow), o01);
        fp4::e2m1x8_to_f16x2((x[2][v] & kLow) | ((x[3][v] << 4) & ~kLow), e23);
        fp4::e2m1x8_to_f16x2(((x[2][v] >> 4) & kLow) | (x[3][v] & ~kLow), o23);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t a[4] = {fp4::hmul2(e01[b], f01), fp4::hmul2(o01[b], f01), fp4::hmul2(e23[b], f23),
                                 fp4::hmul2(o23[b], f23)};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_16816<__half>(acc[4 * v + b][n], a, pb[n][0], pb[n][1]);
        }
      }
    }
  }

  // Complete the sums; the maximum in log2 units.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = l_[n][c];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        l_[n][c] = v;
        m_[n][c] *= hs_[n][c];
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
        const float f = oscale / l_[n][c];
#pragma unroll
        for (int k = 0; k < KS; k += 4) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pack2<T>(acc[k + i][n][c] * f, acc[k + i][n][c + 2] * f);
          *reinterpret_cast<uint4*>(out + h * D + g * (D / 8) + 2 * k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
  }

  __device__ __forceinline__ void store_piece(float* o, float2* ml) const {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = 8 * n + 2 * t4 + c;
#pragma unroll
        for (int k = 0; k < KS; k += 2)
          *reinterpret_cast<float4*>(o + h * D + g * (D / 8) + 2 * k) =
              make_float4(acc[k][n][c], acc[k][n][c + 2], acc[k + 1][n][c], acc[k + 1][n][c + 2]);
        if (g == 0) ml[h] = make_float2(m_[n][c], l_[n][c]);
      }
  }
};

// Head unit u: its kv head, first query head and number of them.
__device__ __forceinline__ void unit_heads(const Fp4DecodeParams& p, int u, int& kvh, int& h0, int& nh) {
  const int per = (p.group + 15) >> 4;
  kvh = u / per;
  h0 = kvh * p.group + (u - kvh * per) * 16;
  nh = min(16, kvh * p.group + p.group - h0);
}

template <typename T, int D, int BS, int NT>
__global__ void __launch_bounds__(Fp4Shape<D, NT>::kWarps * 32, 1) decode_fp4_kernel(const Fp4DecodeParams p) {
  using Sh = Fp4Shape<D, NT>;
  using Math = Fp4Math<T, D, BS, NT>;
  constexpr int WARPS = Sh::kWarps, STAGES = Sh::kStages, TILE = Math::TILE, NB = kChunk / BS;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* ring = smem + warp * STAGES * Sh::kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::kBars) + warp * STAGES;
  uint64_t* never = reinterpret_cast<uint64_t*>(smem + Sh::kBars) + WARPS * STAGES;
  int2* s_seg = reinterpret_cast<int2*>(smem + Sh::kSeg);
  float2* s_ml = reinterpret_cast<float2*>(smem + Sh::kMl);
  int* s_len = reinterpret_cast<int*>(smem + Sh::kLen);
  int* s_pre = reinterpret_cast<int*>(smem + Sh::kPre);
  int* s_sum = s_pre + kMaxSeqsPerLaunch + 1;

  if (lane == 0) {
    for (int st = 0; st < STAGES; ++st) mbar_init(&bars[st], 1);
    if (warp == 0) mbar_init(never, 1);
    fence_barrier_init();
    s_seg[2 * warp] = s_seg[2 * warp + 1] = make_int2(-1, 0);
  }
  griddep_launch_dependents();

  // Lengths (0 when outside [1, max_seq_len]) and the prefix sum of their chunks.  seq_lens
  // is read before the wait on the previous kernel (no kernel of this library writes it).
  const int S = p.num_seqs, U = p.units;
  bool bad = false;
  {
    constexpr int PER = kMaxSeqsPerLaunch / (WARPS * 32);
    int n[PER], sum = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = tid * PER + k;
      int L = i < S ? p.seq_lens[i] : 0;
      if (L < 1 || L > p.max_seq_len) {
        L = 0;
        bad |= i < S;
      }
      if (i < S) s_len[i] = L;
      n[k] = (L + kChunk - 1) / kChunk;
      sum += n[k];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_sum[warp] = incl;
    bad = __syncthreads_or(bad);
    int before = incl - sum;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = tid * PER + k;
      if (i <= S) s_pre[i] = before;
      before += n[k];
    }
    if (tid == WARPS * 32 - 1) s_pre[S] = before;
    __syncthreads();
  }
  griddep_wait();  // from here on: memory the previous kernel may have written

  if (bad && blockIdx.x == 0) {
    if (tid == 0) set_error(p.err, kErrSeqLen);
    for (int s = 0; s < S; ++s) {
      if (s_len[s] != 0) continue;
      uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (long long)s * p.num_heads * D);
      for (int i = tid; i < p.num_heads * D / 8; i += WARPS * 32) out[i] = make_uint4(0, 0, 0, 0);
    }
  }

  // This warp's run of the launch's chunks; with fewer chunks than warps, one each.
  const long long total = (long long)s_pre[S] * U;
  const long long workers = min(total, (long long)gridDim.x * WARPS);
  const long long me = (long long)blockIdx.x * WARPS + warp;
  const long long start = me < workers ? me * total / workers : total;
  const int len = me < workers ? static_cast<int>((me + 1) * total / workers - start) : 0;

  // Position -> (sequence, unit, chunk of it).
  auto locate = [&](long long at, int& s, int& u, int& j) {
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)s_pre[mid] * U <= at) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
    const int n = s_pre[s + 1] - s_pre[s];
    const int r = static_cast<int>(at - (long long)s_pre[s] * U);
    u = r / n;
    j = r - u * n;
  };

  if (len > 0) {
    // Lane i looks up position start + 32 group + i: its blocks (-1: past the sequence) and kv head.
    auto look_up = [&](int group, int (&blk)[NB], int& kvh) {
      const int k = 32 * group + lane;
      kvh = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) blk[b] = -1;
      if (k < len) {
        int s, u, j, h0, nh;
        locate(start + k, s, u, j);
        unit_heads(p, u, kvh, h0, nh);
        const int nblk = (s_len[s] + BS - 1) / BS;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (j * NB + b >= nblk) continue;
          int id = p.block_tables[(long long)s * p.max_blocks_per_seq + j * NB + b];
          if (id < 0 || id >= p.num_blocks) {  // record it, read block 0 instead
            set_error(p.err, kErrBlockId);
            id = 0;
          }
          blk[b] = id;
        }
      }
    };
    int blk_cur[NB], kvh_cur, blk_nxt[NB], kvh_nxt, group = 0;
    look_up(0, blk_cur, kvh_cur);
    look_up(1, blk_nxt, kvh_nxt);
    // Chunk k into its stage: K tiles, then V tiles; lane i < 2 NB issues copy i.
    auto issue = [&](int k) {
      if ((k >> 5) != group) {
#pragma unroll
        for (int b = 0; b < NB; ++b) blk_cur[b] = blk_nxt[b];
        kvh_cur = kvh_nxt;
        look_up(++group + 1, blk_nxt, kvh_nxt);
      }
      int id[NB], n = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        id[b] = __shfl_sync(0xffffffffu, blk_cur[b], k & 31);
        n += id[b] >= 0;
      }
      const int kvh = __shfl_sync(0xffffffffu, kvh_cur, k & 31);
      const int st = k % STAGES;
      if (lane == 0) mbar_arrive_expect_tx(&bars[st], 2 * n * TILE);
      __syncwarp();
      const int b = lane % NB, mine = NB == 1 ? id[0] : (b ? id[NB - 1] : id[0]);
      if (lane < 2 * NB && mine >= 0) {
        const void* pool = lane < NB ? p.k_cache : p.v_cache;
        bulk_copy_g2s(ring + st * Sh::kStage + lane * TILE,
                      static_cast<const unsigned char*>(pool) + ((long long)mine * p.num_kv_heads + kvh) * TILE, TILE,
                      &bars[st]);
      }
    };
    for (int k = 0; k < STAGES && k < len; ++k) issue(k);

    Math math;
    math.init(lane);
    int s, u, j, L, n, h0, nh, kvh;
    locate(start, s, u, j);
    int j0 = j;  // where the current piece starts
    auto enter = [&]() {
      L = s_len[s];
      n = (L + kChunk - 1) / kChunk;
      unit_heads(p, u, kvh, h0, nh);
      math.reset();
      math.load_q(static_cast<const T*>(p.q) + ((long long)s * p.num_heads + h0) * D, nh, p.scale_log2);
    };
    enter();
    for (int k = 0; k < len; ++k) {
      const int st = k % STAGES;
      const bool ok = __all_sync(0xffffffffu, (p.test_wait_ns && k == 0)
                                                  ? mbar_wait_bounded(never, 0, p.test_wait_ns)
                                                  : mbar_wait_bounded(&bars[st], (k / STAGES) & 1, kFp4WaitNs));
      if (!ok) {  // record it, and let the copies in flight land
        if (lane == 0) set_error(p.err, kErrTimeout);
        for (int i = k; i < len && i < k + STAGES; ++i)
          mbar_wait_bounded(&bars[i % STAGES], (i / STAGES) & 1, kFp4WaitNs / 8);
        break;
      }
      const unsigned char* stage = ring + st * Sh::kStage;
      math.chunk(stage, stage + NB * TILE, L - j * kChunk);
      __syncwarp();
      if (k + STAGES < len) {
        fence_proxy_async_smem();
        issue(k + STAGES);
      }
      ++j;
      const bool ends = j == n, last = k + 1 == len;
      if (!ends && !last) continue;
      math.finish();
      if (j0 == 0 && ends) {
        math.store_out(static_cast<T*>(p.out) + ((long long)s * p.num_heads + h0) * D, nh, p.out_scale);
      } else {
        // a piece that ends its segment but did not begin it can only be this warp's first, the other
        // kind only its last, whose room is the ring: its copies have all been read
        const int e = 2 * warp + (ends ? 0 : 1);
        float* o = reinterpret_cast<float*>(ends ? smem + Sh::kFirst + warp * Sh::kPiece : ring);
        __syncwarp();
        math.store_piece(o, s_ml + e * Sh::kRows);
        if (lane == 0) s_seg[e] = make_int2(s * U + u, (j0 == 0 ? kBegins : 0) | (ends ? kEnds : 0));
      }
      if (last) break;
      if (ends && ++u == U) {
        u = 0;
        do {
          ++s;
        } while (s_pre[s + 1] == s_pre[s]);
      }
      j = j0 = 0;
      enter();
    }
  }
  __syncthreads();

  // The CTA's pieces in order: entry e = 2 warp + {0, 1}; runs of entries of one segment are merged.
  // Lane e holds entry e (2 WARPS <= 32).
  const int2 mine = lane < 2 * WARPS ? s_seg[lane] : make_int2(-1, 0);
  const uint32_t have = __ballot_sync(0xffffffffu, mine.x >= 0);
  const uint32_t below = have & ((1u << lane) - 1u);
  const int prev = __shfl_sync(0xffffffffu, mine.x, below ? 31 - __clz(below) : 0);
  const uint32_t heads = __ballot_sync(0xffffffffu, mine.x >= 0 && (below == 0 || prev != mine.x));
  int task = 0;
  int2 out0 = make_int2(-1, 0), out1 = make_int2(-1, 0);
  for (uint32_t hd = heads; hd; hd &= hd - 1) {
    const int e0 = __ffs(hd) - 1;
    const uint32_t next = hd & (hd - 1);
    const uint32_t run = have & ~((1u << e0) - 1u) & (next ? (next & -next) - 1u : 0xffffffffu);
    const int e1 = 31 - __clz(run);
    const int seg = __shfl_sync(0xffffffffu, mine.x, e0);
    const bool begins = __shfl_sync(0xffffffffu, mine.y, e0) & kBegins;
    const bool ends = __shfl_sync(0xffffffffu, mine.y, e1) & kEnds;
    if (!begins) out0 = make_int2(seg, ends);
    else if (!ends) out1 = make_int2(seg, 0);
    const int s = seg / U;
    int kvh, h0, nh;
    unit_heads(p, seg - s * U, kvh, h0, nh);
    for (int r = 0; r < nh; ++r, ++task) {
      if (task % WARPS != warp) continue;
      constexpr int C = D / 32;
      using Vec = std::conditional_t<C == 4, float4, float2>;
      float M = -INFINITY, W = 0.f, O[C] = {};
      const float2 ml = (run >> lane) & 1u ? s_ml[lane * Sh::kRows + r] : make_float2(-INFINITY, 0.f);
      M = ml.x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float f = ml.y > 0.f ? ex2(ml.x - M) : 0.f;
      W = f * ml.y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
      for (uint32_t e = run; e; e &= e - 1) {
        const int i = __ffs(e) - 1;
        const float fi = __shfl_sync(0xffffffffu, f, i);
        const unsigned char* at = i & 1 ? smem + (i >> 1) * STAGES * Sh::kStage
                                        : smem + Sh::kFirst + (i >> 1) * Sh::kPiece;
        const Vec v = *reinterpret_cast<const Vec*>(reinterpret_cast<const float*>(at) + r * D + lane * C);
        const float* vf = reinterpret_cast<const float*>(&v);
#pragma unroll
        for (int c = 0; c < C; ++c) O[c] = fmaf(fi, vf[c], O[c]);
      }
      if (begins && ends) {
        T* out = static_cast<T*>(p.out) + ((long long)s * p.num_heads + h0 + r) * D + lane * C;
        const float il = p.out_scale / W;
#pragma unroll
        for (int c = 0; c < C; c += 2)
          *reinterpret_cast<uint32_t*>(out + c) = pack2<T>(O[c] * il, O[c + 1] * il);
      } else if (p.part_o) {  // (null only in a grid of one CTA, which leaves such a piece only when aborted)
        const long long slot = 2 * (long long)blockIdx.x + (begins ? 1 : 0);
        Vec v;
        float* vf = reinterpret_cast<float*>(&v);
#pragma unroll
        for (int c = 0; c < C; ++c) vf[c] = O[c];
        *reinterpret_cast<Vec*>(p.part_o + (slot * 16 + r) * D + lane * C) = v;
        if (lane == 0) p.part_ml[slot * 16 + r] = make_float2(M, W);
      }
    }
  }
  if (tid == 0 && p.part_seg) {
    p.part_seg[2 * blockIdx.x] = out0;
    p.part_seg[2 * blockIdx.x + 1] = out1;
  }
}

// CTA b merges the segment whose first piece ends CTA b's run (if there is one): that
// piece is slot 2 b + 1, the others are slots 2 (b + 1), 2 (b + 2), ... up to the one
// that ends the segment.  A warp per query head.
constexpr int kFp4MergeWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kFp4MergeWarps * 32) decode_fp4_merge_kernel(const Fp4DecodeParams p, int ctas) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int C = D / 32;
  using Vec = std::conditional_t<C == 4, float4, float2>;
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = p.part_seg[2 * b + 1].x;
  if (seg < 0) return;
  int rest = 0;  // pieces after the first
  for (int i0 = b + 1; i0 < ctas; i0 += 32) {
    const int2 d = i0 + lane < ctas ? p.part_seg[2 * (i0 + lane)] : make_int2(-1, 1);
    const uint32_t stop = __ballot_sync(0xffffffffu, d.x != seg || d.y);
    if (stop) {
      const int at = __ffs(stop) - 1;
      rest += at + (__shfl_sync(0xffffffffu, d.x, at) == seg);  // (another segment: an aborted launch)
      break;
    }
    rest += 32;
  }
  const int s = seg / p.units;
  int kvh, h0, nh;
  unit_heads(p, seg - s * p.units, kvh, h0, nh);
  for (int r = warp; r < nh; r += kFp4MergeWarps) {
    float RM = -INFINITY, RW = 0.f, RO[C] = {};
    for (int i0 = 0; i0 <= rest; i0 += 32) {
      const int cnt = min(32, rest + 1 - i0);
      auto slot = [&](int i) { return i == 0 ? 2 * (long long)b + 1 : 2 * (long long)(b + i); };
      const float2 ml = lane < cnt ? p.part_ml[slot(i0 + lane) * 16 + r] : make_float2(-INFINITY, 0.f);
      float M = fmaxf(ml.x, RM);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float f = ml.y > 0.f ? ex2(ml.x - M) : 0.f;
      float W = f * ml.y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
      const float keep = RW > 0.f ? ex2(RM - M) : 0.f;
      RM = M;
      RW = RW * keep + W;
#pragma unroll
      for (int c = 0; c < C; ++c) RO[c] *= keep;
      for (int i = 0; i < cnt; ++i) {
        const Vec v = *reinterpret_cast<const Vec*>(p.part_o + (slot(i0 + i) * 16 + r) * D + lane * C);
        const float* vf = reinterpret_cast<const float*>(&v);
        const float fi = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
        for (int c = 0; c < C; ++c) RO[c] = fmaf(fi, vf[c], RO[c]);
      }
    }
    const float il = p.out_scale / RW;
    T* out = static_cast<T*>(p.out) + ((long long)s * p.num_heads + h0 + r) * D + lane * C;
#pragma unroll
    for (int c = 0; c < C; c += 2) *reinterpret_cast<uint32_t*>(out + c) = pack2<T>(RO[c] * il, RO[c + 1] * il);
  }
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
  if (grid == 1) return cudaSuccess;  // one CTA: nothing is cut at a CTA's end
  e = launch_pdl(decode_fp4_merge_kernel<T, D>, dim3(grid - 1), dim3(kFp4MergeWarps * 32), 0, stream, p, grid);
  if (e == cudaSuccess) *launches = 2;
  return e;
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

// Chunks a warp should have before another CTA is worth its part of the merge.
constexpr int kFp4MinChunks = 2;

int fp4_decode_grid(int sms, int num_seqs, int num_heads, int num_kv_heads, int max_seq_len) {
  const int group = num_heads / num_kv_heads, warps = group <= 8 ? 16 : 8;
  const long long chunks = (long long)num_seqs * fp4_decode_units(num_heads, num_kv_heads) *
                           ((max_seq_len + kChunk - 1) / kChunk);
  const long long want = (chunks + kFp4MinChunks * warps - 1) / (kFp4MinChunks * warps);
  return static_cast<int>(want < sms ? (want > 0 ? want : 1) : sms);
}

cudaError_t launch_decode_fp4(bool q_is_bf16, int head_size, int block_size, const Fp4DecodeParams& p, int grid,
                              cudaStream_t stream, int* launches) {
  *launches = 0;
  return q_is_bf16 ? launch_shape<__nv_bfloat16>(head_size, block_size, p, grid, stream, launches)
                   : launch_shape<__half>(head_size, block_size, p, grid, stream, launches);
}

}  // namespace pa
