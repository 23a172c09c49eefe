// fp4_decode.cu -- decode attention over FP4 pools (see fp4.cuh).
#include <math.h>

#include <type_traits>

#include "fp4.cuh"
#include "pa_launch.h"

namespace pa {

// One CTA per (query head, sequence); its warps take every fourth token, a lane D/32 dims
// of it, and each keeps a running softmax (m, l, acc); the four are merged at the end.
constexpr int kFp4DecodeWarps = 4;

template <typename T, int D, int BS>
__global__ void __launch_bounds__(kFp4DecodeWarps * 32) decode_fp4_kernel(const Fp4DecodeParams p) {
  constexpr int TILE = fp4::tile_bytes(D, BS), PER = D / 32;
  __shared__ float s_m[kFp4DecodeWarps], s_l[kFp4DecodeWarps], s_o[kFp4DecodeWarps][D];
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.y, h = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T* out = static_cast<T*>(p.out) + ((long long)s * p.num_heads + h) * D;
  const int L = p.seq_lens[s];
  if (L < 1 || L > p.max_seq_len) {
    if (threadIdx.x == 0 && h == 0) set_error(p.err, kErrSeqLen);
    for (int i = threadIdx.x; i < D; i += blockDim.x) out[i] = DType<T>::from_f32(0.f);
    return;
  }
  const T* q = static_cast<const T*>(p.q) + ((long long)s * p.num_heads + h) * D + lane * PER;
  const int kvh = h / p.group, d0 = lane * PER;
  float qv[PER], acc[PER], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    qv[i] = DType<T>::to_f32(q[i]) * p.scale_log2;
    acc[i] = 0.f;
  }
  auto element = [&](const unsigned char* tile, int t, int d, int scale_at) {
    const unsigned two = tile[fp4::code_at<D>(t, d / 2)];
    const __half_raw c = __nv_cvt_fp4_to_halfraw(static_cast<__nv_fp4_storage_t>((d & 1) ? two >> 4 : two & 15), __NV_E2M1);
    const __half_raw f = __nv_cvt_fp8_to_halfraw(tile[scale_at], __NV_E4M3);
    return __half2float(__half(c)) * __half2float(__half(f));
  };
  for (int t = warp; t < L; t += kFp4DecodeWarps) {
    long long blk = p.block_tables[(long long)s * p.max_blocks_per_seq + t / BS];
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) set_error(p.err, kErrBlockId);
      blk = 0;
    }
    const long long at = (blk * p.num_kv_heads + kvh) * TILE;
    const unsigned char* kt = static_cast<const unsigned char*>(p.k_cache) + at;
    const unsigned char* vt = static_cast<const unsigned char*>(p.v_cache) + at;
    const int tt = t % BS;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      dot = fmaf(qv[i], element(kt, tt, d0 + i, fp4::k_scale_at<D, BS>(tt, (d0 + i) / 16)), dot);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float mn = fmaxf(m, dot), corr = exp2f(m - mn), w = exp2f(dot - mn);
    m = mn;
    l = l * corr + w;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      acc[i] = acc[i] * corr + w * element(vt, tt, d0 + i, fp4::v_scale_at<D, BS>(tt, (d0 + i) / 16));
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) s_o[warp][d0 + i] = acc[i];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float M = -INFINITY, W = 0.f, O = 0.f;
    for (int w = 0; w < kFp4DecodeWarps; ++w) M = fmaxf(M, s_m[w]);
    for (int w = 0; w < kFp4DecodeWarps; ++w) {
      const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - M);
      W += s_l[w] * f;
      O += s_o[w][d] * f;
    }
    out[d] = DType<T>::from_f32(O / W * p.out_scale);
  }
}

cudaError_t launch_decode_fp4(bool q_is_bf16, int head_size, int block_size, const Fp4DecodeParams& p,
                              cudaStream_t stream, int* launches) {
  const dim3 grid(p.num_heads, p.num_seqs), block(kFp4DecodeWarps * 32);
  auto go = [&](auto d, auto bs) {
    constexpr int D = decltype(d)::value, BS = decltype(bs)::value;
    return q_is_bf16 ? launch_pdl(decode_fp4_kernel<__nv_bfloat16, D, BS>, grid, block, 0, stream, p)
                     : launch_pdl(decode_fp4_kernel<__half, D, BS>, grid, block, 0, stream, p);
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  using I16 = std::integral_constant<int, 16>;
  using I32 = std::integral_constant<int, 32>;
  const cudaError_t e = head_size == 64 ? (block_size == 16 ? go(I64{}, I16{}) : go(I64{}, I32{}))
                                        : (block_size == 16 ? go(I128{}, I16{}) : go(I128{}, I32{}));
  *launches = e == cudaSuccess;
  return e;
}

}  // namespace pa
