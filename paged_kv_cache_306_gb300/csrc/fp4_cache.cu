// fp4_cache.cu -- the FP4 pools' quantising write and the two reads back (see fp4.cuh).
#include "fp4.cuh"
#include "pa_launch.h"

namespace pa {

// Sixteen values of a row (32 or 64 contiguous bytes).
template <typename T>
struct Group16 {
  static constexpr int kVecs = sizeof(T);
  uint4 raw[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4*>(p)[i] = raw[i];
  }
  __device__ __forceinline__ float get(int i) const { return DType<T>::to_f32(reinterpret_cast<const T*>(raw)[i]); }
  __device__ __forceinline__ void set(int i, float v) { reinterpret_cast<T*>(raw)[i] = DType<T>::from_f32(v); }
};

// The group's scale code and its 16 element codes:
//   u = max|x| / s,  sf = E4M3(u / 6) (at most 448),  code = E2M1(x / (sf s)),
// every fp32 operation rounded to nearest.  A NaN in the group makes sf the NaN code.
template <typename T>
__device__ __forceinline__ unsigned quantise_group(const Group16<T>& x, float s, uint2& codes) {
  uint32_t top = 0;  // the largest |x| by its bits: a NaN's are above every number's
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x.get(i)) & 0x7fffffffu);
  const float u = __fdiv_rn(__uint_as_float(top), s);
  const unsigned sf = __nv_cvt_float_to_fp8(__fdiv_rn(u, 6.f), __NV_SATFINITE, __NV_E4M3);
  __nv_fp8_e4m3 sf8;
  sf8.__x = static_cast<__nv_fp8_storage_t>(sf);
  const float f = __fmul_rn(static_cast<float>(sf8), s);
  float y[2][8];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = x.get(i);
    y[i >> 3][i & 7] = f == 0.f ? copysignf(0.f, v) : __fdiv_rn(v, f);
  }
  codes = make_uint2(fp4::to_e2m1x8(y[0]), fp4::to_e2m1x8(y[1]));
  return sf;
}

// One thread per (token, kv head, group of 16 dims), K and V: 32 or 64 bytes in, 8 code
// bytes and a scale byte out, for each.  A row's groups are consecutive threads, so
// loads and the 64-byte rows of codes are whole sectors.
constexpr int kFp4Threads = 256;

template <typename T, int D, int BS>
__global__ void __launch_bounds__(kFp4Threads)
    reshape_and_cache_fp4_kernel(const T* key, const T* value,
                                 unsigned char* k_cache, unsigned char* v_cache,
                                 const int64_t* slot_mapping, long long items, int num_kv_heads,
                                 long long num_blocks, float k_scale, float v_scale, unsigned* err) {
  constexpr int G = D / 16, TILE = fp4::tile_bytes(D, BS);
  griddep_wait();
  griddep_launch_dependents();
  const long long i = (long long)blockIdx.x * kFp4Threads + threadIdx.x;
  if (i >= items) return;
  const int g = static_cast<int>(i % G);
  const long long row = i / G;
  const long long t = row / num_kv_heads;
  const int h = static_cast<int>(row - t * num_kv_heads);
  const long long slot = slot_mapping[t];
  if (slot < 0) return;  // padding token
  if (slot >= num_blocks * BS) {
    if (g == 0 && h == 0) set_error(err, kErrSlot);
    return;
  }
  Group16<T> k, v;
  k.load(key + row * D + g * 16);
  v.load(value + row * D + g * 16);
  const long long tile = (slot / BS * num_kv_heads + h) * TILE;
  const int off = static_cast<int>(slot % BS);
  uint2 codes;
  const unsigned ks = quantise_group(k, k_scale, codes);
  *reinterpret_cast<uint2*>(k_cache + tile + fp4::code_at<D>(off, 8 * g)) = codes;
  k_cache[tile + fp4::k_scale_at<D, BS>(off, g)] = static_cast<unsigned char>(ks);
  const unsigned vs = quantise_group(v, v_scale, codes);
  *reinterpret_cast<uint2*>(v_cache + tile + fp4::code_at<D>(off, 8 * g)) = codes;
  v_cache[tile + fp4::v_scale_at<D, BS>(off, g)] = static_cast<unsigned char>(vs);
}

// code * sf (exact in fp16) * s, rounded in fp32 and then to T.
template <typename T>
__device__ __forceinline__ void widen_group(uint2 codes, unsigned sf, float s, Group16<T>& x) {
  const uint32_t sf2 = fp4::e4m3x2_to_f16x2(sf | sf << 8);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t h[4];
    fp4::e2m1x8_to_f16x2(w ? codes.y : codes.x, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpack2<__half>(fp4::hmul2(h[i], sf2));
      x.set(8 * w + 2 * i, p.x * s);
      x.set(8 * w + 2 * i + 1, p.y * s);
    }
  }
}

// The write's inverse, with the same threads: the rows of the slots, in T.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kFp4Threads)
    gather_cache_fp4_kernel(T* key, T* value, const unsigned char* k_cache,
                            const unsigned char* v_cache, const int64_t* slot_mapping,
                            long long items, int num_kv_heads, long long num_blocks, float k_scale, float v_scale,
                            unsigned* err) {
  constexpr int G = D / 16, TILE = fp4::tile_bytes(D, BS);
  griddep_wait();
  griddep_launch_dependents();
  const long long i = (long long)blockIdx.x * kFp4Threads + threadIdx.x;
  if (i >= items) return;
  const int g = static_cast<int>(i % G);
  const long long row = i / G;
  const long long t = row / num_kv_heads;
  const int h = static_cast<int>(row - t * num_kv_heads);
  const long long slot = slot_mapping[t];
  if (slot < 0) return;
  if (slot >= num_blocks * BS) {
    if (g == 0 && h == 0) set_error(err, kErrSlot);
    return;
  }
  const long long tile = (slot / BS * num_kv_heads + h) * TILE;
  const int off = static_cast<int>(slot % BS);
  const uint2 kc = *reinterpret_cast<const uint2*>(k_cache + tile + fp4::code_at<D>(off, 8 * g));
  const unsigned ks = k_cache[tile + fp4::k_scale_at<D, BS>(off, g)];
  const uint2 vc = *reinterpret_cast<const uint2*>(v_cache + tile + fp4::code_at<D>(off, 8 * g));
  const unsigned vs = v_cache[tile + fp4::v_scale_at<D, BS>(off, g)];
  Group16<T> x;
  widen_group(kc, ks, k_scale, x);
  x.store(key + row * D + g * 16);
  widen_group(vc, vs, v_scale, x);
  x.store(value + row * D + g * 16);
}

// Whole blocks into a 16-bit pool (k [.., D/8, BS, 8], v [.., D, BS]), a CTA per (pair,
// kv head).  A thread takes 8 dims of 8 tokens: K in 8 stores of 16 bytes (8 dims of a
// token), V transposed in registers into 8 stores of 16 bytes (8 tokens of a dim).
template <typename T, int D, int BS>
__global__ void __launch_bounds__(128)
    expand_blocks_fp4_kernel(T* k_out, T* v_out, const unsigned char* k_cache,
                             const unsigned char* v_cache, const int64_t* src_dst,
                             int num_kv_heads, long long num_out_blocks, long long num_blocks, float k_scale,
                             float v_scale, unsigned* err) {
  constexpr int TILE = fp4::tile_bytes(D, BS), ITEMS = D / 8 * (BS / 8);
  griddep_wait();
  griddep_launch_dependents();
  const long long pair = blockIdx.x;
  const int h = blockIdx.y;
  const long long src = src_dst[2 * pair], dst = src_dst[2 * pair + 1];
  if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_out_blocks) {
    if (threadIdx.x == 0 && h == 0) set_error(err, kErrCopyId);
    return;
  }
  const unsigned char* kt = k_cache + (src * num_kv_heads + h) * TILE;
  const unsigned char* vt = v_cache + (src * num_kv_heads + h) * TILE;
  T* ko = k_out + (dst * num_kv_heads + h) * (D * BS);
  T* vo = v_out + (dst * num_kv_heads + h) * (D * BS);
  for (int i = threadIdx.x; i < 2 * ITEMS; i += 128) {
    const bool is_v = i >= ITEMS;
    const int j = is_v ? i - ITEMS : i, c = j % (D / 8), t0 = j / (D / 8) * 8;  // dims 8c.., tokens t0..
    const unsigned char* tile = is_v ? vt : kt;
    const float s = is_v ? v_scale : k_scale;
    T x[8][8];  // [token][dim]
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + fp4::code_at<D>(t0 + k, 4 * c));
      const unsigned sf = tile[is_v ? fp4::v_scale_at<D, BS>(t0 + k, c / 2) : fp4::k_scale_at<D, BS>(t0 + k, c / 2)];
      const uint32_t sf2 = fp4::e4m3x2_to_f16x2(sf | sf << 8);
      uint32_t hw[4];
      fp4::e2m1x8_to_f16x2(w, hw);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 p = unpack2<__half>(fp4::hmul2(hw[q], sf2));
        x[k][2 * q] = DType<T>::from_f32(p.x * s);
        x[k][2 * q + 1] = DType<T>::from_f32(p.y * s);
      }
    }
    alignas(16) T o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = is_v ? x[q][k] : x[k][q];
      T* to = is_v ? vo + (8 * c + k) * BS + t0 : ko + (c * BS + t0 + k) * 8;
      *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(o);
    }
  }
}

namespace {

template <typename F>
cudaError_t for_shape(int head_size, int block_size, F&& f) {
  if (head_size == 64 && block_size == 16) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
  if (head_size == 64 && block_size == 32) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 32>{});
  if (head_size == 128 && block_size == 16) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 16>{});
  if (head_size == 128 && block_size == 32) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 32>{});
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t write_t(const void* key, const void* value, unsigned char* kc, unsigned char* vc, const int64_t* slots,
                    int64_t num_tokens, int hkv, int head_size, int block_size, int64_t nb, float ks, float vs,
                    unsigned* err, cudaStream_t stream) {
  return for_shape(head_size, block_size, [&](auto d, auto bs) {
    constexpr int D = decltype(d)::value, BS = decltype(bs)::value;
    const long long items = (long long)num_tokens * hkv * (D / 16);
    return launch_pdl(reshape_and_cache_fp4_kernel<T, D, BS>,
                      dim3(static_cast<unsigned>((items + kFp4Threads - 1) / kFp4Threads)), dim3(kFp4Threads), 0,
                      stream, static_cast<const T*>(key), static_cast<const T*>(value), kc, vc, slots, items, hkv,
                      (long long)nb, ks, vs, err);
  });
}

template <typename T>
cudaError_t gather_t(void* key, void* value, const unsigned char* kc, const unsigned char* vc, const int64_t* slots,
                     int64_t num_tokens, int hkv, int head_size, int block_size, int64_t nb, float ks, float vs,
                     unsigned* err, cudaStream_t stream) {
  return for_shape(head_size, block_size, [&](auto d, auto bs) {
    constexpr int D = decltype(d)::value, BS = decltype(bs)::value;
    const long long items = (long long)num_tokens * hkv * (D / 16);
    return launch_pdl(gather_cache_fp4_kernel<T, D, BS>,
                      dim3(static_cast<unsigned>((items + kFp4Threads - 1) / kFp4Threads)), dim3(kFp4Threads), 0,
                      stream, static_cast<T*>(key), static_cast<T*>(value), kc, vc, slots, items, hkv, (long long)nb,
                      ks, vs, err);
  });
}

template <typename T>
cudaError_t expand_t(void* ko, void* vo, const unsigned char* kc, const unsigned char* vc, const int64_t* pairs,
                     int64_t num_pairs, int hkv, int head_size, int block_size, int64_t out_nb, int64_t nb, float ks,
                     float vs, unsigned* err, cudaStream_t stream) {
  return for_shape(head_size, block_size, [&](auto d, auto bs) {
    constexpr int D = decltype(d)::value, BS = decltype(bs)::value;
    return launch_pdl(expand_blocks_fp4_kernel<T, D, BS>,
                      dim3(static_cast<unsigned>(num_pairs), static_cast<unsigned>(hkv)), dim3(128), 0, stream,
                      static_cast<T*>(ko), static_cast<T*>(vo), kc, vc, pairs, hkv, (long long)out_nb, (long long)nb,
                      ks, vs, err);
  });
}

}  // namespace

cudaError_t launch_reshape_and_cache_fp4(const void* key, const void* value, void* k_cache, void* v_cache,
                                         const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads,
                                         int head_size, int block_size, int64_t num_blocks, int key_dtype,
                                         float k_scale, float v_scale, unsigned* err, cudaStream_t stream,
                                         int* launches) {
  auto* kc = static_cast<unsigned char*>(k_cache);
  auto* vc = static_cast<unsigned char*>(v_cache);
  auto* f = key_dtype == 0 ? write_t<float> : key_dtype == 1 ? write_t<__half> : write_t<__nv_bfloat16>;
  const cudaError_t e = f(key, value, kc, vc, slot_mapping, num_tokens, num_kv_heads, head_size, block_size,
                          num_blocks, k_scale, v_scale, err, stream);
  *launches = e == cudaSuccess;
  return e;
}

cudaError_t launch_gather_cache_fp4(void* key, void* value, const void* k_cache, const void* v_cache,
                                    const int64_t* slot_mapping, int64_t num_tokens, int num_kv_heads, int head_size,
                                    int block_size, int64_t num_blocks, int out_dtype, float k_scale, float v_scale,
                                    unsigned* err, cudaStream_t stream, int* launches) {
  const auto* kc = static_cast<const unsigned char*>(k_cache);
  const auto* vc = static_cast<const unsigned char*>(v_cache);
  auto* f = out_dtype == 0 ? gather_t<float> : out_dtype == 1 ? gather_t<__half> : gather_t<__nv_bfloat16>;
  const cudaError_t e = f(key, value, kc, vc, slot_mapping, num_tokens, num_kv_heads, head_size, block_size,
                          num_blocks, k_scale, v_scale, err, stream);
  *launches = e == cudaSuccess;
  return e;
}

cudaError_t launch_expand_blocks_fp4(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                                     const int64_t* src_dst, int64_t num_pairs, int num_kv_heads, int head_size,
                                     int block_size, int64_t num_out_blocks, int64_t num_blocks, int out_dtype,
                                     float k_scale, float v_scale, unsigned* err, cudaStream_t stream, int* launches) {
  const auto* kc = static_cast<const unsigned char*>(k_cache);
  const auto* vc = static_cast<const unsigned char*>(v_cache);
  auto* f = out_dtype == 1 ? expand_t<__half> : expand_t<__nv_bfloat16>;
  const cudaError_t e = f(k_out, v_out, kc, vc, src_dst, num_pairs, num_kv_heads, head_size, block_size,
                          num_out_blocks, num_blocks, k_scale, v_scale, err, stream);
  *launches = e == cudaSuccess;
  return e;
}

}  // namespace pa
