// fp4_cache.cu -- the FP4 pools' quantising write and the two reads back (see fp4.cuh).
//
// All three move 9/16 byte of a pool per element and 2 or 4 bytes of rows, once each, and are
// bound by DRAM where they are large.  Measured on a GB300, calls in a graph: write of 65536
// tokens x 8 heads x 128 dims 58.8 us from bf16 (5.9 TB/s; the quotients still share the time),
// 89.5 us from fp32 (6.9 TB/s); read back 55.5 us as bf16 (6.2 TB/s), 93.0 us as fp32 (6.6 TB/s);
// 8192 blocks of 16 tokens x 8 heads expanded in 111.6 us (6.2 TB/s).  A write of 64 tokens takes
// 2.0 us, a read 1.9 us; a write of 8192 tokens x 4 heads from fp16 4.8 us (floor 3.2): 1024 CTAs
// on 912 places, so a second wave of 112.
#include "fp4.cuh"
#include "pa_launch.h"

namespace pa {

// --- the write ----------------------------------------------------------------------------------

// 32 bytes from an address that is a multiple of 32 (kWide) or of 16.
template <bool kWide>
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  if constexpr (kWide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// Sixteen elements of a row, and the largest magnitude (a NaN if there is one: by its bits it is above every number).
template <typename T, bool kWide>
struct Group16 {
  static constexpr int kWords = 4 * sizeof(T);
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords / 8; ++i)
      load32<kWide>(reinterpret_cast<const char*>(p) + 32 * i, *reinterpret_cast<uint32_t(*)[8]>(w + 8 * i));
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return i & 1 ? unpack2<T>(w[i / 2]).y : unpack2<T>(w[i / 2]).x;
  }
  __device__ __forceinline__ float top() const {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7fffffffu);
      return __uint_as_float(m);
    } else {  // both halves of a word at once
#pragma unroll
      for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
      const float2 v = unpack2<T>(m);
      return __uint_as_float(max(__float_as_uint(v.x), __float_as_uint(v.y)));
    }
  }
};

// a / b rounded to nearest, given r = 1 / b rounded to nearest: the quotient's residual, exact by
// a fused multiply-add, corrects a r to the nearest float (Markstein 1990), as long as nothing
// overflows or leaves the normal range (here: |a / b| between 2^-12 and 2^13 where it matters,
// b at least 2^-73).  With the signs placed so, a zero keeps its sign.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(q, b, -a), -r, q);
}

// The group's scale code and its 16 element codes:
//   u = max|x| / s,  sf = E4M3(u / 6) (at most 448),  code = E2M1(x / (sf s)),
// every fp32 operation rounded to nearest.  A NaN in the group makes sf the NaN code and every code 7.
template <typename G>
__device__ __forceinline__ unsigned quantise_group(const G& x, float s, float inv_s, uint2& codes) {
  const float top = x.top();
  // past 2688 s the scale is 448 whatever the quotient (an infinity too; a NaN passes through)
  const float bounded = top > 4096.f * s ? 4096.f * s : top;
  const float u = quotient(bounded, s, inv_s);
  const float sixth = 1.f / 6.f;
  const unsigned sf = __nv_cvt_float_to_fp8(quotient(u, 6.f, sixth), __NV_SATFINITE, __NV_E4M3);
  __nv_fp8_e4m3 sf8;
  sf8.__x = static_cast<__nv_fp8_storage_t>(sf);
  const float f = __fmul_rn(static_cast<float>(sf8), s);
  float y[2][8];
  if (sf == 0x7eu) {  // the largest scale: quotients may overflow
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i >> 3][i & 7] = __fdiv_rn(x.get(i), f);
  } else {
    const float r = f == 0.f ? 0.f : __frcp_rn(f);  // (scale 0: every code a zero with its element's sign)
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i >> 3][i & 7] = quotient(x.get(i), f, r);
  }
  codes = make_uint2(fp4::to_e2m1x8(y[0]), fp4::to_e2m1x8(y[1]));
  return sf;
}

// One thread per (token, kv head, group of 16 dims), K and V: 32 or 64 bytes in, 8 code
// bytes and a scale byte out, for each.  A row's groups are consecutive threads, so a
// warp's loads are whole rows and its stores whole rows of codes.
constexpr int kFp4Threads = 256;

// The row of this thread's group, its slot and tile; false where there is nothing to do.
template <int D, int BS, int kPerRow>
__device__ __forceinline__ bool locate_row(const int64_t* slot_mapping, int rows, int num_kv_heads,
                                           long long num_blocks, unsigned* err, int& row, int& part, long long& tile,
                                           int& off) {
  const unsigned at = blockIdx.x * (kFp4Threads / kPerRow) + threadIdx.x / kPerRow;
  if (at >= static_cast<unsigned>(rows)) return false;
  row = static_cast<int>(at);
  part = threadIdx.x % kPerRow;
  const int t = row / num_kv_heads, h = row - t * num_kv_heads;
  const long long slot = slot_mapping[t];
  if (slot < 0) return false;  // padding token
  if (slot >= num_blocks * BS) {
    if (part == 0 && h == 0) set_error(err, kErrSlot);
    return false;
  }
  tile = (slot / BS * num_kv_heads + h) * fp4::tile_bytes(D, BS);
  off = static_cast<int>(slot % BS);
  return true;
}

// (16-bit rows: six CTAs of an SM, in 40 registers a thread and a word spilled, hide the loads, 62.9 ->
// 58.9 us for 65536 tokens x 8 heads x 128 dims; fp32 rows are 32 registers a thread and slow down below 50.)
template <typename T, int D, int BS, bool kWide>
__global__ void __launch_bounds__(kFp4Threads, sizeof(T) == 2 ? 6 : 1)
    reshape_and_cache_fp4_kernel(const T* key, const T* value, unsigned char* k_cache, unsigned char* v_cache,
                                 const int64_t* slot_mapping, int rows, int num_kv_heads, long long num_blocks,
                                 float k_scale, float v_scale, float k_inv, float v_inv, unsigned* err) {
  griddep_wait();
  griddep_launch_dependents();
  int row, g, off;
  long long tile;
  if (!locate_row<D, BS, D / 16>(slot_mapping, rows, num_kv_heads, num_blocks, err, row, g, tile, off)) return;
  Group16<T, kWide> k, v;
  k.load(key + (long long)row * D + g * 16);
  v.load(value + (long long)row * D + g * 16);
  uint2 codes;
  const unsigned ks = quantise_group(k, k_scale, k_inv, codes);
  *reinterpret_cast<uint2*>(k_cache + tile + fp4::code_at<D>(off, 8 * g)) = codes;
  k_cache[tile + fp4::k_scale_at<D, BS>(off, g)] = static_cast<unsigned char>(ks);
  const unsigned vs = quantise_group(v, v_scale, v_inv, codes);
  *reinterpret_cast<uint2*>(v_cache + tile + fp4::code_at<D>(off, 8 * g)) = codes;
  v_cache[tile + fp4::v_scale_at<D, BS>(off, g)] = static_cast<unsigned char>(vs);
}

// --- the reads back -------------------------------------------------------------------------------

// 16 bytes of T from codes: code * sf (exact in fp16; sf2: it twice, or two tokens') * s,
// rounded in fp32 and then to T.  A 16-bit T: eight codes; fp32: the four of `codes`' low half.
template <typename T>
__device__ __forceinline__ uint4 widen16(uint32_t codes, uint32_t sf2, float s) {
  uint32_t h[4], o[4];
  fp4::e2m1x8_to_f16x2(codes, h);
#pragma unroll
  for (int i = 0; i < 16 / static_cast<int>(2 * sizeof(T)); ++i) {
    const float2 p = unpack2<__half>(fp4::hmul2(h[i], sf2));
    if constexpr (sizeof(T) == 4) {
      o[2 * i] = __float_as_uint(p.x * s);
      o[2 * i + 1] = __float_as_uint(p.y * s);
    } else {
      o[i] = pack2<T>(p.x * s, p.y * s);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The write's inverse: the rows of the slots, in T.  D/16 threads a row, each 16 bytes of
// every 1/2 (16-bit T) or 1/4 (fp32) of it, K and V, so that each of a warp's stores is whole
// runs of 128 or 64 bytes and a thread has 8 or 16 loads in flight.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kFp4Threads)
    gather_cache_fp4_kernel(T* key, T* value, const unsigned char* k_cache, const unsigned char* v_cache,
                            const int64_t* slot_mapping, int rows, int num_kv_heads, long long num_blocks,
                            float k_scale, float v_scale, unsigned* err) {
  constexpr int kDims = 16 / sizeof(T), TR = D / 16, N = 16 / kDims;  // dims of 16 bytes, threads a row, parts a thread
  using Codes = std::conditional_t<kDims == 8, uint32_t, uint16_t>;
  griddep_wait();
  griddep_launch_dependents();
  int row, part, off;
  long long tile;
  if (!locate_row<D, BS, TR>(slot_mapping, rows, num_kv_heads, num_blocks, err, row, part, tile, off)) return;
  uint32_t kc[N], vc[N], ks[N], vs[N];
#pragma unroll
  for (int x = 0; x < N; ++x) {
    const int c = part + TR * x, g = c * kDims / 16, at = fp4::code_at<D>(off, c * kDims / 2);
    kc[x] = *reinterpret_cast<const Codes*>(k_cache + tile + at);
    vc[x] = *reinterpret_cast<const Codes*>(v_cache + tile + at);
    ks[x] = k_cache[tile + fp4::k_scale_at<D, BS>(off, g)];
    vs[x] = v_cache[tile + fp4::v_scale_at<D, BS>(off, g)];
  }
  const long long to = (long long)row * D + part * kDims;
#pragma unroll
  for (int x = 0; x < N; ++x) {
    *reinterpret_cast<uint4*>(key + to + TR * kDims * x) =
        widen16<T>(kc[x], fp4::e4m3x2_to_f16x2(ks[x] | ks[x] << 8), k_scale);
    *reinterpret_cast<uint4*>(value + to + TR * kDims * x) =
        widen16<T>(vc[x], fp4::e4m3x2_to_f16x2(vs[x] | vs[x] << 8), v_scale);
  }
}

// Whole blocks into a 16-bit pool (k [.., D/8, BS, 8], v [.., D, BS]).  64 threads take a tile
// pair of one kv head (the tiles of a block's heads lie side by side), copied to shared memory
// 16 bytes at a time.  K: a thread takes 8 dims of a token, consecutive threads consecutive
// tokens; V: two dims of 8 tokens, their nibbles interleaved so that the conversion gives token
// pairs.  Every store instruction fills whole 32-byte sectors.
constexpr int kExpandHeads = 2, kExpandThreads = 64 * kExpandHeads;

// (12 CTAs of an SM against the 8 that ptxas chose: 1793 blocks x 4 heads 14.5 -> 13.4 us.)
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kExpandThreads, 12)
    expand_blocks_fp4_kernel(T* k_out, T* v_out, const unsigned char* k_cache, const unsigned char* v_cache,
                             const int64_t* src_dst, int num_kv_heads, long long num_out_blocks, long long num_blocks,
                             float k_scale, float v_scale, unsigned* err) {
  constexpr int TILE = fp4::tile_bytes(D, BS);
  __shared__ __align__(16) unsigned char s_tile[2][kExpandHeads * TILE];
  griddep_wait();
  griddep_launch_dependents();
  const long long pair = blockIdx.x;
  const int h0 = blockIdx.y * kExpandHeads, heads = min(kExpandHeads, num_kv_heads - h0);
  const long long src = src_dst[2 * pair], dst = src_dst[2 * pair + 1];
  if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_out_blocks) {
    if (threadIdx.x == 0 && h0 == 0) set_error(err, kErrCopyId);
    return;
  }
  const long long from = (src * num_kv_heads + h0) * TILE;
  for (int i = threadIdx.x; i < heads * (TILE / 16); i += kExpandThreads) {
    reinterpret_cast<uint4*>(s_tile[0])[i] = reinterpret_cast<const uint4*>(k_cache + from)[i];
    reinterpret_cast<uint4*>(s_tile[1])[i] = reinterpret_cast<const uint4*>(v_cache + from)[i];
  }
  __syncthreads();
  const int h = threadIdx.x / 64, me = threadIdx.x % 64;
  if (h >= heads) return;
  const unsigned char *kt = s_tile[0] + h * TILE, *vt = s_tile[1] + h * TILE;
  const long long to = (dst * num_kv_heads + h0 + h) * (D * BS);
#pragma unroll 4
  for (int i = me; i < D / 8 * BS; i += 64) {
    const int c = i / BS, t = i % BS;
    const uint32_t sf = kt[fp4::k_scale_at<D, BS>(t, c / 2)];
    reinterpret_cast<uint4*>(k_out + to)[i] = widen16<T>(*reinterpret_cast<const uint32_t*>(kt + fp4::code_at<D>(t, 4 * c)),
                                                         fp4::e4m3x2_to_f16x2(sf | sf << 8), k_scale);
  }
#pragma unroll 2
  for (int i = me; i < D / 2 * (BS / 8); i += 64) {
    const int j = i / (BS / 8), t0 = i % (BS / 8) * 8;  // dims 2 j and 2 j + 1, tokens t0 ..
    const uint2 sf = *reinterpret_cast<const uint2*>(vt + fp4::v_scale_at<D, BS>(t0, j / 8));  // of the 8 tokens
    uint32_t even[4], odd[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t a = vt[fp4::code_at<D>(t0 + 2 * x, j)], b = vt[fp4::code_at<D>(t0 + 2 * x + 1, j)];
      const uint32_t two = (a & 15u) | (b & 15u) << 4 | (a >> 4) << 8 | (b & 0xf0u) << 8;  // the even dim's pair, the odd one's
      uint32_t hw[4];
      fp4::e2m1x8_to_f16x2(two, hw);
      const uint32_t f = fp4::e4m3x2_to_f16x2((x < 2 ? sf.x : sf.y) >> (16 * (x & 1)));
      const float2 e = unpack2<__half>(fp4::hmul2(hw[0], f)), o = unpack2<__half>(fp4::hmul2(hw[1], f));
      even[x] = pack2<T>(e.x * v_scale, e.y * v_scale);
      odd[x] = pack2<T>(o.x * v_scale, o.y * v_scale);
    }
    T* out = v_out + to + 2 * j * BS + t0;
    *reinterpret_cast<uint4*>(out) = make_uint4(even[0], even[1], even[2], even[3]);
    *reinterpret_cast<uint4*>(out + BS) = make_uint4(odd[0], odd[1], odd[2], odd[3]);
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

unsigned row_blocks(long long rows, int per_row) {
  const int per_block = kFp4Threads / per_row;
  return static_cast<unsigned>((rows + per_block - 1) / per_block);
}

template <typename T>
cudaError_t write_t(const void* key, const void* value, unsigned char* kc, unsigned char* vc, const int64_t* slots,
                    int rows, int hkv, int head_size, int block_size, int64_t nb, float ks, float vs, unsigned* err,
                    cudaStream_t stream) {
  // 32-byte loads where both row arrays allow them (their rows are multiples of 128 bytes)
  const bool wide = ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value)) & 31) == 0;
  return for_shape(head_size, block_size, [&](auto d, auto bs) {
    constexpr int D = decltype(d)::value, BS = decltype(bs)::value;
    return launch_pdl(wide ? reshape_and_cache_fp4_kernel<T, D, BS, true> : reshape_and_cache_fp4_kernel<T, D, BS, false>,
                      dim3(row_blocks(rows, D / 16)), dim3(kFp4Threads), 0, stream, static_cast<const T*>(key),
                      static_cast<const T*>(value), kc, vc, slots, rows, hkv, (long long)nb, ks, vs, 1.f / ks, 1.f / vs,
                      err);
  });
}

template <typename T>
cudaError_t gather_t(void* key, void* value, const unsigned char* kc, const unsigned char* vc, const int64_t* slots,
                     int rows, int hkv, int head_size, int block_size, int64_t nb, float ks, float vs, unsigned* err,
                     cudaStream_t stream) {
  return for_shape(head_size, block_size, [&](auto d, auto bs) {
    constexpr int D = decltype(d)::value, BS = decltype(bs)::value;
    return launch_pdl(gather_cache_fp4_kernel<T, D, BS>, dim3(row_blocks(rows, D / 16)), dim3(kFp4Threads), 0,
                      stream, static_cast<T*>(key), static_cast<T*>(value), kc, vc, slots, rows, hkv, (long long)nb,
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
                      dim3(static_cast<unsigned>(num_pairs), static_cast<unsigned>((hkv + kExpandHeads - 1) / kExpandHeads)),
                      dim3(kExpandThreads), 0, stream,
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
  const cudaError_t e = f(key, value, kc, vc, slot_mapping, static_cast<int>(num_tokens * num_kv_heads), num_kv_heads,
                          head_size, block_size, num_blocks, k_scale, v_scale, err, stream);
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
  const cudaError_t e = f(key, value, kc, vc, slot_mapping, static_cast<int>(num_tokens * num_kv_heads), num_kv_heads,
                          head_size, block_size, num_blocks, k_scale, v_scale, err, stream);
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
