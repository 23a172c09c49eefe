// prefill_maps.cuh -- the two tensor maps that the prefill kernels' TMA copies read the pools
// through, encoded on the host at every call.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "pa_launch.h"

namespace pa {

// cuTensorMapEncodeTiled, looked up once through the runtime (no link-time libcuda)
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiledFn encoder() {
  static EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// The K pool [NB][Hkv][D/8][bs][8] seen as rows of 16 keys x 8 dims (128 16-bit
// elements, 256 bytes); a box is one row (tile::gather4 takes four of them).
template <int D, int BS>
cudaError_t encode_k_map(const PrefillParams& p, CUtensorMap* map) {
  const EncodeTiledFn enc = encoder();
  if (!enc) return cudaErrorNotSupported;
  const unsigned long long rows = (unsigned long long)p.num_blocks * p.num_kv_heads * (D / 8) * (BS / 16);
  if (rows > 0x7fffffffULL) return cudaErrorInvalidValue;  // rows are addressed with int32 coordinates
  const cuuint64_t dims[2] = {128, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {256};
  const cuuint32_t box[2] = {128, 1};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p.k_cache), dims, strides, box,
                         estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The V pool [NB][Hkv][D][bs] seen as NB * Hkv * D rows of bs 16-bit elements; a box
// is one (block, kv head) tile, [D rows][bs keys], landing with the 32-byte (bs 16) or
// 64-byte (bs 32) swizzle: the K-major layout the P V MMA reads with the same swizzle.
template <int D, int BS>
cudaError_t encode_v_map(const PrefillParams& p, CUtensorMap* map) {
  const EncodeTiledFn enc = encoder();
  if (!enc) return cudaErrorNotSupported;
  const unsigned long long rows = (unsigned long long)p.num_blocks * p.num_kv_heads * D;
  if (rows > 0x7fffffffULL) return cudaErrorInvalidValue;  // box rows are addressed with int32 coordinates
  const cuuint64_t dims[2] = {(cuuint64_t)BS, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)BS * 2};
  const cuuint32_t box[2] = {(cuuint32_t)BS, (cuuint32_t)D};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p.v_cache), dims, strides, box,
                         estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         BS == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace pa
