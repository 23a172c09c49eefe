// decode_masked_f16.cu -- decode with capped or biased scores and windows, for f16 caches.
#include "decode_kernels.cuh"

namespace pa {

int decode_masked_ctas_per_sm_f16(int head_size, int block_size, DecodeKind kind) {
  return decode_ctas_per_sm_dispatch<__half, __half, true>(head_size, block_size, kind);
}

cudaError_t launch_decode_masked_f16(int head_size, int block_size, const DecodeMaskedParams& p, DecodeKind kind, int grid,
                                     cudaStream_t s, int* n) {
  return launch_decode_dispatch<__half, __half, true>(head_size, block_size, p, kind, grid, s, n);
}

}  // namespace pa
