// prefill_masked.cu -- the prefill kernel (prefill_ws.cuh) with scores capped by a tanh or biased
// by distance, sliding windows and prefixes (kMod).
#include "prefill_launch.cuh"

namespace pa {

cudaError_t launch_prefill_masked(int dtype, int head_size, int block_size, const PrefillMaskedParams& p,
                                  cudaStream_t stream, int* launches) {
  if (dtype == 1) return launch_prefill_dispatch<__half, true>(head_size, block_size, p, stream, launches);
  if (dtype == 2) return launch_prefill_dispatch<__nv_bfloat16, true>(head_size, block_size, p, stream, launches);
  return cudaErrorInvalidValue;
}

}  // namespace pa
