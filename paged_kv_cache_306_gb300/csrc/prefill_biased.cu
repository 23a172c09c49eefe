// prefill_biased.cu -- the masked prefill kernel (prefill_masked.cuh) with scores biased by distance.
#include "prefill_masked_launch.cuh"

namespace pa {

cudaError_t launch_prefill_biased(int dtype, int head_size, int block_size, const PrefillMaskedParams& p,
                                  cudaStream_t stream, int* launches) {
  return launch_prefill_masked_kind<wsm::kBiased>(dtype, head_size, block_size, p, stream, launches);
}

}  // namespace pa
