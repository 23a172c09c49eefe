// prefill_capped.cu -- the masked prefill kernel (prefill_masked.cuh) with scores capped by a tanh.
#include "prefill_masked_launch.cuh"

namespace pa {

cudaError_t launch_prefill_capped(int dtype, int head_size, int block_size, const PrefillMaskedParams& p,
                                  cudaStream_t stream, int* launches) {
  return launch_prefill_masked_kind<wsm::kCapped>(dtype, head_size, block_size, p, stream, launches);
}

}  // namespace pa
