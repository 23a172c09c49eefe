// prefill.cu -- chunked-prefill attention over the paged pool, for sm_103a.
//
// What is computed: the step before decode ("vLLM's PagedAttention: why the KV
// cache is paged" §2.3: a prompt is processed and its K/V enter the cache, then
// tokens are generated one by one), read as causal attention of a chunk of new
// query tokens over the sequence's cache: for sequence s with L tokens cached
// (the chunk's own K/V already written) and a chunk of n tokens, query token i
// at position p = L - n + i attends to positions 0..p with
//     out = softmax(scale * q K^T) V
// over K, V gathered through the block table, as decode does for one token.
//
// The kernel is in prefill_ws.cuh (tcgen05 MMAs with accumulators in tensor
// memory, warp-specialised), its host-side launch in prefill_launch.cuh; this file
// instantiates them for plain causal prefill.
#include "prefill_launch.cuh"

namespace pa {

cudaError_t launch_prefill(int dtype, int head_size, int block_size, const PrefillParams& p, cudaStream_t stream,
                           int* launches) {
  if (dtype == 1) return launch_prefill_dispatch<__half>(head_size, block_size, p, stream, launches);
  if (dtype == 2) return launch_prefill_dispatch<__nv_bfloat16>(head_size, block_size, p, stream, launches);
  return cudaErrorInvalidValue;
}

}  // namespace pa
