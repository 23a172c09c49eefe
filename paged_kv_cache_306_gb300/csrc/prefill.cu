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
// memory, warp-specialised); this file holds its host-side launch and the dispatch over
// dtype, head size and block size (the tensor maps its TMA copies read the pools
// through: prefill_maps.cuh).
#include <math.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_launch.h"
#include "prefill_maps.cuh"
#include "prefill_ws.cuh"

namespace pa {

// ---- host side ------------------------------------------------------------------------------

// The warp-specialised tcgen05 kernel (prefill_ws.cuh): clusters of two CTAs, each CTA a pair of 128-row query
// tiles, one CTA per SM.
template <typename T, int D, int BS>
cudaError_t launch_prefill_ws_t(const PrefillParams& p, cudaStream_t stream, int* launches) {
  using Sh = ws::Shape<T, D, BS>;
  *launches = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static unsigned done = 0;
  static int resident[32];  // clusters that fit on device d at once
  const bool cached = dev < 32 && (__atomic_load_n(&done, __ATOMIC_ACQUIRE) & (1u << dev));
  int clusters_resident = cached ? __atomic_load_n(&resident[dev], __ATOMIC_RELAXED) : 0;
  if (!cached) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&ws::prefill_ws_kernel<T, D, BS>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&ws::prefill_ws_kernel<T, D, BS>),
                             cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(ws::kCluster);
    q.blockDim = dim3(ws::kThreads);
    q.dynamicSmemBytes = Sh::kSmem;
    cudaLaunchAttribute ca;
    ca.id = cudaLaunchAttributeClusterDimension;
    ca.val.clusterDim.x = ws::kCluster;
    ca.val.clusterDim.y = 1;
    ca.val.clusterDim.z = 1;
    q.attrs = &ca;
    q.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(&ws::prefill_ws_kernel<T, D, BS>), &q);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    clusters_resident = n;
    if (dev < 32) {
      __atomic_store_n(&resident[dev], n, __ATOMIC_RELAXED);
      __atomic_fetch_or(&done, 1u << dev, __ATOMIC_RELEASE);
    }
  }
  CUtensorMap kmap, vmap;
  e = encode_k_map<D, BS>(p, &kmap);
  if (e != cudaSuccess) return e;
  e = encode_v_map<D, BS>(p, &vmap);
  if (e != cudaSuccess) return e;
  // sequence s has ceil(ceil(n_s G / 128) / 4) units of four tiles per kv head, at most
  // n_s G / 512 + 1 (rounded up); each cluster of two CTAs takes units until none is left
  const long long units = (long long)p.num_kv_heads * (((long long)p.num_query_tokens * p.group + ws::kUnitTiles * ws::kRows - 1) /
                                                           (ws::kUnitTiles * ws::kRows) +
                                                       p.num_seqs);
  long long clusters = units < clusters_resident ? units : clusters_resident;
  if (clusters > 32 * ws::kLoadsPerLane) clusters = 32 * ws::kLoadsPerLane;  // the scheduler's table of loads
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * ws::kCluster));
  cfg.blockDim = dim3(ws::kThreads);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ws::kCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, ws::prefill_ws_kernel<T, D, BS>, p, kmap, vmap);
  if (e == cudaSuccess) *launches = 1;
  return e;
}

template <typename T, int D, int BS>
cudaError_t launch_prefill_t(const PrefillParams& p, cudaStream_t s, int* n) {
  return launch_prefill_ws_t<T, D, BS>(p, s, n);
}

template <typename T>
cudaError_t launch_prefill_dispatch(int head_size, int block_size, const PrefillParams& p, cudaStream_t s, int* n) {
  if (head_size == 64 && block_size == 16) return launch_prefill_t<T, 64, 16>(p, s, n);
  if (head_size == 64 && block_size == 32) return launch_prefill_t<T, 64, 32>(p, s, n);
  if (head_size == 128 && block_size == 16) return launch_prefill_t<T, 128, 16>(p, s, n);
  if (head_size == 128 && block_size == 32) return launch_prefill_t<T, 128, 32>(p, s, n);
  return cudaErrorInvalidValue;
}

cudaError_t launch_prefill(int dtype, int head_size, int block_size, const PrefillParams& p, cudaStream_t stream,
                           int* launches) {
  if (dtype == 1) return launch_prefill_dispatch<__half>(head_size, block_size, p, stream, launches);
  if (dtype == 2) return launch_prefill_dispatch<__nv_bfloat16>(head_size, block_size, p, stream, launches);
  return cudaErrorInvalidValue;
}

}  // namespace pa
