// prefill_masked_launch.cuh -- the host-side launch of a kind of the masked prefill kernel
// (prefill_masked.cuh); included by the translation units that instantiate one each.
#pragma once

#include "pa_launch.h"
#include "prefill_maps.cuh"
#include "prefill_masked.cuh"

namespace pa {

// Clusters of two CTAs, one CTA per SM: as many as fit on the GPU at once, at most one per unit.
template <typename T, int D, int BS, int kKind>
cudaError_t launch_prefill_masked_t(const PrefillMaskedParams& p, cudaStream_t stream, int* launches) {
  using Sh = wsm::Shape<T, D, BS>;
  constexpr auto kernel = &wsm::prefill_masked_kernel<T, D, BS, kKind>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  *launches = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ws::kCluster);
  cfg.blockDim = dim3(wsm::kThreads);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ws::kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;

  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static int resident[32];  // clusters that fit on device d at once; 0: not asked yet
  int clusters_resident = dev < 32 ? __atomic_load_n(&resident[dev], __ATOMIC_ACQUIRE) : 0;
  if (clusters_resident == 0) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, fn);
    if (e != cudaSuccess) return e;
    // the registers that the warpgroups share out anew have to be there, or they would wait for ever
    if (a.numRegs < wsm::kLaunchRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&clusters_resident, fn, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters_resident < 1) return cudaErrorInvalidConfiguration;
    if (dev < 32) __atomic_store_n(&resident[dev], clusters_resident, __ATOMIC_RELEASE);
  }
  CUtensorMap kmap, vmap;
  e = encode_k_map<D, BS>(p, &kmap);
  if (e != cudaSuccess) return e;
  e = encode_v_map<D, BS>(p, &vmap);
  if (e != cudaSuccess) return e;
  // sequence s has ceil(ceil(n_s G / 128) / 4) units of four tiles per kv head, at most n_s G / 512 + 1
  const long long unit_rows = ws::kUnitTiles * ws::kRows;
  const long long units =
      p.num_kv_heads * (((long long)p.num_query_tokens * p.group + unit_rows - 1) / unit_rows + p.num_seqs);
  long long clusters = units < clusters_resident ? units : clusters_resident;
  if (clusters > 32 * ws::kLoadsPerLane) clusters = 32 * ws::kLoadsPerLane;  // the scheduler's table of loads
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * ws::kCluster));
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, p, kmap, vmap);
  if (e == cudaSuccess) *launches = 1;
  return e;
}

template <typename T, int kKind>
cudaError_t launch_prefill_masked_shape(int head_size, int block_size, const PrefillMaskedParams& p, cudaStream_t s,
                                        int* n) {
  if (head_size == 64 && block_size == 16) return launch_prefill_masked_t<T, 64, 16, kKind>(p, s, n);
  if (head_size == 64 && block_size == 32) return launch_prefill_masked_t<T, 64, 32, kKind>(p, s, n);
  if (head_size == 128 && block_size == 16) return launch_prefill_masked_t<T, 128, 16, kKind>(p, s, n);
  if (head_size == 128 && block_size == 32) return launch_prefill_masked_t<T, 128, 32, kKind>(p, s, n);
  return cudaErrorInvalidValue;
}

// Over the dtypes (PA_F16, PA_BF16).
template <int kKind>
cudaError_t launch_prefill_masked_kind(int dtype, int head_size, int block_size, const PrefillMaskedParams& p,
                                       cudaStream_t stream, int* launches) {
  if (dtype == 1) return launch_prefill_masked_shape<__half, kKind>(head_size, block_size, p, stream, launches);
  if (dtype == 2) return launch_prefill_masked_shape<__nv_bfloat16, kKind>(head_size, block_size, p, stream, launches);
  return cudaErrorInvalidValue;
}

}  // namespace pa
