// Thread-block cluster helpers: rank, barrier, reads of another CTA's shared memory.
#pragma once

#include "tv_common.cuh"

namespace tv {
namespace cl {

__device__ __forceinline__ uint32_t rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void sync() {
  arrive();
  wait();
}
// The 32-bit word at the same shared-memory place as *p in CTA `r` of the cluster.
__device__ __forceinline__ uint32_t peek(const uint32_t* p, uint32_t r) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(r));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float peek(const float* p, uint32_t r) {
  return __uint_as_float(peek(reinterpret_cast<const uint32_t*>(p), r));
}
__device__ __forceinline__ int peek(const int* p, uint32_t r) {
  return static_cast<int>(peek(reinterpret_cast<const uint32_t*>(p), r));
}

// launch_pdl with clusters of `c` CTAs along x (grid.x a multiple of c).
template <typename... KArgs, typename... Args>
inline int launch_pdl(void (*kernel)(KArgs...), int c, dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                      Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  int prio = 0;
  if (cudaStreamGetPriority(st, &prio) != cudaSuccess) {
    cudaGetLastError();
    prio = 0;
  }
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributePriority;
  attr[1].val.priority = prio;
  attr[2].id = cudaLaunchAttributeClusterDimension;
  attr[2].val.clusterDim.x = c;
  attr[2].val.clusterDim.y = 1;
  attr[2].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 3;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) == cudaSuccess) return TV_OK;
  cudaGetLastError();
  return TV_ECUDA;
}

}  // namespace cl
}  // namespace tv
