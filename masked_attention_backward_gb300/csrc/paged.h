// paged.h -- shared definitions of the paged-cache translation units.  Not part
// of the public interface.
#pragma once
#include "internal.h"
#include "maskattn.h"

namespace mab {

constexpr int PAGED_MAX_B = 4096;  // requests of one call

cudaError_t launch_paged_plan(const attn_plan_t& p, cudaStream_t st);
cudaError_t launch_paged_store(const attn_pages_t& pg, int T, const void* k, const void* v,
                               long long k_stride, long long v_stride, const long long* slot_map,
                               void* k_pages, void* v_pages, cudaStream_t st);

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Barrier over the cluster's threads; what each wrote before it, in global
// memory too, is seen by the others after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
#endif

}  // namespace mab
