// paged_fwd.cu -- attention over a paged cache of 16-bit rows (paged_fwd.cuh).
#include "paged_fwd.cuh"

namespace mab {

cudaError_t launch_paged_fwd(bool bf16, const PagedParams& p, const CUtensorMap& tQ,
                             const CUtensorMap& tK, const CUtensorMap& tV, cudaStream_t st) {
  using paged_side::ROWS16;
  return bf16 ? launch_paged<true, ROWS16>(p, tQ, tK, tV, st)
              : launch_paged<false, ROWS16>(p, tQ, tK, tV, st);
}

}  // namespace mab
