// paged8_fwd.cu -- attention over a paged cache of 8-bit codes (paged_fwd.cuh).
#include "paged_fwd.cuh"

namespace mab {

cudaError_t launch_paged8_fwd(bool bf16, bool i8, const Paged8Params& p, const CUtensorMap& tQ,
                              const CUtensorMap& tK, const CUtensorMap& tV, cudaStream_t st) {
  using namespace paged_side;
  if (i8)
    return bf16 ? launch_paged<true, CODES_I8>(p, tQ, tK, tV, st)
                : launch_paged<false, CODES_I8>(p, tQ, tK, tV, st);
  return bf16 ? launch_paged<true, CODES_E4M3>(p, tQ, tK, tV, st)
              : launch_paged<false, CODES_E4M3>(p, tQ, tK, tV, st);
}

}  // namespace mab
