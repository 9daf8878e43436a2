// paged.h -- shared definitions of the paged-cache translation units.  Not part
// of the public interface.
#pragma once
#include "internal.h"
#include "maskattn.h"

namespace mab {

constexpr int PAGED_MAX_B = 4096;    // requests of one call
constexpr int PAGED_MAX_CTAS = 152;  // CTAs of the attention grid at most (one per SM)
// A warp's share of a piece in the workspace: O [4][32 rows, 16 columns], then
// (M, l) [32 rows].
constexpr int PAGED_ML = 32 * 64;
constexpr int PAGED_WARP_FLOATS = PAGED_ML + 32 * 2;
// On the line of all units, in steps of 64 keys: what a unit costs beside its
// steps (measured: a causal chunk of 8192 took 465 us at 5, 460 at 6, 462 at 7, a
// chunk of 300 over nothing 14.2, 15.0, 14.4; at 2 the chunk of 8192 took 20 %
// more), the least part that a CTA gets (one token at 8000 keys took 20.6 us at 8,
// 22.7 at 11, 26.8 at 20), and the steps below which a unit is not cut (at 5 and 8
// a chunk of 300 took 16.4 and 14.4 us, 200 single tokens at 300 keys 78 and 70 when
// this was chosen; 13.6 and 67 now).
constexpr int PAGED_UNIT_COST = 7;
constexpr int PAGED_MIN_COST = 8;
constexpr int PAGED_MIN_STEPS = 8;

// Where a CTA's part of the line begins, and what the loader needs there: the
// cuts inside that unit (of CTAs first_cut ..), the request's rows and lengths.
struct __align__(16) PagedStart {
  int b, kvh, tile, step;
  int first_cut, cuts;
  int off, n, L, pad_[3];
};

// Everything the attention over the pages reads besides the tensor maps.
struct PagedParams {
  int B, Hq, Hkv, group, Sq, Skv, total_q;
  int tile_tokens, tile_rows;  // tokens of a query tile, and its rows (times group)
  int causal, window, first;   // window and first keys of the causal rule
  const int* cu_q;
  const int* seqlen_k;
  const int* table;
  int table_stride, num_pages, page_size, box_rows;  // box_rows: rows of one load
  float inv_page_size;
  const float* sink;
  uint16_t* out;
  float* lse;  // or nullptr
  float scale_log2;
  DevStatus* status;      // of the call
  DevStatus* cta_status;  // [grid] of each CTA
  unsigned long long timeout_ns;
  int test_no_loads;
  int grid;          // CTAs
  PagedStart* start; // [grid + 1]
  float* part;       // [2 grid, slot_floats] pieces
  int slot_floats;
};

cudaError_t launch_paged_plan(const attn_plan_t& p, cudaStream_t st);
cudaError_t launch_paged_store(const attn_pages_t& pg, int T, const void* k, const void* v,
                               long long k_stride, long long v_stride, const long long* slot_map,
                               void* k_pages, void* v_pages, cudaStream_t st);
cudaError_t launch_paged_fwd(bool bf16, const PagedParams& p, const CUtensorMap& tQ,
                             const CUtensorMap& tK, const CUtensorMap& tV, cudaStream_t st);

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
