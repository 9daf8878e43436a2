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
  // Requests with more than tokens_lo and at most tokens_hi new tokens take part; the
  // call's other kernels take the rest.  more_status: [grid] statuses of a kernel before
  // this one; keep_status: the call's status word has been written.
  int tokens_lo, tokens_hi;
  const DevStatus* more_status;
  int keep_status;
};

// ... and over a cache of 8-bit codes.
struct Paged8Params : PagedParams {
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  long long scale_page_stride, scale_head_stride;
  int scale_shift;  // log2 of the tokens that share a scale
};

attn_status_t check_paged_shape(const attn_shape_t* sh);
attn_status_t paged_call(const attn_shape_t* shape, int num_pages, int page_size, const void* q,
                         const void* k_pages, const void* v_pages, const int* block_table,
                         int table_stride, int max_pages, const float* sink,
                         const attn_mask_desc_t* mask, float scale, void* o, float* lse, void* ws,
                         size_t ws_bytes, cudaStream_t st, PagedParams* out, CUtensorMap* tQ,
                         bool* work);
size_t paged_workspace(const attn_shape_t* shape);

cudaError_t launch_paged_plan(const attn_plan_t& p, cudaStream_t st);
cudaError_t launch_paged_store(const attn_pages_t& pg, int T, const void* k, const void* v,
                               long long k_stride, long long v_stride, const long long* slot_map,
                               void* k_pages, void* v_pages, cudaStream_t st);
cudaError_t launch_paged_fwd(bool bf16, const PagedParams& p, const CUtensorMap& tQ,
                             const CUtensorMap& tK, const CUtensorMap& tV, cudaStream_t st);
cudaError_t launch_paged8_fwd(bool bf16, bool i8, const Paged8Params& p, const CUtensorMap& tQ,
                              const CUtensorMap& tK, const CUtensorMap& tV, cudaStream_t st);
// Query rows (tokens times query heads of a kv head) over 8-bit codes up to which
// k_paged8_rows takes a call, and requests beside chunks.
constexpr int PAGED8_ROWS = 16;
cudaError_t launch_paged8_rows(bool bf16, bool i8, const Paged8Params& p, const CUtensorMap& tK,
                               const CUtensorMap& tV, const void* q, cudaStream_t st);

// Where the rows of the requests that k_paged8_rows does not take stand in 16 bits for a
// call: pages of PAGED8_PAGE tokens [pages, Hkv, PAGED8_PAGE, 128], a table of them
// [B, cols], and the statuses of the kernel that writes them.
constexpr int PAGED8_PAGE = 64;
struct Expanded {
  uint16_t* k;
  uint16_t* v;
  int* table;
  int cols, pages;
  DevStatus* status;
};
cudaError_t launch_paged8_expand(bool bf16, bool i8, const Paged8Params& p, const void* k_pages,
                                 const void* v_pages, long long page_stride,
                                 long long head_stride, long long token_stride,
                                 const Expanded& e, cudaStream_t st);

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
