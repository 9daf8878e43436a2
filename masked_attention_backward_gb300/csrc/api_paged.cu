// api_paged.cu -- the C ABI of the paged key/value cache (declared in
// include/maskattn.h): argument checks, then the launches, on the caller's
// stream.  Nothing is allocated and nothing is read back.
#include <math.h>
#include <string.h>

#include "paged.h"
#include "tmap.h"

using namespace mab;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Slots of a cache, or -1 when its sizes are out of range.
long long slots_of(int num_pages, int page_size) {
  if (num_pages < 1 || page_size < 1) return -1;
  const long long n = (long long)num_pages * page_size;
  return n < (1ll << 31) ? n : -1;
}

attn_status_t check_page_size(int ps) {
  if (ps < 1 || ps > 65536) return ATTN_ERR_INVALID_ARG;
  return ps % 16 == 0 ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

attn_status_t check_pages(const attn_pages_t* pg) {
  if (!pg) return ATTN_ERR_INVALID_ARG;
  if (pg->dtype != ATTN_F16 && pg->dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (pg->Hkv < 1 || pg->Hkv > 65535 || slots_of(pg->num_pages, pg->page_size) < 0)
    return ATTN_ERR_INVALID_ARG;
  // 16-byte rows for the copies; below 2^39 elements for the tensor maps
  for (long long s : {pg->page_stride, pg->head_stride, pg->token_stride})
    if (s < HEAD_DIM || s % 8 != 0 || s >= (1ll << 39)) return ATTN_ERR_INVALID_ARG;
  return check_page_size(pg->page_size);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

attn_status_t check_paged_shape(const attn_shape_t* sh) {
  if (!sh) return ATTN_ERR_INVALID_ARG;
  if (sh->B < 1 || sh->B > PAGED_MAX_B || sh->Hq < 1 || sh->Hkv < 1 || sh->Sq < 1 ||
      sh->Skv < 1 || sh->D < 1 || sh->Hq % sh->Hkv != 0 || sh->flags != 0)
    return ATTN_ERR_INVALID_ARG;
  if (sh->dtype != ATTN_F16 && sh->dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (sh->Sq > (1 << 24) || sh->Skv > (1 << 24) || sh->Hq > 65535) return ATTN_ERR_INVALID_ARG;
  // the query heads of a kv head are rows of one 128-row tile
  if (sh->D != HEAD_DIM || sh->Hq / sh->Hkv > Q_TILE) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

struct PagedLayout {
  size_t status, cta_status, start, part, total;
  int tile_tokens, tile_rows, slot_floats;
};

PagedLayout paged_layout(const attn_shape_t* sh) {
  PagedLayout L;
  const int group = sh->Hq / sh->Hkv;
  L.tile_tokens = Q_TILE / group < sh->Sq ? Q_TILE / group : sh->Sq;
  L.tile_rows = L.tile_tokens * group;
  L.slot_floats = (L.tile_rows + 31) / 32 * 2 * PAGED_WARP_FLOATS;
  size_t off = 0;
  L.status = off;
  off = align256(off + sizeof(DevStatus));
  L.cta_status = off;
  off = align256(off + PAGED_MAX_CTAS * sizeof(DevStatus));
  L.start = off;
  off = align256(off + (PAGED_MAX_CTAS + 1) * sizeof(PagedStart));
  L.part = off;
  off = align256(off + (size_t)2 * PAGED_MAX_CTAS * L.slot_floats * sizeof(float));
  L.total = off;
  return L;
}

attn_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

}  // namespace

extern "C" {

attn_status_t attn_paged_plan(const attn_plan_t* p, void* stream) {
  if (!p || p->B < 1 || p->B > PAGED_MAX_B || p->max_pages < 1 || p->max_tokens < 0 ||
      p->table_stride < p->max_pages || slots_of(p->num_pages, p->page_size) < 0 ||
      slots_of(p->max_pages, p->page_size) < 0)
    return ATTN_ERR_INVALID_ARG;
  const attn_status_t r = check_page_size(p->page_size);
  if (r != ATTN_OK) return r;
  const void* ints[] = {p->cached,       p->fresh,    p->free_pages,     p->free_count,
                        p->block_table,  p->seqlen_k, p->free_count_out, p->refused,
                        p->cu_seqlens_q};
  for (const void* x : ints)
    if (!x || !aligned(x, 4)) return ATTN_ERR_INVALID_ARG;
  if (p->max_tokens > 0 &&
      (!p->slot_map || !aligned(p->slot_map, 8) || !p->position || !aligned(p->position, 4)))
    return ATTN_ERR_INVALID_ARG;
  return cuda_status(launch_paged_plan(*p, reinterpret_cast<cudaStream_t>(stream)));
}

attn_status_t attn_paged_store(const attn_pages_t* pages, int T, const void* k, const void* v,
                               long long k_stride, long long v_stride, const long long* slot_map,
                               void* k_pages, void* v_pages, void* stream) {
  const attn_status_t r = check_pages(pages);
  if (r != ATTN_OK) return r;
  // rows * heads is a 32-bit index
  if (T < 0 || (long long)T * pages->Hkv >= (1ll << 31) - 16) return ATTN_ERR_INVALID_ARG;
  if (T == 0) return ATTN_OK;
  const long long row = (long long)pages->Hkv * HEAD_DIM;
  if (!k || !v || !slot_map || !k_pages || !v_pages || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(slot_map, 8) || k_stride < row ||
      v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return ATTN_ERR_INVALID_ARG;
  return cuda_status(launch_paged_store(*pages, T, k, v, k_stride, v_stride, slot_map, k_pages,
                                        v_pages, reinterpret_cast<cudaStream_t>(stream)));
}

attn_status_t attn_paged_workspace_size(const attn_shape_t* shape, size_t* bytes) {
  if (!bytes) return ATTN_ERR_INVALID_ARG;
  const attn_status_t r = check_paged_shape(shape);
  if (r != ATTN_OK) return r;
  *bytes = paged_layout(shape).total;
  return ATTN_OK;
}

attn_status_t attn_paged_fwd(const attn_shape_t* shape, const attn_pages_t* pages, const void* q,
                             const void* k_pages, const void* v_pages, const int* block_table,
                             int table_stride, int max_pages, const float* sink,
                             const attn_mask_desc_t* mask, float scale, void* o, float* lse,
                             void* ws, size_t ws_bytes, void* stream) {
  attn_status_t r = check_paged_shape(shape);
  if (r == ATTN_OK) r = check_pages(pages);
  if (r != ATTN_OK) return r;
  if (!mask || pages->dtype != shape->dtype || pages->Hkv != shape->Hkv || !(scale > 0.f) ||
      !isfinite(scale) || max_pages < 1 || table_stride < max_pages ||
      slots_of(max_pages, pages->page_size) < 0)
    return ATTN_ERR_INVALID_ARG;
  PagedParams p;
  memset(&p, 0, sizeof(p));
  p.window = 1 << 25;  // longer than any context
  switch (mask->kind) {
    case ATTN_MASK_NONE:
      break;
    case ATTN_MASK_CAUSAL:
      p.causal = 1;
      break;
    case ATTN_MASK_SLIDING_FIRST:
      if (mask->first < 0) return ATTN_ERR_INVALID_ARG;
      p.first = mask->first;
      [[fallthrough]];
    case ATTN_MASK_SLIDING:
      if (mask->window < 1) return ATTN_ERR_INVALID_ARG;
      p.causal = 1;
      if (mask->window < p.window) p.window = mask->window;
      break;
    case ATTN_MASK_BLOCK:
      return ATTN_ERR_UNSUPPORTED;
    default:
      return ATTN_ERR_INVALID_ARG;
  }
  if (!mask->cu_seqlens_q || !mask->seqlen_k || mask->cu_seqlens_k || mask->seqlen_q ||
      !aligned(mask->cu_seqlens_q, 4) || !aligned(mask->seqlen_k, 4) || mask->total_q < 0)
    return ATTN_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return ATTN_ERR_INVALID_ARG;
  const PagedLayout L = paged_layout(shape);
  if (ws_bytes < L.total) return ATTN_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (mask->total_q == 0)  // no new token anywhere
    return cuda_status(cudaMemsetAsync(w + L.status, 0, sizeof(DevStatus), st));
  if (!q || !k_pages || !v_pages || !block_table || !o || !aligned(q, 16) ||
      !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16) ||
      !aligned(block_table, 4) || (lse && !aligned(lse, 4)) || (sink && !aligned(sink, 4)))
    return ATTN_ERR_INVALID_ARG;
  const bool bf16 = shape->dtype == ATTN_BF16;
  p.B = shape->B;
  p.Hq = shape->Hq;
  p.Hkv = shape->Hkv;
  p.group = shape->Hq / shape->Hkv;
  p.Sq = shape->Sq;
  const long long cap = (long long)max_pages * pages->page_size;
  p.Skv = cap < shape->Skv ? (int)cap : shape->Skv;
  p.total_q = mask->total_q;
  p.tile_tokens = L.tile_tokens;
  p.tile_rows = L.tile_rows;
  p.cu_q = mask->cu_seqlens_q;
  p.seqlen_k = mask->seqlen_k;
  p.table = block_table;
  p.table_stride = table_stride;
  p.num_pages = pages->num_pages;
  p.page_size = pages->page_size;
  p.inv_page_size = 1.0f / (float)pages->page_size;
  p.box_rows = pages->page_size % 64 == 0 ? 64 : pages->page_size % 32 == 0 ? 32 : 16;
  p.sink = sink;
  p.out = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.scale_log2 = scale * LOG2E;
  p.status = reinterpret_cast<DevStatus*>(w + L.status);
  p.cta_status = reinterpret_cast<DevStatus*>(w + L.cta_status);
  p.timeout_ns = wait_timeout_ns();
  p.test_no_loads = test_no_loads();
  p.start = reinterpret_cast<PagedStart*>(w + L.start);
  p.part = reinterpret_cast<float*>(w + L.part);
  p.slot_floats = L.slot_floats;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  p.grid = sms < PAGED_MAX_CTAS ? sms : PAGED_MAX_CTAS;
  CUtensorMap tQ, tK, tV;
  auto pages_map = [&](CUtensorMap* m, const void* base) {
    return make_pages_map(m, base, bf16, pages->num_pages, pages->page_size, pages->Hkv,
                          pages->page_stride, pages->head_stride, pages->token_stride,
                          (uint32_t)p.box_rows);
  };
  if (!make_rows_map(&tQ, q, bf16, p.total_q, p.Hq, (uint32_t)p.group, (uint32_t)p.tile_tokens) ||
      !pages_map(&tK, k_pages) || !pages_map(&tV, v_pages))
    return ATTN_ERR_CUDA;
  return cuda_status(launch_paged_fwd(bf16, p, tQ, tK, tV, st));
}

}  // extern "C"
