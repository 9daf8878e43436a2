// api_paged8.cu -- the C ABI of the 8-bit cache (declared in
// include/maskattn.h): argument checks, then the launches, on the caller's
// stream.  Nothing is allocated and nothing is read back.
#include <stdlib.h>

#include "paged.h"
#include "paged8.h"
#include "tmap.h"

using namespace mab;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

attn_status_t check_pages8(const attn_pages8_t* pg, Pages8* out) {
  if (!pg || (pg->dtype != ATTN_F16 && pg->dtype != ATTN_BF16) ||
      (pg->code != ATTN_E4M3 && pg->code != ATTN_I8) || pg->Hkv < 1 || pg->Hkv > 65535 ||
      pg->num_pages < 1 || pg->page_size < 1 || pg->page_size > 65536 ||
      (long long)pg->num_pages * pg->page_size >= (1ll << 31))
    return ATTN_ERR_INVALID_ARG;
  // 16-byte rows for the copies; below 2^40 bytes for the tensor maps
  for (long long s : {pg->page_stride, pg->head_stride, pg->token_stride})
    if (s < HEAD_DIM || s % 16 != 0 || s >= (1ll << 40)) return ATTN_ERR_INVALID_ARG;
  if (pg->page_size % 16 != 0 ||
      (pg->block != 1 && pg->block != 16 && pg->block != 32 && pg->block != 64))
    return ATTN_ERR_UNSUPPORTED;
  if (pg->page_size % pg->block != 0) return ATTN_ERR_INVALID_ARG;
  // a page's scales of a head lie together; one a token is read 16 at a time
  for (long long s : {pg->scale_page_stride, pg->scale_head_stride})
    if (s < pg->page_size / pg->block || s >= (1ll << 40) || (pg->block == 1 && s % 16 != 0))
      return ATTN_ERR_INVALID_ARG;
  int shift = 0;
  while ((1 << shift) < pg->block) ++shift;
  *out = {pg->num_pages,    pg->page_size,   pg->Hkv,          pg->block,
          shift,            pg->page_stride, pg->head_stride,  pg->token_stride,
          pg->scale_page_stride, pg->scale_head_stride};
  return ATTN_OK;
}

attn_status_t check_buffers8(const attn_pages8_t* pg, const void* k_pages, const void* v_pages,
                             const uint8_t* k_scales, const uint8_t* v_scales) {
  const size_t a = pg->block == 1 ? 16 : 1;
  return k_pages && v_pages && k_scales && v_scales && aligned(k_pages, 16) &&
                 aligned(v_pages, 16) && aligned(k_scales, a) && aligned(v_scales, a)
             ? ATTN_OK
             : ATTN_ERR_INVALID_ARG;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Test hook, read at each call: room for 16-bit rows is used however few steps there are.
bool test_paged8_room() {
  const char* e = getenv("MASKATTN_PAGED8_ROOM");
  return e && e[0] == '1';
}

// New tokens whose rows k_paged8_rows takes.
int few_tokens(const attn_shape_t* sh) { return PAGED8_ROWS / (sh->Hq / sh->Hkv); }

// Steps (64 keys of a query tile) that an SM has at least, going by the call's bounds,
// when its chunks' rows are written in 16 bits first.  Measured at 32/8 heads, e4m3, us with
// tiles made inside the attention and with rows written first:
//   four chunks of 256 over 500 to 4000 keys: 13 steps 35 and 33, 26 52 and 45, 40 64 and 53,
//     53 75 and 63, 106 116 and 97;
//   one chunk of 128, 256, 512 over 8000: 26 steps 40 and 45, 52 62 and 58, 105 105 and 84;
//   15 single tokens and a chunk of 500 over 1000, 2000, 3000: 14 steps 48 and 61, 28 72 and 83,
//     42 92 and 105 (two kernels more, and two joins, for the single tokens);
//   the same under a window of 1024, chunks of 500, 1000, 2000: 23 steps 60 and 66, 57 79 and 82,
//     165 110 and 109.
// So chunks alone gain from 10 to 50 steps on, chunks beside single tokens from some 150; which
// of a call's requests are chunks only the device knows, and 40 is between for the former.
constexpr int EXPAND_STEPS = 40;

// Room for the 16-bit rows of a call's chunks behind the other workspace: pages for as
// many requests as the tokens allow to have more than few, each with all the sub-tiles
// that its tokens may see.  pages = 0: none are wanted (or more than a map can hold).
struct ExpandedLayout {
  size_t status, table, k, v, total;
  long long pages;
  int cols;
};
ExpandedLayout expanded_layout(const attn_shape_t* sh, const attn_mask_desc_t* mask) {
  ExpandedLayout L = {};
  L.total = paged_workspace(sh);
  const int group = sh->Hq / sh->Hkv;
  if ((long long)sh->Sq * group <= Q_TILE) return L;
  const long long chunks = mask->total_q / (few_tokens(sh) + 1);
  L.cols = (sh->Skv + PAGED8_PAGE - 1) / PAGED8_PAGE;
  long long tiles = L.cols;
  if (mask->kind == ATTN_MASK_SLIDING || mask->kind == ATTN_MASK_SLIDING_FIRST) {
    const long long first =
        mask->kind == ATTN_MASK_SLIDING_FIRST && mask->first > 0 ? mask->first : 0;
    const long long seen =
        ((long long)mask->window + sh->Sq + PAGED8_PAGE) / PAGED8_PAGE + 1 + first / PAGED8_PAGE + 1;
    if (seen < tiles) tiles = seen;
  }
  const long long steps =
      ((long long)mask->total_q * group + Q_TILE - 1) / Q_TILE * tiles * sh->Hkv / PAGED_MAX_CTAS;
  if (steps < EXPAND_STEPS && !test_paged8_room()) return L;
  const long long pages = (chunks < sh->B ? chunks : sh->B) * tiles;
  if (pages < 1 || pages * PAGED8_PAGE >= (1ll << 31)) return L;
  L.pages = pages;
  const size_t rows = (size_t)pages * sh->Hkv * PAGED8_PAGE * HEAD_DIM * 2;
  L.status = align256(L.total);
  L.table = align256(L.status + PAGED_MAX_CTAS * sizeof(DevStatus));
  L.k = align256(L.table + (size_t)sh->B * L.cols * sizeof(int));
  L.v = align256(L.k + rows);
  L.total = align256(L.v + rows);
  return L;
}

attn_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

}  // namespace

extern "C" {

attn_status_t attn_paged8_store(const attn_pages8_t* pages, int T, const void* k, const void* v,
                                long long k_stride, long long v_stride, const long long* slot_map,
                                void* k_pages, void* v_pages, uint8_t* k_scales,
                                uint8_t* v_scales, void* stream) {
  Pages8 pg;
  attn_status_t r = check_pages8(pages, &pg);
  if (r != ATTN_OK) return r;
  // rows * heads is a 32-bit index
  if (T < 0 || (long long)T * pages->Hkv >= (1ll << 31) - 16) return ATTN_ERR_INVALID_ARG;
  if (T == 0) return ATTN_OK;
  const long long row = (long long)pages->Hkv * HEAD_DIM;
  if (!k || !v || !slot_map || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8) ||
      k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return ATTN_ERR_INVALID_ARG;
  r = check_buffers8(pages, k_pages, v_pages, k_scales, v_scales);
  if (r != ATTN_OK) return r;
  return cuda_status(launch_paged8_store(pages->dtype == ATTN_BF16, pages->code == ATTN_I8, pg, T,
                                         k, v, k_stride, v_stride, slot_map, k_pages, v_pages,
                                         k_scales, v_scales, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_paged8_load(const attn_pages8_t* pages, int B, int total, const int* start,
                               const int* cu_seqlens, const int* block_table, int table_stride,
                               int max_pages, const void* k_pages, const void* v_pages,
                               const uint8_t* k_scales, const uint8_t* v_scales, void* k, void* v,
                               void* stream) {
  Pages8 pg;
  attn_status_t r = check_pages8(pages, &pg);
  if (r != ATTN_OK) return r;
  if (B < 1 || B > 65536 || total < 0 || max_pages < 1 || table_stride < max_pages ||
      (long long)max_pages * pages->page_size >= (1ll << 31))
    return ATTN_ERR_INVALID_ARG;
  if (total == 0) return ATTN_OK;
  if (!cu_seqlens || !aligned(cu_seqlens, 4) || (start && !aligned(start, 4)) || !block_table ||
      !aligned(block_table, 4) || !k || !v || !aligned(k, 16) || !aligned(v, 16))
    return ATTN_ERR_INVALID_ARG;
  r = check_buffers8(pages, k_pages, v_pages, k_scales, v_scales);
  if (r != ATTN_OK) return r;
  return cuda_status(launch_paged8_load(pages->dtype == ATTN_BF16, pages->code == ATTN_I8, pg, B,
                                        total, start, cu_seqlens, block_table, table_stride,
                                        max_pages, k_pages, v_pages, k_scales, v_scales, k, v,
                                        static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_paged8_workspace_size(const attn_shape_t* shape, const attn_mask_desc_t* mask,
                                         size_t* bytes) {
  if (!bytes) return ATTN_ERR_INVALID_ARG;
  const attn_status_t r = check_paged_shape(shape);
  if (r != ATTN_OK) return r;
  *bytes = paged_workspace(shape);
  if (mask) *bytes = expanded_layout(shape, mask).total;
  return ATTN_OK;
}

attn_status_t attn_paged8_fwd(const attn_shape_t* shape, const attn_pages8_t* pages, const void* q,
                              const void* k_pages, const void* v_pages, const uint8_t* k_scales,
                              const uint8_t* v_scales, const int* block_table, int table_stride,
                              int max_pages, const float* sink, const attn_mask_desc_t* mask,
                              float scale, void* o, float* lse, void* ws, size_t ws_bytes,
                              void* stream) {
  attn_status_t r = check_paged_shape(shape);
  Pages8 pg;
  if (r == ATTN_OK) r = check_pages8(pages, &pg);
  if (r != ATTN_OK) return r;
  if (pages->dtype != shape->dtype || pages->Hkv != shape->Hkv) return ATTN_ERR_INVALID_ARG;
  Paged8Params p;
  CUtensorMap tQ, tK, tV;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // every request has few rows: a kernel that reads q's rows itself
  const bool few = shape->Sq <= few_tokens(shape);
  bool work = false;
  r = paged_call(shape, pages->num_pages, pages->page_size, q, k_pages, v_pages, block_table,
                 table_stride, max_pages, sink, mask, scale, o, lse, ws, ws_bytes, st, &p,
                 few ? nullptr : &tQ, &work);
  if (r != ATTN_OK || !work) return r;
  r = check_buffers8(pages, k_pages, v_pages, k_scales, v_scales);
  if (r != ATTN_OK) return r;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.scale_page_stride = pg.scale_page_stride;
  p.scale_head_stride = pg.scale_head_stride;
  p.scale_shift = pg.shift;
  const bool bf16 = shape->dtype == ATTN_BF16, i8 = pages->code == ATTN_I8;
  auto pages_maps = [&](int rows) {
    for (CUtensorMap* m : {&tK, &tV})
      if (!make_pages8_map(m, m == &tK ? k_pages : v_pages, pg.num_pages, pg.page_size, pg.Hkv,
                           pg.page_stride, pg.head_stride, pg.token_stride, (uint32_t)rows))
        return false;
    return true;
  };
  if (few) {
    if (!pages_maps(16)) return ATTN_ERR_CUDA;
    return cuda_status(launch_paged8_rows(bf16, i8, p, tK, tV, q, st));
  }
  // One query tile a request and kv head (or a workspace without room for 16-bit rows): codes
  // become tiles inside the attention.
  const ExpandedLayout L = expanded_layout(shape, mask);
  if (L.pages == 0 || ws_bytes < L.total) {
    if (!pages_maps(p.box_rows)) return ATTN_ERR_CUDA;
    return cuda_status(launch_paged8_fwd(bf16, i8, p, tQ, tK, tV, st));
  }
  // Chunks: the requests with few rows first, unless q has rows enough for every request to
  // have more.  (It may have rows that no request owns, as a captured call's does: its lengths
  // may be any then too, and the kernels behind take every request.  The room holds them: more
  // than (B - 1) Sq + small rows, Sq > small, are B (small + 1) at least, so it was made for B.)
  const int small = few_tokens(shape);
  const bool split =
      small > 0 && mask->total_q <= (long long)(shape->B - 1) * shape->Sq + small;
  if (split) {
    Paged8Params f = p;
    f.tokens_hi = small;
    f.tile_tokens = small;
    f.tile_rows = small * p.group;
    if (!pages_maps(16)) return ATTN_ERR_CUDA;
    if (launch_paged8_rows(bf16, i8, f, tK, tV, q, st) != cudaSuccess) return ATTN_ERR_CUDA;
    p.keep_status = 1;
  }
  // ... then the others' rows in 16 bits, and the attention over them.
  p.tokens_lo = split ? small : 0;
  uint8_t* w = static_cast<uint8_t*>(ws);
  Expanded e;
  e.k = reinterpret_cast<uint16_t*>(w + L.k);
  e.v = reinterpret_cast<uint16_t*>(w + L.v);
  e.table = reinterpret_cast<int*>(w + L.table);
  e.cols = L.cols;
  e.pages = (int)L.pages;
  e.status = reinterpret_cast<DevStatus*>(w + L.status);
  if (launch_paged8_expand(bf16, i8, p, k_pages, v_pages, pg.page_stride, pg.head_stride,
                           pg.token_stride, e, st) != cudaSuccess)
    return ATTN_ERR_CUDA;
  PagedParams d = p;
  d.more_status = e.status;
  d.table = e.table;
  d.table_stride = e.cols;
  d.num_pages = e.pages;
  d.page_size = PAGED8_PAGE;
  d.inv_page_size = 1.f / PAGED8_PAGE;
  d.box_rows = PAGED8_PAGE;
  const long long head = PAGED8_PAGE * HEAD_DIM;
  for (CUtensorMap* m : {&tK, &tV})
    if (!make_pages_map(m, m == &tK ? e.k : e.v, bf16, e.pages, PAGED8_PAGE, shape->Hkv,
                        head * shape->Hkv, head, HEAD_DIM, PAGED8_PAGE))
      return ATTN_ERR_CUDA;
  return cuda_status(launch_paged_fwd(bf16, d, tQ, tK, tV, st));
}

}  // extern "C"
