// api_paged.cu -- the C ABI of the paged key/value cache (declared in
// include/maskattn.h): argument checks, then the launches, on the caller's
// stream.  Nothing is allocated and nothing is read back.
#include "paged.h"

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

}  // extern "C"
