// paged8.h -- shared definitions of the 8-bit cache's translation units.  Not
// part of the public interface.
#pragma once
#include "internal.h"
#include "maskattn.h"

namespace mab {

// Where an 8-bit cache keeps what; strides in bytes.
struct Pages8 {
  int num_pages, page_size, Hkv, block, shift;  // shift: log2 of block
  long long page_stride, head_stride, token_stride;
  long long scale_page_stride, scale_head_stride;
};

cudaError_t launch_paged8_store(bool bf16, bool i8, const Pages8& pg, int T, const void* k,
                                const void* v, long long k_stride, long long v_stride,
                                const long long* slot_map, void* k_pages, void* v_pages,
                                uint8_t* k_scales, uint8_t* v_scales, cudaStream_t st);
cudaError_t launch_paged8_load(bool bf16, bool i8, const Pages8& pg, int B, int total,
                               const int* start, const int* cu, const int* table,
                               int table_stride, int max_pages, const void* k_pages,
                               const void* v_pages, const uint8_t* k_scales,
                               const uint8_t* v_scales, void* k, void* v, cudaStream_t st);

}  // namespace mab
