// tmap.h -- host-side construction of TMA tensor maps for BHSD tensors.
//
// A [BH, S, 128] tensor of 16-bit elements is described as a 3-D tensor map
// (innermost = head dim) with 128-byte swizzle and a box of 64 x rows x 1, so
// one box fills exactly one 128B-swizzled tile of `rows` rows.  Rows past S
// read as zero on loads, per head.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mab {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Returns nullptr when the driver entry point cannot be found.  Looked up once;
// host threads that make the first calls together wait for the one that does so.
inline EncodeTiledFn get_encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// rows_box in [1, 256]; base must be 16-byte aligned.
inline bool make_bhsd_map(CUtensorMap* m, const void* base, bool bf16, int64_t BH, int64_t S,
                          uint32_t rows_box) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  cuuint64_t dims[3] = {128, (cuuint64_t)S, (cuuint64_t)BH};
  cuuint64_t strides[2] = {128 * 2, (cuuint64_t)S * 128 * 2};
  cuuint32_t box[3] = {64, rows_box, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Token-major [T, H, 128] tensor (the packed variable-length layout) as a
// 3-D tensor map (head dim, head, token) with a box of 64 x 1 x rows: one box
// is `rows` consecutive tokens of one head, laid out in shared memory exactly
// like a box of the BHSD map.  Tokens past T read as zero.
inline bool make_thd_map(CUtensorMap* m, const void* base, bool bf16, int64_t T, int64_t H,
                         uint32_t rows_box) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  cuuint64_t dims[3] = {128, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {128 * 2, (cuuint64_t)H * 128 * 2};
  cuuint32_t box[3] = {64, 1, rows_box};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Rows [T, H, 128] of new tokens, read as (token, head) rows: a box of 64
// columns, `heads` heads and `tokens` tokens is heads * tokens rows in shared
// memory, token by token.
inline bool make_rows_map(CUtensorMap* m, const void* base, bool bf16, int64_t T, int64_t H,
                          uint32_t heads, uint32_t tokens) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  cuuint64_t dims[3] = {128, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {128 * 2, (cuuint64_t)H * 128 * 2};
  cuuint32_t box[3] = {64, heads, tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Cache pages as (head dim, row, kv head, page) with the given strides in
// elements and a box of 64 columns and `rows` rows of one head of one page.
// A page number past the last reads zeros.
inline bool make_pages_map(CUtensorMap* m, const void* base, bool bf16, int64_t pages,
                           int64_t page_size, int64_t heads, int64_t page_stride,
                           int64_t head_stride, int64_t token_stride, uint32_t rows) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return false;
  cuuint64_t dims[4] = {128, (cuuint64_t)page_size, (cuuint64_t)heads, (cuuint64_t)pages};
  cuuint64_t strides[3] = {(cuuint64_t)token_stride * 2, (cuuint64_t)head_stride * 2,
                           (cuuint64_t)page_stride * 2};
  cuuint32_t box[4] = {64, rows, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                   const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace mab
