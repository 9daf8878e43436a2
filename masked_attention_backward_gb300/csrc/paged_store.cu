// paged_store.cu -- keys and values of new tokens into their cache slots.
//
// Bound: HBM (each row is read and written once, 512 B per token, head and
// tensor).  A half-warp moves one 256-byte row of K and the same row of V, 16
// bytes a thread, so that every request of a warp covers whole 128-byte lines
// on both sides whatever the layout; the slot is the same word for all 16.
// Measured (one GB300): 16384 tokens of 8 heads 21.7 us, 6.2 TB/s; 32 tokens
// 1.6 us in a row of calls, the launch.
#include "paged.h"

namespace mab {

namespace {
constexpr int STORE_THREADS = 256;
}

__global__ void __launch_bounds__(STORE_THREADS)
k_paged_store(const uint4* __restrict__ k, const uint4* __restrict__ v, uint4* __restrict__ kp,
              uint4* __restrict__ vp, const long long* __restrict__ slot_map, int rows, int Hkv,
              long long k_stride, long long v_stride, unsigned page_size, unsigned slots,
              long long page_stride, long long head_stride, long long token_stride) {
  const int l16 = threadIdx.x & 15;
  // strides count 16-byte units
  const int row = (int)(blockIdx.x * (STORE_THREADS / 16) + (threadIdx.x >> 4));
  if (row >= rows) return;
  const int t = row / Hkv, h = row % Hkv;
  const long long slot = slot_map[t];
  if (slot < 0 || slot >= (long long)slots) return;
  const unsigned page = (unsigned)slot / page_size, off = (unsigned)slot % page_size;
  const uint4 a = k[t * k_stride + h * 16 + l16];
  const uint4 b = v[t * v_stride + h * 16 + l16];
  const long long dst = page * page_stride + h * head_stride + off * token_stride + l16;
  kp[dst] = a;
  vp[dst] = b;
}

cudaError_t launch_paged_store(const attn_pages_t& pg, int T, const void* k, const void* v,
                               long long k_stride, long long v_stride, const long long* slot_map,
                               void* k_pages, void* v_pages, cudaStream_t st) {
  const int rows = T * pg.Hkv;
  const int per = STORE_THREADS / 16;
  k_paged_store<<<(unsigned)((rows + per - 1) / per), STORE_THREADS, 0, st>>>(
      (const uint4*)k, (const uint4*)v, (uint4*)k_pages, (uint4*)v_pages, slot_map, rows, pg.Hkv,
      k_stride / 8, v_stride / 8, (unsigned)pg.page_size, (unsigned)(pg.num_pages * pg.page_size),
      pg.page_stride / 8, pg.head_stride / 8, pg.token_stride / 8);
  return cudaGetLastError();
}

}  // namespace mab
