// paged8_expand.cu -- the rows of an 8-bit cache that a call's chunks see, in 16 bits.
//
// Every query tile of a chunk walks the same keys, and making 16-bit tiles of their
// codes costs the attention kernel more than the products (paged_fwd.cuh): a chunk of
// 1900 tokens with four heads a group would do it 60 times over.  So a call with
// chunks has their rows written once, into pages of 64 tokens in the workspace, and
// its attention over them is that of a 16-bit cache.  Only sub-tiles with a seen key
// are written; code times scale is exact in 16 bits (quant8.cuh).
//
// Bound: HBM and L2, 256 bytes read and 512 written a key and kv head.  Every block
// counts the requests' sub-tiles for itself (a scan over at most 4096 requests), then
// takes sub-tiles of a kv head in turn: 64 rows of K and of V, a half-warp per row.
// Measured (one GB300): one request's window of 1500 keys, 8 heads, 6.5 us, most of it the
// launch and the scan; chunks of 1900 tokens over 8000 keys with the attention behind it
// 389 us, where that over a 16-bit cache takes 363.
#include "paged_line.cuh"
#include "quant8.cuh"

namespace mab {

namespace expand_side {
constexpr int THREADS = 256;
constexpr int PER_SM = 4;  // blocks
}  // namespace expand_side

struct ExpandParams : Paged8Params {
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  long long page_stride, head_stride, token_stride;
  Expanded to;
};

template <bool BF16, bool I8>
__global__ void __launch_bounds__(expand_side::THREADS, expand_side::PER_SM)
k_paged8_expand(const __grid_constant__ ExpandParams p) {
  using namespace expand_side;
  using namespace paged_side;
  __shared__ int first[PAGED_MAX_B + 1];  // sub-tiles of the requests before each
  __shared__ int sums[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  // (p.tile_tokens is at least any request's tokens: a walk over all that it sees)
  {
    const int per = (p.B + THREADS - 1) / THREADS;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= p.B) break;
      const int n = new_tokens(p, b);
      first[b] = mine;
      // (at most 2^24 / 64 sub-tiles of each of 4096 requests)
      if (n > 0) mine += Walk(p, n, keys_of(p, b), 0).cnt;
    }
    int v = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int before = v - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    for (int i = 0; i < per; ++i)
      if (tid * per + i < p.B) first[tid * per + i] += before;
    if (tid == 0) first[p.B] = total;
    __syncthreads();
  }
  const int total = min(first[p.B], p.to.pages);
  const int l16 = lane & 15, r16 = 2 * warp + (lane >> 4);  // column and row of a slice of 16
  for (long long item = blockIdx.x; item < (long long)total * p.Hkv; item += gridDim.x) {
    const int page = (int)(item / p.Hkv), kvh = (int)(item - (long long)page * p.Hkv);
    int lo = 0, hi = p.B - 1;  // the request: the last with first <= page
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= page) lo = mid;
      else hi = mid - 1;
    }
    const Walk w(p, new_tokens(p, lo), keys_of(p, lo), 0);
    const int tile = w.tile(page - first[lo]);
    if (kvh == 0 && tid == 0) p.to.table[(size_t)lo * p.to.cols + tile] = page;
    uint2 kc[4], vc[4];
    int ks[4], vs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k0 = tile * Q_SUB + 16 * i;
      kc[i] = vc[i] = make_uint2(0u, 0u);
      ks[i] = vs[i] = 127;
      if (!w.any(k0, k0 + 16)) continue;  // whatever is written is not seen
      const int idx = div_by(k0, p.page_size, p.inv_page_size);
      const int pg = __ldg(p.table + (size_t)lo * p.table_stride + idx);
      if ((unsigned)pg >= (unsigned)p.num_pages) {  // stands for zeros
        bad = true;
        continue;
      }
      const int row = k0 - idx * p.page_size + r16;
      const long long at = pg * p.page_stride + kvh * p.head_stride + row * p.token_stride + 8 * l16;
      const long long sat = pg * p.scale_page_stride + kvh * p.scale_head_stride +
                            (row >> p.scale_shift);
      kc[i] = *reinterpret_cast<const uint2*>(p.k_pages + at);
      vc[i] = *reinterpret_cast<const uint2*>(p.v_pages + at);
      ks[i] = p.k_scales[sat];
      vs[i] = p.v_scales[sat];
    }
    const size_t to = (((size_t)page * p.Hkv + kvh) * PAGED8_PAGE + r16) * (HEAD_DIM / 8) + l16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t k2 = scale_pair<BF16>(ks[i]), v2 = scale_pair<BF16>(vs[i]);
      uint2 a = values_of<BF16, I8>(kc[i].x, k2), b = values_of<BF16, I8>(kc[i].y, k2);
      reinterpret_cast<uint4*>(p.to.k)[to + 16 * i * (HEAD_DIM / 8)] = make_uint4(a.x, a.y, b.x, b.y);
      a = values_of<BF16, I8>(vc[i].x, v2);
      b = values_of<BF16, I8>(vc[i].y, v2);
      reinterpret_cast<uint4*>(p.to.v)[to + 16 * i * (HEAD_DIM / 8)] = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
  if (first[p.B] > p.to.pages) bad = true;  // (the host's bound rules that out)
  bad = __syncthreads_or(bad);
  if (tid == 0 && bad) atomicExch(&p.to.status[blockIdx.x / PER_SM].code, (unsigned)ATTN_ERR_INVALID_ARG);
}

cudaError_t launch_paged8_expand(bool bf16, bool i8, const Paged8Params& base, const void* k_pages,
                                 const void* v_pages, long long page_stride,
                                 long long head_stride, long long token_stride,
                                 const Expanded& e, cudaStream_t st) {
  ExpandParams p;
  static_cast<Paged8Params&>(p) = base;
  p.tile_tokens = base.Sq;
  p.k_pages = static_cast<const uint8_t*>(k_pages);
  p.v_pages = static_cast<const uint8_t*>(v_pages);
  p.page_stride = page_stride;
  p.head_stride = head_stride;
  p.token_stride = token_stride;
  p.to = e;
  // a status for each four blocks, as many as the attention's CTAs
  cudaError_t r = cudaMemsetAsync(e.status, 0, PAGED_MAX_CTAS * sizeof(DevStatus), st);
  if (r != cudaSuccess) return r;
  const auto kern = bf16 ? (i8 ? k_paged8_expand<true, true> : k_paged8_expand<true, false>)
                         : (i8 ? k_paged8_expand<false, true> : k_paged8_expand<false, false>);
  kern<<<(unsigned)(base.grid * expand_side::PER_SM), expand_side::THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace mab
