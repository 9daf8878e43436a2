// paged_plan.cu -- page tables, slots and offsets of one serving step, built on
// the device from the requests' lengths.
//
// With held = ceil(cached / ps), need = ceil((cached + fresh) / ps) - held and
// the exclusive sums over the requests in order, T0[b] of the new tokens, R0[b]
// of the pages that ended requests return and N0[b] of the needed pages:
//   free_pages[count + R0[b] + i] = table[b, i]           (ended, i < held)
//   table[b, held + i] = free_pages[count' - 1 - N0[b] - i]   (i < need)
//   slot[t] = table[b, x / ps] * ps + x % ps,  x = cached[b] + t - T0[b]
// where count' counts the returned pages too and requests that can never be
// placed need nothing.
//
// Bound: latency.  A step of 512 requests and 16384 tokens reads and writes
// about 0.3 MB.  One launch of one cluster: every CTA loads all lengths and
// scans them on its own (running sums by warp scans), which costs less than
// handing sums from one CTA to another would; the returned pages are on the
// stack at the cluster barrier, which also ends the reading of every input
// that an output may alias; then all threads of the cluster write the tokens'
// entries, a binary search in shared memory finding each token's request.  A
// new page's number is taken from the stack, not from the table entry another
// CTA may be writing.  Page numbers are moved by all threads too, whichever
// request they belong to, by the same search: a warp per request took 35 us for
// one of 100000 tokens that ended among 64 decodes, now 7.5.  Measured (one GB300, ten
// calls replayed in a row): 8 decodes 4.7 us, 512 requests with 16384 tokens
// 10.7 (13.7 with a warp per request and one token at a time).
#include <limits.h>

#include <type_traits>

#include "internal.h"
#include "paged.h"

namespace mab {

namespace {

constexpr int PLAN_THREADS = 1024;
// Pages or tokens that a thread handles at a time: four when it has several,
// whose searches and loads then overlap (512 requests and 16384 tokens: 13.8 us
// one after another, 11.8 so), else one, the shorter code (8 single tokens: 4.8
// us, 4.9 with the longer).
template <int K>
using Width = std::integral_constant<int, K>;
constexpr int PLAN_INTS = 6;  // shared ints per request

struct Sums {
  long long a, b;
};

__device__ __forceinline__ Sums operator+(Sums x, Sums y) { return {x.a + y.a, x.b + y.b}; }
__device__ __forceinline__ Sums shfl_up(Sums x, int d) {
  return {__shfl_up_sync(0xffffffffu, x.a, d), __shfl_up_sync(0xffffffffu, x.b, d)};
}

// Inclusive scan over the block's threads; warp_tot is shared scratch, whose
// last entry holds the block's total afterwards.
__device__ Sums block_scan(Sums v, Sums* warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums u = shfl_up(v, d);
    if (lane >= d) v = v + u;
  }
  __syncthreads();  // the scratch of an earlier scan has been read
  if (lane == 31) warp_tot[warp] = v;
  __syncthreads();
  if (warp == 0) {
    Sums w = warp_tot[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums u = shfl_up(w, d);
      if (lane >= d) w = w + u;
    }
    warp_tot[lane] = w;
  }
  __syncthreads();
  return warp > 0 ? warp_tot[warp - 1] + v : v;
}

// For K x at a time: how many of n non-decreasing ends are <= x, which is the
// first entry whose range holds x.
template <int K>
__device__ __forceinline__ void find(const int* end, int n, const int (&x)[K], int (&at)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) at[k] = 0;
  for (int s = 1 << (31 - __clz(n)); s > 0; s >>= 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at[k] + s <= n && end[at[k] + s - 1] <= x[k]) at[k] += s;
  }
}

__device__ __forceinline__ int clamp_int(long long x) {
  return x > INT_MAX ? INT_MAX : (int)x;
}

}  // namespace

__global__ void __launch_bounds__(PLAN_THREADS, 1) k_paged_plan(const attn_plan_t p) {
  // per request: the ends of its tokens, of the pages that it returns and of
  // those that it needs, where its pages begin among the needed ones less the
  // held ones, its cached tokens, and the pages that it needs (REFUSED, ENDED:
  // none)
  extern __shared__ int smem[];
  int* s_end = smem;
  int* s_ret = s_end + p.B;
  int* s_need = s_ret + p.B;
  int* s_from = s_need + p.B;
  int* s_cached = s_from + p.B;
  int* s_grant = s_cached + p.B;
  constexpr int REFUSED = -1, ENDED = -2;
  __shared__ Sums warp_tot[PLAN_THREADS / 32];
  __shared__ int s_refused, s_granted;
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = (int)cluster_rank(), nranks = (int)gridDim.x;
  const int gtid = rank * PLAN_THREADS + tid, gthreads = nranks * PLAN_THREADS;
  const unsigned ps = (unsigned)p.page_size;
  const long long cap = (long long)p.max_pages * p.page_size;
  const int count = min(max(*p.free_count, 0), p.num_pages);
  auto pages_of = [&](int n) -> int { return (int)(((unsigned)n + ps - 1) / ps); };
  if (tid == 0) s_refused = s_granted = 0;

  Sums carry{0, 0};          // tokens and returned pages of the chunks before
  long long need_carry = 0;  // and needed pages
  for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
    const int b = b0 + tid;
    int cached = 0, fresh = 0, held = 0;
    if (b < p.B) {
      cached = max(p.cached[b], 0);
      fresh = p.fresh[b];
      held = min(pages_of(cached), p.max_pages);
    }
    const bool ended = fresh < 0;
    const Sums upto =
        block_scan(Sums{ended ? 0 : fresh, ended ? held : 0}, warp_tot) + carry;
    carry = carry + warp_tot[PLAN_THREADS / 32 - 1];
    // what can never be placed needs no page
    const bool bad = !ended && ((long long)cached + fresh > cap || upto.a > p.max_tokens);
    const int need = ended || bad ? 0 : pages_of(cached + fresh) - held;
    const long long need_upto = block_scan(Sums{need, 0}, warp_tot).a + need_carry;
    need_carry += warp_tot[PLAN_THREADS / 32 - 1].a;
    if (b < p.B) {
      s_end[b] = clamp_int(upto.a);
      s_ret[b] = clamp_int(upto.b);
      s_cached[b] = cached;
      s_need[b] = clamp_int(need_upto);
      s_from[b] = clamp_int(need_upto - need) - held;
      s_grant[b] = ended ? ENDED : bad ? REFUSED : need;
    }
  }
  const int avail = (int)min(count + carry.b, (long long)p.num_pages);
  // Copies n page numbers, those of request b up to ends[b], spread over all
  // threads of the cluster: at(b, i, x, from, to) says where number i of request
  // b, x of all, comes from and goes to.
  auto spread = [&](const int* ends, int n, auto at) {
    auto go = [&](auto width) {
      constexpr int K = decltype(width)::value;
      for (unsigned x0 = gtid; x0 < (unsigned)n; x0 += K * gthreads) {
        int x[K], b[K], page[K];
        int* to[K];
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = (int)min(x0 + k * gthreads, (unsigned)n - 1);
        find(ends, p.B, x, b);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int* from;
          at(b[k], x[k] - (b[k] > 0 ? ends[b[k] - 1] : 0), x[k], from, to[k]);
          page[k] = *from;
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (x0 + k * gthreads < (unsigned)n) *to[k] = page[k];
      }
    };
    if (n > gthreads) go(Width<4>());
    else go(Width<1>());
  };
  // the returned pages onto the stack
  __syncthreads();
  const int moved = avail - count;
  spread(s_ret, moved, [&](int b, int i, int x, const int*& from, int*& to) {
    from = &p.block_table[(size_t)b * p.table_stride + i];
    to = &p.free_pages[count + x];
  });
  // every input that an output may alias has been read, and the returned
  // pages are on the stack
  cluster_sync();

  // the needs that fit are the first ones in request order: once one does not,
  // no later one does
  for (int b = tid; b < p.B; b += PLAN_THREADS) {
    const int g = s_grant[b];
    if (g > 0) {
      const long long end = (long long)s_from[b] + pages_of(s_cached[b]) + g;
      if (end > avail) s_grant[b] = REFUSED;
      else atomicMax(&s_granted, (int)end);
    }
    if (s_grant[b] == REFUSED) atomicAdd(&s_refused, 1);
  }
  __syncthreads();
  const int total = min(s_end[p.B - 1], p.max_tokens);
  if (gtid == 0) {
    p.cu_seqlens_q[0] = 0;
    *p.free_count_out = avail - s_granted;
    *p.refused = s_refused;
  }
  for (int b = gtid; b < p.B; b += gthreads) {
    const int g = s_grant[b];
    p.cu_seqlens_q[b + 1] = s_end[b];
    p.seqlen_k[b] = g == ENDED     ? 0
                    : g == REFUSED ? s_cached[b]
                                   : s_cached[b] + s_end[b] - (b > 0 ? s_end[b - 1] : 0);
  }
  spread(s_need, s_granted, [&](int b, int i, int x, const int*& from, int*& to) {
    from = &p.free_pages[avail - 1 - x];
    to = &p.block_table[(size_t)b * p.table_stride + pages_of(s_cached[b]) + i];
  });
  auto place = [&](auto width) {
    constexpr int K = decltype(width)::value;
    const unsigned tokens = (unsigned)p.max_tokens;
    for (unsigned t0 = gtid; t0 < tokens; t0 += K * gthreads) {
      int x[K], at[K], pos[K], off[K];
      const int* src[K];  // where the page of a placed token stands
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] = (int)min(t0 + k * gthreads, tokens - 1);
      // the requests: the first whose tokens end past the token
      find(s_end, p.B, x, at);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        src[k] = nullptr;
        pos[k] = -1;
        off[k] = 0;
        if (x[k] < total) {
          const int b = at[k], cached = s_cached[b];
          pos[k] = clamp_int((long long)cached + (x[k] - (b > 0 ? s_end[b - 1] : 0)));
          if (s_grant[b] >= 0) {
            const int i = (int)((unsigned)pos[k] / ps), first = i * (int)ps;
            off[k] = pos[k] - first;
            src[k] = first < cached ? &p.block_table[(size_t)b * p.table_stride + i]
                                    : &p.free_pages[avail - 1 - s_from[b] - i];
          }
        }
      }
      int page[K];
#pragma unroll
      for (int k = 0; k < K; ++k) page[k] = src[k] ? *src[k] : -1;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t0 + k * gthreads < tokens) {
          p.slot_map[x[k]] = page[k] >= 0 && page[k] < p.num_pages
                                 ? (long long)page[k] * p.page_size + off[k]
                                 : -1;
          p.position[x[k]] = pos[k];
        }
    }
  };
  if (p.max_tokens > gthreads) place(Width<4>());
  else place(Width<1>());
}

cudaError_t launch_paged_plan(const attn_plan_t& p, cudaStream_t st) {
  // four tokens a thread before a second CTA pays; at most the portable eight
  const long long n = ((long long)p.max_tokens + 4 * PLAN_THREADS - 1) / (4 * PLAN_THREADS);
  int ranks = 1;
  while (ranks < n && ranks < 8) ranks *= 2;
  const size_t smem = (size_t)p.B * PLAN_INTS * sizeof(int);
  if (smem + sizeof(Sums) * 64 > (48u << 10)) {
    // past what a launch may use unasked; the most that any call needs, so that
    // calls of several host threads do not lower one another's limit
    const cudaError_t e =
        cudaFuncSetAttribute(k_paged_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(PAGED_MAX_B * PLAN_INTS * sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ranks);
  cfg.blockDim = dim3(PLAN_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_paged_plan, p);
}

}  // namespace mab
