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
// CTA may be writing.  Measured (one GB300, replayed): 8 decodes 6.2 us, 512
// requests with 16384 tokens 16.4 us (41 with a thread, not a warp, moving each
// request's pages).
#include <limits.h>

#include "internal.h"
#include "paged.h"

namespace mab {

namespace {

constexpr int PLAN_THREADS = 1024;

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

__device__ __forceinline__ int clamp_int(long long x) {
  return x > INT_MAX ? INT_MAX : (int)x;
}

}  // namespace

__global__ void __launch_bounds__(PLAN_THREADS, 1) k_paged_plan(const attn_plan_t p) {
  // per request: the end of its tokens, its cached tokens, the needed pages of
  // the requests before it, and its own (REFUSED, ENDED: none)
  extern __shared__ int smem[];
  int* s_end = smem;
  int* s_cached = s_end + p.B;
  int* s_need0 = s_cached + p.B;
  int* s_grant = s_need0 + p.B;
  constexpr int REFUSED = -1, ENDED = -2;
  __shared__ Sums warp_tot[PLAN_THREADS / 32];
  __shared__ int s_refused, s_granted;
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = (int)cluster_rank(), nranks = (int)gridDim.x;
  const int gtid = rank * PLAN_THREADS + tid, gthreads = nranks * PLAN_THREADS;
  const unsigned ps = (unsigned)p.page_size;
  const long long cap = (long long)p.max_pages * p.page_size;
  const int count = min(max(*p.free_count, 0), p.num_pages);
  if (tid == 0) s_refused = s_granted = 0;

  Sums carry{0, 0};          // tokens and returned pages of the chunks before
  long long need_carry = 0;  // and needed pages
  for (int b0 = 0; b0 < p.B; b0 += PLAN_THREADS) {
    const int b = b0 + tid;
    int cached = 0, fresh = 0, held = 0;
    if (b < p.B) {
      cached = max(p.cached[b], 0);
      fresh = p.fresh[b];
      held = min((int)(((unsigned)cached + ps - 1) / ps), p.max_pages);
    }
    const bool ended = fresh < 0;
    const Sums upto =
        block_scan(Sums{ended ? 0 : fresh, ended ? held : 0}, warp_tot) + carry;
    carry = carry + warp_tot[PLAN_THREADS / 32 - 1];
    // one warp of the cluster moves an ended request's pages
    for (unsigned todo = __ballot_sync(0xffffffffu, ended && b % nranks == rank); todo;
         todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const long long at = __shfl_sync(0xffffffffu, count + upto.b - held, src);
      const long long room = max(p.num_pages - at, 0ll);
      const int moved = (int)min((long long)__shfl_sync(0xffffffffu, held, src), room);
      const int* row = p.block_table + (size_t)(b - lane + src) * p.table_stride;
#pragma unroll 4
      for (int i = lane; i < moved; i += 32) p.free_pages[at + i] = row[i];
    }
    // what can never be placed needs no page
    const bool bad = !ended && ((long long)cached + fresh > cap || upto.a > p.max_tokens);
    const int need = ended || bad ? 0 : (int)(((unsigned)(cached + fresh) + ps - 1) / ps) - held;
    const long long need_upto = block_scan(Sums{need, 0}, warp_tot).a + need_carry;
    need_carry += warp_tot[PLAN_THREADS / 32 - 1].a;
    if (b < p.B) {
      s_end[b] = clamp_int(upto.a);
      s_cached[b] = cached;
      s_need0[b] = clamp_int(need_upto - need);
      s_grant[b] = ended ? ENDED : bad ? REFUSED : need;
    }
  }
  const int avail = (int)min(count + carry.b, (long long)p.num_pages);
  // every input that an output may alias has been read, and the returned
  // pages are on the stack
  cluster_sync();

  // the needs that fit are the first ones in request order: once one does not,
  // no later one does
  for (int b = tid; b < p.B; b += PLAN_THREADS) {
    const int g = s_grant[b];
    if (g > 0 && (long long)s_need0[b] + g > avail) s_grant[b] = REFUSED;
    if (s_grant[b] == REFUSED) atomicAdd(&s_refused, 1);
    if (s_grant[b] > 0) atomicMax(&s_granted, s_need0[b] + g);
  }
  __syncthreads();
  const int total = min(s_end[p.B - 1], p.max_tokens);
  if (gtid == 0) {
    p.cu_seqlens_q[0] = 0;
    *p.free_count_out = avail - s_granted;
    *p.refused = s_refused;
  }
  // requests in whole warps: one that gets many pages has all lanes append them
  for (int b0 = gtid - lane; b0 < p.B; b0 += gthreads) {
    const int b = b0 + lane;
    int g = 0, held = 0, need0 = 0;
    if (b < p.B) {
      const int cached = s_cached[b];
      g = s_grant[b];
      need0 = s_need0[b];
      p.cu_seqlens_q[b + 1] = s_end[b];
      p.seqlen_k[b] = g == ENDED     ? 0
                      : g == REFUSED ? cached
                                     : cached + s_end[b] - (b > 0 ? s_end[b - 1] : 0);
      held = (int)(((unsigned)cached + ps - 1) / ps);
    }
    auto append = [&](int to, int have, int first, int i) {
      p.block_table[(size_t)to * p.table_stride + have + i] = p.free_pages[avail - 1 - first - i];
    };
    if (g <= 4)
      for (int i = 0; i < g; ++i) append(b, held, need0, i);
    for (unsigned todo = __ballot_sync(0xffffffffu, g > 4); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int n = __shfl_sync(0xffffffffu, g, src), h = __shfl_sync(0xffffffffu, held, src);
      const int first = __shfl_sync(0xffffffffu, need0, src);
      for (int i = lane; i < n; i += 32) append(b0 + src, h, first, i);
    }
  }
  for (int t = gtid; t < p.max_tokens; t += gthreads) {
    long long slot = -1;
    int pos = -1;
    if (t < total) {
      // the first request whose tokens end past t
      int lo = 0, hi = p.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_end[mid] > t) hi = mid;
        else lo = mid + 1;
      }
      const int cached = s_cached[lo];
      pos = clamp_int((long long)cached + (t - (lo > 0 ? s_end[lo - 1] : 0)));
      if (s_grant[lo] >= 0) {
        const int held = (int)(((unsigned)cached + ps - 1) / ps);
        const int i = (int)((unsigned)pos / ps);
        const int page = i < held ? p.block_table[(size_t)lo * p.table_stride + i]
                                  : p.free_pages[avail - 1 - s_need0[lo] - (i - held)];
        if (page >= 0 && page < p.num_pages)
          slot = (long long)page * p.page_size + pos - i * p.page_size;
      }
    }
    p.slot_map[t] = slot;
    p.position[t] = pos;
  }
}

cudaError_t launch_paged_plan(const attn_plan_t& p, cudaStream_t st) {
  // four tokens a thread before a second CTA pays; at most the portable eight
  const long long n = ((long long)p.max_tokens + 4 * PLAN_THREADS - 1) / (4 * PLAN_THREADS);
  int ranks = 1;
  while (ranks < n && ranks < 8) ranks *= 2;
  const size_t smem = (size_t)p.B * 4 * sizeof(int);
  if (smem + sizeof(Sums) * 64 > (48u << 10)) {
    // past what a launch may use unasked; the most that any call needs, so that
    // calls of several host threads do not lower one another's limit
    const cudaError_t e =
        cudaFuncSetAttribute(k_paged_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(PAGED_MAX_B * 4 * sizeof(int)));
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
