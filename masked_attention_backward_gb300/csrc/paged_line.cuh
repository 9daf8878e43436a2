// paged_line.cuh -- the work line of the attentions over a paged cache, shared by
// their kernels: which keys a query tile sees, the line of all units, its cuts, and
// the join of the pieces that the cuts leave.
#pragma once
#include <math.h>

#include "paged.h"
#include "tiles.cuh"

namespace mab {

namespace paged_side {

constexpr float RESCALE_LOG2 = 8.f;  // M moves when a row maximum exceeds it by this
constexpr unsigned LOAD_SLEEP_NS = 100;  // polling period of the loaders' waits

// The warps' shares of the line: cost and units.
template <int NUM_THREADS>
struct LineSums {
  long long cost[NUM_THREADS / 32];
  int units[NUM_THREADS / 32];
};

// A unit's piece, as the loader publishes it.
struct Unit {
  int kvh, off, n, L, tok0;  // kv head; the request's first row, new tokens, keys; first token
  int s0, N;                 // first step and steps of the piece
  int b;                     // the request
  int whole, slot;           // not cut; else the piece's slot
};

enum { TAG_Q = 0x501, TAG_QA, TAG_KV_EMPTY, TAG_KV_FULL, TAG_S_FULL, TAG_P_FULL, TAG_P_FREE,
       TAG_ACC, TAG_ACC_EMPTY, TAG_UNIT_FREE, TAG_XML, TAG_LD_EMPTY, TAG_LD_FULL };

template <int NS>
struct Cyc {
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++i == NS) {
      i = 0;
      ph ^= 1u;
    }
  }
};

// a / b of non-negative numbers, in 32 bits where they fit.
__device__ __forceinline__ long long quot(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// New tokens (none of a request that another kernel of the call takes) and keys of
// request b.
__device__ __forceinline__ int new_tokens(const PagedParams& p, int b) {
  const int n = packed_len(p.cu_q, b, p.total_q, p.Sq);
  return n > p.tokens_lo && n <= p.tokens_hi ? n : 0;
}
__device__ __forceinline__ int keys_of(const PagedParams& p, int b) {
  return min(max(p.seqlen_k[b], 0), p.Skv);
}

// Keys that some row of a query tile sees, [0, f) and [wlo, hi], and the walk
// over their sub-tiles: the nfirst ones that hold first keys, then those from
// lo on.  cnt = 0 when no row sees a key.
struct Walk {
  int f, wlo, hi, nfirst, lo, cnt;
  __device__ __forceinline__ Walk(const PagedParams& p, int n, int L, int tok0) {
    const int x0 = L - n + tok0;
    hi = p.causal ? L - n + min(tok0 + p.tile_tokens, n) - 1 : L - 1;
    wlo = p.causal ? max(x0 - p.window + 1, 0) : 0;
    f = min(p.first, hi + 1);
    lo = wlo / Q_SUB;
    nfirst = min((max(f, 0) + Q_SUB - 1) / Q_SUB, lo);
    cnt = hi < 0 ? 0 : nfirst + hi / Q_SUB - lo + 1;
  }
  __device__ __forceinline__ int tile(int s) const { return s < nfirst ? s : lo + s - nfirst; }
  // whether a row sees any key of [a, b), or every one
  __device__ __forceinline__ bool any(int a, int b) const { return a < f || (a <= hi && b > wlo); }
  __device__ __forceinline__ bool all(int a, int b) const {
    return b <= f || (a >= wlo && b <= hi + 1);
  }
  __device__ __forceinline__ bool sees(int j) const { return j < f || (j >= wlo && j <= hi); }
};

// What a unit costs on the line that is cut: its steps, and PAGED_UNIT_COST
// for its start and end.
__device__ __forceinline__ int unit_cost(const PagedParams& p, int n, int L, int tile) {
  return Walk(p, n, L, tile * p.tile_tokens).cnt + PAGED_UNIT_COST;
}

// The line of all units as every CTA lays it out for itself, in the memory of
// the K / V ring: cost of the requests before each, and their new tokens, keys
// and first rows.
struct Line {
  long long* base;  // [B + 1]
  int *n, *L, *off; // [B]
};
__device__ __forceinline__ Line line_at(void* mem, int B) {
  Line l;
  l.base = static_cast<long long*>(mem);
  l.n = reinterpret_cast<int*>(l.base + B + 1);
  l.L = l.n + B;
  l.off = l.L + B;
  return l;
}
// Lays the line out (all threads of the block); returns the number of parts it
// is cut into: one per unit while there are CTAs, and parts of at least
// PAGED_MIN_COST, since further cuts would cost more to join.
template <int NUM_THREADS>
__device__ int lay_line(const PagedParams& p, const Line& line, LineSums<NUM_THREADS>& sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + NUM_THREADS - 1) / NUM_THREADS;  // requests of a thread
  long long mine = 0;
  int units = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    int n = 0, L = 0, tiles = 0;
    if (b < p.B) {
      n = new_tokens(p, b);
      L = keys_of(p, b);
      tiles = (n + p.tile_tokens - 1) / p.tile_tokens;
      line.n[b] = n;
      line.L[b] = L;
      line.off[b] = packed_off(p.cu_q, b, p.total_q);
    }
    long long w = tiles > 0 ? unit_cost(p, n, L, 0) : 0;
    // several tiles: the warp adds their costs, one request after another
    for (unsigned todo = __ballot_sync(0xffffffffu, tiles > 1); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int sn = __shfl_sync(0xffffffffu, n, src), sL = __shfl_sync(0xffffffffu, L, src);
      const int st = __shfl_sync(0xffffffffu, tiles, src);
      long long sum = 0;
      for (int t = lane; t < st; t += 32) sum += unit_cost(p, sn, sL, t);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == src) w = sum;
    }
    if (b < p.B) line.base[b] = mine;  // of this thread's requests so far
    mine += w * p.Hkv;
    units = min(units + min(tiles, PAGED_MAX_CTAS) * p.Hkv, 1 << 24);
  }
  // exclusive sums over the block
  long long v = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  units = __reduce_add_sync(0xffffffffu, units);
  if (lane == 31) {
    sums.cost[warp] = v;
    sums.units[warp] = units;
  }
  __syncthreads();
  long long total = 0, before = v - mine;
  units = 0;
#pragma unroll
  for (int w = 0; w < NUM_THREADS / 32; ++w) {
    if (w < warp) before += sums.cost[w];
    total += sums.cost[w];
    units = min(units + sums.units[w], 1 << 24);
  }
  for (int i = 0; i < per; ++i)
    if (tid * per + i < p.B) line.base[tid * per + i] += before;
  if (tid == 0) line.base[p.B] = total;
  __syncthreads();
  const long long most = max(total / PAGED_MIN_COST, (long long)units);
  return (int)(most < 1 ? 1 : most < p.grid ? most : p.grid);
}

// Where cut c of `parts` falls (one warp, all lanes alike).
inline __device__ PagedStart cut_of(const PagedParams& p, const Line& line, int parts, int c) {
  const int lane = threadIdx.x & 31;
  PagedStart r;
  r.b = p.B;  // past the last unit
  r.kvh = r.tile = r.step = r.first_cut = r.cuts = r.off = r.n = r.L = 0;
  const long long total = line.base[p.B];
  const long long cut = c < parts ? quot(total * c, parts) : total;
  if (cut >= total) return r;
  int lo = 0, hi = p.B - 1;  // the request that holds the cut: the last with base <= cut
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (line.base[mid] <= cut) lo = mid;
    else hi = mid - 1;
  }
  int b = lo;
  const int n = line.n[b], L = line.L[b];
  const int tiles = (n + p.tile_tokens - 1) / p.tile_tokens;
  const long long head = quot(line.base[b + 1] - line.base[b], p.Hkv);
  int kvh = (int)quot(cut - line.base[b], head);
  // the cut's distance from the start of the head, then of the unit
  long long rem = (cut - line.base[b]) - kvh * head;
  int tile = 0, cost = (int)head;  // of the only tile
  if (tiles > 1) {
    for (int t0 = 0; t0 < tiles; t0 += 32) {
      const int mine = t0 + lane < tiles ? unit_cost(p, n, L, t0 + lane) : 0;
      int v = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
      }
      const unsigned past = __ballot_sync(0xffffffffu, v > rem);
      if (past) {
        const int at = __ffs(past) - 1;
        tile = t0 + at;
        cost = __shfl_sync(0xffffffffu, mine, at);
        rem -= __shfl_sync(0xffffffffu, v, at) - cost;
        break;
      }
      rem -= __shfl_sync(0xffffffffu, v, 31);
    }
  }
  // the unit's own cost stands before its steps; a cut beside its first or
  // last step moves to the unit's edge, and a cut in a unit of less than
  // PAGED_MIN_STEPS to the nearer edge
  int step = (int)rem - PAGED_UNIT_COST;
  if (step <= 0) step = 0;
  const int steps = cost - PAGED_UNIT_COST;
  const bool small = steps < PAGED_MIN_STEPS;
  if (small && 2 * step <= steps) step = 0;
  if (step > 0 && (small || steps - step <= 1)) {
    step = 0;
    if (++tile == tiles) {
      tile = 0;
      if (++kvh == p.Hkv) {
        kvh = 0;
        ++b;
        while (b < p.B && line.base[b + 1] == line.base[b]) ++b;
      }
    }
  }
  // cuts inside the unit: those that lie more than its own cost past its
  // start and more than one step before its end (cut c is at
  // floor(c total / parts))
  if (step > 0) {
    const long long u0 = cut - rem;
    r.first_cut = (int)quot((u0 + PAGED_UNIT_COST + 1) * parts + total - 1, total);
    r.cuts = (int)quot((u0 + cost - 1) * parts + total - 1, total) - r.first_cut;
  }
  r.b = b;
  r.kvh = kvh;
  r.tile = tile;
  r.step = step;
  if (b < p.B) {
    r.off = line.off[b];
    r.n = line.n[b];
    r.L = line.L[b];
  }
  return r;
}

// Columns 4 j .. 4 j + 3 of a row in a warp's share of a piece: 16 columns of a
// row, then the same of the next row, so that a warp that writes a row per lane
// touches 16 lines a store, not 32 (row by row a piece's end took 5000 cycles,
// a unit's 1800), and one that reads a row 8, not 4 (8 columns: 8 and 16; 15
// single tokens and a chunk of 500: 16 columns 43.2 us, rows 44.2; 5 tokens at
// 100000 keys: 8 columns 76.5, 16 75.0, rows 73.5).
__device__ __forceinline__ float4* part_at(float* part, int row, int j) {
  return reinterpret_cast<float4*>(part + ((j >> 2) * 32 + row) * 16) + (j & 3);
}

// Row sum and LSE of a row with maximum m_row and sum l_row, the sink (log2
// domain) joined; *inv is what the row's O is multiplied by.  A row whose sum is
// NaN (a query or a logit that is not finite), or whose sink is, gives NaN.
__device__ __forceinline__ float finish_row(float m_row, float l_row, float sink2, float* inv) {
  if (l_row != l_row || sink2 != sink2) return *inv = l_row + sink2;
  const float top = fmaxf(m_row, sink2);
  *inv = 0.f;
  if (top == -INFINITY) return INFINITY;  // no key and no sink
  const float e = l_row > 0.f ? fast_exp2(m_row - top) : 0.f;
  float lt = l_row * e;
  if (sink2 > -INFINITY) lt += fast_exp2(sink2 - top);
  if (!(lt > 0.f)) return INFINITY;
  *inv = e / lt;
  return (top + log2f(lt)) * 0.6931471805599453f;
}

}  // namespace paged_side

// Adds up the pieces of the units that a cut fell into, in their order, and
// stores them: block (c, y) the rows 8 y .. 8 y + 7 of the unit whose first
// piece is CTA c's last one, a warp per row, 4 columns a lane.  Latency bound:
// one lane per piece for the weights, and the first two pieces' rows on their
// way before those are known (with 16, whose registers left two blocks on an SM,
// 15 single tokens and a chunk of 500 took 43.1 us, 37.9 with two).  (Joined by the
// last warp to finish inside the kernel above, 19 pieces took 5 to 15 us and the
// code slowed its loop by 5 %; with four rows a warp one after another they took
// 15 us more than now.)
template <bool BF16>
__global__ void __launch_bounds__(256) k_paged_join(const PagedParams p) {
  using namespace paged_side;
  const int lane = threadIdx.x & 31, c = (int)blockIdx.x;
  const int row = (int)blockIdx.y * 8 + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (c == p.grid - 1) {
    // the last CTA's part ends with the line: here the CTAs' statuses are
    // passed on, the first one that is not 0 (behind those of a call's earlier kernels)
    if (blockIdx.y == 0 && threadIdx.x < 32) {
      unsigned code = 0, v[(PAGED_MAX_CTAS + 31) / 32];
#pragma unroll
      for (int k = 0; k < (PAGED_MAX_CTAS + 31) / 32; ++k) {
        v[k] = 32 * k + lane < p.grid ? __ldcg(&p.cta_status[32 * k + lane].code) : 0u;
        if (p.more_status && v[k] == 0u && 32 * k + lane < p.grid)
          v[k] = __ldcg(&p.more_status[32 * k + lane].code);
      }
#pragma unroll
      for (int k = (PAGED_MAX_CTAS + 31) / 32 - 1; k >= 0; --k) {
        const unsigned set = __ballot_sync(0xffffffffu, v[k] != 0u);
        if (set) code = __shfl_sync(0xffffffffu, v[k], __ffs(set) - 1);
      }
      if (lane == 0 && !(p.keep_status && p.status->code != 0u)) {
        DevStatus st{};
        st.code = code;
        *p.status = st;
      }
    }
    return;
  }
  const PagedStart u = p.start[c + 1];
  const int tok0 = u.tile * p.tile_tokens;
  if (u.step == 0 || u.first_cut != c + 1 ||
      row >= min(p.tile_tokens, u.n - tok0) * p.group)
    return;
  const int pieces = u.cuts + 1;
  // this row's warp share in piece i (slots: 2 c + 1, then those of the CTAs
  // that go on), columns from 64 half on
  const int sp = row >> 5, r = row & 31;
  auto piece = [&](int i, int half) -> float* {
    return p.part + (size_t)(2 * (c + i) + (i == 0 ? 1 : 0)) * p.slot_floats +
           (2 * sp + half) * PAGED_WARP_FLOATS;
  };
  auto values = [&](int i) -> float4 {
    return __ldcg(part_at(piece(i, lane >> 4), r, lane & 15));
  };
  constexpr int EARLY = 2;
  float4 v[EARLY];
#pragma unroll
  for (int i = 0; i < EARLY; ++i)
    v[i] = i < pieces ? values(i) : make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int MOST = (PAGED_MAX_CTAS + 31) / 32;  // pieces a lane may know
  float m[MOST], l[MOST], top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    m[k] = -INFINITY;
    l[k] = 0.f;
    if (32 * k + lane < pieces) {
      const float2 x =
          __ldcg(reinterpret_cast<const float2*>(piece(32 * k + lane, 0) + PAGED_ML) + r);
      m[k] = x.x;
      l[k] = x.y;
    }
    top = fmaxf(top, m[k]);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    m[k] = l[k] != 0.f ? fast_exp2(m[k] - top) : 0.f;  // the piece's weight from here on
    sum += l[k] * m[k];
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& x, float w) {
    acc.x = fmaf(x.x, w, acc.x);
    acc.y = fmaf(x.y, w, acc.y);
    acc.z = fmaf(x.z, w, acc.z);
    acc.w = fmaf(x.w, w, acc.w);
  };
#pragma unroll
  for (int i = 0; i < EARLY; ++i)
    add(v[i], i < pieces ? __shfl_sync(0xffffffffu, m[0], i) : 0.f);
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    const int end = min(32, pieces - 32 * k);
#pragma unroll 8
    for (int i = k == 0 ? EARLY : 0; i < end; ++i)
      add(values(32 * k + i), __shfl_sync(0xffffffffu, m[k], i));
  }
  const int tl = row / p.group;
  const int tok = u.off + tok0 + tl, head = u.kvh * p.group + row - tl * p.group;
  float inv;
  const float lse = finish_row(top, sum, p.sink ? p.sink[head] * LOG2E : -INFINITY, &inv);
  if (p.lse && lane == 0) p.lse[(size_t)head * p.total_q + tok] = lse;
  uint2 o;
  o.x = pack2<BF16>(acc.x * inv, acc.y * inv);
  o.y = pack2<BF16>(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.out + ((size_t)tok * p.Hq + head) * HEAD_DIM + 4 * lane) = o;
}

template <bool BF16>
cudaError_t launch_paged_join(const PagedParams& p, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)p.grid, (unsigned)((p.tile_rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, k_paged_join<BF16>, p);
}

}  // namespace mab
