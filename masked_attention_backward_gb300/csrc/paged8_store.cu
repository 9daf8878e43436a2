// paged8_store.cu -- keys and values of new tokens into their slots of an 8-bit
// cache, and rows of the cache back to 16 bits.
//
// A block of tokens of one kv head has one scale 2^e, e the least that its
// largest magnitude fits (quant8.cuh).  The tokens that a call brings for one
// block are a run: consecutive rows of k and v with consecutive slots.  A run
// that begins at its block's row 0 begins the block anew, whatever stood there;
// one that begins at row r0 > 0 joins r0 earlier rows: e is then the larger of
// the block's and the run's, and where it grew the earlier rows' codes are
// rounded again, in units of the new scale.  Values are taken in units of 2^e
// exactly and rounded once, to nearest even.
//
// Bound: HBM (512 bytes read and 256 written a token and head, both tensors; the
// other way when read back), a launch for single tokens.
// Measured (one GB300, 8 heads): 16800 tokens to int8 with a scale each, 16-token pages,
// 19.6 us, 5.3 TB/s (two rows a half-warp 23.3 when this took 20.5), 76 % of the issue
// slots; into 64-token pages 22.5, and with a scale for 16, 32 or 64 tokens 30, 32 and 37
// (3.4 to 2.8 TB/s: a run's rows past the 16th are read twice); 32 tokens of blocks that
// hold others 3.3 us; 70000 rows of 64-token blocks back to 16 bits 68 us, 6.3 TB/s; 16800
// 14.7.
#include "paged8.h"
#include "quant8.cuh"

namespace mab {

namespace {
constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

// Largest magnitude of the eight 16-bit values of v as a bit pattern: their
// patterns without the sign grow with the magnitude, infinity and NaN on top.
__device__ __forceinline__ uint32_t top_of(uint4 v) {
  constexpr uint32_t M = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(v.x & M, v.y & M), __vmaxu2(v.z & M, v.w & M));
}
// ... of a half-warp's rows, on all its lanes.
__device__ __forceinline__ uint32_t half_max(uint32_t m, unsigned mask) {
  m = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(mask, m, d));
  return m;
}

// The scale byte that the pattern `top` needs.
template <bool BF16, bool I8>
__device__ __forceinline__ int scale_of(uint32_t top) {
  if (top >= (BF16 ? 0x7f80u : 0x7c00u)) return SCALE_NAN;
  return scale_for<BF16, I8>(unpack2<BF16>(top).x);
}

// Eight 16-bit values to their codes under scale byte s (zeros under SCALE_NAN,
// where they mean nothing).
template <bool BF16, bool I8>
__device__ __forceinline__ uint2 quantise(uint4 v, int s) {
  if (s == SCALE_NAN) return make_uint2(0u, 0u);
  const float unit = exp2_int(127 - s);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // (two ways, so that the usual one has product and int8 rounding in one instruction:
  // the product is exact)
  auto codes = [&](auto top) {
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 x = unpack2<BF16>(w[2 * i]), y = unpack2<BF16>(w[2 * i + 1]);
      r[i] = codes_of<I8>(top(x.x * unit), top(x.y * unit), top(y.x * unit), top(y.y * unit));
    }
    return make_uint2(r[0], r[1]);
  };
  if (s >= CodeRange<BF16, I8>::big) {
    constexpr float T = CodeRange<BF16, I8>::big_top;
    return codes([](float f) { return fminf(fmaxf(f, -T), T); });
  }
  return codes([](float f) { return f; });
}

// Eight codes moved from scale byte s0 to s1 > s0.  (int8's 127 becomes 63.5, which rounds to
// 64: held back like the new rows' codes where 64 has no finite value.  e4m3's 448 becomes 224,
// below its 240.)
template <bool BF16, bool I8>
__device__ __forceinline__ uint2 rescale(uint2 c, int s0, int s1) {
  const float unit = exp2_int(max(s0 - s1, -126));
  const float top = s1 >= CodeRange<BF16, I8>::big ? CodeRange<BF16, I8>::big_top : 127.f;
  uint32_t r[2];
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f[4];
    const uint2 v = word_pairs<false, I8>(w[i]);
    const float2 x = unpack2<false>(v.x), y = unpack2<false>(v.y);
    f[0] = x.x * unit;
    f[1] = x.y * unit;
    f[2] = y.x * unit;
    f[3] = y.y * unit;
    if (I8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = fminf(fmaxf(f[j], -top), top);
    }
    r[i] = codes_of<I8>(f[0], f[1], f[2], f[3]);
  }
  return make_uint2(r[0], r[1]);
}

}  // namespace

// A scale a token: a half-warp per row of K and the same row of V.
template <bool BF16, bool I8>
__global__ void __launch_bounds__(THREADS)
k_paged8_store_rows(const Pages8 pg, const uint4* __restrict__ k, const uint4* __restrict__ v,
                    long long k_stride, long long v_stride,
                    const long long* __restrict__ slot_map, int rows, uint8_t* __restrict__ kp,
                    uint8_t* __restrict__ vp, uint8_t* __restrict__ ks,
                    uint8_t* __restrict__ vs) {
  const int l16 = threadIdx.x & 15;
  const unsigned mask = 0xffffu << (threadIdx.x & 16);
  const int row = (int)(blockIdx.x * (THREADS / 16) + (threadIdx.x >> 4));
  if (row >= rows) return;
  const int t = row / pg.Hkv, h = row - t * pg.Hkv;
  const long long slot = slot_map[t];
  if (slot < 0 || slot >= (long long)pg.num_pages * pg.page_size) return;
  const unsigned page = (unsigned)slot / pg.page_size, off = (unsigned)slot - page * pg.page_size;
  const uint4 a = k[t * k_stride + h * 16 + l16];
  const uint4 b = v[t * v_stride + h * 16 + l16];
  const int sa = scale_of<BF16, I8>(half_max(top_of(a), mask));
  const int sb = scale_of<BF16, I8>(half_max(top_of(b), mask));
  const long long at = page * pg.page_stride + h * pg.head_stride + off * pg.token_stride;
  reinterpret_cast<uint2*>(kp + at)[l16] = quantise<BF16, I8>(a, sa);
  reinterpret_cast<uint2*>(vp + at)[l16] = quantise<BF16, I8>(b, sb);
  const long long sat = page * pg.scale_page_stride + h * pg.scale_head_stride + off;
  if (l16 == 0) ks[sat] = (uint8_t)sa;
  if (l16 == 1) vs[sat] = (uint8_t)sb;
}

// A scale for 16, 32 or 64 tokens: a warp per run, head and tensor, its halves on
// alternate rows.  A warp looks through `span` (a power of two up to 32)
// consecutive tokens for the first ones of runs and takes these runs to their
// ends.  The first 16 rows of a run stay in registers between the search for the
// maximum and the rounding; the others are read again.
template <bool BF16, bool I8>
__global__ void __launch_bounds__(THREADS)
k_paged8_store_blocks(const Pages8 pg, const uint4* __restrict__ k, const uint4* __restrict__ v,
                      long long k_stride, long long v_stride,
                      const long long* __restrict__ slot_map, int T, int span, long long warps,
                      uint8_t* __restrict__ kp, uint8_t* __restrict__ vp,
                      uint8_t* __restrict__ ks, uint8_t* __restrict__ vs) {
  const int lane = threadIdx.x & 31, l16 = lane & 15, half = lane >> 4;
  const long long w = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (w >= warps) return;
  const int kinds = 2 * pg.Hkv;
  const int t0 = (int)(w / kinds) * span, kind = (int)(w % kinds);
  const int h = kind >> 1;
  const bool is_v = kind & 1;
  const long long slots = (long long)pg.num_pages * pg.page_size;
  // lane l looks at token t0 + l: does a run begin there?
  auto slot_at = [&](int t) -> long long {
    const long long s = t < T ? slot_map[t] : -1;
    return s < slots ? s : -1;
  };
  // whether token t goes on with the run of the one before it
  auto joins = [&](long long before, long long s) {
    return before >= 0 && s == before + 1 && (s >> pg.shift) == (before >> pg.shift);
  };
  bool begins = false;
  long long mine = -1;
  if (lane < span) {
    mine = slot_at(t0 + lane);
    begins = mine >= 0 && (t0 + lane == 0 || !joins(slot_at(t0 + lane - 1), mine));
  }
  const uint4* x = (is_v ? v : k) + h * 16 + l16;
  const long long x_stride = is_v ? v_stride : k_stride;
  uint8_t* pages = is_v ? vp : kp;
  uint8_t* scales = is_v ? vs : ks;
  for (unsigned todo = __ballot_sync(0xffffffffu, begins); todo; todo &= todo - 1) {
    const int i = __ffs(todo) - 1, t = t0 + i;
    const long long slot = __shfl_sync(0xffffffffu, mine, i);
    const int r0 = (int)(slot & (pg.block - 1));
    // its length: tokens that go on with it, up to the block's end
    int n = 1;
    for (int d = 1; d < pg.block - r0; d += 32) {
      const bool on = d + lane < pg.block - r0 && slot_at(t + d + lane) == slot + d + lane;
      const unsigned off = ~__ballot_sync(0xffffffffu, on);
      const int run = off ? __ffs(off) - 1 : 32;
      n += run;
      if (run < 32) break;
    }
    const unsigned page = (unsigned)slot / pg.page_size,
                   row = (unsigned)slot - page * pg.page_size;
    uint8_t* at = pages + page * pg.page_stride + h * pg.head_stride + row * pg.token_stride;
    uint8_t* sat = scales + page * pg.scale_page_stride + h * pg.scale_head_stride +
                   (row >> pg.shift);
    const uint4* src = x + t * x_stride;
    const int had = r0 > 0 ? *sat : 0;
    uint4 keep[8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (2 * j + half < n) keep[j] = src[(2 * j + half) * x_stride];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (2 * j + half < n) top = __vmaxu2(top, top_of(keep[j]));
    for (int j0 = 16; j0 < n; j0 += 16) {
      uint4 y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + 2 * j + half < n) y[j] = src[(j0 + 2 * j + half) * x_stride];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + 2 * j + half < n) top = __vmaxu2(top, top_of(y[j]));
    }
    top = half_max(top, 0xffffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
    const int s = max(scale_of<BF16, I8>(top), had);
    if (r0 > 0 && s > had && s != SCALE_NAN) {
      // the rows that were there, in units of the new scale
      for (int r = half; r < r0; r += 2) {
        uint2* c = reinterpret_cast<uint2*>(at - (r0 - r) * pg.token_stride) + l16;
        *c = rescale<BF16, I8>(*c, had, s);
      }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *sat = (uint8_t)s;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (2 * j + half < n)
        reinterpret_cast<uint2*>(at + (2 * j + half) * pg.token_stride)[l16] =
            quantise<BF16, I8>(keep[j], s);
    for (int j0 = 16; j0 < n; j0 += 16) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + 2 * j + half < n)
          reinterpret_cast<uint2*>(at + (j0 + 2 * j + half) * pg.token_stride)[l16] =
              quantise<BF16, I8>(src[(j0 + 2 * j + half) * x_stride], s);
    }
  }
}

cudaError_t launch_paged8_store(bool bf16, bool i8, const Pages8& pg, int T, const void* k,
                                const void* v, long long k_stride, long long v_stride,
                                const long long* slot_map, void* k_pages, void* v_pages,
                                uint8_t* k_scales, uint8_t* v_scales, cudaStream_t st) {
  const uint4* k4 = static_cast<const uint4*>(k);
  const uint4* v4 = static_cast<const uint4*>(v);
  uint8_t* kp = static_cast<uint8_t*>(k_pages);
  uint8_t* vp = static_cast<uint8_t*>(v_pages);
  if (pg.block == 1) {
    const int rows = T * pg.Hkv, per = THREADS / 16;
    const auto kern = bf16 ? (i8 ? k_paged8_store_rows<true, true> : k_paged8_store_rows<true, false>)
                           : (i8 ? k_paged8_store_rows<false, true>
                                 : k_paged8_store_rows<false, false>);
    kern<<<(unsigned)(((long long)rows + per - 1) / per), THREADS, 0, st>>>(
        pg, k4, v4, k_stride / 8, v_stride / 8, slot_map, rows, kp, vp, k_scales, v_scales);
    return cudaGetLastError();
  }
  // as many tokens a warp as leave 32 warps an SM
  const long long kinds = 2ll * pg.Hkv;
  int span = 1;
  while (span < 32 && T * kinds / (2 * span) >= 32 * 152) span *= 2;
  const long long warps = (T + span - 1) / span * kinds;
  const auto kern = bf16 ? (i8 ? k_paged8_store_blocks<true, true>
                               : k_paged8_store_blocks<true, false>)
                         : (i8 ? k_paged8_store_blocks<false, true>
                               : k_paged8_store_blocks<false, false>);
  kern<<<(unsigned)((warps + WARPS - 1) / WARPS), THREADS, 0, st>>>(
      pg, k4, v4, k_stride / 8, v_stride / 8, slot_map, T, span, warps, kp, vp, k_scales,
      v_scales);
  return cudaGetLastError();
}

// Token t of the packed rows is position start[b] + t - cu[b] of request b: a
// warp per token, its request found by all lanes (a boundary each, 32-fold
// search), a half-warp per row.
template <bool BF16, bool I8>
__global__ void __launch_bounds__(THREADS)
k_paged8_load(const Pages8 pg, int B, int total, const int* __restrict__ start,
              const int* __restrict__ cu, const int* __restrict__ table, int table_stride,
              int max_pages, const uint8_t* __restrict__ kp, const uint8_t* __restrict__ vp,
              const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vs,
              uint4* __restrict__ k, uint4* __restrict__ v) {
  const int lane = threadIdx.x & 31, l16 = lane & 15, half = lane >> 4;
  const long long t = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (t >= total) return;
  // the last b with cu[b] <= t (the offsets ascend; of those before the first,
  // none)
  int lo = 0, len = B;  // b in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int i = lo + lane * step;
    const unsigned le =
        __ballot_sync(0xffffffffu, lane * step < len && __ldg(cu + i) <= (int)t);
    const int at = le ? 31 - __clz(le) : 0;
    const int end = lo + len;
    lo += at * step;
    len = min(step, end - lo);
  }
  const int first = __ldg(cu + lo);
  if (t < first || t >= __ldg(cu + lo + 1)) return;  // no request's
  const long long x = (start ? max(__ldg(start + lo), 0) : 0) + (t - first);
  const long long col = x / pg.page_size;
  const int row = (int)(x - col * pg.page_size);
  const int page = col < max_pages ? __ldg(table + (long long)lo * table_stride + col) : -1;
  const bool there = (unsigned)page < (unsigned)pg.num_pages;
  const long long at = page * pg.page_stride + row * pg.token_stride;
  const long long sat = page * pg.scale_page_stride + (row >> pg.shift);
  uint4* out = (half ? v : k) + t * pg.Hkv * 16 + l16;
  const uint8_t* codes = (half ? vp : kp) + at + l16 * 8;
  const uint8_t* scales = (half ? vs : ks) + sat;
  for (int h0 = 0; h0 < pg.Hkv; h0 += 4) {
    uint2 c[4];
    int s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = make_uint2(0u, 0u);
      s[j] = 127;
      if (there && h0 + j < pg.Hkv) {
        c[j] = *reinterpret_cast<const uint2*>(codes + (h0 + j) * pg.head_stride);
        s[j] = scales[(h0 + j) * pg.scale_head_stride];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (h0 + j < pg.Hkv) {
        const uint32_t s2 = scale_pair<BF16>(s[j]);
        const uint2 a = values_of<BF16, I8>(c[j].x, s2), b = values_of<BF16, I8>(c[j].y, s2);
        out[(h0 + j) * 16] = make_uint4(a.x, a.y, b.x, b.y);
      }
  }
}

cudaError_t launch_paged8_load(bool bf16, bool i8, const Pages8& pg, int B, int total,
                               const int* start, const int* cu, const int* table,
                               int table_stride, int max_pages, const void* k_pages,
                               const void* v_pages, const uint8_t* k_scales,
                               const uint8_t* v_scales, void* k, void* v, cudaStream_t st) {
  const auto kern = bf16 ? (i8 ? k_paged8_load<true, true> : k_paged8_load<true, false>)
                         : (i8 ? k_paged8_load<false, true> : k_paged8_load<false, false>);
  kern<<<(unsigned)(((long long)total + WARPS - 1) / WARPS), THREADS, 0, st>>>(
      pg, B, total, start, cu, table, table_stride, max_pages,
      static_cast<const uint8_t*>(k_pages), static_cast<const uint8_t*>(v_pages), k_scales,
      v_scales, static_cast<uint4*>(k), static_cast<uint4*>(v));
  return cudaGetLastError();
}

}  // namespace mab
