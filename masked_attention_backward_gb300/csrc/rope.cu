// rope.cu -- rotary positions: queries and keys turned by their positions, and
// their gradients turned back (declared in include/maskattn.h).
//
// Pair i of a row at position x is turned by the angle x w_i:
//   y1 = a (x1 cos - x2 sin),  y2 = a (x2 cos + x1 sin);
// the backward is the transpose, the same with the angle negated.  w_i comes as
// turns a position in 64-bit fixed point, so x w_i is one integer product whose
// overflow drops the whole turns: what is left is exact to 2^-64 x of a turn at
// any position, with no table to read.  The fraction goes through sincospif as a
// float (relative error 2^-24) and cos and sin are kept in fp32; the rows are
// rounded once.
//
// Bound: HBM, each row read and written once.  A thread owns 16 elements (eight
// pairs, two 16-byte vectors) of the rows of one token and walks that token's
// heads, so its eight angles are computed once; eight lanes cover a row.  (Two heads
// at a time and 24 blocks an SM; four at a time and 8 blocks: 29.1 and 18.6 us below,
// and 16 blocks 29.0 and 15.9.)
// Measured (one GB300): 8192 tokens of 40 heads, bf16, 27.8 us, 6.0 TB/s; the gradient of
// 5003 packed tokens of 32 heads, half of the head, fp16, 14.9 us, 5.5 TB/s; eight tokens
// 2.7 us, the launch.
#include <math.h>

#include "internal.h"
#include "maskattn.h"

namespace mab {

namespace rope_side {
constexpr int THREADS = 128;
constexpr int TOKENS = THREADS / 8;  // of a block
constexpr int AHEAD = 2;             // heads whose rows a thread has in flight
constexpr int BLOCKS = 24;           // of an SM, where there are heads enough
}  // namespace rope_side

struct RopeTensor {
  const uint16_t* x;
  uint16_t* y;
  int heads;
  long long xb, xh, xt, yb, yh, yt;  // strides in elements
};
struct RopeParams {
  RopeTensor q, k;  // k.heads = 0: none
  const unsigned long long* turns;
  const int* position;  // or nullptr: counted
  long long position_stride;
  float factor;
  int S, rot, interleaved, inverse;
  int heads_per_block;  // of q's and k's together
};

template <bool BF16>
__global__ void __launch_bounds__(rope_side::THREADS) k_rope(const RopeParams p) {
  using namespace rope_side;
  const int c = threadIdx.x & 7;
  const long long t = (long long)blockIdx.x * TOKENS + (threadIdx.x >> 3);
  const long long b = blockIdx.z;
  if (t >= p.S) return;
  const int h0 = (int)blockIdx.y * p.heads_per_block;
  const int h1 = min(h0 + p.heads_per_block, p.q.heads + p.k.heads);
  const bool turned = 16 * c < p.rot;
  // the thread's two vectors of a row
  const int at0 = turned && !p.interleaved ? 8 * c : 16 * c;
  const int at1 = turned && !p.interleaved ? p.rot / 2 + 8 * c : 16 * c + 8;
  auto src = [&](int h) -> const uint16_t* {
    const bool in_q = h < p.q.heads;
    const RopeTensor& r = in_q ? p.q : p.k;
    return r.x + b * r.xb + t * r.xt + (long long)(in_q ? h : h - p.q.heads) * r.xh;
  };
  auto dst = [&](int h) -> uint16_t* {
    const bool in_q = h < p.q.heads;
    const RopeTensor& r = in_q ? p.q : p.k;
    return r.y + b * r.yb + t * r.yt + (long long)(in_q ? h : h - p.q.heads) * r.yh;
  };
  uint4 v0[AHEAD], v1[AHEAD];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (h + i < h1) {
        const uint16_t* x = src(h + i);
        v0[i] = *reinterpret_cast<const uint4*>(x + at0);
        v1[i] = *reinterpret_cast<const uint4*>(x + at1);
      }
  };
  const int pos = p.position ? p.position[b * p.position_stride + t] : (int)t;
  if (pos < 0) return;  // no token: its rows are left
  load(h0);             // under way while the angles are computed
  float cs[8], sn[8];
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // half turns in [-1, 1)
      const unsigned long long frac = p.turns[8 * c + i] * (unsigned long long)(unsigned)pos;
      const float half = (float)(long long)frac * 0x1p-63f;
      sincospif(half, &sn[i], &cs[i]);
      cs[i] *= p.factor;
      sn[i] *= p.inverse ? -p.factor : p.factor;
    }
  }
  for (int h = h0; h < h1; h += AHEAD) {
    if (h > h0) load(h);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (h + i >= h1) break;
      uint32_t a[4] = {v0[i].x, v0[i].y, v0[i].z, v0[i].w};
      uint32_t d[4] = {v1[i].x, v1[i].y, v1[i].z, v1[i].w};
      if (turned) {
        if (p.interleaved) {
          // the pairs of each vector are its words
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = unpack2<BF16>(a[j]), y = unpack2<BF16>(d[j]);
            a[j] = pack2<BF16>(x.x * cs[j] - x.y * sn[j], x.y * cs[j] + x.x * sn[j]);
            d[j] = pack2<BF16>(y.x * cs[4 + j] - y.y * sn[4 + j],
                               y.y * cs[4 + j] + y.x * sn[4 + j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = unpack2<BF16>(a[j]), y = unpack2<BF16>(d[j]);
            a[j] = pack2<BF16>(x.x * cs[2 * j] - y.x * sn[2 * j],
                               x.y * cs[2 * j + 1] - y.y * sn[2 * j + 1]);
            d[j] = pack2<BF16>(y.x * cs[2 * j] + x.x * sn[2 * j],
                               y.y * cs[2 * j + 1] + x.y * sn[2 * j + 1]);
          }
        }
      }
      uint16_t* y = dst(h + i);
      *reinterpret_cast<uint4*>(y + at0) = make_uint4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<uint4*>(y + at1) = make_uint4(d[0], d[1], d[2], d[3]);
    }
  }
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows of 16-byte vectors; rows that are written must not share elements.
attn_status_t rope_tensor(const attn_rope_tensor_t* t, int B, int S, RopeTensor* out) {
  if (!t->x || !t->y || !aligned(t->x, 16) || !aligned(t->y, 16) || t->heads < 1 ||
      t->heads > 65535)
    return ATTN_ERR_INVALID_ARG;
  const int n[3] = {B, t->heads, S};
  const long long xs[3] = {t->x_batch, t->x_head, t->x_token};
  const long long ys[3] = {t->y_batch, t->y_head, t->y_token};
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;  // never used
    if (xs[i] < 0 || xs[i] % 8 != 0 || xs[i] >= (1ll << 40) || ys[i] < HEAD_DIM ||
        ys[i] % 8 != 0 || ys[i] >= (1ll << 40))
      return ATTN_ERR_INVALID_ARG;
  }
  *out = {static_cast<const uint16_t*>(t->x), static_cast<uint16_t*>(t->y), t->heads,
          B > 1 ? xs[0] : 0, t->heads > 1 ? xs[1] : 0, S > 1 ? xs[2] : 0,
          B > 1 ? ys[0] : 0, t->heads > 1 ? ys[1] : 0, S > 1 ? ys[2] : 0};
  return ATTN_OK;
}

}  // namespace
}  // namespace mab

using namespace mab;

extern "C" attn_status_t attn_rope(const attn_rope_desc_t* rope, int dtype, int B, int S,
                                   const attn_rope_tensor_t* q, const attn_rope_tensor_t* k,
                                   const int* position, long long position_stride, int inverse,
                                   void* stream) {
  if (!rope || !q || (dtype != ATTN_F16 && dtype != ATTN_BF16) || B < 1 || B > 65535 || S < 0 ||
      !rope->turns || !aligned(rope->turns, 8) || rope->rotary_dim < 2 ||
      rope->rotary_dim > HEAD_DIM || rope->rotary_dim % 2 != 0 || !isfinite(rope->factor) ||
      (position && (!aligned(position, 4) || position_stride < 0)))
    return ATTN_ERR_INVALID_ARG;
  if (rope->rotary_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if (S == 0) return ATTN_OK;
  RopeParams p = {};
  attn_status_t r = rope_tensor(q, B, S, &p.q);
  if (r == ATTN_OK && k) r = rope_tensor(k, B, S, &p.k);
  if (r != ATTN_OK) return r;
  p.turns = reinterpret_cast<const unsigned long long*>(rope->turns);
  p.position = position;
  p.position_stride = position_stride;
  p.factor = rope->factor;
  p.S = S;
  p.rot = rope->rotary_dim;
  p.interleaved = rope->interleaved != 0;
  p.inverse = inverse != 0;
  const int heads = p.q.heads + p.k.heads;
  const long long tiles = ((long long)S + rope_side::TOKENS - 1) / rope_side::TOKENS;
  // heads a block walks: as many as leave BLOCKS an SM, at least AHEAD
  const long long parts = (rope_side::BLOCKS * 152 + tiles * B - 1) / (tiles * B);
  const int most = (heads + rope_side::AHEAD - 1) / rope_side::AHEAD;
  const int groups = (int)(parts < most ? parts : most);
  p.heads_per_block = ((heads + groups - 1) / groups + rope_side::AHEAD - 1) / rope_side::AHEAD *
                      rope_side::AHEAD;
  const dim3 grid((unsigned)tiles, (unsigned)((heads + p.heads_per_block - 1) / p.heads_per_block),
                  (unsigned)B);
  const auto kern = dtype == ATTN_BF16 ? k_rope<true> : k_rope<false>;
  kern<<<grid, rope_side::THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
