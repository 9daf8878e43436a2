// paged8_rows.cu -- attention of a few new tokens over an 8-bit paged cache.
//
// The same operation, work line, cuts and join as paged_fwd.cuh, for calls whose
// tokens and query heads of a kv head make few rows (single tokens, a few
// speculated ones).  Bound: HBM, 256 bytes a key and kv head.  At the copy rate an
// SM gets 23 codes a cycle, and the way through shared memory that the matrix
// unit's tiles need (codes in, codes out, 16-bit tile in, tile out: 96 KB a step
// of 64 keys, 750 cycles of 700) does not keep up.  So here a code goes from HBM
// to shared memory and to registers, and becomes an operand there:
//   S^T = K Q^T  with the warp's 16 keys as the rows of m16n8k16, so that a
//       thread's codes of a key, whatever their order in d, are its A fragments
//       when Q's B fragments take the same order (kept in registers, a unit long);
//   O^T += V^T P^T  with 16 of d as rows: a thread takes 16 bytes of each of four
//       keys, and a byte of two keys makes an A register; the scores, 16 keys by
//       8 rows, become B fragments by a transposition of 8 x 8 blocks.
// K's scale multiplies the score; V's the probability (bf16, exactly) or the
// values (f16, whose small probabilities times a small scale would lose bits).
//
// Warps share nothing while they walk a unit's keys, 16 at a time each in turn:
// every thread brings its own 16-byte pieces by cp.async into its own slots,
// which are free of bank conflicts and need no barrier.  At a piece's end the
// warps' O, M and l meet in shared memory.
#include "paged_fwd.cuh"

namespace mab {

namespace rows_side {

using namespace paged_side;

template <int NT>
struct Rows {
  static constexpr int WARPS = NT == 1 ? 16 : 8;
  static constexpr int STAGES = NT == 1 ? 2 : 4;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int N = 8 * NT;         // rows of a unit at most
  static constexpr int O_STRIDE = 132;     // floats: rows on other banks
  struct Smem {
    uint4 ring[WARPS][STAGES][8][32];      // K: 4 pieces a lane, V: 4
    uint32_t scales[WARPS][STAGES][8];     // a scale a token: 16 bytes of K, 16 of V
    float O[WARPS][N][O_STRIDE];
    float ml[WARPS][N][2];                 // (M, l)
    LineSums<THREADS> sums;
    PagedStart cut[2];
    unsigned bad_page;
  };
  static_assert((PAGED_MAX_B + 1) * 8 + PAGED_MAX_B * 12 <= sizeof(Smem::ring),
                "the line of the most requests fits the ring");
  static_assert(sizeof(Smem) + 1024 <= 232448, "over the shared memory a CTA may use");
};

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 16-bit matrix, a row a quad of lanes, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16 bytes to shared memory, or zeros where `there` is false (then nothing is read).
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most n of the committed groups are pending (n < 4).
__device__ __forceinline__ void copies_wait(int n) {
  if (n <= 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// The pieces of a CTA's part of the line, one after another (a warp, all lanes
// alike; lane i holds the lengths of request b_base + i).
struct Pieces {
  PagedStart at, end;
  int cta, b_base, l_off, l_n, l_L;

  __device__ __forceinline__ Pieces(const PagedStart& a, const PagedStart& e, int c)
      : at(a), end(e), cta(c), b_base(a.b - 32), l_off(0), l_n(0), l_L(0) {}

  // N < 0: none is left.
  __device__ __forceinline__ Unit next(const PagedParams& p) {
    Unit u;
    u.N = -1;
    const bool in_end = at.b == end.b && at.kvh == end.kvh;
    if (at.b >= p.B || (in_end && end.step <= at.step)) return u;
    u.b = at.b;
    u.kvh = at.kvh;
    u.off = at.off;
    u.n = at.n;
    u.L = at.L;
    u.tok0 = 0;
    u.s0 = at.step;
    u.N = (in_end ? end.step : Walk(p, at.n, at.L, 0).cnt) - at.step;
    u.whole = at.step == 0 && !(in_end && end.step > 0);
    u.slot = 2 * cta + (at.step > 0 ? 0 : 1);
    if (in_end) {
      at.step = end.step;
      return u;
    }
    at.step = 0;
    if (++at.kvh < p.Hkv) return u;
    at.kvh = 0;
    const int lane = threadIdx.x & 31;
    for (at.n = 0; at.n == 0 && ++at.b < p.B;) {
      if (at.b >= b_base + 32) {
        b_base = at.b;
        l_off = l_n = l_L = 0;
        if (b_base + lane < p.B) {
          l_off = packed_off(p.cu_q, b_base + lane, p.total_q);
          l_n = new_tokens(p, b_base + lane);
          l_L = keys_of(p, b_base + lane);
        }
      }
      at.off = __shfl_sync(0xffffffffu, l_off, at.b - b_base);
      at.n = __shfl_sync(0xffffffffu, l_n, at.b - b_base);
      at.L = __shfl_sync(0xffffffffu, l_L, at.b - b_base);
      if (at.b == end.b) break;
    }
    return u;
  }
};

}  // namespace rows_side

// Where the rows of q and of the pages are.
struct RowsParams : Paged8Params {
  const uint16_t* q;
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  long long page_stride, head_stride, token_stride;
};

template <bool BF16, bool I8, int NT>
__global__ void __launch_bounds__(rows_side::Rows<NT>::THREADS, 1)
k_paged8_rows(const __grid_constant__ RowsParams p) {
  using namespace rows_side;
  using R = Rows<NT>;
  constexpr int WARPS = R::WARPS, STAGES = R::STAGES;
  extern __shared__ uint8_t smem_raw[];
  typename R::Smem& s = *reinterpret_cast<typename R::Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;  // row and column pair of the fragments
  grid_launch_dependents();               // the join's blocks may wait beside this grid
  if (threadIdx.x == 0) s.bad_page = 0;
  {
    const Line line = line_at(s.ring, p.B);
    const int parts = lay_line(p, line, s.sums);
    if (warp < 2) {
      const PagedStart at = cut_of(p, line, parts, (int)blockIdx.x + warp);
      if (lane == 0) {
        s.cut[warp] = at;
        if (warp == 1) p.start[blockIdx.x + 1] = at;  // for the join
      }
    }
    __syncthreads();  // the ring is free of the line
  }

  Pieces pieces(s.cut[0], s.cut[1], (int)blockIdx.x);
  Unit cur = pieces.next(p), nxt;
  nxt.N = -1;

  // ---- what this warp brings: slices of 16 keys, warp + WARPS i of a unit
  auto slices = [&](const Unit& u) { return u.N < 0 ? 0 : (4 * u.N - warp + WARPS - 1) / WARPS; };
  auto key_of = [&](const Unit& u, const Walk& w, int i) {
    const int sl = warp + WARPS * i;
    return w.tile(u.s0 + (sl >> 2)) * Q_SUB + 16 * (sl & 3);
  };
  // lane l: the page of slice i + l, -1 where none of its keys is seen or there is
  // no such page
  auto pages_of = [&](const Unit& u, int i) -> int {
    if (i + lane >= slices(u)) return -1;
    const Walk w(p, u.n, u.L, 0);
    const int k0 = key_of(u, w, i + lane);
    if (!w.any(k0, k0 + 16)) return -1;
    const int pg = __ldg(p.table + (size_t)u.b * p.table_stride +
                         div_by(k0, p.page_size, p.inv_page_size));
    if ((unsigned)pg < (unsigned)p.num_pages) return pg;
    s.bad_page = 1;
    return -1;
  };
  int issued = 0, taken = 0;   // slices so far
  bool ahead = false;          // the slices being brought are nxt's
  int bi = 0;                  // the next one to bring
  int page = pages_of(cur, 0), page_next = pages_of(cur, 32), page_nxt = -1;
  // scales of the blocks of the last STAGES - 1 slices (blocks of 16 tokens or more)
  int ksc[STAGES], vsc[STAGES];
#pragma unroll
  for (int i = 0; i < STAGES; ++i) ksc[i] = vsc[i] = 127;
  auto bring = [&]() {
    if (!ahead && bi >= slices(cur) && nxt.N >= 0) {
      ahead = true;
      bi = 0;
      page = page_nxt;
      page_next = pages_of(nxt, 32);
    }
    const Unit& u = ahead ? nxt : cur;
    if (bi >= slices(u)) return;
    const Walk w(p, u.n, u.L, 0);
    const int k0 = key_of(u, w, bi), st = issued % STAGES;
    const int pg = __shfl_sync(0xffffffffu, page, bi & 31);
    const int r0 = k0 - div_by(k0, p.page_size, p.inv_page_size) * p.page_size;
    const bool all = w.all(k0, k0 + 16);
    uint4* to = &s.ring[warp][st][0][lane];
    const long long at = (long long)max(pg, 0) * p.page_stride + u.kvh * p.head_stride +
                         r0 * p.token_stride;
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // K: rows g and g + 8, bytes 16 c and 64 + 16 c on
      const int r = g + 8 * i;
      const bool there = pg >= 0 && (all || w.sees(k0 + r));
      const uint8_t* src = p.k_pages + at + r * p.token_stride + 16 * c;
      copy16(to + 32 * (2 * i), src, there);
      copy16(to + 32 * (2 * i + 1), src + 64, there);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // V: rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9, bytes 16 g on
      const int r = 2 * c + (i & 1) + 8 * (i >> 1);
      const bool there = pg >= 0 && (all || w.sees(k0 + r));
      copy16(to + 32 * (4 + i), p.v_pages + at + r * p.token_stride + 16 * g, there);
    }
    const long long sat = (long long)max(pg, 0) * p.scale_page_stride +
                          u.kvh * p.scale_head_stride + (r0 >> p.scale_shift);
    if (p.scale_shift == 0) {
      if (lane < 8)
        copy4(&s.scales[warp][st][lane],
              (lane < 4 ? p.k_scales : p.v_scales) + sat + 4 * (lane & 3), pg >= 0);
    } else {
#pragma unroll
      for (int i = STAGES - 1; i > 0; --i) {
        ksc[i] = ksc[i - 1];
        vsc[i] = vsc[i - 1];
      }
      ksc[0] = vsc[0] = 127;
      if (pg >= 0) {
        ksc[0] = __ldg(p.k_scales + sat);
        vsc[0] = __ldg(p.v_scales + sat);
      }
    }
    copies_commit();
    ++issued;
    if ((++bi & 31) == 0) {
      page = page_next;
      page_next = pages_of(u, bi + 32);
    }
  };

  for (; cur.N >= 0;) {
    nxt = pieces.next(p);
    page_nxt = nxt.N >= 0 ? pages_of(nxt, 0) : -1;
    const Walk w(p, cur.n, cur.L, 0);
    const int rows = cur.n * p.group, x0 = cur.L - cur.n;
    // Q as B fragments: row n = g of each eight, the elements of this thread's codes
    uint32_t qf[NT][16];
    // the positions of the two rows of each eight that this thread's scores have
    int x[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int n = 8 * t + g;
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (n < rows && cur.N > 0) {
        const int tl = n / p.group;
        const uint16_t* q = p.q + ((long long)(cur.off + tl) * p.Hq + cur.kvh * p.group +
                                   (n - tl * p.group)) * HEAD_DIM + 16 * c;
        v[0] = __ldg(reinterpret_cast<const uint4*>(q));
        v[1] = __ldg(reinterpret_cast<const uint4*>(q + 8));
        v[2] = __ldg(reinterpret_cast<const uint4*>(q + 64));
        v[3] = __ldg(reinterpret_cast<const uint4*>(q + 72));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[t][4 * i] = v[i].x;
        qf[t][4 * i + 1] = v[i].y;
        qf[t][4 * i + 2] = v[i].z;
        qf[t][4 * i + 3] = v[i].w;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = 8 * t + 2 * c + i;
        x[t][i] = m < rows ? x0 + m / p.group : -1;
      }
    }
    float acc[NT][8][4], M[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][i][j] = 0.f;
      M[t][0] = M[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
    const int x_last = x0 + cur.n - 1;
    const int cnt = slices(cur);
    for (int i = 0; i < cnt; ++i) {
      if (issued == taken) bring();
      while (issued - taken < STAGES) {
        const int before = issued;
        bring();
        if (issued == before) break;
      }
      copies_wait(issued - taken - 1);
      __syncwarp();
      const int st = taken % STAGES;
      const uint4* from = &s.ring[warp][st][0][lane];
      const int k0 = key_of(cur, w, i);
      // scales of keys g and g + 8 of K, and of 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of V
      float kf[2];
      int vb[4];
      if (p.scale_shift == 0) {
        const uint8_t* sc = reinterpret_cast<const uint8_t*>(s.scales[warp][st]);
        kf[0] = scale_float<BF16>(sc[g]);
        kf[1] = scale_float<BF16>(sc[g + 8]);
        const uint16_t* sv = reinterpret_cast<const uint16_t*>(sc + 16);
        vb[0] = sv[c] & 255;
        vb[1] = sv[c] >> 8;
        vb[2] = sv[c + 4] & 255;
        vb[3] = sv[c + 4] >> 8;
      } else {
        const int back = issued - taken - 1;
        int a = ksc[0], b = vsc[0];
#pragma unroll
        for (int j = 1; j < STAGES; ++j)
          if (j == back) {
            a = ksc[j];
            b = vsc[j];
          }
        kf[0] = kf[1] = scale_float<BF16>(a);
        vb[0] = vb[1] = vb[2] = vb[3] = b;
      }
      // ---- scores
      float sc[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint4 a = from[32 * hf], b = from[32 * (2 + hf)];
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = code_pair<BF16, I8>(aw[j], aw[j], 0, 1);
          const uint32_t a1 = code_pair<BF16, I8>(bw[j], bw[j], 0, 1);
          const uint32_t a2 = code_pair<BF16, I8>(aw[j], aw[j], 2, 3);
          const uint32_t a3 = code_pair<BF16, I8>(bw[j], bw[j], 2, 3);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma16816<BF16>(sc[t], a0, a1, a2, a3, qf[t][8 * hf + 2 * j],
                           qf[t][8 * hf + 2 * j + 1]);
        }
      }
      kf[0] *= p.scale_log2;
      kf[1] *= p.scale_log2;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[t][j] *= kf[j >> 1];
      // every row sees all 16 keys, or the mask is applied
      const bool whole = (p.causal ? k0 + 16 <= x0 + 1 : k0 + 16 <= cur.L) &&
                         (!p.causal || k0 > x_last - p.window || k0 + 16 <= p.first);
      if (!whole) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = k0 + g + 8 * (j >> 1), xx = x[t][j & 1];
            const bool sees = k < cur.L && (!p.causal || (k <= xx && (xx - k < p.window ||
                                                                      k < p.first)));
            if (!sees) sc[t][j] = -INFINITY;
          }
        // (a block of 16 tokens or more that holds a seen key has a scale for it)
        if (p.scale_shift == 0)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!w.sees(k0 + 2 * c + (j & 1) + 8 * (j >> 1))) vb[j] = 127;
      }
      // ---- the running maximum: moved when a score exceeds it by more than 8
      bool moves = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          moves = moves || fmaxf(sc[t][j], sc[t][j + 2]) > M[t][j] + RESCALE_LOG2;
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = fmaxf(sc[t][j], sc[t][j + 2]);
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            if (mx > M[t][j] + RESCALE_LOG2) {
              const float alpha = M[t][j] == -INFINITY ? 1.f : fast_exp2(M[t][j] - mx);
              M[t][j] = mx;
              l[t][j] *= alpha;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                acc[t][k][j] *= alpha;
                acc[t][k][j + 2] *= alpha;
              }
            }
          }
      }
      // ---- probabilities as B fragments
      uint32_t pf[NT][2];
      float vf[2];  // of this thread's scores' keys, g and g + 8 (bf16)
      if (BF16) {
        if (p.scale_shift == 0) {
          // lane g / 2 of the quad has the bytes of keys g and g + 8
          const int src = (lane & 28) | (g >> 1);
          const int lo = __shfl_sync(0xffffffffu, vb[0] | vb[1] << 8, src);
          const int hi = __shfl_sync(0xffffffffu, vb[2] | vb[3] << 8, src);
          vf[0] = scale_float<BF16>((g & 1) ? lo >> 8 : lo & 255);
          vf[1] = scale_float<BF16>((g & 1) ? hi >> 8 : hi & 255);
        } else {
          vf[0] = vf[1] = scale_float<BF16>(vb[0]);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // a row that has seen nothing keeps its scores at -inf; 0 stands in for M
          const float m = M[t][j & 1];
          e[j] = fast_exp2(sc[t][j] - (m == -INFINITY ? 0.f : m));
          l[t][j & 1] += e[j];
          if (BF16) e[j] *= vf[j >> 1];
        }
        pf[t][0] = transpose8x8(pack2<BF16>(e[0], e[1]));
        pf[t][1] = transpose8x8(pack2<BF16>(e[2], e[3]));
      }
      // ---- O^T += V^T P^T
      const uint4 v0 = from[32 * 4], v1 = from[32 * 5], v2 = from[32 * 6], v3 = from[32 * 7];
      const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
      const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
      uint32_t s01 = 0, s23 = 0;
      if (!BF16) {
        s01 = (scale_pair<BF16>(vb[0]) & 0xffffu) | (scale_pair<BF16>(vb[1]) << 16);
        s23 = (scale_pair<BF16>(vb[2]) & 0xffffu) | (scale_pair<BF16>(vb[3]) << 16);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int wd = k >> 1, by = 2 * (k & 1);
        uint32_t a0 = code_pair<BF16, I8>(w0[wd], w1[wd], by, 4 + by);
        uint32_t a1 = code_pair<BF16, I8>(w0[wd], w1[wd], by + 1, 5 + by);
        uint32_t a2 = code_pair<BF16, I8>(w2[wd], w3[wd], by, 4 + by);
        uint32_t a3 = code_pair<BF16, I8>(w2[wd], w3[wd], by + 1, 5 + by);
        if (!BF16) {
          a0 = mul16x2<false>(a0, s01);
          a1 = mul16x2<false>(a1, s01);
          a2 = mul16x2<false>(a2, s23);
          a3 = mul16x2<false>(a3, s23);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816<BF16>(acc[t][k], a0, a1, a2, a3, pf[t][0], pf[t][1]);
      }
      ++taken;
      __syncwarp();  // the scales' slot is read
    }

    // ---- the piece's end: the warps' shares meet
    __syncthreads();  // the piece before is out of the shared memory
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], d);
        const int n = 8 * t + 2 * c + j;
        if (g == 0) {
          s.ml[warp][n][0] = M[t][j];
          s.ml[warp][n][1] = l[t][j];
        }
        float4* to = reinterpret_cast<float4*>(&s.O[warp][n][16 * g]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          to[k] = make_float4(acc[t][2 * k][j], acc[t][2 * k][j + 2], acc[t][2 * k + 1][j],
                              acc[t][2 * k + 1][j + 2]);
      }
    __syncthreads();
    for (int u = threadIdx.x; u < rows * 64; u += R::THREADS) {
      const int n = u >> 6, d = 2 * (u & 63);
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) top = fmaxf(top, s.ml[k][n][0]);
      float2 o = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        const float lk = s.ml[k][n][1];
        // a warp that saw nothing of the row has no weight (l is never negative, and
        // a NaN stays)
        const float wk = lk != 0.f ? fast_exp2(s.ml[k][n][0] - top) : 0.f;
        sum += lk * wk;
        const float2 y = *reinterpret_cast<const float2*>(&s.O[k][n][d]);
        o.x = fmaf(y.x, wk, o.x);
        o.y = fmaf(y.y, wk, o.y);
      }
      const int tl = n / p.group, head = cur.kvh * p.group + n - tl * p.group;
      const int tok = cur.off + tl;
      if (cur.whole) {
        float inv;
        const float lse = finish_row(top, sum, p.sink ? p.sink[head] * LOG2E : -INFINITY, &inv);
        if (p.lse && d == 0) p.lse[(size_t)head * p.total_q + tok] = lse;
        *reinterpret_cast<uint32_t*>(p.out + ((size_t)tok * p.Hq + head) * HEAD_DIM + d) =
            pack2<BF16>(o.x * inv, o.y * inv);
      } else {
        float* part = p.part + (size_t)cur.slot * p.slot_floats +
                      (2 * (n >> 5) + (d >> 6)) * PAGED_WARP_FLOATS;
        *reinterpret_cast<float2*>(reinterpret_cast<float*>(part_at(part, n & 31, (d & 63) >> 2)) +
                                   (d & 3)) = o;
        if (d == 0) {
          part[PAGED_ML + 2 * (n & 31)] = top;
          part[PAGED_ML + 2 * (n & 31) + 1] = sum;
        }
      }
    }
    cur = nxt;
    if (ahead) {
      ahead = false;
    } else {  // nothing of it was brought yet
      bi = 0;
      page = page_nxt;
      page_next = cur.N >= 0 ? pages_of(cur, 32) : -1;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    DevStatus st{};
    st.code = s.bad_page ? (unsigned)ATTN_ERR_INVALID_ARG : 0u;
    p.cta_status[blockIdx.x] = st;
  }
}

template <bool BF16, bool I8, int NT>
cudaError_t launch_rows(const RowsParams& p, cudaStream_t st) {
  using R = rows_side::Rows<NT>;
  const auto kern = k_paged8_rows<BF16, I8, NT>;
  constexpr int smem = (int)sizeof(typename R::Smem) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)p.grid, R::THREADS, smem, st>>>(p);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_join<BF16>(p, st) : e;
}

template <bool BF16, bool I8>
cudaError_t launch_rows_of(int rows, const RowsParams& p, cudaStream_t st) {
  return rows <= 8 ? launch_rows<BF16, I8, 1>(p, st) : launch_rows<BF16, I8, 2>(p, st);
}

cudaError_t launch_paged8_rows(bool bf16, bool i8, const Paged8Params& base, const void* q,
                               const void* k_pages, const void* v_pages, long long page_stride,
                               long long head_stride, long long token_stride, cudaStream_t st) {
  RowsParams p;
  static_cast<Paged8Params&>(p) = base;
  p.q = static_cast<const uint16_t*>(q);
  p.k_pages = static_cast<const uint8_t*>(k_pages);
  p.v_pages = static_cast<const uint8_t*>(v_pages);
  p.page_stride = page_stride;
  p.head_stride = head_stride;
  p.token_stride = token_stride;
  const int rows = p.tile_rows;
  if (i8) return bf16 ? launch_rows_of<true, true>(rows, p, st) : launch_rows_of<false, true>(rows, p, st);
  return bf16 ? launch_rows_of<true, false>(rows, p, st) : launch_rows_of<false, false>(rows, p, st);
}

}  // namespace mab
