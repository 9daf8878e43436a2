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

// The pieces of a CTA's part of the line, one after another: where the first warp
// stands, kept in shared memory.
struct Pieces {
  PagedStart at, end;
  int cta, b_base;                  // lengths of requests b_base .. b_base + 31
  int l_off[32], l_n[32], l_L[32];

  // The next one, by one whole warp; N < 0: none is left.
  __device__ __noinline__ void next(const PagedParams& p, Unit* out) {
    const int lane = threadIdx.x & 31;
    PagedStart a = at;
    const bool in_end = a.b == end.b && a.kvh == end.kvh;
    Unit u{};
    u.N = -1;
    if (a.b < p.B && !(in_end && end.step <= a.step)) {
      u.b = a.b;
      u.kvh = a.kvh;
      u.off = a.off;
      u.n = a.n;
      u.L = a.L;
      u.s0 = a.step;
      u.N = (in_end ? end.step : Walk(p, a.n, a.L, 0).cnt) - a.step;
      u.whole = a.step == 0 && !(in_end && end.step > 0);
      u.slot = 2 * cta + (a.step > 0 ? 0 : 1);
      if (in_end) {
        a.step = end.step;
      } else {
        a.step = 0;
        if (++a.kvh == p.Hkv) {
          a.kvh = 0;
          // the next request with new tokens
          for (a.n = 0; a.n == 0 && ++a.b < p.B;) {
            if (a.b >= b_base + 32) {
              __syncwarp();
              if (lane == 0) b_base = a.b;
              const int b = a.b + lane;
              l_off[lane] = b < p.B ? packed_off(p.cu_q, b, p.total_q) : 0;
              l_n[lane] = b < p.B ? new_tokens(p, b) : 0;
              l_L[lane] = b < p.B ? keys_of(p, b) : 0;
              __syncwarp();
            }
            a.off = l_off[a.b - b_base];
            a.n = l_n[a.b - b_base];
            a.L = l_L[a.b - b_base];
            if (a.b == end.b) break;
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) {
      at = a;
      *out = u;
    }
    __syncwarp();
  }
};

template <int NT>
struct Rows {
  static constexpr int WARPS = NT <= 2 ? 16 : 8;
  static constexpr int LAG = NT <= 2 ? 1 : 2;   // slices on their way while one is worked on
  static constexpr int STAGES = LAG + 1;
  static constexpr bool Q_REGS = NT == 1;       // Q's fragments in registers, or shared memory
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int N = 8 * NT;              // rows of a unit at most
  static constexpr int MERGE = 128 / WARPS;     // rows whose shares meet at a time
  static constexpr int O_STRIDE = 132;          // floats: rows on other banks
  struct Smem {
    uint4 ring[WARPS][STAGES][8][32];           // K: 4 pieces a lane, V: 4
    uint32_t scales[WARPS][STAGES][8];          // a scale a token: 16 bytes of K, 16 of V
    uint2 q[Q_REGS ? 1 : NT][8][32];            // Q's fragments
    float O[WARPS][MERGE][O_STRIDE];
    float ml[WARPS][N][2];                      // (M, l)
    LineSums<THREADS> sums;
    PagedStart cut[2];
    Unit unit[3];                               // unit j at j % 3, j + 2 known at j's end
    Pieces pieces;
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

// 16 bytes to shared memory; the second form zeros where `there` is false (then
// nothing is read).
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy16_if(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4_if(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most n of the committed groups are pending (n < 3).
__device__ __forceinline__ void copies_wait(int n) {
  if (n <= 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// Unit of a bf16 unit's O: probabilities that meet e4m3's moved bits (2^120 too
// small) come times 2^112.
template <bool I8>
constexpr float V_UNIT = I8 ? 1.f : 0x1p-8f;

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
  constexpr int WARPS = R::WARPS, STAGES = R::STAGES, LAG = R::LAG;
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
  if (warp == 0) {
    if (lane == 0) {
      s.pieces.at = s.cut[0];
      s.pieces.end = s.cut[1];
      s.pieces.cta = (int)blockIdx.x;
      s.pieces.b_base = s.cut[0].b - 32;
    }
    __syncwarp();
    s.pieces.next(p, &s.unit[0]);
    s.pieces.next(p, &s.unit[1]);
  }
  __syncthreads();

  // ---- what this warp brings: slices of 16 keys, warp + WARPS i of a unit, which
  // has u_cnt of them; u_at is the next one
  int u_slot = 0, u_cnt = 0, u_at = 0;
  auto slices = [&](const Unit& x) { return x.N < 0 ? 0 : (4 * x.N - warp + WARPS - 1) / WARPS; };
  // Lane l looks slice i + l up: its page (-1: no seen key, or no such page) ...
  constexpr int ALL = 1, WHOLE = 2, NONE = 4;  // flags below the slice's first key
  auto first_key = [&](const Unit& u, const Walk& w, int i) {
    const int sl = warp + WARPS * (i + lane);
    return w.tile(u.s0 + (sl >> 2)) * Q_SUB + 16 * (sl & 3);
  };
  auto page_of = [&](const Unit& u, int i) -> int {
    if (i + lane >= slices(u)) return -1;
    const Walk w(p, u.n, u.L, 0);
    const int k0 = first_key(u, w, i);
    if (!w.any(k0, k0 + 16)) return -1;
    const int pg = __ldg(p.table + (size_t)u.b * p.table_stride +
                         div_by(k0, p.page_size, p.inv_page_size));
    if ((unsigned)pg < (unsigned)p.num_pages) return pg;
    s.bad_page = 1;
    return -1;
  };
  // ... and where its rows and scales are: batch of the 32 slices from u_at on
  int b_key = 0, b_scale = 0, page_next = -1;
  long long b_base = 0, b_sat = 0;
  auto batch = [&](int page) {
    const Unit& u = s.unit[u_slot];
    const Walk w(p, u.n, u.L, 0);
    const int k0 = first_key(u, w, u_at);
    const int r0 = k0 - div_by(k0, p.page_size, p.inv_page_size) * p.page_size;
    const int x0 = u.L - u.n;
    const bool whole = (p.causal ? k0 + 16 <= x0 + 1 : k0 + 16 <= u.L) &&
                       (!p.causal || k0 > u.L - 1 - p.window || k0 + 16 <= p.first);
    b_key = k0 | (w.all(k0, k0 + 16) ? ALL : 0) | (whole ? WHOLE : 0) | (page < 0 ? NONE : 0);
    b_base = max(page, 0) * p.page_stride + u.kvh * p.head_stride + r0 * p.token_stride;
    b_sat = max(page, 0) * p.scale_page_stride + u.kvh * p.scale_head_stride +
            (r0 >> p.scale_shift);
    b_scale = 127 | 127 << 8;
    if (p.scale_shift > 0 && page >= 0)
      b_scale = __ldg(p.k_scales + b_sat) | __ldg(p.v_scales + b_sat) << 8;
    page_next = page_of(u, u_at + 32);
  };
  // this thread's pieces of a slice: K rows g and g + 8, bytes 16 c and 64 + 16 c on;
  // V rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9, bytes 16 g on
  const int ts = (int)p.token_stride;
  const int k_off = g * ts + 16 * c, v_off = 2 * c * ts + 16 * g;
  // A slice on its way: its first key and flags, and its scales (K's byte, V's the
  // next one) where 16 tokens or more share one.
  struct Slice {
    int key, scale;
  };
  bool more = false;  // the next unit may be taken up
  int page_nxt = -1;  // its first batch's pages
  int stage = 0;      // that the next slice goes to
  auto bring = [&](Slice& sl) -> bool {
    if (u_at == u_cnt) {
      if (!more) return false;
      more = false;
      u_slot = u_slot == 2 ? 0 : u_slot + 1;
      u_at = 0;
      u_cnt = slices(s.unit[u_slot]);
      if (u_cnt == 0) return false;
      batch(page_nxt);
    } else if ((u_at & 31) == 0 && u_at > 0) {
      batch(page_next);
    }
    const int i = u_at & 31;
    sl.key = __shfl_sync(0xffffffffu, b_key, i);
    sl.scale = __shfl_sync(0xffffffffu, b_scale, i);
    const long long base = __shfl_sync(0xffffffffu, b_base, i);
    uint4* to = &s.ring[warp][stage][0][lane];
    const uint8_t* k = p.k_pages + base + k_off;
    const uint8_t* v = p.v_pages + base + v_off;
    if ((sl.key & (ALL | NONE)) == ALL) {
      copy16(to, k);
      copy16(to + 32, k + 64);
      copy16(to + 64, k + 8 * ts);
      copy16(to + 96, k + 8 * ts + 64);
      copy16(to + 128, v);
      copy16(to + 160, v + ts);
      copy16(to + 192, v + 8 * ts);
      copy16(to + 224, v + 9 * ts);
    } else {
      const Walk w(p, s.unit[u_slot].n, s.unit[u_slot].L, 0);
      const int k0 = sl.key & ~15;
#pragma unroll 1
      for (int j = 0; j < 8; ++j) {
        const int r = j < 4 ? g + 8 * (j >> 1) : 2 * c + (j & 1) + 8 * ((j - 4) >> 1);
        const uint8_t* src = (j < 4 ? p.k_pages + 16 * c + 64 * (j & 1) : p.v_pages + 16 * g) +
                             base + (long long)r * ts;
        copy16_if(to + 32 * j, src, !(sl.key & NONE) && w.sees(k0 + r));
      }
    }
    if (p.scale_shift == 0) {
      const long long sat = __shfl_sync(0xffffffffu, b_sat, i);
      if (lane < 8)
        copy4_if(&s.scales[warp][stage][lane],
                 (lane < 4 ? p.k_scales : p.v_scales) + sat + 4 * (lane & 3), !(sl.key & NONE));
    }
    copies_commit();
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    ++u_at;
    return true;
  };

  // slices on their way, the earliest first
  Slice way[LAG + 1];
  int on_way = 0;
  int from_stage = 0;  // of the earliest
#pragma unroll
  for (int i = 0; i <= LAG; ++i) way[i].key = way[i].scale = 0;
  u_cnt = slices(s.unit[0]);
  if (u_cnt > 0) batch(page_of(s.unit[0], 0));
  auto fill = [&]() {
#pragma unroll
    for (int i = 0; i <= LAG; ++i)
      if (on_way == i && bring(way[i])) on_way = i + 1;
  };

  // Q's fragment words of row n = g of eight t: the elements of this thread's codes.
  // f16 products take K's codes as they are, so a bf16 row comes times 2^sh, which
  // puts its largest element below 2^15: exact but for elements 2^-32 of that.
  auto q_row = [&](const Unit& x, int t, uint4 (&v)[4]) {
    const int n = 8 * t + g;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (n < x.n * p.group && x.N > 0) {
      const int tl = n / p.group;
      const uint16_t* q = p.q + ((long long)(x.off + tl) * p.Hq + x.kvh * p.group +
                                 (n - tl * p.group)) * HEAD_DIM + 16 * c;
      v[0] = __ldg(reinterpret_cast<const uint4*>(q));
      v[1] = __ldg(reinterpret_cast<const uint4*>(q + 8));
      v[2] = __ldg(reinterpret_cast<const uint4*>(q + 64));
      v[3] = __ldg(reinterpret_cast<const uint4*>(q + 72));
    }
  };
  for (int slot = 0; s.unit[slot].N >= 0;) {
    const Unit& cur = s.unit[slot];
    const int next_slot = slot == 2 ? 0 : slot + 1;
    if (u_slot != slot) {  // not taken up while the one before was worked on
      u_slot = slot;
      u_at = 0;
      u_cnt = slices(cur);
      if (u_cnt > 0) batch(page_nxt);
    }
    more = s.unit[next_slot].N >= 0;
    page_nxt = more ? page_of(s.unit[next_slot], 0) : -1;
    uint32_t qf[R::Q_REGS ? 16 : 1];
    float col[NT][2];  // what the scores of this thread's two rows are multiplied by
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint4 v[4];
      q_row(cur, t, v);
      uint32_t qw[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qw[4 * i] = v[i].x;
        qw[4 * i + 1] = v[i].y;
        qw[4 * i + 2] = v[i].z;
        qw[4 * i + 3] = v[i].w;
      }
      float back = p.scale_log2;
      if (BF16) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = __vmaxu2(top, qw[i] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent field e: elements below 2^(e - 126) become below 2^15
        const int e = min(max((int)(top >> 7), 20), 254);
        const float up = exp2_int(141 - e);
        back = exp2_int(e - 141) * p.scale_log2;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 y = unpack2<true>(qw[i]);
          qw[i] = pack2<false>(y.x * up, y.y * up);
        }
      }
      if (R::Q_REGS) {
#pragma unroll
        for (int i = 0; i < 16; ++i) qf[i] = qw[i];
      } else if (warp == t % WARPS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s.q[t][i][lane] = make_uint2(qw[2 * i], qw[2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        col[t][i] = __shfl_sync(0xffffffffu, back, 4 * (2 * c + i));
      }
    }
    if (!R::Q_REGS) __syncthreads();
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
    const int cnt = slices(cur);
#pragma unroll 1
    for (int i = 0; i < cnt; ++i) {
      fill();
      copies_wait(on_way - 1);
      __syncwarp();
      const Slice sl = way[0];
      const int st = from_stage;
      const uint4* from = &s.ring[warp][st][0][lane];
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
        kf[0] = kf[1] = scale_float<BF16>(sl.scale & 255);
        vb[0] = vb[1] = vb[2] = vb[3] = sl.scale >> 8;
      }
      // ---- scores: f16 products of the codes themselves
      float sc[NT][4];
      {
        float s1[NT][4];  // of the second half of d: a chain of its own
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[t][j] = s1[t][j] = 0.f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint4 a = from[32 * hf], b = from[32 * (2 + hf)];
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = code_pair<false, I8>(aw[j], aw[j], 0, 1);
            const uint32_t a1 = code_pair<false, I8>(bw[j], bw[j], 0, 1);
            const uint32_t a2 = code_pair<false, I8>(aw[j], aw[j], 2, 3);
            const uint32_t a3 = code_pair<false, I8>(bw[j], bw[j], 2, 3);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              uint2 q;
              if (R::Q_REGS)
                q = make_uint2(qf[(8 * hf + 2 * j) % 16], qf[(8 * hf + 2 * j + 1) % 16]);
              else
                q = s.q[t][4 * hf + j][lane];
              mma16816<false>(hf ? s1[t] : sc[t], a0, a1, a2, a3, q.x, q.y);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            sc[t][j] = (sc[t][j] + s1[t][j]) * (kf[j >> 1] * col[t][j & 1]);
      }
      if (!(sl.key & WHOLE)) {  // some row does not see some key
        const int k0 = sl.key & ~15, rows = cur.n * p.group;
        const Walk w(p, cur.n, cur.L, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int m = 8 * t + 2 * c + i;
            const int x = m < rows ? cur.L - cur.n + m / p.group : -1;  // the row's position
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int k = k0 + g + 8 * j;
              const bool sees = k < cur.L && (!p.causal || (k <= x && (x - k < p.window ||
                                                                       k < p.first)));
              if (!sees) sc[t][i + 2 * j] = -INFINITY;
            }
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
      // ---- probabilities as B fragments; for bf16 times V's scale, in units of
      // 2^V_UNIT (a power of two each, so exactly)
      float vf[2] = {1.f, 1.f};  // of this thread's scores' keys, g and g + 8
      bool raw = true;           // V's codes are taken as moved bits, 2^120 too small
      if (BF16) {
        int lo = vb[0], hi = vb[0];
        if (p.scale_shift == 0) {
          // lane g / 2 of the quad has the bytes of keys g and g + 8
          const int src = (lane & 28) | (g >> 1);
          lo = __shfl_sync(0xffffffffu, vb[0] | vb[1] << 8, src);
          hi = __shfl_sync(0xffffffffu, vb[2] | vb[3] << 8, src);
          lo = (g & 1) ? lo >> 8 : lo & 255;
          hi = (g & 1) ? hi >> 8 : hi & 255;
        }
        // probabilities are at most 2^8, so that times 2^112 they want exponents of
        // at most 7
        if (!I8) raw = !__any_sync(0xffffffffu, max(lo, hi) > 127 + 7);
        vf[0] = scale_float<true>(lo) * V_UNIT<I8>;
        vf[1] = scale_float<true>(hi) * V_UNIT<I8>;
        if (!I8 && raw) {
          vf[0] *= 0x1p120f;
          vf[1] *= 0x1p120f;
        }
      }
      uint32_t pf[NT][2];
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
      auto add_values = [&](auto&& pair) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int wd = k >> 1, by = 2 * (k & 1);
          uint32_t a0 = pair(w0[wd], w1[wd], by, 4 + by);
          uint32_t a1 = pair(w0[wd], w1[wd], by + 1, 5 + by);
          uint32_t a2 = pair(w2[wd], w3[wd], by, 4 + by);
          uint32_t a3 = pair(w2[wd], w3[wd], by + 1, 5 + by);
          if (!BF16) {
            a0 = mul16x2<false>(a0, s01);
            a1 = mul16x2<false>(a1, s01);
            a2 = mul16x2<false>(a2, s23);
            a3 = mul16x2<false>(a3, s23);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma16816<BF16>(acc[t][k], a0, a1, a2, a3, pf[t][0], pf[t][1]);
        }
      };
      auto exact_pair = [](uint32_t a, uint32_t b, int x, int y) {
        return code_pair<BF16, I8>(a, b, x, y);
      };
      if constexpr (BF16 && !I8) {
        if (raw)
          add_values([](uint32_t a, uint32_t b, int x, int y) { return code_bits(a, b, x, y); });
        else
          add_values(exact_pair);
      } else {
        add_values(exact_pair);
      }
      __syncwarp();  // the scales' slot is read
#pragma unroll
      for (int j = 0; j < LAG; ++j) way[j] = way[j + 1];
      --on_way;
      from_stage = from_stage + 1 == STAGES ? 0 : from_stage + 1;
    }

    // ---- the piece's end: the warps' shares meet, MERGE rows at a time
    const int rows = cur.n * p.group;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], d);
#pragma unroll
    for (int t0 = 0; t0 < NT; t0 += R::MERGE / 8) {
      if (8 * t0 >= rows) break;
      __syncthreads();  // what was there is read
      // (nobody is at the unit before this one any more: its slot takes the one
      // after the next)
      if (t0 == 0 && warp == 0) s.pieces.next(p, &s.unit[next_slot == 2 ? 0 : next_slot + 1]);
#pragma unroll
      for (int t = t0; t < t0 + R::MERGE / 8 && t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = 8 * t + 2 * c + j;
          if (g == 0) {
            s.ml[warp][n][0] = M[t][j];
            s.ml[warp][n][1] = l[t][j];
          }
          float4* to = reinterpret_cast<float4*>(&s.O[warp][n - 8 * t0][16 * g]);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            to[k] = make_float4(acc[t][2 * k][j], acc[t][2 * k][j + 2], acc[t][2 * k + 1][j],
                                acc[t][2 * k + 1][j + 2]);
        }
      __syncthreads();
      const int end = min(rows - 8 * t0, R::MERGE) * 64;
      for (int i = threadIdx.x; i < end; i += R::THREADS) {
        const int m = i >> 6, n = 8 * t0 + m, d = 2 * (i & 63);
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
          const float2 y = *reinterpret_cast<const float2*>(&s.O[k][m][d]);
          o.x = fmaf(y.x, wk, o.x);
          o.y = fmaf(y.y, wk, o.y);
        }
        if (BF16) {
          o.x *= 1.f / V_UNIT<I8>;
          o.y *= 1.f / V_UNIT<I8>;
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
          *reinterpret_cast<float2*>(
              reinterpret_cast<float*>(part_at(part, n & 31, (d & 63) >> 2)) + (d & 3)) = o;
          if (d == 0) {
            part[PAGED_ML + 2 * (n & 31)] = top;
            part[PAGED_ML + 2 * (n & 31) + 1] = sum;
          }
        }
      }
    }
    if (!R::Q_REGS) __syncthreads();  // Q is read by all
    slot = next_slot;
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
