// paged8_rows.cu -- attention of a few new tokens over an 8-bit paged cache.
//
// The same operation, work line, cuts and join as paged_fwd.cu, for calls whose
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
// each brings its own slices into a ring of its own.  At a piece's end the warps'
// O, M and l meet in shared memory.
//
// An m16n8k16 occupies its quarter of the SM for 8 cycles: eight rows want 128 of the
// 706 that a quarter has for a slice at the copy rate, and the conversions and the rest
// 466 instructions, 198 of them on the half-rate integer pipe.  Sixteen rows leave 12
// warps' registers, forty 8, whose latencies then show: 64 requests of five tokens (40
// rows) took 551 us in this form, 403 with the tiles of the tcgen05 kernel
// (paged_fwd.cuh), which takes more than 16.
//
// Measured (one GB300), 64 single tokens at 9000 keys on average, 64/8 heads, 1.14 GB: e4m3
// bf16 195 us, 5.9 TB/s (copy rate 6.7), e4m3 fp16 184, int8 fp16 193, int8 bf16 197, a
// scale a token 211; two tokens each 295.  One token at 1000 keys 15 us: the line 2.5, the
// first slices, the join.  On the way there: the tcgen05 kernel 719 us; this one with
// cp.async of 16 bytes a lane, every code times 2^120 and bf16 scores 329; with f16 scores
// of the codes themselves and V's codes as moved bits 237; slices by TMA 202.
#include <cfloat>
#include <type_traits>

#include "paged_line.cuh"
#include "quant8.cuh"

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
  // (NT 1 with 12 warps and two slices on their way: 64 tokens at 2000 to 16000 keys
  // 223 us when this took 207; NT 2 with 16 and one 447, with 8 and two 332, when this
  // took 319)
  static constexpr int WARPS = NT == 1 ? 16 : 12;
  static constexpr int LAG = NT == 1 ? 1 : 2;   // slices on their way while one is worked on
  static constexpr int STAGES = LAG + 1;
  static constexpr bool Q_REGS = NT == 1;       // Q's fragments in registers, or shared memory
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int N = 8 * NT;              // rows of a unit at most
  static constexpr int O_STRIDE = 132;          // floats: rows on other banks
  struct Smem {
    // K's and V's rows of a slice (128B swizzle), and 16 scales of each where every
    // token has its own
    uint8_t ring[WARPS][STAGES][2][16 * 128];
    uint8_t scales[WARPS][STAGES][2][16];
    uint64_t full[WARPS][STAGES];
    uint2 q[Q_REGS ? 1 : NT][8][32];            // Q's fragments
    uint4 rows[2][N][16];                       // the rows of q of a unit and of the next
    float O[WARPS][8][O_STRIDE];                // eight rows meet at a time
    float ml[WARPS][N][2];                      // (M, l)
    LineSums<THREADS> sums;
    PagedStart cut[2];
    Unit unit[3];                               // unit j at j % 3, j + 2 known at j's end
    Pieces pieces;
    unsigned bad_page;
    int abort_flag;
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

// 16 bytes to shared memory, asynchronously.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The maximum of a row that has seen nothing: above no finite score, and finite, so that
// -inf less it is -inf.
constexpr float NO_MAX = -FLT_MAX;

// Unit of a bf16 unit's O: probabilities that meet e4m3's moved bits (2^120 too
// small) come times 2^112.
template <bool I8>
constexpr float V_UNIT = I8 ? 1.f : 0x1p-8f;

}  // namespace rows_side

template <bool BF16, bool I8, int NT>
__global__ void __launch_bounds__(rows_side::Rows<NT>::THREADS, 1)
k_paged8_rows(const __grid_constant__ CUtensorMap tK, const __grid_constant__ CUtensorMap tV,
              const uint16_t* __restrict__ q_rows, const __grid_constant__ Paged8Params p) {
  using namespace rows_side;
  using R = Rows<NT>;
  constexpr int WARPS = R::WARPS, STAGES = R::STAGES, LAG = R::LAG;
  extern __shared__ uint8_t smem_raw[];
  typename R::Smem& s = *reinterpret_cast<typename R::Smem*>(smem_align1024(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;  // row and column pair of the fragments
  grid_launch_dependents();               // the join's blocks may wait beside this grid
  WaitCtx wc{p.cta_status + blockIdx.x, &s.abort_flag, p.timeout_ns};
  if (threadIdx.x == 0) {
    s.bad_page = 0;
    s.abort_flag = 0;
    *wc.status = DevStatus{};
    for (int i = 0; i < WARPS * STAGES; ++i) mbar_init(smem_u32(&s.full[0][0] + i), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tK);
    tma_prefetch_desc(&tV);
  }
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
    // the loads into the ring come after these generic accesses to it
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
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
  constexpr int WHOLE = 1, NONE = 2;  // flags below the slice's first key
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
  // ... and where its rows and scales are: batch of the 32 slices from u_at on.
  // (Flags: every row sees all 16 keys; no page, zeros stand in.)
  int b_key = 0, b_page = 0, b_row = 0, page_next = -1;
  long long b_sat = 0;            // a scale a token: their offset
  // a scale for 16 tokens or more: the scales, V's negative where its exponent is past
  // what the moved bits take
  float b_ks = 1.f, b_vs = 1.f;
  auto batch = [&](int page) {
    const Unit& u = s.unit[u_slot];
    const Walk w(p, u.n, u.L, 0);
    const int k0 = first_key(u, w, u_at);
    b_row = k0 - div_by(k0, p.page_size, p.inv_page_size) * p.page_size;
    const int x0 = u.L - u.n;
    const bool whole = (p.causal ? k0 + 16 <= x0 + 1 : k0 + 16 <= u.L) &&
                       (!p.causal || k0 > u.L - 1 - p.window || k0 + 16 <= p.first);
    b_key = k0 | (whole ? WHOLE : 0) | (page < 0 ? NONE : 0);
    b_page = page < 0 ? p.num_pages : page;  // past the tensor's end a load reads zeros
    const long long sat = max(page, 0) * p.scale_page_stride + u.kvh * p.scale_head_stride +
                          (b_row >> p.scale_shift);
    if (p.scale_shift == 0) {
      b_sat = sat;
    } else {
      b_ks = b_vs = 1.f;
      if (page >= 0) {
        const int v = __ldg(p.v_scales + sat);
        b_ks = scale_float<BF16>(__ldg(p.k_scales + sat));
        b_vs = scale_float<BF16>(v);
        if (v > 127 + 7) b_vs = -b_vs;
      }
    }
    page_next = page_of(u, u_at + 32);
  };
  // A slice on its way: its first key and flags, and its scales where 16 tokens or
  // more share one.
  struct Slice {
    int key;
    float ks, vs;
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
    const int i = u_at & 31, kvh = s.unit[u_slot].kvh;
    sl.key = __shfl_sync(0xffffffffu, b_key, i);
    const int page = __shfl_sync(0xffffffffu, b_page, i);
    const int row = __shfl_sync(0xffffffffu, b_row, i);
    const uint32_t fb = smem_u32(&s.full[warp][stage]);
    const uint32_t to = smem_u32(s.ring[warp][stage][0]);
    const bool own_scales = p.scale_shift == 0 && !(sl.key & NONE);
    if (!p.test_no_loads) {
      if (lane == 0) mbar_arrive_expect_tx(fb, 2 * 16 * 128 + (own_scales ? 32 : 0));
      __syncwarp();
      tma_load_4d_w(to, &tK, 0, row, kvh, page, fb);
      tma_load_4d_w(to + 16 * 128, &tV, 0, row, kvh, page, fb);
    }
    if (p.scale_shift == 0) {
      const long long sat = __shfl_sync(0xffffffffu, b_sat, i);
      if (lane < 2 && own_scales && !p.test_no_loads)
        bulk_load(smem_u32(s.scales[warp][stage][lane]), (lane ? p.v_scales : p.k_scales) + sat,
                  16, fb);
    } else {
      sl.ks = __shfl_sync(0xffffffffu, b_ks, i);
      sl.vs = __shfl_sync(0xffffffffu, b_vs, i);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    ++u_at;
    return true;
  };

  // slices on their way, the earliest first
  Slice way[LAG + 1];
  int on_way = 0;
  int from_stage = 0;  // of the earliest, and the parity of its use
  uint32_t from_ph = 0;
  bool ok = true;
#pragma unroll
  for (int i = 0; i <= LAG; ++i) way[i] = {0, 1.f, 1.f};
  u_cnt = slices(s.unit[0]);
  if (u_cnt > 0) batch(page_of(s.unit[0], 0));
  auto fill = [&]() {
#pragma unroll
    for (int i = 0; i <= LAG; ++i)
      if (on_way == i && bring(way[i])) on_way = i + 1;
  };

  // Brings the rows of q of unit x (the block; there once its copies are waited for and
  // the block has met); rows that are no token's are left as they are, nobody reads them.
  auto bring_q = [&](const Unit& x, int to) {
    const int rows = x.N > 0 ? x.n * p.group : 0;
    for (int i = threadIdx.x; i < rows * 16; i += R::THREADS) {
      const int n = i >> 4, tl = n / p.group;
      copy16(&s.rows[to][n][i & 15],
             q_rows + ((long long)(x.off + tl) * p.Hq + x.kvh * p.group + (n - tl * p.group)) *
                          HEAD_DIM + 8 * (i & 15));
    }
    copies_commit();
  };
  bring_q(s.unit[0], 0);
  copies_wait();
  __syncthreads();
  // Q's fragment words of row n = g of eight t: the elements of this thread's codes.
  // f16 products take K's codes as they are, so a bf16 row comes times 2^sh, which
  // puts its largest element below 2^15: exact but for elements 2^-31 of that.
  int parity = 0;  // of s.rows
  auto q_row = [&](const Unit& x, int t, uint4 (&v)[4]) {
    const int n = 8 * t + g;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (n < x.n * p.group && x.N > 0) {
      const uint4* q = &s.rows[parity][n][2 * c];
      v[0] = q[0];
      v[1] = q[1];
      v[2] = q[8];
      v[3] = q[9];
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
    bring_q(s.unit[next_slot], parity ^ 1);
    more = s.unit[next_slot].N >= 0;
    page_nxt = more ? page_of(s.unit[next_slot], 0) : -1;
    uint32_t qf[R::Q_REGS ? 16 : 1];
    float col[NT][2];  // what the scores of this thread's two rows of each eight are multiplied by
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
      M[t][0] = M[t][1] = NO_MAX;
      l[t][0] = l[t][1] = 0.f;
    }
    const int cnt = slices(cur), rows = cur.n * p.group;
#pragma unroll 1
    for (int i = 0; i < cnt && ok; ++i) {
      fill();
      ok = mbar_wait_warp(smem_u32(&s.full[warp][from_stage]), from_ph, wc, TAG_KV_FULL);
      if (!ok) break;
      const Slice sl = way[0];
      const uint8_t* rk = s.ring[warp][from_stage][0];
      const uint8_t* rv = s.ring[warp][from_stage][1];
      // scales of keys g and g + 8 of K, and of V: of these, or (f16) of 2 c, 2 c + 1,
      // 2 c + 8 and 2 c + 9 as pairs
      float kf[2] = {sl.ks, sl.ks}, vf[2] = {fabsf(sl.vs), fabsf(sl.vs)};
      bool big = !(sl.vs > 0.f);
      uint32_t s01 = 0, s23 = 0;
      if (p.scale_shift == 0) {
        // lane l makes the scale of K's key l, or V's key l - 16, of the bytes
        const int sb = sl.key & NONE ? 127 : (&s.scales[warp][from_stage][0][0])[lane];
        const float sf = scale_float<BF16>(sb);
        kf[0] = __shfl_sync(0xffffffffu, sf, g);
        kf[1] = __shfl_sync(0xffffffffu, sf, g + 8);
        if (BF16) {
          vf[0] = __shfl_sync(0xffffffffu, sf, g + 16);
          vf[1] = __shfl_sync(0xffffffffu, sf, g + 24);
          if (!I8) big = __any_sync(0xffffffffu, lane >= 16 && sb > 127 + 7);
        } else {
          const uint32_t h = scale_pair<false>(sb);
          s01 = __byte_perm(__shfl_sync(0xffffffffu, h, 2 * c + 16),
                            __shfl_sync(0xffffffffu, h, 2 * c + 17), 0x5410);
          s23 = __byte_perm(__shfl_sync(0xffffffffu, h, 2 * c + 24),
                            __shfl_sync(0xffffffffu, h, 2 * c + 25), 0x5410);
        }
      } else if (!BF16) {
        s01 = s23 = pack2<false>(vf[0], vf[0]);
      }
      // ---- scores: f16 products with K's codes as A fragments, bytes 16 c on of rows g
      // and g + 8, then bytes 64 + 16 c on; one tile in two chains
      float sc[NT][4], s1[4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[t][j] = s1[j] = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint8_t* at = rk + ((g * 128 + ((c ^ g) << 4)) ^ (64 * hf));
        const uint4 a = *reinterpret_cast<const uint4*>(at);
        const uint4 b = *reinterpret_cast<const uint4*>(at + 1024);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint2 pa = word_pairs<false, I8>(aw[j]), pb = word_pairs<false, I8>(bw[j]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint2 q = R::Q_REGS ? make_uint2(qf[(8 * hf + 2 * j) % 16],
                                                   qf[(8 * hf + 2 * j + 1) % 16])
                                      : s.q[R::Q_REGS ? 0 : t][4 * hf + j][lane];
            mma16816<false>(NT == 1 && hf ? s1 : sc[t], pa.x, pb.x, pa.y, pb.y, q.x, q.y);
          }
        }
      }
      const bool masked = !(sl.key & WHOLE);  // some row does not see some key
      if (masked && p.scale_shift == 0) {
        // keys that no row sees may have any scale, and 0 * NaN is NaN (a block of 16
        // tokens or more that holds a seen key has a scale for it)
        const int k0 = sl.key & ~15;
        const Walk w(p, cur.n, cur.L, 0);
        if (BF16) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (!w.sees(k0 + g + 8 * j)) vf[j] = 0.f;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!w.sees(k0 + 2 * c + (j & 1) + 8 * (j >> 1))) {
              uint32_t& pair = j < 2 ? s01 : s23;
              pair &= (j & 1) ? 0x0000ffffu : 0xffff0000u;
            }
        }
      }
      // probabilities for bf16 come times V's scale (a power of two, so exactly), in O's
      // unit: at most 2^8 each, so that times 2^112 they want exponents of at most 7
      if (BF16) {
        const float unit = V_UNIT<I8> * (!I8 && !big ? 0x1p120f : 1.f);
        vf[0] *= unit;
        vf[1] *= unit;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sc[t][j] = (NT == 1 ? sc[t][j] + s1[j] : sc[t][j]) * (kf[j >> 1] * col[t][j & 1]);
      }
      if (masked) {
        const int k0 = sl.key & ~15;
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
      }
      // ---- the running maxima: moved when a score exceeds one by more than 8
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
              const float alpha = fast_exp2(M[t][j] - mx);
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
      // ---- probabilities as B fragments: rounded to 16 bits, as the products take them (l sums
      // the unrounded ones).  With o's own rounding o is off by 2.0e-3 of its norm in bf16 and
      // 2.5e-4 in fp16; 32-bit probabilities, 1.7e-3 and 2.1e-4, would take a second product
      // of what the rounding leaves.
      uint32_t pf[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = fast_exp2(sc[t][j] - M[t][j & 1]);
        l[t][0] += e[0] + e[2];
        l[t][1] += e[1] + e[3];
        if (BF16) {
          e[0] *= vf[0];
          e[1] *= vf[0];
          e[2] *= vf[1];
          e[3] *= vf[1];
        }
        pf[t][0] = transpose8x8(pack2<BF16>(e[0], e[1]));
        pf[t][1] = transpose8x8(pack2<BF16>(e[2], e[3]));
      }
      // ---- O^T += V^T P^T
      // V: bytes 16 g on of rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9
      const uint8_t* av = rv + 2 * c * 128 + ((g ^ (2 * c)) << 4);
      const uint8_t* bv = rv + (2 * c + 1) * 128 + ((g ^ (2 * c + 1)) << 4);
      uint4 v[4] = {*reinterpret_cast<const uint4*>(av), *reinterpret_cast<const uint4*>(bv),
                    *reinterpret_cast<const uint4*>(av + 1024),
                    *reinterpret_cast<const uint4*>(bv + 1024)};
      if (masked) {  // what no row sees may be anything
        const int k0 = sl.key & ~15;
        const Walk w(p, cur.n, cur.L, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (!w.sees(k0 + 2 * c + (j & 1) + 8 * (j >> 1))) v[j] = make_uint4(0u, 0u, 0u, 0u);
      }
      auto add_values = [&](auto bits) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = k == 0 ? v[j].x : k == 1 ? v[j].y : k == 2 ? v[j].z : v[j].w;
          uint32_t lo[4], hi[4];
          cross_pairs<BF16, I8, decltype(bits)::value>(w[0], w[1], lo);
          cross_pairs<BF16, I8, decltype(bits)::value>(w[2], w[3], hi);
          if (!BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              lo[j] = mul16x2<false>(lo[j], s01);
              hi[j] = mul16x2<false>(hi[j], s23);
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16816<BF16>(acc[t][2 * k], lo[0], lo[1], hi[0], hi[1], pf[t][0], pf[t][1]);
            mma16816<BF16>(acc[t][2 * k + 1], lo[2], lo[3], hi[2], hi[3], pf[t][0], pf[t][1]);
          }
        }
      };
      if constexpr (BF16 && !I8) {
        if (big)
          add_values(std::false_type());
        else
          add_values(std::true_type());
      } else {
        add_values(std::false_type());
      }
      __syncwarp();  // the stage is read
#pragma unroll
      for (int j = 0; j < LAG; ++j) way[j] = way[j + 1];
      --on_way;
      if (++from_stage == STAGES) {
        from_stage = 0;
        from_ph ^= 1u;
      }
    }
    if (!ok) {  // gives up: its copies in flight land first
      for (; on_way > 0 && !p.test_no_loads; --on_way) {
        mbar_drain_warp(smem_u32(&s.full[warp][from_stage]), from_ph, wc.timeout_ns);
        if (++from_stage == STAGES) {
          from_stage = 0;
          from_ph ^= 1u;
        }
      }
      on_way = 0;
      more = false;
      u_at = u_cnt;
    }

    // ---- the piece's end: the warps' shares meet, eight rows at a time (and the next
    // unit's rows of q are there behind the meeting)
    copies_wait();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], d);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (8 * t >= rows) break;
      __syncthreads();  // what was there is read
      // (nobody is at the unit before this one any more: its slot takes the one
      // after the next)
      if (t == 0 && warp == 0) s.pieces.next(p, &s.unit[next_slot == 2 ? 0 : next_slot + 1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = 8 * t + 2 * c + j;
        if (g == 0) {
          s.ml[warp][n][0] = M[t][j];
          s.ml[warp][n][1] = l[t][j];
        }
        float4* to = reinterpret_cast<float4*>(&s.O[warp][2 * c + j][16 * g]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          to[k] = make_float4(acc[t][2 * k][j], acc[t][2 * k][j + 2], acc[t][2 * k + 1][j],
                              acc[t][2 * k + 1][j + 2]);
      }
      __syncthreads();
      const int end = min(rows - 8 * t, 8) * 64;
      for (int i = threadIdx.x; i < end; i += R::THREADS) {
        const int m = i >> 6, n = 8 * t + m, d = 2 * (i & 63);
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
    parity ^= 1;
  }
  __syncthreads();
  if (threadIdx.x == 0 && s.bad_page) atomicCAS(&wc.status->code, 0u, (unsigned)ATTN_ERR_INVALID_ARG);
}

template <bool BF16, bool I8, int NT>
cudaError_t launch_rows(const Paged8Params& p, const CUtensorMap& tK, const CUtensorMap& tV,
                        const void* q, cudaStream_t st) {
  using R = rows_side::Rows<NT>;
  const auto kern = k_paged8_rows<BF16, I8, NT>;
  constexpr int smem = (int)sizeof(typename R::Smem) + 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)p.grid, R::THREADS, smem, st>>>(tK, tV, static_cast<const uint16_t*>(q), p);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_join<BF16>(p, st) : e;
}

template <bool BF16, bool I8>
cudaError_t launch_rows_of(const Paged8Params& p, const CUtensorMap& tK, const CUtensorMap& tV,
                           const void* q, cudaStream_t st) {
  return p.tile_rows <= 8 ? launch_rows<BF16, I8, 1>(p, tK, tV, q, st)
                          : launch_rows<BF16, I8, 2>(p, tK, tV, q, st);
}

cudaError_t launch_paged8_rows(bool bf16, bool i8, const Paged8Params& p, const CUtensorMap& tK,
                               const CUtensorMap& tV, const void* q, cudaStream_t st) {
  if (i8)
    return bf16 ? launch_rows_of<true, true>(p, tK, tV, q, st)
                : launch_rows_of<false, true>(p, tK, tV, q, st);
  return bf16 ? launch_rows_of<true, false>(p, tK, tV, q, st)
              : launch_rows_of<false, false>(p, tK, tV, q, st);
}

}  // namespace mab
