// paged8_chunk.cu -- attention of chunks of new tokens over an 8-bit paged cache.
//
// The same operation, work line, cuts and join as over 16-bit pages (paged_fwd.cu
// gives the formulas), on the tensor cores: S = Q K^T and O += P V over 64 keys a
// step, with Q and P in TMEM.  The matrix unit reads 16-bit tiles of K and V from
// shared memory, so eight warps make them of the codes that the loads bring: code
// times scale, exactly (quant8.cuh), zeros for rows that no row of the unit sees.
//
// What bounds it is that way through shared memory beside the matrix unit's own:
// a step brings 16 KB of codes in and out, writes 32 KB of tiles and reads them once
// for each 128 query rows.  So a unit is a tile of 256 query rows (token, head of the
// group), two halves that share the tiles: 128 KB and 1024 cycles either way, of
// which the tensor pipe's work is 1024 too.  (With 128 rows a step, alternate steps
// to two softmax groups, chunks of 1900 over 8000 keys took 813 us.)
//
// Each half has an issuing warp, a group of four softmax warps, its own S buffer,
// accumulator, maximum and sum, and nothing to say to the other.  One S buffer is
// enough: O += P V of a step and S of the next are issued together, in that order,
// so the commit after S also says that P has been read and O is complete, which is
// all that the next step's P and rescaling need.  While a half's softmax runs, the
// other half's 512 cycles of products do.
//
// Warps: loader; an issuing warp per half; four softmax warps per half; four
// converting warps for K and four for V, each 16 rows of every step, half a row a
// thread, whose pages and scales it looks up 32 steps at a time, a batch ahead.  The
// softmax warps' registers come from the other warps' (setmaxnreg).
#include <type_traits>

#include "paged_line.cuh"
#include "quant8.cuh"

namespace mab {

namespace chunk_side {

using namespace paged_side;

constexpr int HALF = PAGED8_TILE / 2;  // 128 rows, the matrix unit's
constexpr int STAGES = 3;              // ring of 16-bit K / V tiles
constexpr int LD_STAGES = 3;           // ring of codes
constexpr int COL_O = 0;               // accumulator of half t at COL_O + 128 t
constexpr int COL_Q = 256;             // Q as the A operand, 64 columns of pairs, + 64 t
constexpr int COL_S = 384;             // S, then P, + 64 t
constexpr int SM_WARP0 = 4, SM_WARPS = 8;
constexpr int CV_WARP0 = 12, CV_WARPS = 8;
constexpr int NUM_THREADS = 32 * (CV_WARP0 + CV_WARPS);
constexpr int AHEAD = 8;  // steps of a unit issued before the next one's Q
// registers of the warps that wait and convert (12), and of the softmax warps (8):
// of 20 * 96 that are launched
constexpr int REGS_FEW = 56, REGS_SOFTMAX = 152;
static_assert(12 * REGS_FEW + 8 * REGS_SOFTMAX <= 20 * 96 && NUM_THREADS == 20 * 32,
              "shares of the launch's registers");

struct __align__(1024) Smem {
  uint8_t Q[2][PAGED8_TILE * 128];  // two 64-column chunks, 128B swizzle; once copied into
                                    // TMEM, the epilogue staging
  uint8_t K[STAGES][2 * Q_SUB * 128];
  uint8_t V[STAGES][2 * Q_SUB * 128];
  uint8_t K8[LD_STAGES][Q_SUB * 128];
  uint8_t V8[LD_STAGES][Q_SUB * 128];
  uint8_t scales[CV_WARPS][2][32][16];  // [warp][batch][step][row]
  LineSums<NUM_THREADS> sums;
  PagedStart cut[2];            // where this CTA's part begins and ends
  Unit unit;                    // piece of the latest Q load, N < 0: none left
  uint64_t bar_q_full;
  uint64_t bar_qa_full;         // Q copied into TMEM (all softmax warps)
  uint64_t bar_ld_full[LD_STAGES];
  uint64_t bar_ld_empty[LD_STAGES];
  uint64_t bar_kv_full[STAGES];
  uint64_t bar_kv_empty[STAGES];  // both halves' O += P V that read the stage complete
  uint64_t bar_s_full[2];       // [half]: S of a step complete, and all before it
  uint64_t bar_p_full[2];       // P packed (the half's four warps)
  uint64_t bar_acc_full[2];     // every MMA of the half's piece complete
  uint64_t bar_acc_empty;       // both accumulators read (all softmax warps)
  uint64_t bar_unit_free;       // every other warp took the unit (and, softmax warps,
                                // left the previous unit's rows)
  uint64_t bar_x_done[2];       // every MMA of an issuing warp complete
  uint32_t tmem_base;
  int abort_flag;
};

constexpr size_t SMEM_BYTES = sizeof(Smem) + 1024;
static_assert(SMEM_BYTES <= 232448, "over the 227 KB of shared memory a CTA may use");
static_assert((PAGED_MAX_B + 1) * 8 + PAGED_MAX_B * 12 <= sizeof(Smem::K) + sizeof(Smem::V),
              "the line of the most requests fits the ring");

}  // namespace chunk_side

template <bool BF16, bool I8>
__global__ void __launch_bounds__(chunk_side::NUM_THREADS, 1)
k_paged8_chunk(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
               const __grid_constant__ CUtensorMap tV, const __grid_constant__ Paged8Params p) {
  using namespace chunk_side;
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                     ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's own status word, which the join passes on
  WaitCtx wc{p.cta_status + blockIdx.x, &s.abort_flag, p.timeout_ns};

  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    *wc.status = DevStatus{};
    mbar_init(smem_u32(&s.bar_q_full), 1);
    mbar_init(smem_u32(&s.bar_qa_full), SM_WARPS);
    for (int i = 0; i < LD_STAGES; ++i) {
      mbar_init(smem_u32(&s.bar_ld_full[i]), 1);
      mbar_init(smem_u32(&s.bar_ld_empty[i]), CV_WARPS);
    }
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&s.bar_kv_full[i]), CV_WARPS);
      mbar_init(smem_u32(&s.bar_kv_empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.bar_s_full[i]), 1);
      mbar_init(smem_u32(&s.bar_p_full[i]), SM_WARPS / 2);
      mbar_init(smem_u32(&s.bar_acc_full[i]), 1);
      mbar_init(smem_u32(&s.bar_x_done[i]), 1);
    }
    mbar_init(smem_u32(&s.bar_acc_empty), SM_WARPS);
    mbar_init(smem_u32(&s.bar_unit_free), SM_WARPS + 2 + CV_WARPS);
    fence_mbar_init();
    tma_prefetch_desc(&tQ);
    tma_prefetch_desc(&tK);
    tma_prefetch_desc(&tV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = s.tmem_base;
  grid_launch_dependents();  // the join's blocks may wait beside this grid
  {
    const Line line = line_at(s.K, p.B);
    const int parts = lay_line(p, line, s.sums);
    if (warp < 2) {
      const PagedStart at = cut_of(p, line, parts, (int)blockIdx.x + warp);
      if (lane == 0) {
        s.cut[warp] = at;
        if (warp == 1) p.start[blockIdx.x + 1] = at;  // for the join
      }
    }
    __syncthreads();
  }
  if (warp >= SM_WARP0 && warp < CV_WARP0)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_FEW));

  if (warp == 0) {
    // ------------------------------------------------------------ loader of Q and codes
    const int cta = (int)blockIdx.x;
    const PagedStart at0 = s.cut[0], end = s.cut[1];
    int b = at0.b, kvh = at0.kvh, tile = at0.tile, step = at0.step;  // where this CTA stands
    int off = at0.off, n = at0.n, L = at0.L;                         // of request b
    bool ok = !p.test_no_loads;
    int q_loaded = -1;  // last unit whose Q tile was loaded
    int m_load = 0;     // steps issued, across units
    Cyc<LD_STAGES> rg;
    // lane i holds the lengths of request b_base + i (none yet: the first
    // request's came with the start)
    int b_base = b - 32, l_off = 0, l_n = 0, l_L = 0;
    const uint32_t qbar = smem_u32(&s.bar_q_full);
    // Publishes unit j and loads its Q once the slot and the Q tile are free;
    // then stands at the unit after it.
    Unit next;
    auto publish = [&](int j) -> bool {
      if (j >= 1 &&
          !mbar_wait_sleep_warp(smem_u32(&s.bar_unit_free), (j - 1) & 1, wc, TAG_UNIT_FREE,
                                LOAD_SLEEP_NS))
        return false;
      const bool in_end = b == end.b && kvh == end.kvh && tile == end.tile;
      if (b >= p.B || (in_end && end.step <= step)) {
        next.N = -1;  // none is left
        if (lane == 0) {
          s.unit.N = -1;
          mbar_arrive(qbar);
        }
        return true;
      }
      next.b = b;
      next.kvh = kvh;
      next.off = off;
      next.n = n;
      next.L = L;
      next.tok0 = tile * p.tile_tokens;
      next.s0 = step;
      next.N = (in_end ? end.step : Walk(p, n, L, next.tok0).cnt) - step;
      // slots: 2 c for a piece that goes on with a unit, 2 c + 1 for its first one
      next.whole = step == 0 && !(in_end && end.step > 0);
      next.slot = 2 * cta + (step > 0 ? 0 : 1);
      if (lane == 0) {
        s.unit = next;
        if (next.N == 0) {
          mbar_arrive(qbar);  // no key to see: no Q either
        } else {
          const int row = off + next.tok0;
          mbar_arrive_expect_tx(qbar, 2 * p.tile_rows * 128);
          tma_load_3d(smem_u32(s.Q[0]), &tQ, 0, kvh * p.group, row, qbar);
          tma_load_3d(smem_u32(s.Q[1]), &tQ, 64, kvh * p.group, row, qbar);
        }
      }
      __syncwarp();
      if (next.N > 0) q_loaded = j;
      if (in_end) {  // nothing of this CTA is left
        step = end.step;
        return true;
      }
      step = 0;
      if (++tile * p.tile_tokens < n) return true;
      tile = 0;
      if (++kvh < p.Hkv) return true;
      kvh = 0;
      // the next request with new tokens
      for (n = 0; n == 0 && ++b < p.B;) {
        if (b >= b_base + 32) {
          b_base = b;
          l_off = l_n = l_L = 0;
          if (b_base + lane < p.B) {
            l_off = packed_off(p.cu_q, b_base + lane, p.total_q);
            l_n = new_tokens(p, b_base + lane);
            l_L = keys_of(p, b_base + lane);
          }
        }
        off = __shfl_sync(0xffffffffu, l_off, b - b_base);
        n = __shfl_sync(0xffffffffu, l_n, b - b_base);
        L = __shfl_sync(0xffffffffu, l_L, b - b_base);
        if (b == end.b) break;
      }
      return true;
    };
    // Steps [s0, s0 + N) of a unit: the boxes of each step into its stage, once
    // that is free; the unit after it is published before step AHEAD.
    auto load_steps = [&](const Unit un, int j, bool* ahead) -> bool {
      const Walk w(p, un.n, un.L, un.tok0);
      const int runs = Q_SUB / p.box_rows;
      const int batch = 32 / runs;  // steps whose pages the lanes look up at once
      const int* row = p.table + (size_t)un.b * p.table_stride;
      // lane l has run l % runs of step i + l / runs: its first key, whether it
      // holds a seen one, and its page (past the last where it holds none) and
      // first row there
      const int l_step = lane / runs, l_run = lane - l_step * runs;
      auto key_of = [&](int i) { return w.tile(i + l_step) * Q_SUB + l_run * p.box_rows; };
      auto seen = [&](int i, int k0) {
        return i + l_step < un.s0 + un.N && w.any(k0, k0 + p.box_rows);
      };
      int row0 = 0;
      auto pages_of = [&](int i) -> int {
        const int k0 = key_of(i);
        const int idx = div_by(k0, p.page_size, p.inv_page_size);
        row0 = k0 - idx * p.page_size;
        return seen(i, k0) ? __ldg(row + idx) : p.num_pages;
      };
      int page = p.num_pages, prow = 0, nxt = pages_of(un.s0), next_row = row0, left = 0;
      for (int i = un.s0; i < un.s0 + un.N; ++i, ++m_load, rg.next(), --left) {
        if (i == un.s0 + AHEAD) {
          *ahead = true;
          if (!publish(j + 1)) return false;
        }
        if (left == 0) {
          page = nxt;
          prow = next_row;
          left = batch;
          if ((unsigned)page >= (unsigned)p.num_pages) {
            // past the tensor's end, where a load reads zeros
            if (seen(i, key_of(i)))
              atomicCAS(&wc.status->code, 0u, (unsigned)ATTN_ERR_INVALID_ARG);
            page = p.num_pages;
          }
          nxt = pages_of(i + batch);  // a batch ahead
          next_row = row0;
        }
        if (m_load >= LD_STAGES &&
            !mbar_wait_sleep_warp(smem_u32(&s.bar_ld_empty[rg.i]), rg.ph ^ 1u, wc, TAG_LD_EMPTY,
                                  LOAD_SLEEP_NS))
          return false;
        const uint32_t fb = smem_u32(&s.bar_ld_full[rg.i]);
        if (lane == 0) mbar_arrive_expect_tx(fb, 2 * Q_SUB * 128);
        __syncwarp();
        const uint32_t dst_k = smem_u32(s.K8[rg.i]), dst_v = smem_u32(s.V8[rg.i]);
        for (int r = 0; r < runs; ++r) {
          const int src = (batch - left) * runs + r;
          const int pg = __shfl_sync(0xffffffffu, page, src);
          const int pr = __shfl_sync(0xffffffffu, prow, src);
          tma_load_4d_w(dst_k + r * p.box_rows * 128, &tK, 0, pr, un.kvh, pg, fb);
          tma_load_4d_w(dst_v + r * p.box_rows * 128, &tV, 0, pr, un.kvh, pg, fb);
        }
      }
      return true;
    };
    bool ahead = false;  // the unit after the one being loaded is published
    for (int j = 0; ok; ++j) {
      if (!ahead) ok = publish(j);
      if (!ok || next.N < 0) break;
      ahead = false;
      ok = load_steps(next, j, &ahead);
    }
    if (!ok) {  // a CTA that gives up lets the copies still in flight land first
      if (q_loaded >= 0) mbar_drain_warp(qbar, q_loaded & 1, wc.timeout_ns);
      for (int k = m_load > LD_STAGES ? m_load - LD_STAGES : 0; k < m_load; ++k)
        mbar_drain_warp(smem_u32(&s.bar_ld_full[k % LD_STAGES]), (k / LD_STAGES) & 1,
                        wc.timeout_ns);
    }
  } else if (warp < 3) {
    // ------------------------------------------------------------ MMA issuers (whole warps)
    constexpr uint32_t ID_S = idesc_f16(BF16, HALF, Q_SUB, false, false);
    constexpr uint32_t ID_O = idesc_f16(BF16, HALF, HEAD_DIM, false, true);
    const int t = warp - 1;
    const uint32_t col_s = tbase + COL_S + 64 * t, col_o = tbase + COL_O + 128 * t;
    bool ok = true;
    int cnt = 0;  // steps of this half so far
    Cyc<STAGES> rg;
    auto issue_s = [&](int st) {
      const uint64_t bK = sdesc_sw128(smem_u32(s.K[st]), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < HEAD_DIM / 16; ++kk)
        mma_ts_w(col_s, tbase + COL_Q + 64 * t + 8 * kk,
                 bK + (uint64_t)(((kk >> 2) * (Q_SUB * 128) + (kk & 3) * 32) >> 4), ID_S,
                 kk > 0 ? 1u : 0u);
      mma_commit_w(smem_u32(&s.bar_s_full[t]));
    };
    for (int j = 0; ok; ++j) {
      if (!mbar_wait_warp(smem_u32(&s.bar_q_full), j & 1, wc, TAG_Q)) break;
      const int N = s.unit.N;
      if (N < 0) break;
      // rows of the second half are there
      const bool active =
          t == 0 || min(p.tile_tokens, s.unit.n - s.unit.tok0) * p.group > HALF;
      ok = mbar_wait_warp(smem_u32(&s.bar_qa_full), j & 1, wc, TAG_QA);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.bar_unit_free));
      if (!ok) break;
      if (active && N > 0) {
        ok = mbar_wait_warp(smem_u32(&s.bar_kv_full[rg.i]), rg.ph, wc, TAG_KV_FULL);
        if (!ok) break;
        tc_fence_after();
        issue_s(rg.i);
      }
      for (int i = 0; ok && i < N; ++i) {
        const int st = rg.i;
        const uint32_t ph = rg.ph;
        rg.next();
        if (!active) {  // the stage is free of this half once it is there
          ok = mbar_wait_warp(smem_u32(&s.bar_kv_full[st]), ph, wc, TAG_KV_FULL);
          if (ok && lane == 0) mbar_arrive(smem_u32(&s.bar_kv_empty[st]));
          continue;
        }
        if (i + 1 < N) ok = mbar_wait_warp(smem_u32(&s.bar_kv_full[rg.i]), rg.ph, wc, TAG_KV_FULL);
        // the unit's first accumulation overwrites the accumulator: the softmax warps
        // must have read the previous unit's
        if (ok && i == 0 && j >= 1)
          ok = mbar_wait_warp(smem_u32(&s.bar_acc_empty), (j - 1) & 1, wc, TAG_ACC_EMPTY);
        ok = ok && mbar_wait_warp(smem_u32(&s.bar_p_full[t]), cnt & 1, wc, TAG_P_FULL);
        ++cnt;
        if (!ok) break;
        tc_fence_after();
        const uint64_t bV = sdesc_sw128(smem_u32(s.V[st]), Q_SUB * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < Q_SUB / 16; ++kk)
          mma_ts_w(col_o, col_s + 8 * kk, bV + (uint64_t)((kk * 2048) >> 4), ID_O,
                   (i > 0 || kk > 0) ? 1u : 0u);
        mma_commit_w(smem_u32(&s.bar_kv_empty[st]));
        if (i + 1 < N) issue_s(rg.i);  // over P, after the MMAs that read it
      }
      // (a unit without accumulations here: the signal must not come a phase before the
      // softmax warps wait for the previous unit's)
      if (ok && j >= 1 && !(active && N > 0))
        ok = mbar_wait_warp(smem_u32(&s.bar_acc_empty), (j - 1) & 1, wc, TAG_ACC_EMPTY);
      if (ok) mma_commit_w(smem_u32(&s.bar_acc_full[t]));  // the accumulator is complete
    }
    // this warp's MMAs must be complete before TMEM is freed (also when the
    // CTA gave up, hence a wait that ignores the abort flag)
    const uint32_t done = smem_u32(&s.bar_x_done[t]);
    mma_commit_w(done);
    mbar_drain_warp(done, 0, wc.timeout_ns);
  } else if (warp >= SM_WARP0 && warp < CV_WARP0) {
    // ------------------------------------------------------------ softmax warps
    const int sp = warp & 3, t = (warp - SM_WARP0) >> 2;
    const int row0 = t * HALF + sp * 32, rloc = row0 + lane;  // of the tile
    const int tl = rloc / p.group, hh = rloc - tl * p.group;  // the row's token and head
    const uint32_t lane_base = tbase + ((uint32_t)(sp * 32) << 16);
    const uint32_t col_o = lane_base + COL_O + 128 * t, col_s = lane_base + COL_S + 64 * t;
    // Scales the accumulator of unit j and stores it (a whole unit), or leaves it in the
    // workspace for the join (a piece); staged through the Q rows this warp itself
    // copies.  Arrives on acc_empty, and on unit_free of the unit after it (whose Q this
    // warp has copied) once the staging space is not needed any more.
    auto epilogue = [&](int j, const Unit& un, float M, float l, bool ok) {
      // rows of this warp that are a token of the request
      const int nr = min(32, min(p.tile_tokens, un.n - un.tok0) * p.group - row0);
      const bool mine = lane < nr;
      const int tok = un.off + un.tok0 + tl, head = un.kvh * p.group + hh;
      const long long row_at = mine ? (long long)tok * p.Hq + head : -1;
      float* part = p.part + (size_t)un.slot * p.slot_floats +
                    2 * (row0 >> 5) * PAGED_WARP_FLOATS;
      float inv = 1.f;
      if (un.whole) {
        const float lse =
            finish_row(M, l, p.sink && mine ? p.sink[head] * LOG2E : -INFINITY, &inv);
        if (p.lse && mine && ok) p.lse[(size_t)head * p.total_q + tok] = lse;
      } else if (mine) {
        part[PAGED_ML + 2 * lane] = M;
        part[PAGED_ML + 2 * lane + 1] = l;
      }
      // a row that saw nothing has zeros in its accumulator, or nothing was computed
      ok = ok && mbar_wait_warp(smem_u32(&s.bar_acc_full[t]), j & 1, wc, TAG_ACC);
      tc_fence_after();
      // 16 columns at a time, in a loop: this code runs once a unit, and as one straight
      // piece most of its time would go into fetching it
      if (ok && nr > 0) {
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          float a[16];
          if (un.N > 0) {
            tmem_ld16(col_o + 16 * q, a);
            tmem_wait_ld_regs(a);
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) a[c] = 0.f;
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 x = fmul2(make_float2(a[2 * c], a[2 * c + 1]), inv2);
            a[2 * c] = x.x;
            a[2 * c + 1] = x.y;
          }
          if constexpr (BF16) {  // back from the converted tiles' order of d
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float x = a[4 * c + 1];
              a[4 * c + 1] = a[4 * c + 2];
              a[4 * c + 2] = x;
            }
          }
          if (un.whole) {
            // through shared memory, so that a row's 128 bytes leave together
            uint8_t* stage = s.Q[q >> 2] + rloc * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<uint4*>(stage + (((2 * (q & 3) + h) ^ (lane & 7)) << 4)) =
                  make_uint4(pack2<BF16>(a[8 * h], a[8 * h + 1]),
                             pack2<BF16>(a[8 * h + 2], a[8 * h + 3]),
                             pack2<BF16>(a[8 * h + 4], a[8 * h + 5]),
                             pack2<BF16>(a[8 * h + 6], a[8 * h + 7]));
          } else if (mine) {
            float* to = part + (q >> 2) * PAGED_WARP_FLOATS;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *part_at(to, lane, 4 * (q & 3) + c) =
                  make_float4(a[4 * c], a[4 * c + 1], a[4 * c + 2], a[4 * c + 3]);
          }
        }
      }
      // the accumulator is read: the next unit's O may begin
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.bar_acc_empty));
      if (ok && nr > 0 && un.whole) {
#pragma unroll 4
        for (int k = 0; k < 16; ++k) {
          const int row = (k >> 1) * 4 + (lane >> 3), c = lane & 7;
          const long long to = __shfl_sync(0xffffffffu, row_at, row);
          const uint4 v = *reinterpret_cast<const uint4*>(s.Q[k & 1] + (row0 + row) * 128 +
                                                          ((c ^ (row & 7)) << 4));
          if (to >= 0)
            *reinterpret_cast<uint4*>(p.out + to * HEAD_DIM + 64 * (k & 1) + c * 8) = v;
        }
      }
      // the next TMA load into the Q tile comes after this warp's generic
      // accesses to it
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.bar_unit_free));
    };
    bool ok = true;
    int cnt = 0;  // steps of this half so far
    Unit prev{};
    float prev_M = -INFINITY, prev_l = 0.f;
    for (int j = 0;; ++j) {
      ok = ok && mbar_wait_warp(smem_u32(&s.bar_q_full), j & 1, wc, TAG_Q);
      const Unit un = s.unit;
      const bool last = !ok || un.N < 0;  // no unit: only the previous one's epilogue
      const int rows = min(p.tile_tokens, un.n - un.tok0) * p.group;
      const bool busy = row0 < rows;                   // some row of this warp is a token's
      const bool active = t == 0 || rows > HALF;       // ... of this half
      // Q rows into TMEM as 16-bit pairs (every S of this half's previous unit has been
      // waited for)
      if (!last && busy && un.N > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* src = s.Q[h] + rloc * 128;
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + ((c ^ (rloc & 7)) << 4));
            w[4 * c] = v.x;
            w[4 * c + 1] = v.y;
            w[4 * c + 2] = v.z;
            w[4 * c + 3] = v.w;
          }
          if constexpr (BF16) {  // the order of d in the converted tiles
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const uint32_t a = w[2 * c], b = w[2 * c + 1];
              w[2 * c] = __byte_perm(a, b, 0x5410);
              w[2 * c + 1] = __byte_perm(a, b, 0x7632);
            }
          }
          tmem_st32(lane_base + COL_Q + 64 * t + 32 * h, w);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.bar_qa_full));
      // the previous unit's epilogue overlaps this unit's first MMAs
      if (j >= 1) {
        epilogue(j - 1, prev, prev_M, prev_l, ok);
      } else if (lane == 0) {
        mbar_arrive(smem_u32(&s.bar_unit_free));
      }
      if (last) break;

      // this row's running maximum M (log2 domain) and sum (the sink joins in the
      // epilogue)
      float M = -INFINITY, l = 0.f;
      const Walk w(p, un.n, un.L, un.tok0);
      // the row's position and the end of the keys it may see; rows that are no
      // token's see nothing
      const int x0 = un.L - un.n + un.tok0, x = x0 + tl;
      const int key_end = rloc >= rows ? 0 : p.causal ? max(x + 1, 0) : un.L;
      // sub-tiles that every row of this warp sees whole: [full_lo, full_hi] (before the
      // first row's position and within the last one's window), and those up to
      // full_first among the first keys
      const int x_first = x0 + row0 / p.group;
      const int x_last = x0 + (min(rows, row0 + 32) - 1) / p.group;
      const int all_end = p.causal ? x_first + 1 : un.L;
      const int full_hi = all_end < Q_SUB ? -1 : all_end / Q_SUB - 1;
      const int full_lo =
          !p.causal || x_last < p.window ? 0 : (x_last - p.window + Q_SUB) / Q_SUB;
      const int full_first = min(full_hi, p.first / Q_SUB - 1);
      // sub-tiles that no row of this warp sees a key of: past the last row's position, or
      // before the first row's window and past the first keys
      auto unseen = [&](int tile) {
        if (!p.causal) return false;
        const int k0 = tile * Q_SUB;
        return k0 > x_last || (k0 + Q_SUB <= x_first - p.window + 1 && k0 >= p.first);
      };
      // Takes a step's row maximum mx (raw logits; the scale is positive, so it is applied
      // once here).  M moves when mx exceeds it by more than 8; a row that has seen nothing
      // yet (M = -inf, so O and l are still zero) just takes the new value.  The O rows of a
      // warp in which some M moved are rescaled: O += P V of every step before is complete
      // (the unit's first accumulation overwrites instead).
      auto move_max = [&](int i, float mx) {
        const float mx2 = mx == -INFINITY ? -INFINITY : mx * p.scale_log2;
        float alpha = 1.f;
        if (mx2 > M + RESCALE_LOG2) {
          if (M != -INFINITY) alpha = fast_exp2(M - mx2);
          M = mx2;
          l *= alpha;
        }
        if (i >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t v[32];
            tmem_ld32(col_o + 32 * q, reinterpret_cast<float(&)[32]>(v));
            tmem_wait_ld_regs(reinterpret_cast<float(&)[32]>(v));
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * alpha);
            tmem_st32(col_o + 32 * q, v);
          }
        }
      };
      // P = exp2(S scale log2e - M): an invisible logit (-inf) gives 0; a row
      // with nothing visible keeps M = -inf and all its logits at -inf, and the
      // finite stand-in keeps -inf - (-inf) out
      auto minus_max = [&]() { return M == -INFINITY ? 0.f : -M; };
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
      // A sub-tile that every row of the warp sees whole: P packed over S.
      auto whole_step = [&](int i) {
        float sv[64];
        tmem_ld32(col_s, *reinterpret_cast<float(*)[32]>(&sv[0]));
        tmem_ld32(col_s + 32, *reinterpret_cast<float(*)[32]>(&sv[32]));
        tmem_wait_ld_regs(sv);
        // eight partial maxima and four sums keep the dependency chains short
        float mp[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mp[c] = fmaxf(sv[2 * c], sv[2 * c + 1]);
#pragma unroll
        for (int c = 8; c < 32; ++c) mp[c & 7] = fmax3f(mp[c & 7], sv[2 * c], sv[2 * c + 1]);
        move_max(i, fmax3f(fmax3f(mp[0], mp[1], mp[2]), fmax3f(mp[3], mp[4], mp[5]),
                           fmaxf(mp[6], mp[7])));
        const float nm = minus_max();
        const float2 nm2 = make_float2(nm, nm);
        uint32_t pk[32];
        float2 lp[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) lp[c] = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 xx = ffma2(make_float2(sv[2 * c], sv[2 * c + 1]), sc2, nm2);
          const float2 pp = make_float2(fast_exp2(xx.x), fast_exp2(xx.y));
          lp[c & 3] = fadd2(lp[c & 3], pp);
          pk[c] = pack2<BF16>(pp.x, pp.y);
        }
        const float2 ls = fadd2(fadd2(lp[0], lp[1]), fadd2(lp[2], lp[3]));
        l += ls.x + ls.y;
        tmem_st32(col_s, pk);
      };
      // A sub-tile from key j0 on that some row does not see whole: two passes of 32
      // columns at a time, in loops (it runs a few times a unit).
      auto masked_step = [&](int i, int j0) {
        auto load32 = [&](int q, float (&v)[32]) {
          tmem_ld32(col_s + 32 * q, v);
          const int k0 = j0 + 32 * q;
          uint32_t vis = bit_range(0, key_end - 1 - k0);
          if (p.causal)
            vis &= bit_range(x - p.window + 1 - k0, 31) | bit_range(0, p.first - 1 - k0);
          tmem_wait_ld_regs(v);
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = ((vis >> c) & 1u) ? v[c] : -INFINITY;
        };
        float mx = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          float v[32];
          load32(q, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) mx = fmax3f(mx, v[2 * c], v[2 * c + 1]);
        }
        move_max(i, mx);
        const float nm = minus_max();
        const float2 nm2 = make_float2(nm, nm);
        float2 ls = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          float v[32];
          load32(q, v);
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 xx = ffma2(make_float2(v[2 * c], v[2 * c + 1]), sc2, nm2);
            const float2 pp = make_float2(fast_exp2(xx.x), fast_exp2(xx.y));
            ls = fadd2(ls, pp);
            pk[c] = pack2<BF16>(pp.x, pp.y);
          }
          // over columns that have been read: 16 q + 15 < 32 q + 32
          tmem_st16(col_s + 16 * q, pk);
        }
        l += ls.x + ls.y;
      };
      if (active) {
        for (int i = 0; ok && i < un.N; ++i) {
          const int tile = w.tile(un.s0 + i);
          // warp-uniform: every row of the warp sees every key of the sub-tile
          const bool full = (tile >= full_lo && tile <= full_hi) || tile <= full_first;
          ok = mbar_wait_warp(smem_u32(&s.bar_s_full[t]), cnt & 1, wc, TAG_S_FULL);
          if (!ok) break;
          ++cnt;
          if (busy) {
            tc_fence_after();
            if (full) {
              whole_step(i);
            } else if (unseen(tile)) {
              uint32_t zero[32];
#pragma unroll
              for (int c = 0; c < 32; ++c) zero[c] = 0u;
              tmem_st32(col_s, zero);
            } else {
              masked_step(i, tile * Q_SUB);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.bar_p_full[t]));
        }
      }
      prev = un;
      prev_M = M;
      prev_l = l;
    }
  } else if (warp >= CV_WARP0) {
    // ------------------------------------------------------------ converting warps
    const int cw = warp - CV_WARP0, slice = cw & 3;
    const bool is_v = cw >= 4;
    const uint8_t* all_scales = is_v ? p.v_scales : p.k_scales;
    // this thread's row of a step, and which half of it
    const int srow = lane >> 1, row = 16 * slice + srow, half = lane & 1;
    bool ok = true;
    Cyc<LD_STAGES> lg;
    Cyc<STAGES> rg;
    int m = 0;  // step counter across units
    for (int j = 0; ok; ++j) {
      if (!mbar_wait_warp(smem_u32(&s.bar_q_full), j & 1, wc, TAG_Q)) break;
      const int N = s.unit.N, s0 = s.unit.s0, kvh = s.unit.kvh;
      if (N < 0) break;
      const Walk w(p, s.unit.n, s.unit.L, s.unit.tok0);
      const int* table = p.table + (size_t)s.unit.b * p.table_stride;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.bar_unit_free));
      // Lane l looks up step i + l of the piece: the page of this warp's 16 rows there
      // (-1 where none of them is seen, or the page is not there), and their scales.
      auto page_of = [&](int i) -> int {
        const int k0 = w.tile(s0 + i + lane) * Q_SUB + 16 * slice;
        if (i + lane >= N || !w.any(k0, k0 + 16)) return -1;
        const int pg = __ldg(table + div_by(k0, p.page_size, p.inv_page_size));
        return (unsigned)pg < (unsigned)p.num_pages ? pg : -1;
      };
      auto scales_of = [&](int i, int pg) -> uint4 {
        if (pg < 0) return make_uint4(0u, 0u, 0u, 0u);
        const int k0 = w.tile(s0 + i + lane) * Q_SUB + 16 * slice;
        const int r = k0 - div_by(k0, p.page_size, p.inv_page_size) * p.page_size;
        const long long at =
            pg * p.scale_page_stride + kvh * p.scale_head_stride + (r >> p.scale_shift);
        if (p.scale_shift == 0) return __ldg(reinterpret_cast<const uint4*>(all_scales + at));
        const uint32_t a = __ldg(all_scales + at) * 0x01010101u;
        return make_uint4(a, a, a, a);
      };
      uint4 sc = scales_of(0, page_of(0));
      int page = page_of(32);
      for (int i = 0; ok && i < N; ++i, ++m, lg.next(), rg.next()) {
        if ((i & 31) == 0) {
          __syncwarp();  // the batch before the last is read
          *reinterpret_cast<uint4*>(s.scales[cw][(i >> 5) & 1][lane]) = sc;
          __syncwarp();
          sc = scales_of(i + 32, page);  // a batch ahead
          page = page_of(i + 64);
        }
        const int sb = s.scales[cw][(i >> 5) & 1][i & 31][srow];
        const bool seen = w.sees(w.tile(s0 + i) * Q_SUB + row);
        // e4m3 to bf16: one product while every exponent is at most 7
        const bool small = BF16 && !I8 && !__any_sync(0xffffffffu, seen && sb > 127 + 7);
        const uint32_t scale2 = scale_pair<BF16>(small ? min(max(sb, 1) + 120, 254) : sb);
        ok = mbar_wait_warp(smem_u32(&s.bar_ld_full[lg.i]), lg.ph, wc, TAG_LD_FULL);
        if (ok && m >= STAGES)
          ok = mbar_wait_warp(smem_u32(&s.bar_kv_empty[rg.i]), rg.ph ^ 1u, wc, TAG_KV_EMPTY);
        if (!ok) break;
        const uint8_t* from = (is_v ? s.V8[lg.i] : s.K8[lg.i]) + row * 128;
        uint8_t* to = (is_v ? s.V[rg.i] : s.K[rg.i]) + half * (Q_SUB * 128) + row * 128;
        auto convert = [&](auto one) {
          constexpr bool SMALL = decltype(one)::value;
          // 16-byte units: 4 half + c of the code row become 2 c and 2 c + 1 of the
          // half's 128-byte row, both swizzled by the row; the halves take them in
          // orders that keep them off each other's banks
          uint4 v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[c] = *reinterpret_cast<const uint4*>(
                from + (((4 * half + (c ^ (half << 1))) ^ (row & 7)) << 4));
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            const int c = cc ^ (half << 1);
            uint2 a = tile_words<BF16, I8, SMALL>(v[cc].x, scale2);
            uint2 b = tile_words<BF16, I8, SMALL>(v[cc].y, scale2);
            uint2 d = tile_words<BF16, I8, SMALL>(v[cc].z, scale2);
            uint2 e = tile_words<BF16, I8, SMALL>(v[cc].w, scale2);
            if (!seen) a = b = d = e = make_uint2(0u, 0u);
            *reinterpret_cast<uint4*>(to + (((2 * c) ^ (row & 7)) << 4)) =
                make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4*>(to + (((2 * c + 1) ^ (row & 7)) << 4)) =
                make_uint4(d.x, d.y, e.x, e.y);
          }
        };
        if constexpr (BF16 && !I8) {
          if (small)
            convert(std::true_type());
          else
            convert(std::false_type());
        } else {
          convert(std::false_type());
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&s.bar_kv_full[rg.i]));
          mbar_arrive(smem_u32(&s.bar_ld_empty[lg.i]));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <bool BF16, bool I8>
cudaError_t launch_chunk(const Paged8Params& p, const CUtensorMap& tQ, const CUtensorMap& tK,
                         const CUtensorMap& tV, cudaStream_t st) {
  using namespace chunk_side;
  const auto kern = k_paged8_chunk<BF16, I8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)SMEM_BYTES);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)p.grid, NUM_THREADS, SMEM_BYTES, st>>>(tQ, tK, tV, p);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_join<BF16>(p, st) : e;
}

cudaError_t launch_paged8_chunk(bool bf16, bool i8, const Paged8Params& p, const CUtensorMap& tQ,
                                const CUtensorMap& tK, const CUtensorMap& tV, cudaStream_t st) {
  if (i8)
    return bf16 ? launch_chunk<true, true>(p, tQ, tK, tV, st)
                : launch_chunk<false, true>(p, tQ, tK, tV, st);
  return bf16 ? launch_chunk<true, false>(p, tQ, tK, tV, st)
              : launch_chunk<false, false>(p, tQ, tK, tV, st);
}

}  // namespace mab
