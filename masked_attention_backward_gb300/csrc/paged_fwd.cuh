// paged_fwd.cuh -- attention of each request's new tokens over its paged cache,
// of 16-bit rows (paged_fwd.cu) or of 8-bit codes and scales (paged8_fwd.cu).
//
// Request b brings n new tokens (rows cu_q[b] .. of q) and has L keys in its
// cache, the new tokens' own among them; new token i stands at position
// x = L - n + i and sees key j < L when
//   j <= x and (x - j < window or j < first)      (or every key, MK_NONE)
//   O = sum_j P_j v_j / l,  P_j = exp2(s_j scale log2e - M),
//   l = sum_j P_j + exp2(sink log2e - M),  LSE = (M + log2 l) ln 2.
//
// One kernel for single tokens and long chunks.  The rows of a query tile are
// (token, query head of the group) pairs, so that one pass over a kv head's
// keys serves all of its query heads: 128 / group tokens fill the 128 rows of
// the matrix unit for a chunk, and a single token has `group` rows, the rest
// of the tile idle.  Work: unit = (request, kv head, query tile), walked over
// key sub-tiles of 64.
//
// Bounds: chunks, the tensor cores (4 * 128 FLOP per pair and query head);
// single tokens, HBM (512 bytes per key and kv head).  A step of a single
// token moves 32 KB and costs the tensor pipe 540 cycles, an SM's share of the
// HBM rate 1400, so the idle rows cost nothing there.
//
// Balance: every CTA of a persistent grid lays all units end to end, in steps,
// for itself, cuts the line into equal parts, one per CTA, and takes its own: a
// unit that a cut falls into is done in pieces, each leaving its fp32 O, M and l
// in the workspace, which k_paged_join adds up in order.  So a single request's
// keys spread over the whole GPU, ragged batches load every SM alike, and the
// workspace is bounded by two pieces per CTA whatever the lengths, which stay
// on the device.  (The line laid once, by a kernel before this one: 4 to 9 us
// until the first CTA had its part, 2.5 to 4 now: a window of 1024 over 8192
// keys took 197 us so and 189 without, 15 single tokens and a chunk of 500 51
// and 49, 4096 requests of 64 keys 99 and 102.)  The join's blocks wait beside the
// attention's last CTAs (programmatic launch).
//
// The inner loop is that of the BHSD forward kernel (attn_fwd.cu): warp 0 loads
// (a box per run of keys in a page, the page numbers looked up 32 at a time, a
// batch ahead), warp 1 issues S = Q K^T, warp 2 O += P V, two groups of four
// softmax warps take alternate steps.  Rows of V that no row of the unit sees
// (past the last key, before the window, between the first keys and it) may
// hold anything, NaN included, and 0 * NaN is NaN in the matrix unit: the page
// runs without a seen key are not loaded (zeros stand in), and warp 2 clears
// the other unseen rows in shared memory before it multiplies.
//
// Measured (one GB300, bf16 unless stated): 64 single tokens at 9000 keys, 64/8
// heads, 0.345 ms, 6.84 TB/s (16-token pages, [page, row, head], 6.6); 2 at
// 100000 keys, 32/4 heads, 73 us, 5.6 TB/s; 200 at 300 keys, 32/8 heads, 65 us,
// latency bound (a unit's start and end, about 5000 cycles, beside 5 steps);
// chunks of 2048 over 9000 keys, 32/8 heads, 0.44 ms, 1215 TFLOP/s, bound by
// the latency of S, softmax and P V over three buffers (tensor pipe 56 %
// active); one token at 1000 keys (fp16) 16 us, of which the line takes 2.5
// and the join 3.  Kept out, measured: one lane per box in place of an elected
// lane per load (a chunk's loader 940 cycles a step of 1140), a second loader
// warp for V, four epilogue warps of their own (every polling warp slows the
// softmax: a chunk 10 %), the join at the end of the last piece.
//
// The 8-bit cache: the loads bring codes into a ring of their own, and eight
// more warps make the 16-bit tiles of them that the matrix unit reads, two sets
// that take steps in turn, each warp 16 rows of K and of V, half a row a thread:
// code times scale, exactly (quant8.cuh), zeros for the rows that no row of the
// unit sees.  Each looks the pages and scales of 16 of its steps up a batch ahead.
// Bound by these warps beside the softmax: 3200 warp instructions a step, half of
// them theirs, on pipes of half rate, and a chain of tile, S, softmax and P V over
// four tiles (a step takes 1600 cycles; its bytes 700, the products 540).
// Measured: 2 requests of 5 and 4 tokens at 99770 and 107923 keys, 32/4 heads, int8, 89 us;
// 64 requests of 5 tokens at 9000, 64/8 heads, e4m3, 403; 15 requests of 1 to 4 tokens
// and a chunk of 500 under a window of 1024, 32/8 heads, fp16, 51; chunks of 1900 tokens
// over 8000 keys 603, which is why chunks take paged8_expand.cu where the workspace has
// room.  What made the two requests 109 to 88: shared memory reached as such
// (smem_align1024) 93, int8's masks in one instruction each 88.  Kept out: K's and V's
// tiles in rings of their own, 3 and 5 stages (chunks 768 when this took 626); three
// tiles and five stages of codes (two requests 118 of 109); a warp to K or to V alone,
// every step (122 of 109); K's tile reported before V's (90 of 88.7, the window of 1024
// 54 of 51); the codes read ahead so that their stage is free sooner (91 of 88.7,
// 64 requests 400 of 403); more registers to the softmax warps from the others
// (setmaxnreg; 88 and 88, 64 requests 413 and 403); 256 query rows in two halves that
// share the tiles, one S buffer each (chunks 619 of 813, the two requests 120), or S
// beside P with half of Q in shared memory (839).
#pragma once
#include <type_traits>

#include "paged_line.cuh"
#include "quant8.cuh"

namespace mab {

namespace paged_side {

// What the cache holds.
enum Form { ROWS16 = 0, CODES_E4M3 = 1, CODES_I8 = 2 };

constexpr int NBUF = 3;          // S / P buffers
constexpr int COL_O = 0;         // O accumulator of group g at COL_O + 128 g
constexpr int COL_QA = 256;      // Q as the A operand, 64 columns of 16-bit pairs
constexpr int COL_S = 320;       // S buffer b at COL_S + 64 b
constexpr int SM_WARPS = 8;      // softmax warps, two groups of four
constexpr int CV_WARPS = 8;      // converting warps, two sets of four
constexpr int CV_BATCH = 16;     // steps of a set whose pages and scales are looked up at once
// Warps and rings of a form.
template <int FORM>
struct Cfg {
  static constexpr bool Q8 = FORM != ROWS16;
  static constexpr int STAGES = Q8 ? 4 : 5;     // ring of 16-bit K / V tiles
  static constexpr int LD_STAGES = Q8 ? 3 : 5;  // ring that the loads go to
  // Barriers of the loads: step m's is m % LD_BARS.  A warp may wait for a phase only
  // when it has seen the one before it complete (a parity says no more), and the two
  // converting sets take steps in turn: an even number gives each its own barriers.
  // (With one a stage a set came to the third step after another one's whose load was
  // still under way, took it for complete, and freed a stage that was being filled.)
  static constexpr int LD_BARS = Q8 ? 2 * LD_STAGES : LD_STAGES;
  static constexpr int SM_WARP0 = Q8 ? 4 : 3;   // first softmax warp
  static constexpr int CV_WARP0 = SM_WARP0 + SM_WARPS;
  static constexpr int NUM_THREADS = 32 * (CV_WARP0 + (Q8 ? CV_WARPS : 0));
  static constexpr int AHEAD = 8;               // steps of a unit issued before the next one's Q
};

// What the converting warps add: the codes' ring (128B swizzle), and the scales
// of each warp's 16 rows, two batches: [warp][batch][step][K, V][row]; which of the
// rows are seen (bits 0 to 15), and whether some exponent is above 7 (bit 16).
template <int LD_STAGES>
struct __align__(1024) Smem8 {
  uint8_t K8[LD_STAGES][Q_SUB * 128];
  uint8_t V8[LD_STAGES][Q_SUB * 128];
  uint8_t scales[CV_WARPS][2][CV_BATCH][2][16];
  uint32_t seen[CV_WARPS][2][CV_BATCH];
  uint64_t bar_ld_full[2 * LD_STAGES];
  uint64_t bar_ld_empty[LD_STAGES];
};
struct Smem16 {};

template <int FORM>
struct __align__(1024) Smem
    : std::conditional_t<Cfg<FORM>::Q8, Smem8<Cfg<FORM>::LD_STAGES>, Smem16> {
  static constexpr int STAGES = Cfg<FORM>::STAGES;
  alignas(1024) uint8_t Q[2 * Q_TILE * 128];  // two 64-column chunks, 128B swizzle; once copied
                                // into TMEM, the epilogue staging (4 KB per warp)
  uint8_t K[STAGES][2 * Q_SUB * 128];
  uint8_t V[STAGES][2 * Q_SUB * 128];
  float xml[2][2][Q_TILE][2];   // [unit parity][group][row]: (M, l) at the piece's end
  LineSums<Cfg<FORM>::NUM_THREADS> sums;
  PagedStart cut[2];            // where this CTA's part begins and ends
  Unit unit;                    // piece of the latest Q load, N < 0: none left
  uint64_t bar_q_full;
  uint64_t bar_qa_full;         // Q copied into TMEM (all softmax warps)
  uint64_t bar_kv_full[STAGES];
  uint64_t bar_kv_empty[STAGES];
  uint64_t bar_s_full[2][2];    // [group][its step count parity]: S of the step complete
  uint64_t bar_p_full[NBUF];    // P of the buffer packed (the four warps of its group)
  uint64_t bar_p_free[NBUF];    // O += P V that read the buffer complete
  uint64_t bar_xml[4][2];       // [row quarter][unit parity]: both groups posted (M, l)
  uint64_t bar_acc_full;        // every O MMA of the piece complete
  uint64_t bar_acc_empty;       // its accumulators read (all softmax warps)
  uint64_t bar_unit_free;       // every other warp took the unit (and, softmax warps,
                                // left the previous unit's rows)
  uint64_t bar_x_done[2];       // every MMA of the S / O warp complete
  uint32_t tmem_base;
  int abort_flag;
};

template <int FORM>
constexpr size_t SMEM_BYTES = sizeof(Smem<FORM>) + 1024;
static_assert(SMEM_BYTES<ROWS16> <= 232448 && SMEM_BYTES<CODES_I8> <= 232448,
              "over the 227 KB of shared memory a CTA may use");

static_assert((PAGED_MAX_B + 1) * 8 + PAGED_MAX_B * 12 <=
                  sizeof(Smem<CODES_I8>::K) + sizeof(Smem<CODES_I8>::V),
              "the line of the most requests fits the smaller ring");

}  // namespace paged_side

template <int FORM>
using paged_params_t = std::conditional_t<FORM == paged_side::ROWS16, PagedParams, Paged8Params>;

template <bool BF16, int FORM>
__global__ void __launch_bounds__(paged_side::Cfg<FORM>::NUM_THREADS, 1)
k_paged_fwd(const __grid_constant__ CUtensorMap tQ, const __grid_constant__ CUtensorMap tK,
            const __grid_constant__ CUtensorMap tV,
            const __grid_constant__ paged_params_t<FORM> p) {
  using namespace paged_side;
  using C = Cfg<FORM>;
  constexpr bool Q8 = C::Q8;
  constexpr int STAGES = C::STAGES, LD_STAGES = C::LD_STAGES;
  constexpr int SM_WARP0 = C::SM_WARP0, AHEAD = C::AHEAD;
  extern __shared__ uint8_t smem_raw[];
  Smem<FORM>& s = *reinterpret_cast<Smem<FORM>*>(smem_align1024(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's own status word, which the join passes on
  WaitCtx wc{p.cta_status + blockIdx.x, &s.abort_flag, p.timeout_ns};

  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    *wc.status = DevStatus{};
    mbar_init(smem_u32(&s.bar_q_full), 1);
    mbar_init(smem_u32(&s.bar_qa_full), SM_WARPS);
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&s.bar_kv_full[i]), Q8 ? CV_WARPS / 2 : 1);
      mbar_init(smem_u32(&s.bar_kv_empty[i]), 1);
    }
    if constexpr (Q8)
      for (int i = 0; i < C::LD_BARS; ++i) {
        mbar_init(smem_u32(&s.bar_ld_full[i]), 1);
        if (i < LD_STAGES) mbar_init(smem_u32(&s.bar_ld_empty[i]), CV_WARPS / 2);
      }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s.bar_s_full[i >> 1][i & 1]), 1);
      mbar_init(smem_u32(&s.bar_xml[i][0]), 2);
      mbar_init(smem_u32(&s.bar_xml[i][1]), 2);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(smem_u32(&s.bar_p_full[i]), SM_WARPS / 2);
      mbar_init(smem_u32(&s.bar_p_free[i]), 1);
    }
    mbar_init(smem_u32(&s.bar_acc_full), 1);
    mbar_init(smem_u32(&s.bar_acc_empty), SM_WARPS);
    mbar_init(smem_u32(&s.bar_unit_free), SM_WARPS + 2 + (Q8 ? CV_WARPS : 0));
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&s.bar_x_done[i]), 1);
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
    // the loads into the ring come after these generic accesses to it
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }

  // Steps [s0, s0 + N) of a unit: the boxes of each step into its stage, once
  // that is free; midway() before step AHEAD.
  int m_load = 0;  // steps issued, across units
  Cyc<LD_STAGES> rg_load;
  Cyc<C::LD_BARS> rg_bar;
  uint64_t *ld_full = s.bar_kv_full, *ld_empty = s.bar_kv_empty;
  if constexpr (Q8) {
    ld_full = s.bar_ld_full;
    ld_empty = s.bar_ld_empty;
  }
  auto load_steps = [&](const Walk& w, int b, int kvh, int s0, int N, auto&& midway) -> bool {
    const int runs = Q_SUB / p.box_rows;
    const int batch = 32 / runs;  // steps whose pages the lanes look up at once
    const int* row = p.table + (size_t)b * p.table_stride;
    // lane l has run l % runs of step i + l / runs: its first key, whether it
    // holds a seen one, and its page (past the last where it holds none) and
    // first row there
    const int l_step = lane / runs, l_run = lane - l_step * runs;
    auto key_of = [&](int i) { return w.tile(i + l_step) * Q_SUB + l_run * p.box_rows; };
    auto seen = [&](int i, int k0) {
      return i + l_step < s0 + N && w.any(k0, k0 + p.box_rows);
    };
    int row0 = 0;
    auto pages_of = [&](int i) -> int {
      const int k0 = key_of(i);
      const int idx = div_by(k0, p.page_size, p.inv_page_size);
      row0 = k0 - idx * p.page_size;
      return seen(i, k0) ? __ldg(row + idx) : p.num_pages;
    };
    int page = p.num_pages, prow = 0, next = pages_of(s0), next_row = row0, left = 0;
    for (int i = s0; i < s0 + N; ++i, ++m_load, rg_load.next(), rg_bar.next(), --left) {
      const int st = rg_load.i;
      if (i == s0 + AHEAD && !midway()) return false;
      if (left == 0) {
        page = next;
        prow = next_row;
        left = batch;
        if ((unsigned)page >= (unsigned)p.num_pages) {
          // past the tensor's end, where a load reads zeros
          if (seen(i, key_of(i))) atomicCAS(&wc.status->code, 0u, (unsigned)ATTN_ERR_INVALID_ARG);
          page = p.num_pages;
        }
        next = pages_of(i + batch);  // a batch ahead
        next_row = row0;
      }
      if (m_load >= LD_STAGES &&
          !mbar_wait_sleep_warp(smem_u32(&ld_empty[st]), rg_load.ph ^ 1u, wc,
                                Q8 ? TAG_LD_EMPTY : TAG_KV_EMPTY, LOAD_SLEEP_NS))
        return false;
      const uint32_t fb = smem_u32(&ld_full[rg_bar.i]);
      if (lane == 0) mbar_arrive_expect_tx(fb, (Q8 ? 2 : 4) * Q_SUB * 128);
      __syncwarp();
      uint32_t dst_k, dst_v;
      if constexpr (Q8) {
        dst_k = smem_u32(s.K8[st]);
        dst_v = smem_u32(s.V8[st]);
      } else {
        dst_k = smem_u32(s.K[st]);
        dst_v = smem_u32(s.V[st]);
      }
      for (int r = 0; r < runs; ++r) {
        const int src = (batch - left) * runs + r;
        const int pg = __shfl_sync(0xffffffffu, page, src);
        const int pr = __shfl_sync(0xffffffffu, prow, src);
        const uint32_t k = dst_k + r * p.box_rows * 128, v = dst_v + r * p.box_rows * 128;
        tma_load_4d_w(k, &tK, 0, pr, kvh, pg, fb);
        if constexpr (!Q8) tma_load_4d_w(k + Q_SUB * 128, &tK, 64, pr, kvh, pg, fb);
        tma_load_4d_w(v, &tV, 0, pr, kvh, pg, fb);
        if constexpr (!Q8) tma_load_4d_w(v + Q_SUB * 128, &tV, 64, pr, kvh, pg, fb);
      }
    }
    return true;
  };
  // a CTA that gives up lets the copies still in flight land first
  auto drain_loads = [&]() {
    for (int k = m_load > LD_STAGES ? m_load - LD_STAGES : 0; k < m_load; ++k)
      mbar_drain_warp(smem_u32(&ld_full[k % C::LD_BARS]), (k / C::LD_BARS) & 1, wc.timeout_ns);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ loader of Q and K
    const int cta = (int)blockIdx.x;
    const PagedStart at0 = s.cut[0], end = s.cut[1];
    int b = at0.b, kvh = at0.kvh, tile = at0.tile, step = at0.step;  // where this CTA stands
    int off = at0.off, n = at0.n, L = at0.L;                         // of request b
    bool ok = !p.test_no_loads;
    int q_loaded = -1;  // last unit whose Q tile was loaded
    // lane i holds the lengths of request b_base + i (none yet: the first
    // request's came with the start)
    int b_base = b - 32, l_off = 0, l_n = 0, l_L = 0;
    auto load_lengths = [&]() {
      l_off = l_n = l_L = 0;
      if (b_base + lane < p.B) {
        l_off = packed_off(p.cu_q, b_base + lane, p.total_q);
        l_n = new_tokens(p, b_base + lane);
        l_L = keys_of(p, b_base + lane);
      }
    };
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
          tma_load_3d(smem_u32(s.Q), &tQ, 0, kvh * p.group, row, qbar);
          tma_load_3d(smem_u32(s.Q + Q_TILE * 128), &tQ, 64, kvh * p.group, row, qbar);
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
          load_lengths();
        }
        off = __shfl_sync(0xffffffffu, l_off, b - b_base);
        n = __shfl_sync(0xffffffffu, l_n, b - b_base);
        L = __shfl_sync(0xffffffffu, l_L, b - b_base);
        if (b == end.b) break;
      }
      return true;
    };
    bool ahead = false;  // the unit after the one being loaded is published
    for (int j = 0; ok; ++j) {
      if (!ahead) ok = publish(j);
      if (!ok || next.N < 0) break;
      const Walk w(p, next.n, next.L, next.tok0);
      ahead = false;
      // a long unit's successor is published, and its Q loaded, while this
      // one is still being worked on: its consumers have then taken it
      ok = load_steps(w, next.b, next.kvh, next.s0, next.N, [&]() {
        ahead = true;
        return publish(j + 1);
      });
    }
    if (!ok) {
      if (q_loaded >= 0) mbar_drain_warp(qbar, q_loaded & 1, wc.timeout_ns);
      drain_loads();
    }
  } else if (warp < 3) {
    // ------------------------------------------------------------ MMA issuers (whole warps)
    bool ok = true;
    int m = 0;  // step counter across units
    Cyc<STAGES> rg;
    Cyc<NBUF> bc;
    if (warp == 1) {
      // S(m) = Q K^T into buffer m % NBUF (A = Q from TMEM, B = K tile, K-major)
      constexpr uint32_t ID_S = idesc_f16(BF16, Q_TILE, Q_SUB, false, false);
      int cnt0 = 0, cnt1 = 0;  // steps of each group so far
      for (int j = 0; ok; ++j) {
        if (!mbar_wait_warp(smem_u32(&s.bar_q_full), j & 1, wc, TAG_Q)) break;
        const int N = s.unit.N;
        if (N < 0) break;
        ok = mbar_wait_warp(smem_u32(&s.bar_qa_full), j & 1, wc, TAG_QA);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.bar_unit_free));
        for (int i = 0; ok && i < N; ++i, ++m, rg.next(), bc.next()) {
          const int st = rg.i, bf = bc.i, grp = i & 1;
          ok = mbar_wait_warp(smem_u32(&s.bar_kv_full[st]), rg.ph, wc, TAG_KV_FULL);
          // the buffer held P(m - NBUF), read by O += P V
          if (ok && m >= NBUF)
            ok = mbar_wait_warp(smem_u32(&s.bar_p_free[bf]), bc.ph ^ 1u, wc, TAG_P_FREE);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bK = sdesc_sw128(smem_u32(s.K[st]), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < HEAD_DIM / 16; ++kk)
            mma_ts_w(tbase + COL_S + 64 * bf, tbase + COL_QA + 8 * kk,
                     bK + (uint64_t)(((kk >> 2) * (Q_SUB * 128) + (kk & 3) * 32) >> 4), ID_S,
                     kk > 0 ? 1u : 0u);
          const int c = grp ? cnt1 : cnt0;
          mma_commit_w(smem_u32(&s.bar_s_full[grp][c & 1]));
          if (grp) ++cnt1; else ++cnt0;
        }
      }
    } else {
      // O_{i % 2} += P(m) V (A = P packed in buffer m % NBUF, B = V tile, MN-major)
      constexpr uint32_t ID_O = idesc_f16(BF16, Q_TILE, HEAD_DIM, false, true);
      for (int j = 0; ok; ++j) {
        // the unit's first accumulations overwrite the accumulators: the
        // softmax warps must have read the previous unit's
        if (j >= 1 &&
            !mbar_wait_warp(smem_u32(&s.bar_acc_empty), (j - 1) & 1, wc, TAG_ACC_EMPTY))
          break;
        if (!mbar_wait_warp(smem_u32(&s.bar_q_full), j & 1, wc, TAG_Q)) break;
        const int N = s.unit.N;
        if (N < 0) break;
        const Walk w(p, s.unit.n, s.unit.L, s.unit.tok0);
        const int s0 = s.unit.s0;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.bar_unit_free));
        for (int i = 0; ok && i < N; ++i, ++m, rg.next(), bc.next()) {
          const int st = rg.i, bf = bc.i;
          // unseen rows of V cleared while S and the softmax of the step run
          // (only these steps wait for their loads here: a wait costs an
          // issuing warp 150 to 300 cycles)
          const int k0 = w.tile(s0 + i) * Q_SUB;
          if (!Q8 && !w.all(k0, k0 + Q_SUB)) {
            ok = mbar_wait_warp(smem_u32(&s.bar_kv_full[st]), rg.ph, wc, TAG_KV_FULL);
            if (!ok) break;
            // 8 lanes per 128-byte row: four rows of a half at a time
            for (int r = lane >> 3; r < Q_SUB; r += 4)
              if (!w.sees(k0 + r)) {
                uint4* row = reinterpret_cast<uint4*>(s.V[st] + r * 128) + (lane & 7);
                row[0] = make_uint4(0u, 0u, 0u, 0u);
                row[Q_SUB * 128 / 16] = make_uint4(0u, 0u, 0u, 0u);
              }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          ok = mbar_wait_warp(smem_u32(&s.bar_p_full[bf]), bc.ph, wc, TAG_P_FULL);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = tbase + COL_S + 64 * bf;
          const uint64_t bV = sdesc_sw128(smem_u32(s.V[st]), Q_SUB * 128, 1024);
#pragma unroll
          for (int kk = 0; kk < Q_SUB / 16; ++kk)
            mma_ts_w(tbase + COL_O + 128 * (i & 1), a + 8 * kk,
                     bV + (uint64_t)((kk * 2048) >> 4), ID_O, (i >= 2 || kk > 0) ? 1u : 0u);
          // S(m) completed before the softmax warps could signal step m, so
          // this commit also frees the K / V stage
          mma_commit_w(smem_u32(&s.bar_kv_empty[st]));
          mma_commit_w(smem_u32(&s.bar_p_free[bf]));
        }
        if (ok) mma_commit_w(smem_u32(&s.bar_acc_full));  // the accumulators are complete
      }
    }
    // this warp's MMAs must be complete before TMEM is freed (also when the
    // CTA gave up, hence a wait that ignores the abort flag)
    const uint32_t done = smem_u32(&s.bar_x_done[warp - 1]);
    mma_commit_w(done);
    mbar_drain_warp(done, 0, wc.timeout_ns);
  } else if (!Q8 || (warp >= SM_WARP0 && warp < C::CV_WARP0)) {
    // ------------------------------------------------------------ softmax warps
    const int sp = warp & 3, grp = (warp - SM_WARP0) >> 2;
    const int rloc = sp * 32 + lane;
    const int tl = rloc / p.group, hh = rloc - tl * p.group;  // the row's token and head
    const uint32_t lane_base = tbase + ((uint32_t)(sp * 32) << 16);
    // the epilogue stages through the Q rows this warp itself copies
    uint8_t* stage = s.Q + grp * (Q_TILE * 128) + sp * 4096;
    // Combines both groups' accumulators of unit j into columns [64 grp,
    // 64 grp + 64) of this warp's 32 rows, and stores them (a whole unit), or
    // leaves them in the workspace for the join (a piece).
    // Arrives on acc_empty, and on unit_free of the unit after it (whose Q this
    // warp has copied) once the staging space is not needed any more.  (M, l)
    // of the own group come in, the other group's through shared memory.
    auto epilogue = [&](int j, const Unit& un, float M, float l, bool ok) {
      s.xml[j & 1][grp][rloc][0] = M;
      s.xml[j & 1][grp][rloc][1] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.bar_xml[sp][j & 1]));
      const int N = un.N;
      // rows of this warp that are a token of the request
      const int nr = min(32, min(p.tile_tokens, un.n - un.tok0) * p.group - sp * 32);
      const bool mine = lane < nr, whole = un.whole;
      const int tok = un.off + un.tok0 + tl, head = un.kvh * p.group + hh;
      const float sink2 = p.sink && mine ? p.sink[head] * LOG2E : -INFINITY;
      const long long row_at = mine ? (long long)tok * p.Hq + head : -1;
      const size_t lse_at = (size_t)head * p.total_q + tok;
      const int wq = sp * 2 + grp;
      // (a piece without steps waits too, so that no wait meets these barriers
      // two phases late)
      ok = ok && mbar_wait_warp(smem_u32(&s.bar_xml[sp][j & 1]), (j >> 1) & 1, wc, TAG_XML);
      // weights of O_0 and O_1: group 1 has steps only when the piece has two
      // or more, and a group that saw nothing of a row (l = 0) has none (l is
      // never negative, and a NaN stays)
      float w0 = 0.f, w1 = 0.f, top = -INFINITY, lsum = 0.f;
      if (ok && N > 0) {
        const float mo = s.xml[j & 1][grp ^ 1][rloc][0], lo = s.xml[j & 1][grp ^ 1][rloc][1];
        const float l0 = grp == 0 ? l : lo, l1 = grp == 0 ? lo : l;
        top = fmaxf(M, mo);
        if (l0 != 0.f) w0 = fast_exp2((grp == 0 ? M : mo) - top);
        if (N >= 2 && l1 != 0.f) w1 = fast_exp2((grp == 0 ? mo : M) - top);
        lsum = l0 * w0 + l1 * w1;
      }
      float* part = p.part + (size_t)un.slot * p.slot_floats + wq * PAGED_WARP_FLOATS;
      if (whole) {
        float inv;
        const float lse = finish_row(top, lsum, sink2, &inv);
        if (p.lse && grp == 0 && mine && ok) p.lse[lse_at] = lse;
        w0 *= inv;
        w1 *= inv;
      } else if (mine) {
        part[PAGED_ML + 2 * lane] = top;
        part[PAGED_ML + 2 * lane + 1] = lsum;
      }
      ok = ok && mbar_wait_warp(smem_u32(&s.bar_acc_full), j & 1, wc, TAG_ACC);
      tc_fence_after();
      // 16 columns at a time, in a loop: this code runs once a unit, and as one
      // straight piece most of its time went into fetching it.  (O of a group
      // that saw nothing of a row is zero there; group 1 without a step has the
      // weight zero, and O_0 stands in.)
      if (ok && nr > 0) {
        const uint32_t o1 = N >= 2 ? 128u : 0u;
        const float2 w02 = make_float2(w0, w0), w12 = make_float2(w1, w1);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float a0[16], a1[16];
          const uint32_t col = lane_base + COL_O + 64 * grp + 16 * q;
          if (N > 0) {
            tmem_ld16(col, a0);
            tmem_ld16(col + o1, a1);
            tmem_wait_ld_regs(a0);
#pragma unroll
            for (int c = 0; c < 16; ++c) asm volatile("" : "+f"(a1[c]));
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) a0[c] = a1[c] = 0.f;
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 x = ffma2(make_float2(a1[2 * c], a1[2 * c + 1]), w12,
                                   fmul2(make_float2(a0[2 * c], a0[2 * c + 1]), w02));
            a0[2 * c] = x.x;
            a0[2 * c + 1] = x.y;
          }
          if constexpr (Q8 && BF16) {  // back from the converted tiles' order of d
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float x = a0[4 * c + 1];
              a0[4 * c + 1] = a0[4 * c + 2];
              a0[4 * c + 2] = x;
            }
          }
          if (whole) {
            // through shared memory, so that a row's 128 bytes leave together
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((2 * q + h) ^ (lane & 7)) << 4)) =
                  make_uint4(pack2<BF16>(a0[8 * h], a0[8 * h + 1]),
                             pack2<BF16>(a0[8 * h + 2], a0[8 * h + 3]),
                             pack2<BF16>(a0[8 * h + 4], a0[8 * h + 5]),
                             pack2<BF16>(a0[8 * h + 6], a0[8 * h + 7]));
          } else if (mine) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *part_at(part, lane, 4 * q + c) =
                  make_float4(a0[4 * c], a0[4 * c + 1], a0[4 * c + 2], a0[4 * c + 3]);
          }
        }
      }
      // the accumulators are read: the next unit's O may begin
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.bar_acc_empty));
      if (ok && nr > 0 && whole) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = k * 4 + (lane >> 3), c = lane & 7;
          const long long to = __shfl_sync(0xffffffffu, row_at, row);
          const uint4 v =
              *reinterpret_cast<const uint4*>(stage + row * 128 + ((c ^ (row & 7)) << 4));
          if (to >= 0) *reinterpret_cast<uint4*>(p.out + to * HEAD_DIM + 64 * grp + c * 8) = v;
        }
      }
      // the next TMA load into the Q tile comes after this warp's generic
      // accesses to it
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.bar_unit_free));
    };
    bool ok = true;
    int cnt = 0, oth = 0;  // steps of this group and of the other one so far
    Cyc<NBUF> bc;
    Unit prev{};
    float prev_M = -INFINITY, prev_l = 0.f;
    for (int j = 0;; ++j) {
      ok = ok && mbar_wait_warp(smem_u32(&s.bar_q_full), j & 1, wc, TAG_Q);
      const Unit un = s.unit;
      const bool last = !ok || un.N < 0;  // no unit: only the previous one's epilogue
      const int rows = min(p.tile_tokens, un.n - un.tok0) * p.group;
      const bool busy = sp * 32 < rows;  // some row of this warp is a token's
      // Q rows into TMEM as 16-bit pairs (element 2c in the low half of
      // column c): this warp copies d columns 64 grp .. 64 grp + 63 of its
      // rows.  S of this group's last step is complete; the other group's last
      // one, which may be the later of the two, is waited for.
      if (!last && oth > 0)
        ok = mbar_wait_warp(smem_u32(&s.bar_s_full[grp ^ 1][(oth - 1) & 1]), ((oth - 1) >> 1) & 1,
                            wc, TAG_S_FULL);
      tc_fence_after();
      if (!last && ok && busy && un.N > 0) {
        const uint8_t* src = s.Q + grp * (Q_TILE * 128) + rloc * 128;
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + ((c ^ (rloc & 7)) << 4));
          w[4 * c] = v.x;
          w[4 * c + 1] = v.y;
          w[4 * c + 2] = v.z;
          w[4 * c + 3] = v.w;
        }
        if constexpr (Q8 && BF16) {  // the order of d in the converted tiles
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint32_t a = w[2 * c], b = w[2 * c + 1];
            w[2 * c] = __byte_perm(a, b, 0x5410);
            w[2 * c + 1] = __byte_perm(a, b, 0x7632);
          }
        }
        tmem_st32(lane_base + COL_QA + 32 * grp, w);
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

      // this group's running maximum M (log2 domain) and its row sum (the sink
      // joins in the epilogue)
      float M = -INFINITY, l = 0.f;
      const Walk w(p, un.n, un.L, un.tok0);
      // the row's position and the end of the keys it may see; rows that are no
      // token's see nothing
      const int x0 = un.L - un.n + un.tok0, x = x0 + tl;
      const int key_end = rloc >= rows ? 0 : p.causal ? max(x + 1, 0) : un.L;
      // sub-tiles that every row sees whole: [full_lo, full_hi] (before the
      // first row's position and within the last one's window), and those up to
      // full_first among the first keys
      const int all_end = p.causal ? x0 + 1 : un.L;
      const int x_last = x0 + min(p.tile_tokens, un.n - un.tok0) - 1;
      const int full_hi = all_end < Q_SUB ? -1 : all_end / Q_SUB - 1;
      const int full_lo =
          !p.causal || x_last < p.window ? 0 : (x_last - p.window + Q_SUB) / Q_SUB;
      const int full_first = min(full_hi, p.first / Q_SUB - 1);
      int last_bf = 0;       // buffer of this group's previous step of the unit
      uint32_t last_ph = 0;  // and the parity of its use
      // Takes a step's row maximum mx (raw logits; the scale is positive, so it
      // is applied once here).  M moves when mx exceeds it by more than 8; a row
      // that has seen nothing yet (M = -inf, so O and l are still zero) just
      // takes the new value.  The group's O rows whose M moved are rescaled once
      // its previous O += P V of the unit has completed (the unit's first
      // accumulation of the group overwrites instead).
      auto move_max = [&](int i, float mx) -> bool {
        const float mx2 = mx == -INFINITY ? -INFINITY : mx * p.scale_log2;
        float alpha = 1.f;
        if (mx2 > M + RESCALE_LOG2) {
          if (M != -INFINITY) alpha = fast_exp2(M - mx2);
          M = mx2;
          l *= alpha;
        }
        if (i >= 2 && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (!mbar_wait_warp(smem_u32(&s.bar_p_free[last_bf]), last_ph, wc, TAG_P_FREE))
            return false;
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t v[32];
            tmem_ld32(lane_base + COL_O + 128 * grp + 32 * q, reinterpret_cast<float(&)[32]>(v));
            tmem_wait_ld_regs(reinterpret_cast<float(&)[32]>(v));
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * alpha);
            tmem_st32(lane_base + COL_O + 128 * grp + 32 * q, v);
          }
        }
        return true;
      };
      // P = exp2(S scale log2e - M): an invisible logit (-inf) gives 0; a row
      // with nothing visible keeps M = -inf and all its logits at -inf, and the
      // finite stand-in keeps -inf - (-inf) out
      auto minus_max = [&]() { return M == -INFINITY ? 0.f : -M; };
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
      // A sub-tile that every row sees whole, from TMEM buffer column `col`: P
      // packed over it, rounded to 16 bits as O += P V takes it (l sums the unrounded
      // ones).  With o's own rounding o is off by 2.1e-3 of its norm in bf16 and 2.6e-4 in
      // fp16; 32-bit probabilities, 1.7e-3 and 2.1e-4, would take a second product of
      // what the rounding leaves.
      auto whole_step = [&](int i, uint32_t col) -> bool {
        float sv[64];
        tmem_ld32(col, *reinterpret_cast<float(*)[32]>(&sv[0]));
        tmem_ld32(col + 32, *reinterpret_cast<float(*)[32]>(&sv[32]));
        tmem_wait_ld_regs(sv);
        // eight partial maxima and four sums keep the dependency chains short
        float mp[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mp[c] = fmaxf(sv[2 * c], sv[2 * c + 1]);
#pragma unroll
        for (int c = 8; c < 32; ++c) mp[c & 7] = fmax3f(mp[c & 7], sv[2 * c], sv[2 * c + 1]);
        if (!move_max(i, fmax3f(fmax3f(mp[0], mp[1], mp[2]), fmax3f(mp[3], mp[4], mp[5]),
                                fmaxf(mp[6], mp[7]))))
          return false;
        const float nm = minus_max();
        const float2 nm2 = make_float2(nm, nm);
        if constexpr (Q8) {
          // the logits are read again, 32 at a time: 64 beside their probabilities are
          // more than the registers of 20 warps hold
          float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float v[32];
            tmem_ld32(col + 32 * q, v);
            tmem_wait_ld_regs(v);
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 xx = ffma2(make_float2(v[2 * c], v[2 * c + 1]), sc2, nm2);
              const float2 pp = make_float2(fast_exp2(xx.x), fast_exp2(xx.y));
              ls[c & 1] = fadd2(ls[c & 1], pp);
              pk[c] = pack2<BF16>(pp.x, pp.y);
            }
            // over columns that have been read: 16 q + 15 < 32 q + 32
            tmem_st16(col + 16 * q, pk);
          }
          const float2 x = fadd2(ls[0], ls[1]);
          l += x.x + x.y;
        } else {
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
          tmem_st32(col, pk);
        }
        tmem_wait_st();
        return true;
      };
      // A sub-tile from key j0 on that some row does not see whole: two passes
      // of 32 columns at a time, in loops.  It runs once or twice a unit; the
      // masking among the code above cost whole sub-tiles 5 %, and a masked copy
      // of that code the time to fetch it.
      auto masked_step = [&](int i, uint32_t col, int j0) -> bool {
        auto load32 = [&](int q, float (&v)[32]) {
          tmem_ld32(col + 32 * q, v);
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
        if (!move_max(i, mx)) return false;
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
          tmem_st16(col + 16 * q, pk);
        }
        l += ls.x + ls.y;
        tmem_wait_st();
        return true;
      };
      for (int i = 0; ok && i < un.N; ++i, bc.next()) {
        if ((i & 1) != grp) {
          ++oth;
          continue;
        }
        const int bf = bc.i;
        const int t = w.tile(un.s0 + i);
        // warp-uniform: every row of the tile sees every key of the sub-tile
        const bool full = (t >= full_lo && t <= full_hi) || t <= full_first;
        ok = mbar_wait_warp(smem_u32(&s.bar_s_full[grp][cnt & 1]), (cnt >> 1) & 1, wc, TAG_S_FULL);
        if (!ok) break;
        ++cnt;
        if (busy) {
          tc_fence_after();
          const uint32_t col = lane_base + COL_S + 64 * bf;
          ok = full ? whole_step(i, col) : masked_step(i, col, t * Q_SUB);
          if (!ok) break;
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.bar_p_full[bf]));
        last_bf = bf;
        last_ph = bc.ph;
      }
      prev = un;
      prev_M = M;
      prev_l = l;
    }
  } else if constexpr (Q8) {
    // ------------------------------------------------------------ converting warps
    if (warp >= C::CV_WARP0) {
      constexpr bool I8 = FORM == CODES_I8;
      const int cw = warp - C::CV_WARP0, slice = cw & 3, set = cw >> 2;
      // this thread's row of a step, and which half of it
      const int srow = lane >> 1, row = 16 * slice + srow, half = lane & 1;
      bool ok = true;
      static_assert(STAGES % 2 == 0 && C::LD_BARS % 2 == 0, "a barrier belongs to one set");
      int m0 = 0;  // steps of the units so far; a set takes every other one
      for (int j = 0; ok; ++j) {
        if (!mbar_wait_warp(smem_u32(&s.bar_q_full), j & 1, wc, TAG_Q)) break;
        const int N = s.unit.N, s0 = s.unit.s0, kvh = s.unit.kvh;
        if (N < 0) break;
        const Walk w(p, s.unit.n, s.unit.L, s.unit.tok0);
        const int* table = p.table + (size_t)s.unit.b * p.table_stride;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.bar_unit_free));
        const int first = (m0 ^ set) & 1;  // the set's first step of the piece
        // Lanes l and l + 16 look up the set's step i + 2 l: the page of this warp's 16 rows
        // there (-1 where none of them is seen, or the page is not there), and K's and V's
        // scales.
        auto key_of = [&](int i) {
          return w.tile(s0 + i + 2 * (lane & (CV_BATCH - 1))) * Q_SUB + 16 * slice;
        };
        auto page_of = [&](int i) -> int {
          const int k0 = key_of(i);
          if (i + 2 * (lane & (CV_BATCH - 1)) >= N || !w.any(k0, k0 + 16)) return -1;
          const int pg = __ldg(table + div_by(k0, p.page_size, p.inv_page_size));
          return (unsigned)pg < (unsigned)p.num_pages ? pg : -1;
        };
        auto scales_of = [&](int i, int pg) -> uint4 {
          if (pg < 0) return make_uint4(0u, 0u, 0u, 0u);
          const int k0 = key_of(i);
          const int r = k0 - div_by(k0, p.page_size, p.inv_page_size) * p.page_size;
          const uint8_t* at = (lane < CV_BATCH ? p.k_scales : p.v_scales) +
                              pg * p.scale_page_stride + kvh * p.scale_head_stride +
                              (r >> p.scale_shift);
          if (p.scale_shift == 0) return __ldg(reinterpret_cast<const uint4*>(at));
          const uint32_t a = __ldg(at) * 0x01010101u;
          return make_uint4(a, a, a, a);
        };
        uint4 sc = scales_of(first, page_of(first));
        int page = page_of(first + 2 * CV_BATCH);
        int at = 0;  // own steps so far
        for (int i = first; ok && i < N; i += 2, ++at) {
          const int bt = (at / CV_BATCH) & 1, bi = at & (CV_BATCH - 1);
          if (bi == 0) {
            // which rows some row of the unit sees; unseen ones count as small
            const int k0 = key_of(i);
            uint32_t bits = 0;
            const uint32_t sw[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (w.sees(k0 + r)) {
                bits |= 1u << r;
                if (((sw[r >> 2] >> (8 * (r & 3))) & 255u) > 127 + 7) bits |= 1u << 16;
              }
            bits |= __shfl_xor_sync(0xffffffffu, bits, CV_BATCH);
            __syncwarp();  // the batch before the last is read
            *reinterpret_cast<uint4*>(
                s.scales[cw][bt][lane & (CV_BATCH - 1)][lane / CV_BATCH]) = sc;
            if (lane < CV_BATCH) s.seen[cw][bt][lane] = bits;
            __syncwarp();
            sc = scales_of(i + 2 * CV_BATCH, page);  // a batch ahead
            page = page_of(i + 4 * CV_BATCH);
          }
          const int m = m0 + i, ld = m % LD_STAGES, kv = m % STAGES;
          const uint32_t bits = s.seen[cw][bt][bi];
          const bool small = BF16 && !I8 && !(bits >> 16);
          ok = mbar_wait_warp(smem_u32(&s.bar_ld_full[m % C::LD_BARS]), (m / C::LD_BARS) & 1, wc,
                              TAG_LD_FULL);
          if (ok && m >= STAGES)
            ok = mbar_wait_warp(smem_u32(&s.bar_kv_empty[kv]), (m / STAGES + 1) & 1, wc,
                                TAG_KV_EMPTY);
          if (!ok) break;
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {  // K, then V
            const int sb = s.scales[cw][bt][bi][x][srow];
            // e4m3 to bf16: one product while every exponent is at most 7
            uint32_t scale2 = scale_pair<BF16>(small ? min(max(sb, 1) + 120, 254) : sb);
            const uint8_t* from = (x ? s.V8[ld] : s.K8[ld]) + row * 128;
            uint8_t* to = (x ? s.V[kv] : s.K[kv]) + half * (Q_SUB * 128) + row * 128;
            // 16-byte units: 4 half + c of the code row become 2 c and 2 c + 1 of the
            // half's 128-byte row, both swizzled by the row; the halves take them in
            // orders that keep them off each other's banks
            uint4 v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              v[c] = *reinterpret_cast<const uint4*>(
                  from + (((4 * half + (c ^ (half << 1))) ^ (row & 7)) << 4));
            // a row that nobody sees may hold anything: zeros
            if ((bits & 0xffffu) != 0xffffu && !((bits >> srow) & 1u)) {
#pragma unroll
              for (int c = 0; c < 4; ++c) v[c] = make_uint4(0u, 0u, 0u, 0u);
              scale2 = 0u;
            }
            auto convert = [&](auto one) {
              constexpr bool SMALL = decltype(one)::value;
#pragma unroll
              for (int cc = 0; cc < 4; ++cc) {
                const int c = cc ^ (half << 1);
                const uint2 a = tile_words<BF16, I8, SMALL>(v[cc].x, scale2);
                const uint2 b = tile_words<BF16, I8, SMALL>(v[cc].y, scale2);
                const uint2 d = tile_words<BF16, I8, SMALL>(v[cc].z, scale2);
                const uint2 e = tile_words<BF16, I8, SMALL>(v[cc].w, scale2);
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
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&s.bar_kv_full[kv]));
            mbar_arrive(smem_u32(&s.bar_ld_empty[ld]));
          }
        }
        m0 += N;
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

template <bool BF16, int FORM>
cudaError_t launch_paged(const paged_params_t<FORM>& p, const CUtensorMap& tQ,
                         const CUtensorMap& tK, const CUtensorMap& tV, cudaStream_t st) {
  using namespace paged_side;
  const auto kern = k_paged_fwd<BF16, FORM>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)SMEM_BYTES<FORM>);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3(Cfg<FORM>::NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES<FORM>;
  cfg.stream = st;
  e = cudaLaunchKernelEx(&cfg, kern, tQ, tK, tV, p);
  if (e != cudaSuccess) return e;
  return launch_paged_join<BF16>(p, st);
}

}  // namespace mab
