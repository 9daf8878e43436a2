/*
 * maskattn.h -- C ABI of libmaskattn: masked attention forward and backward
 * (GQA/MHA, BHSD, head dim 128, fp16 or bf16, fp32 accumulation) with a
 * per-head attention sink, for one NVIDIA GB300 GPU (sm_103a).
 *
 * The operation (restated from the pages this library follows):
 *   - tilelang-ascend PR #1 "Add GQA Sink Backward BHSD", Summary: online
 *     softmax with an attention sink and a sliding-window mask; commit notes
 *     of the 2-kernel design: Phase0 Delta = sum(O*dO), a KV loop of five
 *     contractions + softmax + dS, Phase5 dSink.  The sink is one logit per
 *     head that joins only the softmax denominator (it has no value row).
 *   - cannbot-knowledge PR #174, BlockSparseAttentionGrad runbook, task
 *     features: a uint8 block mask [B,N,ceil(Sq/bx),ceil(Skv/by)] with bx and
 *     by chosen independently and not required to divide the sequence
 *     lengths; optimisations 1-2: the host only checks shapes and carves
 *     memory, the mask is transposed and compacted into select tables on the
 *     device; optimisation 3: dK/dV are written back contiguously, without
 *     atomics; precision notes: p = exp(s - lse), ds = p * (dp - delta), a row
 *     that sees no key gets zeros.
 *
 * With g = Hq / Hkv, query head h reads key/value head floor(h / g).
 * Visibility of key j to query i (0-based):
 *   ATTN_MASK_NONE     every j
 *   ATTN_MASK_CAUSAL   j <= i                        (requires Sq == Skv)
 *   ATTN_MASK_SLIDING  j <= i and i - j < window     (requires Sq == Skv)
 *   ATTN_MASK_BLOCK    block_mask[b, h, i / bx, j / by] != 0
 *   ATTN_MASK_SLIDING_FIRST  j <= i and (i - j < window or j < first)
 *                                                    (requires Sq == Skv)
 *
 * Memory: every tensor argument is a DEVICE pointer owned by the caller,
 * contiguous, 16-byte aligned.  q, o, dO, dq: [B,Hq,Sq,128]; k, v, dk, dv:
 * [B,Hkv,Skv,128], all of `dtype`; lse: float32 [B,Hq,Sq] (natural log);
 * sink, dsink: float32 [Hq]; block_mask: uint8 [B,Hq,ceil(Sq/bx),ceil(Skv/by)].
 * The library allocates no device memory: scratch comes from the caller's
 * workspace `ws` (size from attn_workspace_size, 256-byte aligned).
 * Limits: Sq, Skv <= 2^24 and B * Hq <= 65535.
 *
 * Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 * default stream), returns a status at once, and may be enqueued again on the
 * same stream with the same workspace.  Calls that share a workspace must not
 * overlap in time (use one stream, or one workspace per stream).
 *
 * Errors: arguments are checked on the host before anything is enqueued; on
 * an error nothing is enqueued and the outputs are left untouched.  Device
 * waits inside the kernels are bounded: a wait that runs out records
 * ATTN_ERR_TIMEOUT in the workspace status word, which attn_get_device_status
 * reads back; the outputs of such a call are undefined.  The limit is 2 s per
 * wait, or MASKATTN_WAIT_TIMEOUT_NS nanoseconds from the environment at the
 * time of the call.  Test hooks, off unless set in the environment at the time
 * of a call: MASKATTN_TEST_NO_LOADS=1 makes the kernels' loader warps issue
 * nothing, so the call's waits run out and it ends with ATTN_ERR_TIMEOUT;
 * MASKATTN_PAGED8_ROOM=1 makes attn_paged8_fwd use room for its chunks' rows
 * however little work there is (and attn_paged8_workspace_size ask for it);
 * MASKATTN_DKDV_SCHEDULE=tile or =units forces the per-tile or the persistent
 * form of the dK/dV kernel (otherwise chosen by the walk lengths; the results
 * are the same bit for bit).
 */
#ifndef MASKATTN_H_
#define MASKATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1, /* bad shape, null or misaligned pointer, bad mask fields */
  ATTN_ERR_UNSUPPORTED = 2, /* valid request the library does not implement (D != 128) */
  ATTN_ERR_WORKSPACE = 3,   /* ws_bytes smaller than attn_workspace_size() */
  ATTN_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed */
  ATTN_ERR_TIMEOUT = 5      /* a device-side wait ran out (read back by attn_get_device_status) */
} attn_status_t;

typedef enum { ATTN_F16 = 0, ATTN_BF16 = 1 } attn_dtype_t;

typedef enum {
  ATTN_MASK_NONE = 0,
  ATTN_MASK_CAUSAL = 1,
  ATTN_MASK_SLIDING = 2, /* causal with a window of `window` keys including the diagonal */
  ATTN_MASK_BLOCK = 3,
  ATTN_MASK_SLIDING_FIRST = 4 /* the same window, and the first `first` keys stay visible */
} attn_mask_kind_t;

/* Shapes of one call; tensors are contiguous BHSD.  flags: 0, or
 * ATTN_FLAG_COMPENSATED or ATTN_FLAG_SINGLE_PASS (not both). */
typedef struct {
  int B, Hq, Hkv, Sq, Skv, D;
  int dtype; /* attn_dtype_t */
  int flags; /* attn_flag_t bits */
} attn_shape_t;

/* ATTN_FLAG_COMPENSATED (attn_bwd): P and dS enter the 16-bit contractions
 * dV += P^T dO, dK += dS^T Q and dQ += dS K as a 16-bit high part plus a
 * 16-bit remainder (two contractions each), so they are rounded to about 22
 * bits instead of 11 (fp16) or 8 (bf16) before the fp32 accumulation --
 * the compensated ("hi + lo") mode for tighter tolerances.  It costs 1.3x
 * the tensor work and 1.1x to 1.35x the time.  attn_fwd ignores it. */
/* ATTN_FLAG_SINGLE_PASS (attn_bwd): the single-pass design of the backward.
 * The key-stationary kernel also computes, for every visible (key tile,
 * query sub-tile) step, that step's dq partial dS K in fp32 and stores it in
 * the workspace; a second kernel sums each query sub-tile's partials in
 * ascending key-tile order (deterministic) and rounds.  S and dP are then
 * computed once per tile instead of twice (the default split design computes
 * them again in its query-stationary dq kernel), at the price of 32 KB of
 * partials written and read per step: the workspace grows by 32 KB + 1 byte
 * per (query head, key tile, query sub-tile) step the key tiles can take at
 * the full lengths (all of them for block masks).  Same results up to
 * rounding order.  ATTN_ERR_UNSUPPORTED with ATTN_FLAG_COMPENSATED, the
 * packed layout or ATTN_MASK_SLIDING_FIRST.  attn_fwd ignores it (its workspace need is unchanged). */
typedef enum { ATTN_FLAG_COMPENSATED = 1, ATTN_FLAG_SINGLE_PASS = 2 } attn_flag_t;

/* Mask description.  window is read for ATTN_MASK_SLIDING and
 * ATTN_MASK_SLIDING_FIRST only; bx, by and block_mask for ATTN_MASK_BLOCK only
 * (block_mask is a device pointer); first (>= 0) for ATTN_MASK_SLIDING_FIRST
 * only.  first counts from each sequence's start, as the window does; with
 * first = 0 the mask is ATTN_MASK_SLIDING.
 *
 * Variable lengths: seqlen_q and seqlen_k, when not NULL, are device int32
 * arrays [B] of the valid query rows and keys of each batch element (values
 * are clamped to [0, Sq] and [0, Skv]); NULL means all rows / keys.  Rows
 * i >= seqlen_q[b] and keys j >= seqlen_k[b] are outside the problem: no pair
 * with either is visible (the mask rules count i and j from the start of the
 * sequence, as without lengths), such a row has O = 0 and LSE = +inf in the
 * forward, dQ = 0 and no part in dSink in the backward whatever finite values
 * q, O, dO and LSE hold there, and such a key has dK = dV = 0 whatever finite
 * values k and v hold there.  This is the variable-length
 * batch on the padded BHSD layout: each sequence starts at row 0 of its batch
 * element.  4-byte aligned.
 *
 * Packed variable lengths: cu_seqlens_q and cu_seqlens_k, when not NULL (both,
 * with seqlen_q and seqlen_k NULL), are device int32 arrays [B + 1] of
 * cumulative sequence offsets: sequence b owns tokens [cu_seqlens_q[b],
 * cu_seqlens_q[b + 1]) of q, o, dO and dq, which are then token-major
 * [total_q, Hq, 128] tensors, and tokens [cu_seqlens_k[b], cu_seqlens_k[b + 1])
 * of k, v, dk and dv, [total_k, Hkv, 128]; lse is float32 [Hq, total_q].
 * total_q and total_k (>= 1) are the token counts of those tensors, known to
 * the caller; Sq and Skv of the shape are the longest sequence lengths (they
 * size the workspace and the block mask, whose rows and columns count from
 * each sequence's start, as the causal and sliding-window rules do).  Offsets
 * are clamped to [0, total] and lengths to [0, Sq] / [0, Skv]; every write
 * stays inside the sequence's own tokens, and tokens no sequence owns are not
 * written.  4-byte aligned. */
typedef struct {
  int kind; /* attn_mask_kind_t */
  int window;
  int bx, by;
  const uint8_t* block_mask;
  const int* seqlen_q;     /* device [B] or NULL */
  const int* seqlen_k;     /* device [B] or NULL */
  const int* cu_seqlens_q; /* device [B + 1] or NULL: packed layout */
  const int* cu_seqlens_k; /* device [B + 1] or NULL */
  int total_q, total_k;    /* packed layout: tokens in the query / key tensors */
  int first;               /* ATTN_MASK_SLIDING_FIRST: first keys that stay visible */
} attn_mask_desc_t;

/* Workspace bytes needed by attn_fwd and attn_bwd for this shape and mask.
 * Host only; never touches the GPU.  Errors: ATTN_ERR_INVALID_ARG,
 * ATTN_ERR_UNSUPPORTED (same checks as attn_bwd, pointers not required). */
attn_status_t attn_workspace_size(const attn_shape_t* shape, const attn_mask_desc_t* mask,
                                  size_t* bytes);

/* Forward: O = softmax_with_sink(scale * q k^T, masked) v, and
 * lse[b,h,i] = log(sum_j exp(scale*s_ij) + exp(sink_h)) over visible j.
 * sink may be NULL (no sink).  A row with no visible key and no sink gets
 * O = 0 and lse = +inf.  A row of q that is not finite gets NaN in its own o
 * and lse alone; where every logit that it sees is -inf, these weigh nothing,
 * as for a row with no visible key.  Outputs: o (dtype), lse (float32). */
attn_status_t attn_fwd(const attn_shape_t* shape, const void* q, const void* k, const void* v,
                       const float* sink, const attn_mask_desc_t* mask, float scale, void* o,
                       float* lse, void* ws, size_t ws_bytes, void* stream);

/* Backward from the forward's o and lse (taken as given):
 *   Delta_i = sum_d dO_id o_id;  P_ij = exp(scale*s_ij - lse_i);
 *   dS_ij = P_ij (dO_i . v_j - Delta_i);
 *   dq_i = scale sum_j dS_ij k_j;  dk_j = scale sum_{h in group} sum_i dS_ij q_i;
 *   dv_j = sum_{h in group} sum_i P_ij dO_i;
 *   dsink_h = - sum_b sum_i exp(sink_h - lse_i) Delta_i.
 * sink NULL means no sink; dsink is then not written and may be NULL.
 * Every element of dq, dk, dv (and dsink) is written.  Outputs dq, dk, dv
 * have `dtype` (fp32 accumulation, round to nearest even). */
attn_status_t attn_bwd(const attn_shape_t* shape, const void* q, const void* k, const void* v,
                       const void* o, const void* dO, const float* lse, const float* sink,
                       const attn_mask_desc_t* mask, float scale, void* dq, void* dk, void* dv,
                       float* dsink, void* ws, size_t ws_bytes, void* stream);

/* Backward for callers that cannot allocate device memory (operator or plugin
 * interfaces that receive no workspace, services that forbid allocation while
 * running).  The pages describe no such variant; this is an addition of this
 * library.  Same arguments and results as attn_bwd, without ws / ws_bytes:
 * the scratch lives in a fixed 32 MiB device array inside the library, held
 * on every GPU that loads it until the process exits.  The first call on a
 * device looks up that array's address (make that first call before any
 * stream capture on the device).  Errors: those of attn_bwd, and
 * ATTN_ERR_WORKSPACE when attn_workspace_size() for the shape exceeds 32 MiB.
 * All calls on a device share the array: calls whose GPU work overlaps in
 * time race on it and give wrong results, so order them on one stream.
 * `stream` must belong to the current device (ATTN_ERR_INVALID_ARG
 * otherwise).  The array's address is cached per device for the life of the
 * process: after cudaDeviceReset on a device this entry point must not be
 * used on it again.  A device wait that runs out is recorded in the array's
 * status word: read it with attn_noalloc_get_device_status. */
attn_status_t attn_bwd_noalloc(const attn_shape_t* shape, const void* q, const void* k,
                               const void* v, const void* o, const void* dO, const float* lse,
                               const float* sink, const attn_mask_desc_t* mask, float scale,
                               void* dq, void* dk, void* dv, float* dsink, void* stream);

/* ---- paged key/value cache (serving) ----
 *
 * A cache holds `num_pages` pages of `page_size` tokens for each of K and V.
 * Request b's token at position x lives in row x % page_size of page
 * block_table[b, x / page_size]; its slot is page * page_size + row.  The
 * K and the V pages are two device tensors of the same strides (in elements):
 * element (page, kv head, row, d) is at page * page_stride + head * head_stride
 * + row * token_stride + d, so that [pages, Hkv, page_size, 128],
 * [pages, page_size, Hkv, 128] and both halves of one interleaved tensor are
 * all described.  Strides are at least 128 and multiples of 8; page_size is a
 * multiple of 16 up to 65536; num_pages * page_size < 2^31. */
typedef struct {
  int num_pages, page_size, Hkv;
  int dtype; /* attn_dtype_t */
  long long page_stride, head_stride, token_stride;
} attn_pages_t;

/* One step's page planning, from request lengths on the device: which pages
 * the new tokens get, and where each token goes.  Every pointer is a device
 * pointer; nothing is read back to the host, so the call can be captured.
 *
 *   cached[b]      tokens of request b in the cache before the step
 *   fresh[b]       its new tokens of this step; negative: the request has ended
 *   free_pages     [num_pages] stack of free pages, of which the first
 *                  *free_count are free (the top is the last of them)
 *   block_table    [B, max_pages], rows table_stride apart
 *
 * In request order, ended requests first put their ceil(cached / page_size)
 * pages on the stack; then every other request takes the pages that its new
 * tokens need from the top, appended to its row of the table.  Written:
 *
 *   cu_seqlens_q   [B + 1] offsets of the requests' new tokens (ended: none)
 *   seqlen_k       [B] cached + fresh; 0 for ended requests
 *   free_count_out [1] free pages left
 *   slot_map       [max_tokens] int64: each new token's slot, -1 past the last
 *   position       [max_tokens] its position in its request, -1 past the last
 *   refused        [1] requests that were refused
 *
 * A request is refused, and keeps its pages and its cached length, when
 * cached + fresh exceeds max_pages * page_size, when its tokens end past
 * max_tokens (a request without new tokens: when those before it do), or when
 * it needs pages and those that the requests up to and with it need (but for
 * those refused by the first two rules) exceed the free ones: its slots are -1
 * and its rows of the step's attention mean nothing.
 * Entries of the table past a request's pages are left as they were.
 * seqlen_k may be `cached`, free_count_out may be `free_count`; with outputs
 * of their own the call may be repeated and does the same again.  Negative
 * cached counts as 0, *free_count is clamped to [0, num_pages], a page number
 * outside [0, num_pages) gives slots of -1, and pages that do not fit the
 * stack are dropped.  Limits: B <= 4096; max_pages * page_size and
 * num_pages * page_size < 2^31. */
typedef struct {
  int B, page_size, num_pages, max_pages, table_stride, max_tokens;
  const int* cached;
  const int* fresh;
  int* free_pages;
  const int* free_count;
  int* block_table;
  int* cu_seqlens_q;
  int* seqlen_k;
  int* free_count_out;
  long long* slot_map;
  int* position;
  int* refused;
} attn_plan_t;
attn_status_t attn_paged_plan(const attn_plan_t* plan, void* stream);

/* Writes the keys and values of T tokens into their slots: row t of k and v
 * ([T, Hkv, 128] of the pages' dtype; rows k_stride / v_stride elements apart,
 * heads 128 apart) goes to slot_map[t] of k_pages / v_pages.  A slot outside
 * [0, num_pages * page_size) is skipped (-1: a padded row).  Slots must be
 * distinct: of two rows for one slot either, or parts of each, may stay. */
attn_status_t attn_paged_store(const attn_pages_t* pages, int T, const void* k, const void* v,
                               long long k_stride, long long v_stride, const long long* slot_map,
                               void* k_pages, void* v_pages, void* stream);

/* Workspace bytes of attn_paged_fwd for this shape (host only): B requests
 * (<= 4096), Sq the longest run of new tokens, Skv the longest context.  The
 * need does not grow with the lengths.  Errors: ATTN_ERR_INVALID_ARG, and
 * ATTN_ERR_UNSUPPORTED for D != 128 or Hq / Hkv > 128. */
attn_status_t attn_paged_workspace_size(const attn_shape_t* shape, size_t* bytes);

/* Attention of each request's new tokens over its paged cache, in which their
 * own keys and values are stored already (attn_paged_store).
 *
 * q and o are packed rows [total_q, Hq, 128]; request b's new tokens are rows
 * [cu_seqlens_q[b], cu_seqlens_q[b + 1]), its keys are the first seqlen_k[b]
 * of its pages, and of n new tokens over L keys token i stands at position
 * x = L - n + i (the masks' i): the new tokens end where the keys end.  lse is
 * float32 [Hq, total_q], or NULL when it is not wanted.  A row that sees no
 * key (L = 0, or x < 0 unless the kind is NONE) gets O = 0 and LSE = the sink,
 * or +inf without one.
 *
 * mask: kind NONE, CAUSAL, SLIDING or SLIDING_FIRST (Sq and Skv need not be
 * equal); cu_seqlens_q, seqlen_k and total_q are set, seqlen_q and
 * cu_seqlens_k NULL.  Offsets are clamped to [0, total_q], new tokens to Sq,
 * keys to min(Skv, max_pages * page_size); rows of q that no request owns
 * leave o and lse as they were.  block_table is int32 [B, max_pages], rows
 * table_stride apart; only entries that hold a seen key are read.
 *
 * Pages may hold anything, NaN included, in rows past a request's keys, and in
 * those that none of its new tokens sees any more (before the window, past the
 * first keys): pages that left the window may be given back.  Keys and values
 * that some new token sees must be finite.  A row of q that is not finite gets
 * NaN in its own o and lse alone; where every logit that it sees is -inf (an
 * infinite element against keys of the other sign there) these weigh nothing,
 * and it gets what a row that sees no key does.  A page number outside [0,
 * num_pages) that holds seen keys is not read: it stands for zeros, and
 * attn_get_device_status then returns ATTN_ERR_INVALID_ARG.
 *
 * The lengths stay on the device: one call's grid and workspace serve any
 * lengths within the shape, so a captured call may be replayed with others.
 * Results do not depend on the order in which CTAs finish.  shape.flags must
 * be 0 and scale positive. */
attn_status_t attn_paged_fwd(const attn_shape_t* shape, const attn_pages_t* pages, const void* q,
                             const void* k_pages, const void* v_pages, const int* block_table,
                             int table_stride, int max_pages, const float* sink,
                             const attn_mask_desc_t* mask, float scale, void* o, float* lse,
                             void* ws, size_t ws_bytes, void* stream);

/* ---- rotary positions ----
 *
 * Pair i of a row at position x is turned by the angle x * w_i and multiplied by
 * `factor`: (x1, x2) -> factor (x1 cos - x2 sin, x2 cos + x1 sin).  The pairs are
 * elements (i, i + rotary_dim / 2), or (2 i, 2 i + 1) when `interleaved` is not 0;
 * elements from rotary_dim on stay as they are.  rotary_dim is a multiple of 16 up
 * to 128.  `turns` is a device array [rotary_dim / 2] of w_i / (2 pi) in units of
 * 2^-64 (modulo 2^64), so that the angle is exact at every position. */
typedef struct {
  int rotary_dim;
  int interleaved;
  float factor;
  const unsigned long long* turns;
} attn_rope_desc_t;

/* A tensor that is turned: element (b, head, token, d) of x is at b * x_batch +
 * head * x_head + token * x_token + d, and so for y, so that [T, heads, 128] rows
 * (possibly slices of a wider tensor) and [B, heads, S, 128] are both described.
 * Strides are in elements, multiples of 8, those of y at least 128; the stride of a
 * dimension of one is not read.  y may be x with the same strides; otherwise the two
 * must not overlap, nor may rows of y. */
typedef struct {
  const void* x;
  void* y;
  int heads;
  long long x_batch, x_head, x_token;
  long long y_batch, y_head, y_token;
} attn_rope_tensor_t;

/* Turns q, and k unless it is NULL, both of `dtype`: B sequences of S tokens.
 * position: device int32, token t of sequence b stands at position[b *
 * position_stride + t] (position_stride 0: one row for all); NULL: at t.  Rows at a
 * negative position are no tokens and are left as y had them.  inverse not 0: the
 * angles negated, which turns the gradients of y into those of x.  Results are
 * rounded once.  ATTN_ERR_UNSUPPORTED for an even rotary_dim that is no multiple of
 * 16. */
attn_status_t attn_rope(const attn_rope_desc_t* rope, int dtype, int B, int S,
                        const attn_rope_tensor_t* q, const attn_rope_tensor_t* k,
                        const int* position, long long position_stride, int inverse,
                        void* stream);

/* ---- paged key/value cache held in 8 bits ----
 *
 * Pages as in attn_pages_t, of one-byte codes, and a scale for each block of
 * `block` (1, 16, 32 or 64, a divisor of page_size) tokens of each kv head: a byte
 * s that stands for 2^(s - 127), or for NaN when it is 255.  A value is code * scale,
 * the code an e4m3 number or an int8 from -127 to 127; `dtype` is the 16-bit type of
 * the values, in which code * scale is exact for every scale that attn_paged8_store
 * writes.  (Scales of other origin: for ATTN_F16 exponents outside [-24, 15] count as
 * the nearest of these, for ATTN_BF16 byte 0 as 1.  What the e4m3 codes 0x7f and 0xff
 * and the int8 code -128 stand for is not defined.)
 *
 * Element (page, kv head, row, d) of the K or the V pages is at page * page_stride +
 * head * head_stride + row * token_stride + d, in bytes, strides multiples of 16 and
 * at least 128.  Its scale is byte page * scale_page_stride + head *
 * scale_head_stride + row / block of the K or V scales; these strides are at least
 * page_size / block, for block = 1 multiples of 16 (and the scales 16-byte aligned).
 * Other limits as for attn_pages_t. */
typedef enum { ATTN_E4M3 = 0, ATTN_I8 = 1 } attn_code_t;
typedef struct {
  int num_pages, page_size, Hkv;
  int dtype; /* attn_dtype_t: the values' type */
  int code;  /* attn_code_t */
  int block;
  long long page_stride, head_stride, token_stride;
  long long scale_page_stride, scale_head_stride;
} attn_pages8_t;

/* attn_paged_store into an 8-bit cache.  A block's scale is 2^e with the least e for
 * which its largest magnitude is at most 448 * 2^e (e4m3) or 127 * 2^e (int8), but at
 * least -15 (e4m3) or -24 (int8) for ATTN_F16 and -110 for ATTN_BF16; codes are
 * value / scale rounded to nearest even, held back to the largest code whose value is
 * finite in `dtype`.
 *
 * The rows of one call that go to one block must be consecutive, with consecutive
 * slots, as attn_paged_plan gives them (of other orders the block's content is
 * undefined, nothing else).  Where they begin at the block's row 0 the block begins
 * anew, whatever it held.  Where they begin at a row r > 0 its rows before r stay:
 * the block keeps the larger of its scale and the one that the new rows need, and if
 * that is the new one the earlier rows' codes are rounded in units of it, held back
 * as the new ones are.  Rows of the block past the new ones mean nothing afterwards.
 * A value that is not finite makes the scale 255: the block reads as NaN until it
 * begins anew.
 *
 * So a block does not forget tokens that are taken back (speculated ones that failed):
 * those stored in their place share the scale that they left, and are rounded in its
 * units, or read as NaN after a value that was not finite, until the block is stored
 * from row 0 again.  With block 1 every row begins its block. */
attn_status_t attn_paged8_store(const attn_pages8_t* pages, int T, const void* k, const void* v,
                                long long k_stride, long long v_stride, const long long* slot_map,
                                void* k_pages, void* v_pages, uint8_t* k_scales,
                                uint8_t* v_scales, void* stream);

/* Rows of an 8-bit cache back to 16 bits: row t of k and v ([total, Hkv, 128] of the
 * pages' dtype) is position start[b] + t - cu_seqlens[b] of the request b whose rows
 * [cu_seqlens[b], cu_seqlens[b + 1]) hold t (start NULL: all 0; negative ones count
 * as 0).  cu_seqlens is int32 [B + 1], ascending; rows of no request are left as they
 * were.  block_table is int32 [B, max_pages], rows table_stride apart; a position
 * past its pages, or in a page outside [0, num_pages), reads zeros.  B <= 65536. */
attn_status_t attn_paged8_load(const attn_pages8_t* pages, int B, int total, const int* start,
                               const int* cu_seqlens, const int* block_table, int table_stride,
                               int max_pages, const void* k_pages, const void* v_pages,
                               const uint8_t* k_scales, const uint8_t* v_scales, void* k, void* v,
                               void* stream);

/* Workspace bytes of attn_paged8_fwd: the least for mask = NULL, as
 * attn_paged_workspace_size; with the call's mask (of which kind, window, first and
 * total_q are read) with room besides for the rows that chunks see, in 16 bits: 512
 * bytes for each key (up to Skv, or those of the window) of each kv head and request
 * that may have a chunk, where the bounds say that there is work enough.  With that much
 * attn_paged8_fwd writes them there once; with less every query tile makes them anew
 * (chunks of 1900 tokens over 8000 keys: 389 and 603 us).  The results of both differ by
 * roundings. */
attn_status_t attn_paged8_workspace_size(const attn_shape_t* shape, const attn_mask_desc_t* mask,
                                         size_t* bytes);

/* attn_paged_fwd over an 8-bit cache: the attention over the values that the codes
 * and scales stand for, exactly (attn_paged8_load gives the same ones); masks,
 * lengths, results and statuses as attn_paged_fwd has them.  A block whose scale is
 * 255 reads as NaN, which a new token must not see, as it must not see other values
 * that are not finite. */
attn_status_t attn_paged8_fwd(const attn_shape_t* shape, const attn_pages8_t* pages, const void* q,
                              const void* k_pages, const void* v_pages, const uint8_t* k_scales,
                              const uint8_t* v_scales, const int* block_table, int table_stride,
                              int max_pages, const float* sink, const attn_mask_desc_t* mask,
                              float scale, void* o, float* lse, void* ws, size_t ws_bytes,
                              void* stream);

/* Synchronizes `stream`, then reads the status word that the last call which
 * used `ws` left in the workspace: ATTN_OK, or ATTN_ERR_TIMEOUT when a device
 * wait ran out, or ATTN_ERR_INVALID_ARG when attn_paged_fwd met a page
 * number outside the cache.  ATTN_ERR_CUDA if the synchronization itself fails. */
attn_status_t attn_get_device_status(const void* ws, void* stream);

/* Synchronizes `stream` (which must belong to the current device), then
 * reads the status word that the last attn_bwd_noalloc call on the current
 * device left in the library's scratch array: ATTN_OK or ATTN_ERR_TIMEOUT.
 * ATTN_ERR_INVALID_ARG for a stream of another device, ATTN_ERR_CUDA if the
 * synchronization or the read fails. */
attn_status_t attn_noalloc_get_device_status(void* stream);

/* Per-kernel timing, for diagnostics and benchmarks.  attn_profile_enable(1)
 * makes later attn_fwd / attn_bwd calls on this process bracket every kernel
 * they enqueue with CUDA events (created on first use, on the current device,
 * and kept until the process exits); attn_profile_enable(0) stops it.
 * attn_profile_read waits for the events of the most recent profiled call and
 * writes up to `capacity` kernel names (static strings) and elapsed times in
 * milliseconds, in launch order; *count receives the number of kernels.
 * Errors: ATTN_ERR_INVALID_ARG (null count, or names/ms null with capacity >
 * 0), ATTN_ERR_CUDA (event creation or synchronization failed). */
attn_status_t attn_profile_enable(int on);
attn_status_t attn_profile_read(const char** names, float* ms, int capacity, int* count);

/* Static string naming a status code ("ATTN_OK", ...). Never NULL. */
const char* attn_status_string(attn_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* MASKATTN_H_ */
