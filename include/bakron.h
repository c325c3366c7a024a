/*
 * bakron.h -- C ABI of libbakron.so: two-sided (Kronecker-factored) GPTQ
 * rounding on one AMD Instinct MI355X (gfx950).
 *
 * The method (arXiv 2608.06291, "BaKron: Efficient Quantization with
 * Kronecker-Factored Hessians", also published as "FastKron"; described on
 * the pith.science review page and the mlsanity.com index page):
 *   A weight matrix W (m x n; rows = outputs, columns = inputs) is rounded
 *   under the quadratic loss ||vec(W) - vec(V)||^2_H with H = A (x) B, where A
 *   (n x n) is the input-side and B (m x m) the output-side factor (review
 *   page, "Assumptions").  With LA, LB the lower Cholesky factors of A^-1 and
 *   B^-1 ("What carries the argument"), rounding entry (i,j) with current
 *   value P produces e = (P - Q(P)) / (LB[i][i] LA[j][j]) and the update
 *   W -= e LB[:,i] LA[:,j]^T (Proposition 3.1), which touches only rows >= i
 *   and columns >= j.  Entries on one anti-diagonal i + j = k are
 *   independent, and a recursion over anti-diagonal ranges batches the
 *   postponed updates into two matrix products (Algorithm 6; "Core claim",
 *   Theorem 3.2; O(m+n) sequential steps, O(mn(m+n)) work).
 *
 * Conventions for every call:
 *   - All matrices are dense, row-major, contiguous, 32-bit float unless noted,
 *     and live in device memory of the current HIP device.  They are owned by
 *     the caller; the library never keeps a pointer after the call returns.
 *   - Inputs are never written.  Outputs must not overlap inputs or each other.
 *   - `ws` is caller-owned device scratch of at least *_workspace_size() bytes,
 *     256-byte aligned.  Its contents on entry do not matter.
 *   - Every call enqueues work on `stream` (a hipStream_t; NULL = the null
 *     stream) and returns without waiting, unless a flag below asks for
 *     timing.  Overlapping calls that share a workspace race.
 *   - The return value reports argument and launch errors (BAKRON_ERR_*), and
 *     bakron_last_error() gives a message for the calling thread.  Errors
 *     found by the kernels are OR-ed as BAKRON_DEV_* bits into the optional
 *     device word `dev_status` (caller zeroes it; read it after synchronising).
 */
#ifndef BAKRON_H
#define BAKRON_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* return codes */
#define BAKRON_OK 0
#define BAKRON_ERR_INVALID_ARG 1
#define BAKRON_ERR_WORKSPACE 2
#define BAKRON_ERR_HIP 5
#define BAKRON_ERR_UNSUPPORTED_DEVICE 6

/* bits OR-ed into *dev_status by the kernels */
#define BAKRON_DEV_NONFINITE 1  /* a non-finite weight or error term was met */
#define BAKRON_DEV_NOT_PD 2     /* a non-positive pivot in bakron_factor */
#define BAKRON_DEV_SPIN_LIMIT 4 /* a bounded wait inside a kernel gave up (results invalid) */
#define BAKRON_DEV_BAD_INDEX 8  /* a target or a group offset out of range */

/* base quantizer kinds (the solver is modular in the base quantizer; review
 * page abstract).  Per-row (output channel) parameters from the ORIGINAL W:
 *   SYM  b in {2,3,4,8}: s_i = max_j |W_ij| / (2^(b-1) - 1), z_i = 0,
 *        codes in [-2^(b-1), 2^(b-1) - 1]
 *   ASYM b in {2,3,4}:   s_i = (max_j W_ij - min_j W_ij) / (2^b - 1),
 *        z_i = clamp(rint(-min_j W_ij / s_i), 0, 2^b - 1), codes in [0, 2^b - 1]
 *   UNIT (bits ignored): s_i = 1, z_i = 0, codes in [-128, 127] (unit grid)
 * s_i = 0 is replaced by 1.  The scale is IEEE fp32 arithmetic on fp32 data.
 * An entry with value P gets code c = clamp(rint(P / s_i) + z_i) (round half
 * to even) and dequantised value v = s_i (c - z_i). */
#define BAKRON_Q_SYM 0
#define BAKRON_Q_ASYM 1
#define BAKRON_Q_UNIT 2

/* flags for bakron_quantize */
#define BAKRON_ORDER_AUTO 0        /* pick the product order with fewer executed flops */
#define BAKRON_ORDER_LA_FIRST 1    /* band update as LB (E_S LA^T) */
#define BAKRON_ORDER_LB_FIRST 2    /* band update as (LB E_S) LA^T */
#define BAKRON_ORDER_MASK 3
#define BAKRON_FLAG_PHASE_TIMING 4 /* time each phase with HIP events; the call
                                      then synchronises the stream before it
                                      returns.  See bakron_last_phase_ms(). */
#define BAKRON_FLAG_NO_GRAPH 8     /* launch kernel by kernel instead of replaying
                                      the cached executable graph of the solve */
#define BAKRON_FLAG_MSE_SCALE 16   /* per-row scale shrink by MSE search (review
                                      page, free parameters: up to a factor 2).
                                      The row's range is scaled by p = 1, 0.99,
                                      ..., 0.50; each candidate takes the plain
                                      parameters of the shrunk range; the first p
                                      with the least sum over the row of
                                      (w - v)^2 (v the clamped base-quantizer value
                                      of w, fp32; sum in fp64) wins.  Symmetric and
                                      asymmetric kinds; ignored for BAKRON_Q_UNIT. */
#define BAKRON_FLAG_SPLIT_COLS 32  /* hybrid schedule (review "Circularity Check":
                                      BaKron-recursive's recurrence, Appendix C): solve
                                      the tile columns 0 .. N/2-1, apply their updates to
                                      the rest (W2 -= LB E1 LA21^T), solve the rest;
                                      each half by the recursion over anti-diagonals.
                                      Same result (Theorem 3.2). */
#define BAKRON_FLAG_SPLIT_ROWS 64  /* the same with the tile rows 0 .. M/2-1 first
                                      (W2 -= LB21 E1 LA^T).  At most one split flag;
                                      neither with BAKRON_FLAG_PHASE_TIMING. */

/*
 * bakron_hessian -- Kronecker factor from samples, with damping.
 *   H = X^T X / N + damp_rel * mean(diag(X^T X / N)) * I
 * (input side: X = activation samples, giving A; output side: output-side
 * samples, giving B.  Gram regularisation by a multiple of the mean diagonal:
 * review page, free parameters.)
 *   X  N x d, row-major (one sample per row), device.   H  d x d, full
 *   symmetric, device.  N >= 1, d >= 1, damp_rel >= 0 and finite.
 * Computed with fp32 matrix cores, fp32 accumulation.
 */
size_t bakron_hessian_workspace_size(int64_t N, int64_t d);
int32_t bakron_hessian(const float *X, int64_t N, int64_t d, float damp_rel,
                       float *H, void *ws, size_t ws_bytes, void *stream);

/*
 * bakron_factor -- L = lower Cholesky factor of H^-1 (L L^T = H^-1), the
 * "normalised Cholesky factor" the solver consumes (review page, "What
 * carries the argument": lower-triangular Cholesky factors of A^-1, B^-1).
 *   H  d x d symmetric positive definite (only the lower triangle is read).
 *   L  d x d lower triangular, strictly-upper part written as 0.
 * Computed in fp64 as the reverse-order factorisation H = U U^T (U upper),
 * L = U^-T.  A non-positive pivot sets BAKRON_DEV_NOT_PD in *dev_status (may
 * be NULL) and leaves L undefined.
 */
size_t bakron_factor_workspace_size(int64_t d);
int32_t bakron_factor(const float *H, int64_t d, float *L, int32_t *dev_status,
                      void *ws, size_t ws_bytes, void *stream);

/*
 * bakron_quantize -- the solver (BaKron, Algorithm 6).
 *   W      m x n input weights.
 *   LA     n x n, lower Cholesky factor of A^-1 (only the lower triangle is read).
 *   LB     m x m, lower Cholesky factor of B^-1 (only the lower triangle is read).
 *   qkind, qbits  base quantizer (BAKRON_Q_*).
 *   codes  m x n int8 output codes.
 *   scales m output per-row scales.       zeros  m per-row zero points or NULL.
 *   V      m x n dequantised output (v = s_i (c - z_i)), or NULL.
 *   E      m x n normalised errors e_ij, or NULL.
 *   sum_e2 device double, receives sum e_ij^2 (= the proxy loss when LA, LB
 *          are exact; fixed-order reduction), or NULL.
 *   flags  BAKRON_ORDER_* | BAKRON_FLAG_*.
 * Any m, n >= 1 is accepted; inside, W is handled in 64 x 64 tiles with
 * zero padding.  The result equals the raster-order naive solver up to fp32
 * rounding order (Theorem 3.2).
 * The static schedule of a solve (see bakron_schedule_plan) runs on two
 * streams: `stream` carries the leaves and the band products that feed the
 * next target diagonals; the rest of the wide recursion nodes' products runs
 * on a side stream of the library's, forked and joined with events, while the
 * leaves occupy few CUs.  The results do not depend on the interleaving (the
 * plan orders every pair of steps that share data) and are the same bit for
 * bit with and without BAKRON_FLAG_NO_GRAPH and BAKRON_FLAG_PHASE_TIMING (the
 * latter runs the plan in order on `stream`).
 * The schedule is captured once into an executable HIP graph, cached per
 * (device, sizes, quantizer, order, every pointer argument, ws) -- at most 16
 * graphs, least recently used dropped -- and replayed on `stream`.  The first
 * call with a new key pays the capture.  Calls from several host threads are
 * safe when they use distinct workspaces and outputs: the cache is locked from
 * lookup through launch, and an evicted graph is destroyed only after its
 * last launch has completed.  Calls that share a workspace race on it.
 */
size_t bakron_quantize_workspace_size(int64_t m, int64_t n, int32_t qkind, int32_t qbits);
int32_t bakron_quantize(const float *W, int64_t m, int64_t n, const float *LA,
                        const float *LB, int32_t qkind, int32_t qbits,
                        int8_t *codes, float *scales, float *zeros, float *V,
                        float *E, double *sum_e2, int32_t *dev_status,
                        int32_t flags, void *ws, size_t ws_bytes, void *stream);

/*
 * bakron_quantize_noalloc -- bakron_quantize for callers that cannot allocate
 * device memory: code under HIP stream capture, tight serving loops, harnesses
 * that forbid hipMalloc.  Same arguments and results as bakron_quantize, without
 * the workspace; the flags BAKRON_ORDER_*, BAKRON_FLAG_MSE_SCALE and
 * BAKRON_FLAG_SPLIT_* (BAKRON_FLAG_NO_GRAPH is accepted and changes nothing).
 *   - The solve's scratch is a fixed array of BAKRON_NOALLOC_SCRATCH_BYTES in
 *     device memory, inside the library: each GPU it runs on holds one copy
 *     until the process ends.  A shape whose workspace
 *     (bakron_quantize_workspace_size) exceeds it is rejected with
 *     BAKRON_ERR_WORKSPACE before anything is enqueued (2048 x 2048 fits,
 *     4096 x 4096 does not).
 *   - The plan runs in order on `stream` alone: no side stream, no event, no
 *     graph.  The results equal bakron_quantize's bit for bit.
 *   - It calls no hipMalloc, hipFree or other allocating routine.
 *   - Every call on one GPU uses that GPU's array, which keeps the last call's
 *     contents (what must start at zero is cleared by each call).  Calls that
 *     overlap on one GPU (other streams, other host threads) race on it and
 *     give wrong results: serialise them.
 * Returns as bakron_quantize; BAKRON_FLAG_PHASE_TIMING is rejected.
 */
#define BAKRON_NOALLOC_SCRATCH_BYTES ((size_t)256 << 20)
int32_t bakron_quantize_noalloc(const float *W, int64_t m, int64_t n, const float *LA,
                                const float *LB, int32_t qkind, int32_t qbits, int8_t *codes,
                                float *scales, float *zeros, float *V, float *E, double *sum_e2,
                                int32_t *dev_status, int32_t flags, void *stream);

/*
 * bakron_quantize_antidiag -- BaKron-antidiagonal, the pages' comparison
 * variant (review page "If this is right": BaKron runs about 27x faster than
 * it at 4096 x 4096; "Core claim", Theorem 3.2: both give the same output).
 * Every entry anti-diagonal d = i + j is rounded at once, then its rank-|d|
 * update W[i'][j'] -= sum_{(i,j) on d} LB[i'][i] e_ij LA[j'][j] is applied to
 * the rest of the matrix: O(m + n) steps, O(m^2 n^2) work.  Arguments,
 * quantizer and outputs as for bakron_quantize (no sum_e2; no flags); two
 * kernel launches per anti-diagonal on `stream`, no graph.  Its own workspace
 * (bakron_quantize_antidiag_workspace_size).  Returns as bakron_quantize.
 */
size_t bakron_quantize_antidiag_workspace_size(int64_t m, int64_t n, int32_t qkind, int32_t qbits);
int32_t bakron_quantize_antidiag(const float *W, int64_t m, int64_t n, const float *LA,
                                 const float *LB, int32_t qkind, int32_t qbits, int8_t *codes,
                                 float *scales, float *zeros, float *V, float *E,
                                 int32_t *dev_status, void *ws, size_t ws_bytes, void *stream);

/*
 * bakron_schedule_info -- the static schedule for an m x n solve, without
 * touching the GPU.  out[0..14]:
 *   0 tile size b           1 leaf launches (tile anti-diagonals M+N-1)
 *   2 band GEMM launches    3 sequential in-kernel diagonal steps ((M+N-1)(2b-1))
 *   4 order used (1 = LA first, 2 = LB first)
 *   5 algorithmic band flops: two products per recursion node at single
 *     anti-diagonal granularity (the exact staircase count of Algorithm 6)
 *   6 flops the band GEMM launches execute with dense b x b tiles (order of out[4])
 *   7 the paper's count F = m n (m + n)
 *   8 in-tile leaf flops executed (two length-b dot products per entry)
 *   9 recursion depth (levels)
 *  10 useful flops of the band GEMM launches: out[6] without the zero half of
 *     the triangular diagonal factor blocks
 *  11 flops of the two-diagonal nodes: a recursion node over two tile
 *     diagonals has no launch of its own; its update (up to four dense
 *     b x b x b products per tile) runs inside the leaves of its two diagonals
 *  12 leaf launches that pull
 *  13 of the band launches in out[2]: deferred ones (side stream)
 *  14 useful flops of the deferred launches (part of out[10])
 * Returns BAKRON_OK or BAKRON_ERR_INVALID_ARG.
 */
int32_t bakron_schedule_info(int64_t m, int64_t n, int32_t flags, double *out);

/*
 * bakron_schedule_plan -- the ordered steps of an m x n solve, for inspection
 * and tests; touches no GPU.  Writes *count; with ops != NULL (cap >= *count
 * entries of 16 int32, else BAKRON_ERR_INVALID_ARG) entry k is step k:
 *   [0] kind: 0 leaf, 1 band product, 2 record event, 3 wait for event
 *   [1] band: 1 = deferred (side stream); record / wait: 1 = on the side stream
 *   [2] record / wait: event index
 *   leaf:  [3] tile diagonal K, [4] 1 = applies the previous leaf's
 *          two-diagonal update, 2 = computes it for the next leaf
 *   band:  [3] K, [5] L, [6] H of the recursion node (split at K + H), [7] its
 *          T buffer (its recursion depth; the nodes below the deepest level
 *          that defers products share one), [8] product (0 first, 1 second),
 *          [9..10] diagonal range lo, hi (T diagonals for the first product,
 *          W target diagonals for the second), then the launch grid for the
 *          order given in flags: [11] mode, [12] first band offset, [13] offsets,
 *          [14] first row, [15] rows (-1 when the range holds no tile).
 * Unused fields are -1.  Returns BAKRON_OK or BAKRON_ERR_INVALID_ARG.
 */
int32_t bakron_schedule_plan(int64_t m, int64_t n, int32_t flags, int32_t *ops, int64_t cap,
                             int64_t *count);

/* Per-phase times (ms) of the calling thread's last bakron_quantize call made
 * with BAKRON_FLAG_PHASE_TIMING.  That call runs the plan in order on one
 * stream with an event after every step: out[0] quantizer parameters +
 * relayout, out[1] leaf kernels, out[2] band GEMM kernels on the critical
 * stream, out[3] finalise, out[4] leaf launches, out[5] critical band GEMM
 * launches, out[6] deferred band kernels, out[7] deferred band launches.
 * These intervals include each launch's dispatch latency.  The call then
 * replays the critical band launches alone, and then the deferred ones alone,
 * each as a one-off graph whose kernels start back to back, timed by events
 * around the graph launch: out[8] and out[9] (kernel time without dispatch
 * gaps; the replays rewrite the workspace, not the outputs).  Returns
 * BAKRON_ERR_INVALID_ARG if no such call was made. */
int32_t bakron_last_phase_ms(double *out);

/* ---------------------------------------------------------------------------
 * Operators for rounded layers: what multiplies with the solver's result, by
 * expert where a layer has experts, and what says how a model's answers moved.
 * For these calls a matrix's rows may be `ld` elements apart (ld >= its width;
 * any ld and any alignment of one element are accepted, rows that begin on 16
 * bytes are faster).  Sizes are 1 to 2^24 unless noted, groups 1 to 4096; groups
 * may be empty.  A product whose tiles need 2^32 threads or more is refused.
 */

/* element types */
#define BAKRON_T_F32 0
#define BAKRON_T_BF16 1
#define BAKRON_T_F16 2

/*
 * bakron_fp8_quantize -- X in 8-bit floating point (e4m3: 3 mantissa bits,
 * largest value 448) with a scale for each row and 128 columns (block_rows 1:
 * activations) or each 128 x 128 block (block_rows 128: weights); the blocks at
 * the right and lower edge may be smaller.
 *   amax = max |x| of the block, at least 2^-100;  scale = amax / 448 (1 for a
 *   block of zeros);  Q = e4m3(clamp(x (448 / amax), -448, 448)), to nearest even
 *   X       rows x cols, `type` BAKRON_T_*, row stride ldx.  rows, cols <= 2^22.
 *   Q       rows x cols codes, row stride ldq.
 *   scales  ceil(cols / 128) x ceil(rows / block_rows), contiguous: the scales
 *           of one block of columns lie together, as the product reads them.
 * A block that holds a NaN or an infinity gets NaN codes and a NaN scale, and
 * sets BAKRON_DEV_NONFINITE in *dev_status (may be NULL).
 */
int32_t bakron_fp8_quantize(const void *X, int32_t type, int64_t rows, int64_t cols, int64_t ldx,
                            int32_t block_rows, uint8_t *Q, int64_t ldq, float *scales,
                            int32_t *dev_status, void *stream);

/*
 * bakron_fp8_from_codes -- a solve's codes as e4m3 weights, exactly: Q = c - z,
 * an integer in [-15, 15] for every kind and width accepted here (BAKRON_Q_SYM
 * and BAKRON_Q_ASYM with 2 to 4 bits).  With the solve's row scales,
 * bakron_fp8_matmul (BAKRON_SCALE_ROW) multiplies with V itself.
 *   codes  m x n (contiguous, as bakron_quantize writes them); m, n <= 2^22,
 *          m n <= 2^40
 *   zeros  m zero points for BAKRON_Q_ASYM, else NULL
 *   Q      m x n, row stride ldq
 */
int32_t bakron_fp8_from_codes(const int8_t *codes, const float *zeros, int64_t m, int64_t n, int32_t qkind,
                              int32_t qbits, uint8_t *Q, int64_t ldq, void *stream);

/* scales of fp8 weights */
#define BAKRON_SCALE_ROW 0   /* one for each row */
#define BAKRON_SCALE_BLOCK 1 /* one for each 128 x 128 block */

/*
 * Rows by group.  `offsets` (device, groups + 1 values, from 0 on, not falling,
 * the last at most rows) gives group g the rows offsets[g] .. offsets[g+1] - 1
 * of X and Y; groups may be empty.  Rows after the last group's get 0.  Offsets
 * that fall or leave [0, rows] set BAKRON_DEV_BAD_INDEX in *dev_status; nothing
 * outside the matrices and the workspace is touched, and the result is undefined.  `offsets` NULL
 * goes with groups = 1: all rows.  The host never reads offsets.
 * Products are summed on the matrix cores in fp32; the order is fixed, so equal
 * inputs give equal bits.
 *
 * bakron_fp8_matmul -- Y = X W_g^T, both operands in e4m3 with scales:
 *   Y[r][n] = sum_b sx[b][r] sw(g, b, n) sum_{k in block b} X[r][k] W_g[n][k]
 * over blocks b of 128 of k.
 *   X   rows x K codes, row stride ldx;   sx  ceil(K / 128) x rows
 *   W   groups x N x K codes, row stride ldw, groups N ldw apart
 *   sw  wscale BAKRON_SCALE_ROW:   groups x N
 *       wscale BAKRON_SCALE_BLOCK: groups x ceil(K / 128) x ceil(N / 128)
 *   Y   rows x N in ytype (bf16 or fp16; the fp8 matrix cores keep too few bits
 *       of a sum for an fp32 result), row stride ldy
 *   ws  bakron_fp8_matmul_workspace_size() bytes
 */
size_t bakron_fp8_matmul_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t groups);
int32_t bakron_fp8_matmul(const uint8_t *X, int64_t ldx, const float *sx, const uint8_t *W, int64_t ldw,
                          const float *sw, int32_t wscale, int64_t rows, int64_t N, int64_t K,
                          int32_t groups, const int32_t *offsets, void *Y, int32_t ytype, int64_t ldy,
                          int32_t *dev_status, void *ws, size_t ws_bytes, void *stream);

/*
 * bakron_grouped_matmul -- Y[r] = X[r] W_g(r)^T, and its gradients
 *   grad_x:  dX[r] = dY[r] W_g(r)        grad_w:  dW_g = dY_g^T X_g (0 for an empty group)
 *   X, dX rows x K;  W, dW groups x N x K (groups N ldw apart);  Y, dY rows x N
 * Inputs are bf16 or fp16 (`type`); the output is of that type or fp32.
 *   ws  *_workspace_size() bytes
 */
size_t bakron_grouped_matmul_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t groups);
int32_t bakron_grouped_matmul(const void *X, int32_t type, int64_t ldx, const void *W, int64_t ldw,
                              int64_t rows, int64_t N, int64_t K, int32_t groups, const int32_t *offsets,
                              void *Y, int32_t ytype, int64_t ldy, int32_t *dev_status, void *ws,
                              size_t ws_bytes, void *stream);
int32_t bakron_grouped_matmul_grad_x(const void *dY, int32_t type, int64_t lddy, const void *W, int64_t ldw,
                                     int64_t rows, int64_t N, int64_t K, int32_t groups,
                                     const int32_t *offsets, void *dX, int32_t dxtype, int64_t lddx,
                                     int32_t *dev_status, void *ws, size_t ws_bytes, void *stream);
int32_t bakron_grouped_matmul_grad_w(const void *dY, int32_t type, int64_t lddy, const void *X, int64_t ldx,
                                     int64_t rows, int64_t N, int64_t K, int32_t groups,
                                     const int32_t *offsets, void *dW, int32_t dwtype, int64_t lddw,
                                     int32_t *dev_status, void *ws, size_t ws_bytes, void *stream);

/*
 * bakron_token_logprobs -- log probabilities of given tokens, with entropy and
 * the k likeliest tokens.  Per row of logits x:
 *   lse = log sum_j e^x_j;  logprob = x_target - lse;  entropy = -sum_j p_j log p_j
 *        (log probabilities are not taken from the rounded lse: with |lse| large,
 *        as in a row of the type's lowest value, they hold more than it does)
 *   top: the k largest log probabilities and their tokens, in falling order,
 *        equal values by lowest index.
 *   logits   rows x vocab, `type` BAKRON_T_*, row stride ld.  -inf masks a token.
 *            vocab <= 2^21, k <= min(64, vocab).
 *   targets  rows token numbers; a negative one gives logprob 0.  One >= vocab
 *            gives NaN and sets BAKRON_DEV_BAD_INDEX.
 *   logprob, lse, entropy  rows fp32.   top_logprob, top_ids  rows x k (k > 0).
 * A row of -inf only has no distribution: lse = logprob = top_logprob = -inf,
 * entropy 0.  A row with a NaN or +inf gives NaN and sets BAKRON_DEV_NONFINITE
 * (its top_ids are tokens of the row, in no order that is defined).
 */
size_t bakron_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int32_t k);
int32_t bakron_token_logprobs(const void *logits, int32_t type, int64_t rows, int64_t vocab, int64_t ld,
                              const int64_t *targets, int32_t k, float *logprob, float *lse, float *entropy,
                              float *top_logprob, int64_t *top_ids, int32_t *dev_status, void *ws,
                              size_t ws_bytes, void *stream);

/*
 * bakron_token_logprobs_grad -- the gradient of sum_r (g_logprob logprob +
 * g_entropy entropy) with respect to the logits:
 *   dlogits_j = g_logprob ([j = target] - p_j) - g_entropy p_j (log p_j + entropy)
 * from the forward call's lse and entropy.  p_j = e^(x_j - lse) of lse as given,
 * an fp32 value: its rounding is p's relative error, 2^-15 at |lse| = 1024, and
 * a row of fp32's or bf16's lowest value only, where lse holds nothing of log s,
 * has p = 1 throughout; such rows should be masked with -inf.
 * Rows without a target have no first term, rows of -inf only get 0.  A target
 * >= vocab sets BAKRON_DEV_BAD_INDEX; its row then has the terms in p only.
 * g_entropy may be NULL (then entropy may be).
 * dlogits has the logits' type, row stride ldd.  With g_logprob = 1 its rows are
 * the last layer's output-side samples (bakron_hessian).
 */
int32_t bakron_token_logprobs_grad(const void *logits, int32_t type, int64_t rows, int64_t vocab, int64_t ld,
                                   const int64_t *targets, const float *lse, const float *entropy,
                                   const float *g_logprob, const float *g_entropy, void *dlogits,
                                   int64_t ldd, int32_t *dev_status, void *stream);

/* ---------------------------------------------------------------------------
 * Rows by group and back: what stands around a product by expert, or by adapter.
 * A batch has `tokens` rows with k choices of a group each, hence n = tokens k pairs;
 * pair t k + j is the j-th choice of token t.  n <= 2^24, k <= 64, groups <= 4096.
 *
 * bakron_group_sort -- a stable sort of the pairs by group:
 *   ids      n group numbers, 32- or 64-bit (`id_bits`), contiguous.  A negative one
 *            belongs to no group (a choice that was dropped, a row without adapter).
 *            One >= groups is taken as negative and sets BAKRON_DEV_BAD_INDEX.
 *   offsets  groups + 1 values: group g has the places offsets[g] .. offsets[g+1] - 1;
 *            pairs of no group have those from offsets[groups] on.
 *   order    n values: the pair at each place; pairs of one group keep their order
 *   slots    n values: the place of each pair (order and slots are permutations, each
 *            the other's inverse)
 *   ws       bakron_group_sort_workspace_size() bytes
 */
size_t bakron_group_sort_workspace_size(int64_t n, int32_t groups);
int32_t bakron_group_sort(const void *ids, int32_t id_bits, int64_t n, int32_t groups, int32_t *offsets,
                          int32_t *order, int32_t *slots, int32_t *dev_status, void *ws, size_t ws_bytes,
                          void *stream);

/*
 * The calls below take the slots (tokens x k, each place once) and offsets of a
 * sort.  Of the offsets they read the last.  A slot outside [0, n) is left out and sets
 * BAKRON_DEV_BAD_INDEX; a place that no slot names is not written.
 *
 * bakron_group_gather -- out[slots[t][j]] = X[t], and 0 for pairs of no group.
 *   X tokens x cols, out n x cols, of one type.  The gradient of X is
 *   bakron_group_combine of out's, without weights.
 * bakron_group_gather_fp8 -- the same in e4m3 with a scale for each row and 128
 *   columns, as bakron_fp8_quantize rounds (each token once).  Q n x cols, scales
 *   ceil(cols / 128) x n; pairs of no group get codes 0 and scales 1.
 * bakron_group_combine -- out[t] = sum_j weights[t][j] Y[slots[t][j]] over the choices
 *   that have a group, in fp32, in the order of j, rounded once.  weights tokens x k
 *   fp32, or NULL for 1.  Y n x cols, out tokens x cols, of one type.  Rows of Y of no
 *   group are not read.
 * bakron_group_combine_grad -- its gradients: dY[slots[t][j]] = weights[t][j] dout[t] (0
 *   for pairs of no group), dweights[t][j] = <dout[t], Y[slots[t][j]]> (fp32, 0 for pairs
 *   of no group).
 */
int32_t bakron_group_gather(const void *X, int32_t type, int64_t tokens, int32_t k, int64_t cols, int64_t ldx,
                            const int32_t *slots, int32_t groups, const int32_t *offsets, void *out, int64_t ldo,
                            int32_t *dev_status, void *stream);
int32_t bakron_group_gather_fp8(const void *X, int32_t type, int64_t tokens, int32_t k, int64_t cols, int64_t ldx,
                                const int32_t *slots, int32_t groups, const int32_t *offsets, uint8_t *Q,
                                int64_t ldq, float *scales, int32_t *dev_status, void *stream);
int32_t bakron_group_combine(const void *Y, int32_t type, int64_t tokens, int32_t k, int64_t cols, int64_t ldy,
                             const int32_t *slots, int32_t groups, const int32_t *offsets, const float *weights,
                             void *out, int64_t ldo, int32_t *dev_status, void *stream);
int32_t bakron_group_combine_grad(const void *dout, int64_t ldd, const void *Y, int32_t type, int64_t tokens,
                                  int32_t k, int64_t cols, int64_t ldy, const int32_t *slots, int32_t groups,
                                  const int32_t *offsets, const float *weights, void *dY, int64_t lddy,
                                  float *dweights, int32_t *dev_status, void *stream);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection.  Places of a
 * bakron_group_sort of the rows' adapters (k = 1): group g has the places offsets[g] ..
 * offsets[g+1] - 1, order[place] is the row there (NULL: the place itself; each row once),
 * rows from offsets[groups] on have no adapter.  offsets NULL goes with groups = 1.
 * Offsets as for the products by group; an order outside [0, rows) is left out and sets
 * BAKRON_DEV_BAD_INDEX.
 *
 * bakron_adapter_matmul -- out[r] = base[r] + scale_g B_g (A_g X[r]) for row r of adapter
 * g, base[r] for a row without one
 *   X  rows x K;  A  groups x rank x K;  B  groups x N x rank (A and B contiguous): bf16 or
 *      fp16 (`type`).  rank 1 .. 256; rows, N and K up to 2^24, where tiles of 16 rows by 256
 *      columns (64 rows, of large batches) fit a launch: (rows / 16 + groups) max(N, K) below
 *      about 2^32, in the gradients also 4 groups max(N, K).
 *   scale  groups fp32, or NULL for 1
 *   base, out  rows x N of that type or fp32 (`otype`); base NULL counts as 0, and base
 *      may be out: then rows without adapter are left as they are
 *   ws  *_workspace_size() bytes
 * Sums are in fp32.  The rank values between the two products keep fp32's 24 bits where
 * the result is fp32, and 16 (a relative 2^-16) where it is of 16 bits; the result is
 * rounded once.  What depends on a value that is not finite is not finite (where the
 * formula has an infinity it may be a NaN).
 *
 * bakron_adapter_matmul_grad -- for dY (rows x N), with U = scale dY B and
 * P = scale X A^T:
 *   dX = base + U A (base as above, of dX's type);  dA_g = U_g^T X_g;  dB_g = dY_g^T P_g
 *   dX, dA and dB of the inputs' type or fp32 (`xtype`, `wtype`).  dX may be NULL, dA and dB
 *   too (both; then X may be).  Adapters without rows get 0.
 */
size_t bakron_adapter_matmul_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups);
int32_t bakron_adapter_matmul(const void *X, int32_t type, int64_t ldx, const void *A, const void *B, int64_t rows,
                              int64_t N, int64_t K, int32_t rank, int32_t groups, const int32_t *offsets,
                              const int32_t *order, const float *scale, const void *base, int64_t ldb, void *out,
                              int32_t otype, int64_t ldo, int32_t *dev_status, void *ws, size_t ws_bytes,
                              void *stream);
size_t bakron_adapter_matmul_grad_workspace_size(int64_t rows, int64_t N, int64_t K, int32_t rank, int32_t groups);
int32_t bakron_adapter_matmul_grad(const void *dY, int64_t lddy, const void *X, int32_t type, int64_t ldx,
                                   const void *A, const void *B, int64_t rows, int64_t N, int64_t K, int32_t rank,
                                   int32_t groups, const int32_t *offsets, const int32_t *order, const float *scale,
                                   const void *base, int64_t ldb, void *dX, int32_t xtype, int64_t lddx, void *dA,
                                   void *dB, int32_t wtype, int32_t *dev_status, void *ws, size_t ws_bytes,
                                   void *stream);

/* ---------------------------------------------------------------------------
 * bakron_verify_drafts -- which drafted tokens a target model keeps, and the token that
 * follows them, from given random numbers; a rounded model drafts for its original.  Per
 * request, with drafts d_i drawn from q_i and the target's probabilities p_i:
 *   draft i is accepted where u_i q_i(d_i) < p_i(d_i) and all before it are;
 *   at the first refusal the token is drawn from max(p_i - q_i, 0) (from p_i where that
 *   has no weight), after the last draft from the p that follows: the first token whose
 *   cumulated weight is above v times the whole.
 * Products, differences and sums are in 64 bits.
 *   p  batch x (drafts + 1) rows of vocab probabilities, row stride ldp
 *   q  batch x drafts rows, row stride ldq; NULL where drafts were not drawn: then q(d_i)
 *      counts as 1 and a refused token is left out of p_i
 *      (both `type` BAKRON_T_*; rows need not sum to 1, only to be finite and >= 0)
 *   draft_tokens  batch x drafts; a negative one ends a request's drafts
 *   u batch x drafts, v batch: uniform in [0, 1), fp32
 *   accepted  batch;  tokens  batch x (drafts + 1): the accepted drafts, the drawn token,
 *             then -1
 *   ws  *_workspace_size() bytes.  batch <= 2^20, drafts 0 .. 64, vocab <= 2^24.
 * Rows after the first refusal are not read.  A draft >= vocab is refused and sets
 * BAKRON_DEV_BAD_INDEX.  A NaN or an infinity of a p or q that was compared, and a sum of
 * weights that is not finite, set BAKRON_DEV_NONFINITE; the drawn token is -1 for such a
 * sum, and where a row of p has no weight at all.
 */
size_t bakron_verify_drafts_workspace_size(int64_t batch, int32_t drafts, int64_t vocab);
int32_t bakron_verify_drafts(const void *p, int64_t ldp, const void *q, int64_t ldq, int32_t type, int64_t batch,
                             int32_t drafts, int64_t vocab, const int64_t *draft_tokens, const float *u,
                             const float *v, int32_t *accepted, int64_t *tokens, int32_t *dev_status, void *ws,
                             size_t ws_bytes, void *stream);

const char *bakron_status_string(int32_t status);
const char *bakron_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* BAKRON_H */
