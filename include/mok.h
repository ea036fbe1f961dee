/*
 * mok.h — C ABI of the MI355X (gfx950) MoE-layer library.
 *
 * One GPU's share of a deterministic mixture-of-experts training layer,
 * forward and backward: top-k ids -> schedule table -> drop-free permute of
 * token rows through a fixed ring buffer in mini-batches -> SwiGLU experts as
 * grouped GEMMs -> weighted combine back to token order; the backward pass
 * mirrors these steps and computes the router-weight gradient inside the
 * SwiGLU backward.
 *
 * Sources: "Mixture-of-Kittens (MoK)" project summary (Functional API; Key
 * concepts table), "Cursor Open-Sources Mixture-of-Kittens (MoK)" digest
 * (English abstract) and "Mixture-of-Kittens(MoK)란?" explainer (sections 1,
 * 4 ①-③). Each call below names the passage that defines it.
 *
 * Conventions for every call:
 *  - Every buffer is allocated and freed by the caller. The library never
 *    allocates, frees, synchronises or copies device memory back to the host.
 *  - Device pointers must be 16-byte aligned. Work is enqueued on `stream`
 *    (a hipStream_t; NULL = the legacy default stream) and the call returns
 *    without waiting for it.
 *  - Host-checkable problems (bad sizes, misaligned or NULL pointers, a buffer
 *    smaller than mok_query_sizes reports, fewer than 2 ring slots) return a
 *    non-zero mok_status and enqueue nothing.
 *  - Data-dependent problems set bits in the device status word (uint32 at
 *    byte 0 of the schedule buffer): MOK_SCHEDULE_OVERFLOW, MOK_BAD_EXPERT_ID.
 *    mok_forward / mok_backward then do no work and their outputs are
 *    undefined. The caller reads the word whenever it synchronises; no
 *    routed row is ever dropped silently.
 *  - Calls are re-entrant; concurrent calls need distinct workspaces.
 *  - bf16 tensors are raw 16-bit patterns; all tensors are dense row-major.
 */
#ifndef MOK_H
#define MOK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mok_status {
    MOK_OK = 0,
    MOK_ERROR_INVALID_VALUE = 1,
    MOK_ERROR_UNSUPPORTED = 2,
    MOK_ERROR_BUFFER_TOO_SMALL = 3,
    MOK_ERROR_LAUNCH_FAILED = 4
} mok_status;

/* precision modes ("Mixture-of-Kittens (MoK)" project summary, Overview) */
#define MOK_BF16 0
#define MOK_MXFP8 1
/* MXFP8 with the weight gradients on the block-scaled MFMA as well: their
   operands (x, dh, g*a, dy) are quantized along the token axis, 32 rows of one
   expert per E8M0 scale in canonical order, each expert's rows zero-padded to
   a multiple of 128 ("Mixture-of-Kittens (MoK)" project summary, Key-concepts
   table: MXFP8 mode; the pages leave the weight-gradient precision open). */
#define MOK_MXFP8_WGRAD 2

/* device status word bits */
#define MOK_SCHEDULE_OVERFLOW 1u
#define MOK_BAD_EXPERT_ID 2u
/* a persistent kernel's work queue made no progress within its spin limit
   (never expected; outputs are then undefined and the kernel has exited) */
#define MOK_SCHEDULER_STALLED 4u
/* mok_forward / mok_backward got a schedule table built for another layout:
   a different shape, minibatch_rows, macrobatch_tokens, capacity_multiplier
   or m-tile height (set by the precision). The builder writes a fingerprint of
   these into the table and each reader checks it before reading anything
   else; no work is done after a mismatch. */
#define MOK_SCHEDULE_MISMATCH 8u

/* debug_flags: replace every expert by the identity on its rows (forward only;
   out_t = sum_j g_tj * x_t). Used to test permute followed by unpermute. */
#define MOK_DEBUG_IDENTITY_EXPERT 1u
/* debug_flags: run each grouped GEMM of a ring round as its own launch
   instead of the persistent producer/consumer kernel (same results, bit for
   bit; used to cross-check the scheduler and to time GEMMs one by one).
   BF16 only: MXFP8 rounds always launch their GEMMs one by one. */
#define MOK_DEBUG_SEPARATE_LAUNCHES 2u
/* debug_flags (k == 1 only): run each whole forward / dgrad pass as one
   persistent launch in which gathers and both GEMMs of every ring round
   follow the in-kernel ring protocol (slot full / release counters) instead
   of stream order between rounds. Currently switched off: every call that
   sets it returns MOK_ERROR_UNSUPPORTED and enqueues nothing, because runs
   that included this mode hung twice without a shown cause. */
#define MOK_DEBUG_WHOLE_PASS 4u
/* debug_flags: every wait inside the persistent kernels gives up at once, as
   if its poll budget were spent. The call then ends with
   MOK_SCHEDULER_STALLED in the status word, leaving the outputs that depend
   on the abandoned waits unwritten. Tests the stall exit path; never for
   production use. */
#define MOK_DEBUG_FORCE_STALL 8u

/*
 * Layer knobs ("Mixture-of-Kittens (MoK)" project summary, Key-concepts table:
 * mini-batch granularity, macro-batch size, schedule capacity multiplier; the
 * communication-SM knob has no meaning without peers and is not present).
 * No knob changes any output bit.
 *   minibatch_rows      rows per mini-batch, a multiple of 16 (default 512)
 *   macrobatch_tokens   tokens per macro-batch; 0 = one macro-batch
 *   ring_bytes          size of the ring token buffer; must hold >= 2 mini-batches
 *   capacity_multiplier schedule capacity relative to the worst case, in (0, 4]
 *   precision           MOK_BF16, MOK_MXFP8 or MOK_MXFP8_WGRAD
 *   debug_flags         0 in production
 *   persistent_workgroups  workgroups of each persistent-kernel launch, in
 *                       [0, 65535]; 0 (the default) = one per compute unit.
 *                       Fewer leave units idle, more wait behind the resident
 *                       ones; the work queues give every value the same bits
 *                       (a grid-size sweep is part of the race tests).
 */
typedef struct mok_config {
    int32_t minibatch_rows;
    int32_t precision;
    int64_t macrobatch_tokens;
    int64_t ring_bytes;
    float capacity_multiplier;
    uint32_t debug_flags;
    int32_t persistent_workgroups;
} mok_config;

/*
 * Layer shape: T rows handed to the layer (tokens; for an expert-parallel
 * share, the received routed rows with k = 1), hidden size H, expert
 * intermediate size I, E local experts, k routed rows per token.
 * H and I are multiples of 64; 1 <= k <= E <= 4096; T >= 0;
 * T*k < 2^31. Activations are addressed with 32-bit byte offsets, so also
 * T*H*2 < 2^31 (x, dy, out, dx), T*k*I*4 < 2^31 (h, dh) and (H+256)*I*2 <
 * 2^31 (one expert's weight gradient). A shape outside these bounds makes
 * every call that takes it return MOK_ERROR_INVALID_VALUE.
 */
typedef struct mok_shape {
    int64_t T;
    int32_t H, I, E, k;
} mok_shape;

/*
 * Expert weights.
 * BF16 mode: w_gate, w_up [E,H,I] and w_down [E,I,H], bf16.
 * MXFP8 mode (weights pre-quantized by mok_mxfp8_quantize; "Mixture-of-Kittens
 * (MoK)" project summary, Key-concepts table), elements E4M3 bytes and scales
 * E8M0 bytes, one scale per 32 contiguous elements along the contraction axis:
 *   for mok_forward : gate/up elems [E,I,H] scales [E,I,H/32]   (W^T, along H)
 *                     down    elems [E,H,I] scales [E,H,I/32]   (W_down^T, along I)
 *   for mok_backward: gate/up elems [E,H,I] scales [E,H,I/32]   (along I)
 *                     down    elems [E,I,H] scales [E,I,H/32]   (along H)
 * In MXFP8 mode the bf16 pointers are ignored: the weight gradients use
 * activations only.
 */
typedef struct mok_weights {
    const void *w_gate, *w_up, *w_down;
    const uint8_t *gate_elems, *gate_scales;
    const uint8_t *up_elems, *up_scales;
    const uint8_t *down_elems, *down_scales;
} mok_weights;

/*
 * Byte offsets of the schedule table's fields inside the schedule buffer, and
 * its sizes, for inspection by tests and tools. Fields are int32 arrays:
 *   counts[E]            rows per expert (sum = T*k: nothing is dropped)
 *   offsets[E+1]         exclusive scan of counts
 *   mcounts[NM*E]        rows per (macro-batch, expert)
 *   moffsets[NM*(E+1)]   first processing position of each (macro-batch, expert)
 *   perm[R]              processing position q -> routed row f = t*k + j
 *   inv[R]               routed row f -> processing position q
 *   canon[R]             position in (expert, f) order -> processing position
 *   mb_start[G+1]        first processing position of each mini-batch
 *   segments[cap*4]      (mini-batch g, expert e, first position q0, rows) for
 *                        each non-empty (mini-batch, expert) intersection
 * plus uint32 status (byte 0) and int32 n_seg (byte 4).
 */
typedef struct mok_schedule_layout {
    int64_t R, NM, G, cap;
    size_t status, n_seg, counts, offsets, mcounts, moffsets, perm, inv, canon,
           mb_start, segments;
    size_t total_bytes;
} mok_schedule_layout;

/* Fill *cfg with the defaults: 512-row mini-batches, one macro-batch, a
   256 MiB ring, capacity multiplier 1, BF16, no debug flags, one persistent
   workgroup per compute unit. */
mok_status mok_config_default(mok_config *cfg);

/*
 * Host-only: size the mini-batch by the two-wave rule ("Mixture-of-Kittens(MoK)
 * 란?" explainer, section 4 ②: the overlap unit is the smallest that still
 * gives every expert-grouped GEMM at least two full waves of compute units;
 * its worked example is 2,368 tokens for a Kimi 2.5-shaped layer).
 * The gate/up GEMM of r rows has r*2I/(BM*256) output tiles counted
 * fractionally, BM being the layer's m-tile rows (256, or 128 for BF16 layers
 * of many small groups) and 256 the n-tile width; two waves over n_cu compute
 * units need r >= 2*n_cu*BM*256/(2I). minibatch_rows becomes that minimum
 * rounded up to whole m-tiles (m-tiles are cut at mini-batch boundaries),
 * capped at one macro-batch's routed rows rounded up to 16; ring_bytes is
 * raised to two slots of that size if it holds fewer and otherwise kept (it is
 * the caller's memory budget). Every other field is kept.
 *   cfg    in/out: the caller's knobs; written only on MOK_OK
 *   shape  the layer shape, validated as by mok_query_sizes
 *   n_cu   compute units to fill; <= 0 means 256 (one MI355X)
 * Returns MOK_ERROR_INVALID_VALUE for a null pointer or a shape or knob
 * mok_query_sizes would reject. Results never depend on the knobs it sets.
 */
mok_status mok_config_autosize(mok_config *cfg, const mok_shape *shape, int32_t n_cu);

/*
 * Host-only size query (the pages' get_workspace sizing, "Mixture-of-Kittens
 * (MoK)" project summary, Functional API; the workspace is made once and
 * reused, Key-concepts table). Writes the byte sizes of the workspace
 * (ring + scratch, reusable across calls), the schedule buffer (one per
 * routing) and fwd_ctx (forward saves for backward). Any output pointer may
 * be NULL. Enqueues nothing; needs no GPU.
 */
mok_status mok_query_sizes(const mok_config *cfg, const mok_shape *shape,
                           size_t *workspace_bytes, size_t *schedule_bytes,
                           size_t *fwd_ctx_bytes);

/* Host-only: the schedule buffer's field offsets for cfg and shape. */
mok_status mok_schedule_layout_query(const mok_config *cfg, const mok_shape *shape,
                                     mok_schedule_layout *layout);

/*
 * Build the schedule table on the device from top-k expert ids
 * ("Mixture-of-Kittens (MoK)" project summary, Functional API: build_schedule;
 * "Mixture-of-Kittens(MoK)란?" explainer, section 4 ①: one table drives both
 * passes; section 4 ③: drop-free, no CPU-GPU synchronisation).
 *   topk_ids  device int32 [T,k], each in [0,E) (else MOK_BAD_EXPERT_ID)
 *   schedule  device buffer of schedule_bytes >= mok_query_sizes' value
 * Processing order sorts routed rows by (macro-batch, expert, row); the table
 * is a pure function of (topk_ids, shape, config).
 */
mok_status mok_build_schedule(const mok_config *cfg, const mok_shape *shape,
                              const int32_t *topk_ids, void *schedule,
                              size_t schedule_bytes, void *stream);

/*
 * Forward pass ("Mixture-of-Kittens (MoK)" project summary, Functional API:
 * forward -> (out, fwd_ctx); "Mixture-of-Kittens(MoK)란?" explainer, section
 * 4 ③: ring token buffer consumed in mini-batches).
 *   schedule the table mok_build_schedule wrote (schedule_bytes long) for
 *            the same shape, minibatch_rows, macrobatch_tokens,
 *            capacity_multiplier and precision; checked against a layout
 *            fingerprint before use (MOK_SCHEDULE_MISMATCH)
 *   x        device bf16 [T,H]
 *   topk_w   device fp32 [T,k] gate weights
 *   w        expert weights (see mok_weights)
 *   out      device bf16 [T,H]: out_t = sum_j topk_w[t,j] * SwiGLU_e(x_t),
 *            accumulated in fp32 in order j = 0..k-1
 *   fwd_ctx  device buffer (fwd_ctx_bytes), written; read by mok_backward
 */
mok_status mok_forward(const mok_config *cfg, const mok_shape *shape,
                       const void *schedule, size_t schedule_bytes,
                       void *workspace, size_t workspace_bytes,
                       const void *x, const float *topk_w, const mok_weights *w,
                       void *out, void *fwd_ctx, size_t fwd_ctx_bytes, void *stream);

/*
 * Backward pass for upstream gradient dy of out ("Mixture-of-Kittens (MoK)"
 * project summary, Functional API: backward -> grads; "Mixture-of-Kittens(MoK)
 * 란?" explainer, section 4 ③: the ring is walked in reverse; "Cursor
 * Open-Sources Mixture-of-Kittens (MoK)" digest, English abstract: the
 * router-weight gradient is fused into the SwiGLU backward).
 *   x, topk_w, w, schedule, fwd_ctx   as given to mok_forward (the schedule
 *            is checked as there)
 *   dy       device bf16 [T,H]
 *   dx       device bf16 [T,H]
 *   dw_gate, dw_up [E,H,I] and dw_down [E,I,H], device bf16, overwritten
 *            (experts that received no rows get zeros)
 *   dtopk_w  device fp32 [T,k]: d loss / d topk_w[t,j] = <dy_t, y_{t,j}>
 */
mok_status mok_backward(const mok_config *cfg, const mok_shape *shape,
                        const void *schedule, size_t schedule_bytes,
                        void *workspace, size_t workspace_bytes,
                        const void *x, const float *topk_w, const mok_weights *w,
                        const void *fwd_ctx, size_t fwd_ctx_bytes, const void *dy,
                        void *dx, void *dw_gate, void *dw_up, void *dw_down,
                        float *dtopk_w, void *stream);

/*
 * mok_forward without a workspace argument: the forward pass's scratch (ring,
 * a-ring, combine staging, work-queue counters) lives in a static device array
 * of MOK_NOALLOC_SCRATCH_BYTES inside the library, one per GPU, held until the
 * process ends. For callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * The call itself allocates nothing (no hipMalloc, hipFree or allocating
 * library routine); its first call on a device looks up that device's copy
 * of the array. Arguments and results are mok_forward's, bit for bit.
 * A layer whose forward needs more scratch than the array holds (about
 * ring_bytes + ring_bytes * I / H + the k > 1 combine staging) returns
 * MOK_ERROR_BUFFER_TOO_SMALL, with the sizes in mok_last_error(); a smaller
 * ring_bytes knob changes no output bit. Every call on one GPU shares that
 * GPU's array and leaves its contents behind: calls that overlap on one GPU
 * (concurrent streams or threads) race and must be serialised by the caller.
 */
#define MOK_NOALLOC_SCRATCH_BYTES (64u << 20)
mok_status mok_forward_noalloc(const mok_config *cfg, const mok_shape *shape,
                               const void *schedule, size_t schedule_bytes,
                               const void *x, const float *topk_w, const mok_weights *w,
                               void *out, void *fwd_ctx, size_t fwd_ctx_bytes, void *stream);

/*
 * MXFP8 quantization ("Mixture-of-Kittens (MoK)" project summary, Key-concepts
 * table: weights are pre-quantized before the kernel; block format: OCP MX
 * v1.0 MXFP8). For each run of 32 contiguous values along K:
 *   scale byte = clamp(floor(log2 amax) - 8, -127, 127) + 127  (127 if amax = 0)
 *   element    = E4M3FN(v * 2^-(scale-127)), nearest-even, saturating to +-448
 *   src            device bf16; [batch, rows, K] if src_is_k_by_rows == 0,
 *                  [batch, K, rows] if 1 (quantizes the transpose)
 *   elems          device uint8 [batch, rows, K]
 *   scales         device uint8 [batch, rows, K/32]
 * A run that holds a NaN or an infinity becomes NaN throughout (elements 0x7F or
 * 0xFF); the same holds wherever the library quantizes rows itself.
 * K must be a multiple of 32.
 */
mok_status mok_mxfp8_quantize(const void *src, int64_t batch, int64_t rows, int64_t K,
                              int32_t src_is_k_by_rows, uint8_t *elems, uint8_t *scales,
                              void *stream);

/*
 * Router front-end: the step before schedule building, which takes the top-k
 * expert choice as input ("Mixture-of-Kittens (MoK)" project summary,
 * Functional API; "Mixture-of-Kittens(MoK)란?" explainer, section 1: each
 * token activates a few experts). The pages leave the router's formula open;
 * this is softmax over all E experts, the k largest logits, and weights
 * renormalised over the chosen k:
 *   topk_ids[t, j]  the j-th largest logit of row t (the lower expert index
 *                   first among equal logits)
 *   topk_w[t, j]    exp(l_j - m) / sum_i exp(l_i - m) over the chosen i,
 *                   m = the row's largest logit (fp32)
 *   logits          device fp32 [T, E], row-major, finite
 *   topk_ids        device int32 [T, k];  topk_w  device fp32 [T, k]
 * 1 <= k <= min(E, 64), E <= 1024; T == 0 is a no-op. Bitwise deterministic.
 */
mok_status mok_route(const float *logits, int64_t T, int32_t E, int32_t k, int32_t *topk_ids,
                     float *topk_w, void *stream);

/*
 * Logit gradient of mok_route (the choice is piecewise constant):
 *   dlogits[t, e] = w_e * (dtopk_w_e - sum_j w_j * dtopk_w_j)  for chosen e,
 *                   0 for every other expert
 * topk_ids and topk_w as mok_route returned them, dtopk_w device fp32 [T, k]
 * (for instance mok_backward's dtopk_w); dlogits device fp32 [T, E], every
 * entry written. Same limits as mok_route.
 */
mok_status mok_route_backward(const int32_t *topk_ids, const float *topk_w, const float *dtopk_w,
                              int64_t T, int32_t E, int32_t k, float *dlogits, void *stream);

/*
 * Operators around the routed experts in a transformer block. The pages
 * describe the routed layer alone; these take the plainest readings: dropout of
 * a branch, the residual's addition with a root-mean-square norm, and the
 * dense gated feed-forward block (a shared expert).
 *
 * Conventions beside the ones at the top of this file:
 *  - The residual stream (residual, sum, their gradients) is bf16 or fp32:
 *    stream_dtype. Branches, normalised rows and weights are bf16.
 *  - Dropout masks come from a counter-based generator and are never stored.
 *    rng points to two device uint64, {seed, offset}; element i of a call is
 *    word i % 4 of the Philox4x32-10 block with key seed and 64-bit counter
 *    offset + i / 4 (the counter's upper 64 bits are 0), and is kept when the
 *    word is at least floor(p * 2^32). A kept value is multiplied by the fp32
 *    value of 1 / (1 - p); a dropped one contributes nothing, whatever it
 *    holds. A call of n elements uses (n + 3) / 4 counters; the caller advances
 *    offset by at least that much before the next draw, and keeps the old pair
 *    for the backward. Both are read when the call's kernels run, so replays of
 *    a captured graph follow the pair's current value. With p == 0 rng is
 *    ignored and may be NULL.
 *  - An output may be the same buffer as an input of the same type and shape
 *    only where a call says so; otherwise buffers must not overlap (refused).
 *  - Calls can be captured into a HIP graph once they have run eagerly (kernels
 *    are loaded and their attributes set on first use). They enqueue kernels
 *    only. Graphs that share a workspace must not run at the same time.
 */
#define MOK_STREAM_BF16 0
#define MOK_STREAM_F32 1

/*
 * out = residual + dropout(x).
 *   x         device bf16 [n], any n in [0, 2^37 - 8192]
 *   residual  device stream_dtype [n], or NULL (then out = dropout(x))
 *   p         drop probability in [0, 1)
 *   out       device stream_dtype [n]; may be residual's buffer, or x's when
 *             the stream is bf16
 */
mok_status mok_dropout(const void *x, const void *residual, int64_t n, float p, const uint64_t *rng,
                       int32_t stream_dtype, void *out, void *stream);

/*
 * Gradient of mok_dropout with respect to x: dx = dy / (1 - p) where the
 * forward kept the element, 0 elsewhere. (The residual's gradient is dy.)
 *   dy  device stream_dtype [n];  dx  device bf16 [n], may be dy's buffer when
 *   the stream is bf16. p and rng as the forward had them.
 */
mok_status mok_dropout_backward(const void *dy, int64_t n, float p, const uint64_t *rng, int32_t stream_dtype,
                                void *dx, void *stream);

/*
 * Residual addition and root-mean-square norm. T >= 0 rows (below 2^31) of H
 * elements, H a multiple of 8 (of 32 for MXFP8 rows) up to 16384; eps >= 0.
 */
typedef struct mok_norm_shape {
    int64_t T;
    int32_t H;
    int32_t stream_dtype;
    float eps;
    float p;   /* drop probability of the branch, in [0, 1) */
} mok_norm_shape;

/*
 * s = residual + dropout(x) in fp32 (element i of the dropout is t * H + h),
 * rstd = 1 / sqrt(mean over h of s^2 + eps), y = s * rstd * weight. Statistics
 * and y come from the fp32 s; sum is its copy in the stream's type.
 *   x         device bf16 [T,H], the branch
 *   residual  device stream_dtype [T,H], or NULL (then s = dropout(x))
 *   weight    device bf16 [H]
 *   sum       device stream_dtype [T,H], or NULL; may be residual's buffer, or
 *             x's when the stream is bf16
 *   y         device bf16 [T,H], or NULL
 *   y_elems, y_scales   y as MXFP8 (mok_mxfp8_quantize's block format along H,
 *             rounded from the fp32 y): device uint8 [T,H] and [T,H/32], or
 *             both NULL. At least one of y and y_elems is given.
 *   rstd      device fp32 [T]
 * s^2 must not overflow fp32 (|s| up to about 10^17).
 */
mok_status mok_add_rmsnorm(const mok_norm_shape *shape, const void *x, const void *residual, const void *weight,
                           const uint64_t *rng, void *sum, void *y, uint8_t *y_elems, uint8_t *y_scales,
                           float *rstd, void *stream);

/* Host-only: workspace bytes of mok_add_rmsnorm_backward for shape (a
   workspace for T rows also serves fewer). */
mok_status mok_add_rmsnorm_backward_size(const mok_norm_shape *shape, size_t *workspace_bytes);

/*
 * Backward of mok_add_rmsnorm from its sum and rstd:
 *   ds = dsum + rstd * (dy * weight - sum * rstd^2 * mean over h of dy * weight * sum)
 *   dy         device bf16 [T,H], gradient of y
 *   sum, rstd  as the forward wrote them
 *   dsum       device stream_dtype [T,H], the gradient that reaches s along
 *              the residual stream, or NULL (zero)
 *   dresidual  device stream_dtype [T,H]: ds; or NULL. May be dsum's buffer.
 *   dx         device bf16 [T,H]: the branch's gradient, ds through the
 *              dropout; or NULL. May be dy's buffer.
 *   dweight    device fp32 [H]: sum over t of dy * sum * rstd (zeros for T == 0)
 *   workspace  at least mok_add_rmsnorm_backward_size bytes
 * p, eps and rng as the forward had them. Bitwise deterministic.
 */
mok_status mok_add_rmsnorm_backward(const mok_norm_shape *shape, void *workspace, size_t workspace_bytes,
                                    const void *dy, const void *sum, const void *weight, const float *rstd,
                                    const void *dsum, const uint64_t *rng, void *dresidual, void *dx,
                                    float *dweight, void *stream);

/*
 * Dense gated feed-forward block (SwiGLU), the shared expert beside the routed
 * ones: T rows of H through an intermediate size I.
 * H and I are multiples of 64 (128 in MXFP8), at most 2^20; T >= 0; the
 * layer's bounds on byte offsets hold: T*H*2 < 2^31, T*I*4 < 2^31,
 * (H+256)*I*2 < 2^31 and (I+256)*H*2 < 2^31.
 * precision is MOK_BF16 or MOK_MXFP8 (weight gradients in BF16).
 * Weights are a mok_weights for one expert (E = 1), in the orientations that
 * struct describes.
 * Between the products, a = silu(x W_gate) * (x W_up) and dh are operands of
 * fewer bits than their fp32 sums: in MOK_BF16 both are rounded to bf16 once (the
 * forward of one row, and of two at the smaller sizes, keeps a in fp32); in
 * MOK_MXFP8 both, and dy, are quantized from fp32 (dy from bf16) for the products
 * with a weight and rounded to bf16 for the weight gradients.
 */
typedef struct mok_ffn_shape {
    int64_t T;
    int32_t H, I;
    int32_t precision;
} mok_ffn_shape;

/* Host-only: workspace bytes that mok_ffn_forward and mok_ffn_backward need (a
   workspace for T rows also serves fewer). */
mok_status mok_ffn_query_size(const mok_ffn_shape *shape, size_t *workspace_bytes);

/*
 * out = addend + (silu(x W_gate) * (x W_up)) W_down.
 *   x         BF16: device bf16 [T,H]. MXFP8: NULL
 *   x_elems, x_scales   MXFP8: device uint8 [T,H], [T,H/32], the rows quantized
 *             along H (mok_add_rmsnorm or mok_mxfp8_quantize). BF16: NULL
 *   addend    device bf16 [T,H] added to the block's output in fp32 (for
 *             instance mok_forward's out), or NULL; its gradient is out's
 *   out       device bf16 [T,H]; may be addend's buffer
 *   h         device bf16 [T,2I]: x [W_gate | W_up], which the backward needs,
 *             or NULL
 * Bitwise deterministic.
 */
mok_status mok_ffn_forward(const mok_ffn_shape *shape, void *workspace, size_t workspace_bytes, const void *x,
                           const uint8_t *x_elems, const uint8_t *x_scales, const mok_weights *w,
                           const void *addend, void *out, void *h, void *stream);

/*
 * Backward of mok_ffn_forward for the gradient dy of out.
 *   x         device bf16 [T,H] in either precision (the weight gradients'
 *             operand)
 *   w         the weights; MXFP8: in the backward's orientation
 *   h         device bf16 [T,2I], as the forward wrote it
 *   dy        device bf16 [T,H]
 *   addend    device bf16 [T,H] added to dx in fp32 (for instance mok_backward's
 *             dx), or NULL
 *   dx        device bf16 [T,H]; may be addend's buffer
 *   dw_gate, dw_up [H,I] and dw_down [I,H], device bf16, overwritten (zeros
 *             for T == 0)
 * Bitwise deterministic.
 */
mok_status mok_ffn_backward(const mok_ffn_shape *shape, void *workspace, size_t workspace_bytes, const void *x,
                            const mok_weights *w, const void *h, const void *dy, const void *addend, void *dx,
                            void *dw_gate, void *dw_up, void *dw_down, void *stream);

/*
 * The routed experts taken apart, for experts of another form than the layer's,
 * or for weights that come in 8-bit blocks of 128: token rows sorted by expert
 * and back, quantization into such blocks, and the products on them. The pages
 * describe the fused layer alone; these take the plainest readings.
 * The conventions above hold: on buffers, on overlaps, on graphs.
 *
 * A sort gives every routed slot f = t*k + j that names an expert here a row.
 * Rows are ordered by (expert, f); each expert's run of rows is rounded up to a
 * multiple of `align` by padding rows at its end. A slot whose id lies outside
 * [0, E) (an expert on another GPU, say -1) has no row. A token may name an
 * expert twice; each slot has its own row.
 * `rows` below is the number of rows that the row buffers hold; a sort fills at
 * most (T*k + min(E, T*k) * (align - 1)) / align * align of them
 * (mok_sort_tokens_size). Rows behind the last expert's run are left as they
 * were by every call that writes rows, and read by none.
 */
typedef struct mok_sort_shape {
    int64_t T;
    int32_t k, E, align;
} mok_sort_shape;

/* Host-only: the most rows that a sort of this shape fills, and the workspace
   bytes of mok_sort_tokens (0 below 65,536 slots of at most 512 experts: the
   workspace may then be NULL). Either pointer may be NULL. T >= 0, k >= 1, 1 <= E <=
   4096, 1 <= align <= 1024; T*k and the rows stay below 2^31. */
mok_status mok_sort_tokens_size(const mok_sort_shape *shape, int64_t *rows, size_t *workspace_bytes);

/*
 *   topk_ids   device int32 [T,k]
 *   offsets    device int32 [E+1]: first row of each expert, then the end
 *   slots      device int32 [T,k]: the slot's row, or -1
 *   row_slots  device int32 [rows of mok_sort_tokens_size]: the row's slot f, or
 *              -1 (padding, and rows behind the last run)
 * Every entry of the three is written. The result is a pure function of the ids.
 */
mok_status mok_sort_tokens(const mok_sort_shape *shape, void *workspace, size_t workspace_bytes,
                           const int32_t *topk_ids, int32_t *offsets, int32_t *slots, int32_t *row_slots,
                           void *stream);

/*
 * Rows of H elements of a sort: T tokens, k slots each, row buffers of `rows`
 * rows (mok_sort_tokens_size's, or any other number: a slot past it counts as
 * one without a row). dtype is MOK_STREAM_BF16 or MOK_STREAM_F32. H is a multiple
 * of 8, at most 2^20; T, rows and T*k are below 2^31; 1 <= E <= 4096.
 */
typedef struct mok_rows_shape {
    int64_t T, rows;
    int32_t k, E, H, dtype;
} mok_rows_shape;

/*
 * rows[slots[t,j]] = x[t] for every slot that has a row; padding rows get zeros.
 *   x          device dtype [T,H]
 *   offsets, slots, row_slots   as mok_sort_tokens wrote them
 *   rows       device dtype [rows,H], or NULL
 *   elems, scales   the rows quantized (mok_fp8_quantize's rows; H is then a
 *              multiple of 16): device uint8 [rows,H] and fp32 [(H+127)/128, rows],
 *              or both NULL. At least one of rows and elems is given.
 */
mok_status mok_permute(const mok_rows_shape *shape, const void *x, const int32_t *offsets, const int32_t *slots,
                       const int32_t *row_slots, void *rows, uint8_t *elems, float *scales, void *stream);

/* Gradient of mok_permute: dx[t] = sum over j of drows[slots[t,j]] in fp32, in
   ascending order of j, rounded once.  drows device dtype [rows,H], dx device
   dtype [T,H]. */
mok_status mok_permute_backward(const mok_rows_shape *shape, const void *drows, const int32_t *slots, void *dx,
                                void *stream);

/*
 * out[t] = addend[t] + sum over j of w[t,j] * y[slots[t,j]] in fp32, in ascending
 * order of j, rounded once; slots without a row contribute nothing, whatever
 * their w.
 *   y       device dtype [rows,H]
 *   w       device fp32 [T,k], or NULL (ones)
 *   addend  device dtype [T,H], or NULL; its gradient is out's
 *   out     device dtype [T,H]; may be addend's buffer
 */
mok_status mok_unpermute(const mok_rows_shape *shape, const void *y, const int32_t *slots, const float *w,
                         const void *addend, void *out, void *stream);

/*
 * Gradient of mok_unpermute with weights (without them it is mok_permute of dout):
 *   dy[slots[t,j]] = w[t,j] * dout[t], zeros in padding rows
 *   dw[t,j]        = sum over h of dout[t,h] * y[slots[t,j],h] (fp32), 0 for a slot without a row
 *   dout    device dtype [T,H];  y as the forward read it
 *   dy      device dtype [rows,H]; may be y's buffer
 *   dw      device fp32 [T,k]
 * Bitwise deterministic.
 */
mok_status mok_unpermute_backward(const mok_rows_shape *shape, const void *dout, const void *y,
                                  const int32_t *offsets, const int32_t *slots, const int32_t *row_slots,
                                  const float *w, void *dy, float *dw, void *stream);

/*
 * Quantization into blocks of 128 with one fp32 scale each. A block is 128
 * contiguous values along K (the last one of a row may be shorter), or with
 * MOK_FP8_TILE 128 rows x 128 values (shorter at the ends). With
 *   m = max(largest magnitude of the block, 2^-52)
 * and both divisions and the product in fp32:
 *   scale   = m / 448
 *   element = E4M3FN(v * (448 / m)), nearest-even, saturating to +-448
 * A block that holds a NaN or an infinity becomes NaN throughout (elements 0x7F)
 * with scale 1.
 *   src     device dtype (MOK_STREAM_BF16 or MOK_STREAM_F32) [batch, rows, K], or
 *           with MOK_FP8_TURNED [batch, K, rows] (quantizes the transpose).
 *           With MOK_FP8_GLU the rows in memory are twice as long ([batch, rows, 2K]
 *           or [batch, K, 2*rows]): g then u, and v = silu(g) * u in fp32 is
 *           quantized. GLU takes bf16 and no TILE.
 *   elems   device uint8 [batch, rows, K]
 *   scales  device fp32 [batch, (K+127)/128, rows]: block by block, so that a
 *           product's K-step reads its rows' scales in one run; with MOK_FP8_TILE
 *           [batch, (rows+127)/128, (K+127)/128]
 * K is a multiple of 16; with MOK_FP8_TURNED rows is a multiple of 8. K and rows
 * stay below 2^31, batch below 65536, a matrix below 2^40 values.
 */
#define MOK_FP8_TURNED 1u
#define MOK_FP8_TILE 2u
#define MOK_FP8_GLU 4u
mok_status mok_fp8_quantize(const void *src, int32_t dtype, int64_t batch, int64_t rows, int64_t K, uint32_t flags,
                            uint8_t *elems, float *scales, void *stream);

/*
 * Gradient of the gated activation a = silu(g) * u for h = [g | u]:
 *   dh = [da * u * s * (1 + g * (1 - s)) | da * g * s],  s = 1 / (1 + e^-g)
 *   da device bf16 [T,I], h and dh device bf16 [T,2I] (dh may be h's buffer). I is
 *   a multiple of 8; T*I stays below 2^40.
 */
mok_status mok_glu_backward(const void *da, const void *h, int64_t T, int32_t I, void *dh, void *stream);

/*
 * Products on operands in blocks of 128. A K-step's product of 128 values is
 * multiplied by the two scales as it is added to the fp32 sum, which asks that
 * the product of two scales be an fp32 number (below 2^128).
 * A bf16 result is computed on the fp8 matrix cores, which cut each product of a
 * group of 16 at 2^-13 of the binade of the group's largest before they add it
 * (1.5e-5 of the result's norm for normal values, under its own rounding). An
 * fp32 result is computed on the bf16 matrix cores, where E4M3 values are exact
 * and all sums keep fp32, at half the rate.
 * M: rows of `a` (mok_fp8_matmul), or the contraction's length (mok_fp8_wgrad).
 * N and K are multiples of 16, at most 2^20; 0 <= M < 2^31, for mok_fp8_wgrad a
 * multiple of 16 below 2^23. E = 0: one product; 1 <= E <= 4096: one for each
 * expert's run of rows. out_dtype is MOK_STREAM_BF16 or MOK_STREAM_F32.
 * offsets (E > 0): device int32 [E+1], ascending, in [0, M] (values outside count
 * as the nearest one inside); NULL for E = 0.
 */
typedef struct mok_fp8_shape {
    int64_t M;
    int32_t N, K, E, out_dtype;
} mok_fp8_shape;

/* Host-only: workspace bytes of mok_fp8_matmul and mok_fp8_wgrad (0 where the
   contraction is not cut into runs: the workspace may then be NULL). */
mok_status mok_fp8_matmul_size(const mok_fp8_shape *shape, size_t *workspace_bytes);
mok_status mok_fp8_wgrad_size(const mok_fp8_shape *shape, size_t *workspace_bytes);

/*
 * out[m][n] = sum over k of a[m][k] * b_e[n][k] for the rows m of expert e's run;
 * rows of no run are left as they were.
 *   a_elems, a_scales   rows: device uint8 [M,K] and fp32 [(K+127)/128, M]
 *   b_elems, b_scales   tiles: device uint8 [E or 1, N, K] and fp32
 *                       [E or 1, (N+127)/128, (K+127)/128]
 *   out                 device out_dtype [M,N]
 * Bitwise deterministic; the gradient with respect to a is the same call with the
 * transposed weights quantized (MOK_FP8_TURNED).
 */
mok_status mok_fp8_matmul(const mok_fp8_shape *shape, void *workspace, size_t workspace_bytes,
                          const uint8_t *a_elems, const float *a_scales, const uint8_t *b_elems,
                          const float *b_scales, const int32_t *offsets, void *out, void *stream);

/*
 * Weight gradient: out[e][n][k] = addend[e][n][k] + sum over the rows r of e's run
 * of dy[n][r] * x[k][r], for operands quantized along the rows (mok_fp8_quantize
 * with MOK_FP8_TURNED, 128 rows a block). The runs start at multiples of 128 (a
 * sort with align = 128) and end at any row: the codes behind an end count for
 * nothing, whatever they are. (The scale of the block it lies in counts them, if
 * mok_fp8_quantize made it.) A run that starts elsewhere gives NaN throughout: its
 * first block's scales hold for another expert's rows too. An expert without rows
 * gets its addend, or zeros, wherever its offset lies.
 *   dy_elems, dy_scales   device uint8 [N,M] and fp32 [(M+127)/128, N]
 *   x_elems, x_scales     device uint8 [K,M] and fp32 [(M+127)/128, K]
 *   addend                device out_dtype [E or 1, N, K], or NULL
 *   out                   the same; may be addend's buffer
 * Bitwise deterministic.
 */
mok_status mok_fp8_wgrad(const mok_fp8_shape *shape, void *workspace, size_t workspace_bytes,
                         const uint8_t *dy_elems, const float *dy_scales, const uint8_t *x_elems,
                         const float *x_scales, const int32_t *offsets, const void *addend, void *out, void *stream);

/*
 * Measurement aid, not part of the layer: per-kernel durations for tools such
 * as benchmarks. While enabled, every kernel launch of the library is
 * bracketed by two HIP events recorded on the launch's own stream (the
 * schedule builder's launches count as one "schedule" entry).
 * mok_kernel_timing_enable(1) discards earlier records and starts recording;
 * mok_kernel_timing_enable(0) discards records and stops. mok_kernel_timing_read
 * waits for the recorded events, writes up to `capacity` per-kernel sums in
 * first-launch order, sets *count to the number of distinct kernels, and
 * discards the records. Off by default; not meant for production loops.
 */
typedef struct mok_kernel_stat {
    char name[32];
    int64_t launches;
    double total_ms;
    double max_ms;
} mok_kernel_stat;

mok_status mok_kernel_timing_enable(int32_t enable);
mok_status mok_kernel_timing_read(mok_kernel_stat *stats, int32_t capacity, int32_t *count);

/*
 * Measurement aid, not part of the layer: a per-item trace of the GEMM
 * kernels, to see how the tiles of a pass overlap and where a compute unit's
 * time goes ("Mixture-of-Kittens(MoK)란?" explainer, section 4 ②: the overlap
 * granularity is checked against its estimate). One record per tile of the
 * persistent pair kernels (forward gate/up + down, backward dA + dX) and of
 * the weight-gradient kernels. Times are the GPU's constant 100 MHz clock
 * (s_memrealtime). While tracing is off a kernel pays one scalar branch per
 * tile.
 */
typedef struct mok_item_record {
    uint64_t t_claim;    /* the workgroup began to claim the item (other kernels: the tile started) */
    uint64_t t_start;    /* the item was claimed and its inputs were ready */
    uint64_t t_kloop;    /* its K loop ended (the epilogue begins) */
    uint64_t t_end;      /* its outputs were stored (and, in a pair kernel, published) */
    uint32_t launch;     /* launches since tracing was enabled, in issue order */
    uint8_t kernel;      /* MOK_TRACE_* */
    uint8_t item_class;  /* pair kernels: 1 producer tile, 2 consumer tile; otherwise 0 */
    uint16_t xcd;        /* workgroup index mod 8, its XCD */
    uint32_t item;       /* pair kernels: index in its class's queue; otherwise the workgroup's tile */
    uint32_t workgroup;  /* workgroup index */
} mok_item_record;
#define MOK_TRACE_FWD_GEMMS 0
#define MOK_TRACE_BWD_GEMMS 1
#define MOK_TRACE_WGRAD_GATE_UP 2
#define MOK_TRACE_WGRAD_DOWN 3
#define MOK_TRACE_OTHER 4
#define MOK_ITEM_TRACE_CAPACITY 65536
/* enable(1): discard earlier records and start recording into a device
   buffer of MOK_ITEM_TRACE_CAPACITY records inside the library (later ones are
   dropped); enable(0): stop. read: wait for the device, copy up to `capacity`
   records in completion order, set *count to the number recorded (it may
   exceed MOK_ITEM_TRACE_CAPACITY when records were dropped). Single device,
   not for production loops. */
mok_status mok_item_trace_enable(int32_t enable);
mok_status mok_item_trace_read(mok_item_record *records, int32_t capacity, int32_t *count);

/* Text of the calling thread's last HIP error reported as
   MOK_ERROR_LAUNCH_FAILED ("" if none); valid until the thread's next call. */
const char *mok_last_error(void);

/* Static string naming a status code. */
const char *mok_status_string(mok_status status);

#ifdef __cplusplus
}
#endif

#endif /* MOK_H */
