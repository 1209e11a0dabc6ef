/*
 * moe.h -- C ABI of the GB300 (sm_103a) dropless mixture-of-experts expert
 * layer: training forward and backward on one GPU.
 *
 * The layer (dropless MoE; "NVIDIA lleva el MoE de DeepSeek-V3 de 103 a 1.068
 * TFLOPS", sections on dropless vs capacity MoE, grouped GEMM and expert-
 * parallel dispatch/combine; the Mega MoE kernel description in "Prime
 * Intellect dopisal backward pass do kernela Mega MoE"):
 *   route:    p = softmax(logits_t) over E experts; S_t = the k largest logits
 *             (ties: lower expert index first); w_tj = p_{S_tj} / sum_S p.
 *   dispatch: counts[e] = tokens that chose e; offsets = exclusive prefix;
 *             row(t,j) = offsets[e] + #{t' < t that chose e}  (stable, no
 *             capacity, no dropped token, no padding).
 *   experts:  for every permuted row r of expert e, with x_r = x[token(r)]:
 *             G = x_r W_gate[e], U = x_r W_up[e], A = silu(G) * U,
 *             Y = A W_down[e]                      (SwiGLU MLP, no biases)
 *   combine:  out_t = sum_j w_tj * Y[row(t,j)]      (token order restored)
 *   backward: the same chain transposed -- dyw = w * dy (permuted), dA =
 *             dyw W_down^T, dSwiGLU, dX = dG W_gate^T + dU W_up^T, un-permute
 *             sum into dx, dW_* = grouped X^T-style products over each
 *             expert's rows, and d_logits[t, S_tj] = w_tj (g_tj - sum_i w_ti
 *             g_ti) with g_tj = <dy_t, Y[row(t,j)]>, zero for other experts.
 *
 * Conventions (all calls):
 *   - Memory: the caller owns and allocates every buffer; the library never
 *     allocates, frees or synchronises (only moe_get_device_status waits).
 *     Pointers named "device" are CUDA device pointers; `stream` is a
 *     cudaStream_t passed as void*; every kernel is enqueued on it, so the
 *     calls can be captured into a CUDA graph.
 *   - Counts and offsets stay on the device: no call copies routing results
 *     to the host.
 *   - Layouts are row-major, dense, as given per argument.  bf16 tensors are
 *     IEEE bfloat16 bit patterns.
 *   - Every device pointer must be 16-byte aligned.
 *   - Shapes: T >= 0, H % 64 == 0 and I % 64 == 0 (both >= 64), 1 <= E <= 256,
 *     1 <= k <= min(E, 16), T * k < 2^31; with MOE_PREC_FP8_BWD or
 *     MOE_PREC_MXFP8 also H % 128 == 0 and I % 128 == 0.
 *   - Errors found on the host (null pointer, bad shape, misalignment, a
 *     too-small workspace) return a negative moe_status with nothing launched.
 *     Anomalies found on the device (non-finite logits, a pipeline wait that
 *     ran out of time) set flags in a status word at the start of the call's
 *     scratch buffer; kernels never trap.  Read it with moe_get_device_status.
 *   - The library holds no per-call state; calls on different streams with
 *     disjoint buffers may run concurrently.  Two exceptions, both opt-in:
 *     the per-kernel timing hook (moe_timing_attach, process-wide while
 *     attached) and moe_route_static_scratch's one shared scratch array.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1, /* null pointer, bad shape or precision */
  MOE_ERR_ALIGNMENT = -2,   /* a pointer is not 16-byte aligned */
  MOE_ERR_WORKSPACE = -3,   /* a scratch/saved buffer is smaller than moe_query_workspace says */
  MOE_ERR_UNSUPPORTED = -4, /* no sm_103a device, or a precision this build does not provide */
  MOE_ERR_CUDA = -5,        /* a CUDA runtime/driver call failed */
  MOE_ERR_DEVICE = -6       /* moe_get_device_status: the device reported an anomaly */
} moe_status;

typedef enum {
  MOE_PREC_BF16 = 0,    /* bf16 operands, fp32 accumulation, everywhere */
  MOE_PREC_FP8_BWD = 1, /* bf16 forward; backward grouped GEMMs in MXFP8 (E4M3 values,
                           one UE8M0 scale per 32 elements along each GEMM's K) */
  MOE_PREC_MXFP8 = 2    /* the forward grouped GEMMs in MXFP8 too ("mxfp8" in the Prime
                           Mega MoE write-ups' precision switch): x and W_gate/W_up
                           along H, A (as bf16) and W_down along I; the activations the
                           forward saves stay bf16; the backward is fp8_bwd's */
} moe_precision;

/* Device status flags (moe_get_device_status *host_code). */
#define MOE_DEV_NONFINITE_LOGIT 0x1 /* a logit was NaN or +-Inf; routing outputs unspecified */
#define MOE_DEV_WAIT_TIMEOUT 0x2    /* a pipeline wait exceeded its bound; outputs unspecified */
#define MOE_DEV_NONFINITE_UPDATE 0x4 /* moe_ortho_update: a matrix's sum of squares, or its result, is not finite */
#define MOE_DEV_BAD_INDEX 0x8       /* moe_balance_forward: an expert index outside [0, E); that slot is not counted */

typedef struct {
  int32_t T;         /* tokens */
  int32_t H;         /* hidden size */
  int32_t I;         /* expert intermediate size */
  int32_t E;         /* experts */
  int32_t k;         /* experts per token */
  int32_t precision; /* moe_precision */
} moe_config;

/* Routing results, written by moe_route, read by moe_forward/moe_backward.
 * All device pointers, caller-owned, M = T*k. */
typedef struct {
  int32_t *topk_idx;    /* [T,k]  chosen experts, ordered by (logit desc, index asc) */
  float *topk_w;        /* [T,k]  renormalised router weights */
  int32_t *counts;      /* [E]    rows per expert */
  int32_t *offsets;     /* [E+1]  exclusive prefix of counts; offsets[E] = M */
  int32_t *row_of_slot; /* [T*k]  permuted row of slot t*k+j */
  int32_t *slot_of_row; /* [M]    inverse: slot t*k+j held by permuted row r */
  float *w_row;         /* [M]    router weight of permuted row r */
} moe_routing;

/* Byte sizes of the caller-provided buffers for a configuration.  The fused
 * kernel of the pages works through preallocated GPU scratch space instead of
 * allocating intermediates per call (the MarkTechPost article in Thai
 * translation, "how the fused kernel works"); here the caller allocates that
 * space once, sized by this call, and passes it to every call:
 *   route_scratch: moe_route's scratch;
 *   saved:        activations moe_forward keeps for moe_backward (layout below);
 *   fwd_scratch:  moe_forward's scratch;  bwd_scratch: moe_backward's scratch.
 * Returns MOE_ERR_INVALID_ARG for an unsupported shape.  Host only. */
moe_status moe_query_workspace(const moe_config *cfg, size_t *route_scratch, size_t *saved,
                               size_t *fwd_scratch, size_t *bwd_scratch);

/* Offsets (bytes) of the saved activations inside `saved`, for inspection:
 * x_perm [M,H], G [M,I], U [M,I], A [M,I], Y [M,H] (unweighted), A_w [M,I]
 * (A times the row's router weight: the weight-gradient operand), all bf16.
 * A_w is written in MOE_PREC_BF16 only: the MXFP8 backwards read w * A
 * quantised along tokens instead (moe_fp8_layout's aw_t, also in `saved`).
 * x_perm is not written in MOE_PREC_MXFP8, whose GEMMs read x's codes and whose
 * backward reads x itself. */
typedef struct {
  size_t x_perm, G, U, A, Y, A_w;
} moe_saved_layout;
moe_status moe_saved_offsets(const moe_config *cfg, moe_saved_layout *layout);

/* MOE_PREC_FP8_BWD and MOE_PREC_MXFP8: byte offsets of the backward GEMMs' MXFP8
 * operands, for inspection after the call: inside moe_backward's scratch, except
 * the ones the forward writes (inside `saved`, listed below).  m_pad is the padded
 * token capacity (a multiple of 128): expert e's rows start at padded row
 * pad_offsets[e] = sum over e' < e of ceil(count/128)*128 (int32 [E+1]); rows
 * past an expert's count are zero codes with zero scale codes; padded rows at
 * and past pad_offsets[E] are left unwritten.
 *   *_q     E4M3 codes, K-major: dy_q [m_pad,H] (padded rows), wd_q [E*I,H],
 *           dg_q/du_q [m_pad,I], wg_q/wu_q [E*H,I];
 *   *_t     token-axis operands transposed, tokens contiguous: aw_t (w*A) and
 *           dg_t/du_t [I,m_pad], dy_t and x_t [H,m_pad];
 *   written by the forward (moe_forward and moe_forward_recompute), so their
 *   offsets are inside `saved`, not the scratch: aw_t (the gate/up epilogue), x_t
 *   (in MOE_PREC_FP8_BWD by the forward's permute, which gathers x into x_perm
 *   and quantises it along tokens in one pass) and the weights' wd_q, wg_q, wu_q
 *   with their scales (in MOE_PREC_FP8_BWD the two bf16 GEMMs quantise each
 *   weight tile as it passes through them, so only the experts that received
 *   rows are written -- no backward GEMM reads the others; in MOE_PREC_MXFP8 the
 *   forward's weight passes write every expert);
 *   *_sf    their UE8M0 scale codes (2^(code-127)), one per 32 elements along
 *           K, in 512-byte atoms of 128 rows x 128 K, the order the tensor core
 *           reads them: row w of atom row-block rb, K-block b, sits at byte
 *           (rb*(K/128) + b/4)*512 + (w%32)*16 + (w/32)*4 + b%4.  For dy_q,
 *           dg_q, du_q, aw_t and x_t (the GEMMs' M side) row r is row r%128 of
 *           block r/128.  For wd_q, wg_q, wu_q, dy_t, dg_t and du_t (the N side,
 *           read in 192-row tiles) rows are cut into segments of S rows (S = I
 *           for wd_q, H for wg_q/wu_q, all rows for the transposed ones), each
 *           segment into groups of 192 rows, each group into two blocks: row r
 *           with s = r/S, g = (r%S)/192, j = (r%S)%192 is row j%128 of block
 *           (s*ceil(S/192) + g)*2 + j/128.  Scale bytes of groups' rows past a
 *           segment's end are left unwritten.
 * Returns MOE_ERR_INVALID_ARG for other precisions or unsupported shapes. */
typedef struct {
  size_t m_pad, pad_offsets;
  size_t dy_q, dy_sf, wd_q, wd_sf, dg_q, dg_sf, du_q, du_sf, wg_q, wg_sf, wu_q, wu_sf;
  size_t aw_t, aw_t_sf, dy_t, dy_t_sf, x_t, x_t_sf, dg_t, dg_t_sf, du_t, du_t_sf;
} moe_fp8_layout;
moe_status moe_fp8_scratch_offsets(const moe_config *cfg, moe_fp8_layout *layout);

/* MOE_PREC_MXFP8 only: byte offsets, inside moe_forward's scratch, of the MXFP8
 * operands of the two forward GEMMs, for inspection after the call (padded row
 * space, pad_offsets, codes and 512-byte scale atoms as in moe_fp8_layout):
 *   x_q   [m_pad,H]  the permuted x along H (M side: row r in block r/128);
 *   a_q   [m_pad,I]  A along I, from its bf16 value (M side);
 *   wgu_q [E*2I,H]   W_gate and W_up along H, transposed and interleaved by 32:
 *                    row e*2I + (i/32)*64 + i%32 holds W_gate[e][:, i] and the
 *                    row 32 after it W_up[e][:, i] (N side, segments of 2I rows);
 *   wdt_q [E*H,I]    W_down along I, transposed: row e*H + h holds W_down[e][:, h]
 *                    (N side, segments of H rows).
 * The same passes over the weights also write the backward GEMMs' weight
 * operands, which live in `saved` (moe_backward does not quantise the weights
 * again; moe_fp8_scratch_offsets reports the same offsets):
 *   bwd_wd_q [E*I,H], bwd_wg_q and bwd_wu_q [E*H,I] and their scales, laid
 *   out as moe_fp8_layout's wd_q, wg_q, wu_q (offsets inside `saved`).
 * Returns MOE_ERR_INVALID_ARG for other precisions or unsupported shapes. */
typedef struct {
  size_t m_pad, pad_offsets, x_q, x_sf, a_q, a_sf, wgu_q, wgu_sf, wdt_q, wdt_sf;
  size_t bwd_wd_q, bwd_wd_sf, bwd_wg_q, bwd_wg_sf, bwd_wu_q, bwd_wu_sf;
} moe_mxfp8_fwd_layout;
moe_status moe_mxfp8_forward_offsets(const moe_config *cfg, moe_mxfp8_fwd_layout *layout);

/* Router and dispatch indices.  logits: device fp32 [T,E].  Writes every field
 * of *routing.  Dropless routing gives per-expert group sizes that change
 * every step; they stay on the device and the grouped GEMMs read them there,
 * so no host copy breaks CUDA-graph capture (NVIDIA article "DeepSeek-V3 MoE
 * from 103 to 1,068 TFLOPS", "optimisations dropless needs" and "grouped
 * GEMM").  Two kernels: the first reads the logits once and writes the top k,
 * the per-block expert histograms and every slot's rank, and its last blocks
 * to finish scan the histograms (counts, offsets, per-block bases); the second
 * writes every slot's row.  Work and scratch grow linearly with T.
 * Non-finite logits set MOE_DEV_NONFINITE_LOGIT; the indices written are still
 * in range. */
moe_status moe_route(const moe_config *cfg, const float *logits, const moe_routing *routing,
                     void *scratch, size_t scratch_bytes, void *stream);

/* Forward.  x: device bf16 [T,H]; W_gate, W_up: device bf16 [E,H,I];
 * W_down: device bf16 [E,I,H]; out: device bf16 [T,H].
 * saved: device, at least moe_query_workspace's `saved` bytes; moe_backward
 * reads it, so keep it unchanged between the two calls. */
moe_status moe_forward(const moe_config *cfg, const void *x, const moe_routing *routing,
                       const void *W_gate, const void *W_up, const void *W_down, void *out,
                       void *saved, size_t saved_bytes, void *scratch, size_t scratch_bytes,
                       void *stream);

/* Activation checkpointing (the pages' "2 fwd + bwd" layer step: the forward
 * runs once without keeping its activations and again just before the
 * backward).  Same arguments and errors as moe_forward.
 * moe_forward_nosave writes out like moe_forward but skips what only the
 * backward reads (bf16 and fp8_bwd: GEMM1's G, U and w*A are not written;
 * mxfp8: GEMM1 writes only A's codes, not the bf16 A, G, U, w*A, and the
 * weights are quantised for the forward GEMMs only); `saved` is used as
 * scratch and is not
 * valid for moe_backward afterwards.  out is bit-identical to moe_forward's.
 * moe_forward_recompute writes everything moe_backward reads into `saved`,
 * and not out (bf16: the permute and GEMM1 only -- the bf16 backward never
 * reads Y; the fp8 modes: GEMM2's Y too, no combine).  moe_backward after it
 * gives results bit-identical to moe_backward after moe_forward. */
moe_status moe_forward_nosave(const moe_config *cfg, const void *x, const moe_routing *routing,
                              const void *W_gate, const void *W_up, const void *W_down, void *out,
                              void *saved, size_t saved_bytes, void *scratch, size_t scratch_bytes,
                              void *stream);
moe_status moe_forward_recompute(const moe_config *cfg, const void *x, const moe_routing *routing,
                                 const void *W_gate, const void *W_up, const void *W_down, void *saved,
                                 size_t saved_bytes, void *scratch, size_t scratch_bytes, void *stream);

/* Backward.  dy: device bf16 [T,H] (gradient of out); x: the forward's input
 * (must be unchanged); routing and saved as left by moe_route/moe_forward.
 * Outputs (device): dx bf16 [T,H]; dW_gate, dW_up bf16 [E,H,I]; dW_down bf16
 * [E,I,H] (overwritten, not accumulated; experts with no token get zeros);
 * d_logits fp32 [T,E]; d_topk_w fp32 [T,k] = g_tj (may be NULL). */
moe_status moe_backward(const moe_config *cfg, const void *dy, const void *x,
                        const moe_routing *routing, const void *W_gate, const void *W_up,
                        const void *W_down, const void *saved, size_t saved_bytes, void *dx,
                        void *dW_gate, void *dW_up, void *dW_down, float *d_logits,
                        float *d_topk_w, void *scratch, size_t scratch_bytes, void *stream);

/* Router projection: the learned router's linear layer in front of moe_route,
 *   logits [T,E] fp32 = x [T,H] bf16 . W_r [H,E] bf16   (fp32 accumulation),
 * and its backward for the d_logits moe_backward returns,
 *   dW_r [H,E] fp32 = x^T . d_logits,   dx [T,H] bf16 += d_logits . W_r^T
 * (dx is updated in place: pass the dx moe_backward wrote to get the layer
 * input's full gradient).  d_logits enters both products rounded to bf16 (the
 * tensor cores' operand type); accumulation is fp32.  cfg->k and cfg->I are not
 * used; requires E % 8 == 0 (8 <= E <= 256) and H % 64 == 0.  Scratch sizes from
 * moe_router_workspace; a status header at the start of the scratch as for the
 * other calls.  With T == 0, logits is untouched and dW_r is zeroed. */
moe_status moe_router_workspace(const moe_config *cfg, size_t *fwd_scratch, size_t *bwd_scratch);
moe_status moe_router_forward(const moe_config *cfg, const void *x, const void *W_r, float *logits,
                              void *scratch, size_t scratch_bytes, void *stream);
moe_status moe_router_backward(const moe_config *cfg, const void *x, const void *W_r,
                               const float *d_logits, void *dx, float *dW_r, void *scratch,
                               size_t scratch_bytes, void *stream);

/* ---- what surrounds the layer in a training step: the norm in front of it,
 * the router's balance loss, and the update of the expert weights.  These
 * three take configurations of their own; everything else is as above (the
 * caller's buffers, dense row-major layouts, 16-byte aligned device pointers,
 * one stream, capturable, nothing allocated). */

typedef enum {
  MOE_DTYPE_BF16 = 0,
  MOE_DTYPE_FP32 = 1
} moe_dtype;

/* Layer norm (or RMS norm) over rows of H elements, with the residual sum in
 * front of it.  Any 1 <= H <= 8192, 0 <= T <= 2^30; H a multiple of 8 (bf16) or
 * 4 (fp32) is fastest.  x, residual, weight, bias, y, sum, dy, d_sum and dx are
 * of the configuration's type, statistics and weight gradients fp32.
 * Forward: h = x + residual (rounded to the type and written to sum; residual
 * and sum are both NULL when there is none, and then h = x),
 *   mu = mean h (MOE_NORM_RMS: 0), r = 1 / sqrt(mean (h - mu)^2 + eps),
 *   y = (h - mu) r weight + bias   (bias may be NULL),
 * stats [T,2] = mu, r, which the backward reads.  sum may be x or residual
 * itself; y overlaps no input.
 * Backward, from dy, h (the forward's sum, or x), weight and stats, with
 * xh = (h - mu) r and g = dy weight:
 *   dx = r (g - mean g - xh mean(g xh)) + d_sum   (MOE_NORM_RMS: no mean g)
 *   dweight [H] = sum_t dy xh,  dbias [H] = sum_t dy   (overwritten)
 * d_sum (may be NULL) is the gradient that reaches h past the norm; dx may be
 * d_sum itself.  dbias may be NULL.  Sums run in a fixed order: the same bits
 * every time.  With T == 0 the weight gradients are zeroed. */
typedef enum {
  MOE_NORM_LAYER = 0,
  MOE_NORM_RMS = 1
} moe_norm_kind;
typedef struct {
  int32_t T;     /* rows */
  int32_t H;     /* elements per row */
  int32_t kind;  /* moe_norm_kind */
  int32_t dtype; /* moe_dtype */
  float eps;     /* >= 0 */
} moe_norm_config;
moe_status moe_norm_workspace(const moe_norm_config *cfg, size_t *bwd_scratch);
moe_status moe_norm_forward(const moe_norm_config *cfg, const void *x, const void *residual, const void *weight,
                            const void *bias, void *y, void *sum, float *stats, void *stream);
moe_status moe_norm_backward(const moe_norm_config *cfg, const void *dy, const void *h, const void *weight,
                             const float *stats, const void *d_sum, void *dx, float *dweight, float *dbias,
                             void *scratch, size_t scratch_bytes, void *stream);

/* The router's auxiliary losses, from the logits and the experts chosen
 * (moe_routing's topk_idx).  The T tokens are `sequences` sequences of T /
 * sequences tokens each (1 <= sequences, a divisor of T; 1 for the whole batch);
 * 1 <= E <= 256, 1 <= k <= min(E, 16), T <= 2^30.  mask [T] (may be NULL): tokens
 * with a zero byte are padding.  Padding, and tokens whose logits are all -inf,
 * have no part in any sum or count, whatever they hold.  With c_se = the slots of
 * sequence s's tokens that chose e, N_s its tokens, N their sum, S' the sequences
 * that have any, f_se = c_se / (k N_s), P_se = the mean softmax probability:
 *   loss[0] = (1/S') sum_s E sum_e f_se P_se     (1 when the load is even)
 *   loss[1] = (1/N) sum_t lse_t^2                (the z loss; lse: log sum exp)
 *   counts [sequences,E] = c, probs [sequences,E] = P (0 where N_s = 0),
 *   tokens [sequences] = N_s, lse [T] (+inf for tokens without a part).
 * Single logits of -inf are experts that a token may not choose.  A NaN or
 * +inf logit makes the losses NaN and sets MOE_DEV_NONFINITE_LOGIT; the status
 * word is at the start of the scratch.
 * Backward, from what the forward left, for the training loss g_balance *
 * loss[0] + g_z * loss[1] (counts are constants):
 *   d_logits_te (+)= g_balance E / (S' N_s) p_te (f_se - sum_e' f_se' p_te')
 *                    + g_z (2/N) lse_t p_te,     0 for tokens without a part,
 * added to d_logits (as moe_backward leaves it) when accumulate is nonzero,
 * else written. */
typedef struct {
  int32_t T;         /* tokens */
  int32_t E;         /* experts */
  int32_t k;         /* experts per token */
  int32_t sequences; /* equal parts of the tokens, each balanced by itself */
} moe_balance_config;
moe_status moe_balance_workspace(const moe_balance_config *cfg, size_t *fwd_scratch);
moe_status moe_balance_forward(const moe_balance_config *cfg, const float *logits, const int32_t *topk_idx,
                               const uint8_t *mask, float *loss, int32_t *counts, float *probs, int32_t *tokens,
                               float *lse, void *scratch, size_t scratch_bytes, void *stream);
moe_status moe_balance_backward(const moe_balance_config *cfg, const float *logits, const int32_t *counts,
                                const int32_t *tokens, const float *lse, float g_balance, float g_z,
                                float *d_logits, int32_t accumulate, void *stream);

/* The orthogonalised update of a batch of matrices by Newton-Schulz products
 * (the Muon optimiser's, for example of dW_gate, dW_up [E,H,I] or dW_down
 * [E,I,H]).  g: device [batch,R,C] of the configuration's type; momentum: device
 * fp32 [batch,R,C], updated in place, or NULL.  Per matrix, in fp32,
 *   u = g, or with momentum:  m <- beta m + g,  u = g + beta m (nesterov) or m;
 *   X = u / max(|u|_F, eps);
 *   steps times, with step i's (a, b, c) = coefs[3i .. 3i+2] (host memory, read
 *   during the call):  S = X X^T (R <= C) or X^T X,  P = a I + b S + c S^2,
 *   X <- P X or X P;
 *   out = scale X, bf16 [batch,R,C].
 * X, S and P are rounded to fp16 between products, whose sums are fp32.  The
 * coefficients are to keep it all in fp16's range: with s a singular value of X in
 * front of a step and p = |a + b s^2 + c s^4|, s has to stay below 255, and p, p s^2
 * and the product of two steps' p in succession below 65504 (the usual quintic,
 * 3.4445 -4.7750 2.0315 five times, keeps s below 1.3 and p below 3.5).  A result that
 * is not finite sets MOE_DEV_NONFINITE_UPDATE.  Singular values far below
 * |u|_F / 1000 grow out of the roundings as they do out of a bf16 gradient's own; where
 * eps is above |u|_F, values of u / eps below about 1e-7 lose exactness, those below
 * 1e-10 become zero.
 * 1 <= R, C <= 16384, 0 <= batch <= 65535, 1 <= steps <= 64, any alignment of rows
 * (multiples of 8 columns are fastest).  out may not overlap g or momentum.  The
 * sum of squares is formed in fp32: values of u below about 1e-22 have no part in
 * it.  A matrix of zeros gives zeros; one whose sum of squares is not finite gives NaN
 * and sets MOE_DEV_NONFINITE_UPDATE (status word at the start of the scratch), and
 * no other matrix is touched by it. */
typedef struct {
  int32_t batch; /* matrices */
  int32_t R, C;  /* rows and columns of each */
  int32_t steps; /* Newton-Schulz steps */
  int32_t dtype; /* moe_dtype of g */
  float eps;     /* >= 0: the least norm divided by */
} moe_ortho_config;
moe_status moe_ortho_workspace(const moe_ortho_config *cfg, size_t *scratch);
moe_status moe_ortho_update(const moe_ortho_config *cfg, const float *coefs, const void *g, float *momentum,
                            float beta, int32_t nesterov, float scale, void *out, void *scratch,
                            size_t scratch_bytes, void *stream);

/* The gate: a routing from the router's logits [T,E] fp32, in the forms that moe_route does not have.
 * Per token, with l its logits:
 *   s = softmax(l) or sigmoid(l);   c = s + bias (fp32 [E], or NULL: the order of l)
 *   groups: the E experts are `groups` equal runs; a group's score is the sum of its group_best (1 or 2)
 *   largest c; the top_groups best groups stay (ties: the lower group)
 *   S = the k largest c among the experts of those groups (ties: the lower expert)
 *   w_j = scale s_{S_j} / sum_i s_{S_i}   (renormalise), or scale s_{S_j}
 * The bias enters the choice alone, not the weights.  topk_idx is ordered by (c desc, index asc), and all
 * fields of *routing are written as moe_route writes them, so that moe_forward and moe_backward take it.
 * The choice is that of exact scores: tokens whose scores lie closer together than fp32 resolves are
 * chosen again from scores in 64 bits, so that a recomputed forward, or another program, chooses the same.
 * (Sums of two softmax scores that are equal but for the last of those bits may go by their roundings.)
 * The time depends on the inputs for that: a token that is chosen again keeps a warp busy for some 5 us.  Of
 * ordinary fp32 logits that is about one in a thousand; it is many
 *   - without a bias, where two of the first k + 1 logits agree in their upper 24 bits: a third of the tokens whose
 *     logits were rounded to bf16 (1.2 to 1.7 times the time of a call, 4 times with k = 16);
 *   - in rows of equal logits, padding for instance, with a bias or without (3 to 9 times, where all rows are that);
 *   - by softmax with a bias on nearly even logits (a spread of 0.01 among 256 experts: 1.4 times);
 *   - with a bias far larger than the scores (1e3: 1.5 to 2.6 times, 1e4: 8 to 20, 1e6: 14 to 45).
 * A logit of -inf, or a bias of -inf or NaN, is an expert that may not be chosen; a group's score goes over
 * the others, and a group without any comes last.  Slots that no expert is left for are filled with the
 * remaining experts by index, at weight zero.  A NaN logit counts as -inf, +inf as the largest float, and
 * both set MOE_DEV_NONFINITE_LOGIT (status word at the start of the scratch).
 * 0 <= T <= 2^30, T * k < 2^31, 1 <= E <= 256, 1 <= k <= min(E, 16), 1 <= groups <= 32, a divisor of E,
 * 1 <= top_groups <= groups, top_groups * (E / groups) >= k, 0 < scale, finite.
 * Backward: d_logits [T,E] (overwritten) from d_topk_w [T,k], the gradient of the weights (moe_backward's
 * d_topk_w; its d_logits are those of moe_route's weights and not used), and the routing's topk_idx and
 * topk_w.  A token's indices are distinct; a slot whose index is outside [0, E), or whose weight is zero,
 * has no part.  The bias has no gradient; its step
 *   bias_e += rate * sign(mean over experts of the load - load_e)
 * takes the load from counts [rows,E], added up over the rows: a routing's counts (rows = 1), or
 * moe_balance_forward's (rows = sequences), which leave padding out.  d_logits may not overlap an input. */
typedef enum {
  MOE_SCORE_SOFTMAX = 0,
  MOE_SCORE_SIGMOID = 1
} moe_score;
typedef struct {
  int32_t T;           /* tokens */
  int32_t E;           /* experts */
  int32_t k;           /* experts per token */
  int32_t score;       /* moe_score */
  int32_t groups;      /* groups of E / groups experts; 1: none */
  int32_t top_groups;  /* groups that a token may use */
  int32_t group_best;  /* scores that a group is judged by: 1 or 2 */
  int32_t renormalise; /* nonzero: the weights of a token add up to scale */
  float scale;         /* factor of the weights */
} moe_gate_config;
moe_status moe_gate_workspace(const moe_gate_config *cfg, size_t *fwd_scratch);
moe_status moe_gate_forward(const moe_gate_config *cfg, const float *logits, const float *bias,
                            const moe_routing *routing, void *scratch, size_t scratch_bytes, void *stream);
moe_status moe_gate_backward(const moe_gate_config *cfg, const float *logits, const int32_t *topk_idx,
                             const float *topk_w, const float *d_topk_w, float *d_logits, void *stream);
moe_status moe_gate_update_bias(const moe_gate_config *cfg, float *bias, const int32_t *counts, int32_t rows,
                                float rate, void *stream);

/* One AdamW step over a list of tensors (for parameters that are no expert matrices: norms, router,
 * embeddings; or for all of them).  Tensor i has n[i] >= 0 elements (at most 2^40 in all): params[i] of
 * param_dtype, updated in place; grads[i] of grad_dtype; copies (NULL: none; fp32 parameters only)
 * with copies[i], or NULL, a bf16 copy of the new parameter; decay[i] >= 0 its weight decay (decay NULL: 0).
 * The arrays of sizes, decays and addresses are host memory, read during the call.  In fp32,
 *   g = grads * *grad_scale (device fp32; NULL: 1),   t = the step's number, from 1
 *   m <- beta1 m + (1 - beta1) g,   v <- beta2 v + (1 - beta2) g^2
 *   p <- p (1 - lr decay) - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * with lr from *lr_device (device fp32) where that is given, so that a captured step follows a schedule.
 * States, in one array each over all tensors, a tensor's from a multiple of 256 elements on
 * (moe_adamw_state_elements gives the elements of an array; the padding is not touched):
 *   state_bits 32: m, v fp32;
 *   state_bits 8: m and the root of v as e4m3 codes, m_scale and v_scale fp32, one per 256 elements: a value
 *   is its code's times the scale, which is the block's largest (1e-30 at least) times 1/448; the code is the
 *   value times 448 times the reciprocal of that largest, rounded to nearest even, a root above zero to 2^-9 of the scale at least.  This step uses m and v from before the rounding.
 *   step: int32 [4]: the status word, the number of steps so far, and two words that are zero between
 *   calls.  A call adds one to the steps.
 * All of it starts as zeros.  A step after which a parameter (as it is stored: bf16 rounds what is too large to
 * infinity) or v is not finite sets MOE_DEV_NONFINITE_UPDATE in the status word (of the last call;
 * moe_get_device_status reads it from step); with 8 bits such an element's m and v are stored as e4m3's NaN and
 * leave the scales of their block alone.  Where *grad_scale is not finite the step
 * is left out: nothing changes but the status word, which gets that flag.
 * Tensors overlap neither each other nor the states.  Calls of up to 64 tensors with elements are one launch. */
typedef struct {
  int32_t tensors;
  int32_t param_dtype; /* moe_dtype */
  int32_t grad_dtype;  /* moe_dtype */
  int32_t state_bits;  /* 8 or 32 */
  double beta1, beta2; /* in [0, 1) */
  double eps;          /* >= 0 */
} moe_adamw_config;
typedef struct {
  void *m, *v;              /* device [elements], fp32 or e4m3 */
  float *m_scale, *v_scale; /* device [elements / 256]; state_bits 8 only */
  int32_t *step;            /* device [4] */
} moe_adamw_state;
moe_status moe_adamw_state_elements(const moe_adamw_config *cfg, const int64_t *n, int64_t *elements);
moe_status moe_adamw_step(const moe_adamw_config *cfg, const int64_t *n, const double *decay, void *const *params,
                          const void *const *grads, void *const *copies, const moe_adamw_state *state, double lr,
                          const float *lr_device, const float *grad_scale, void *stream);

/* A dense layer (a shared expert beside the routed ones, a projection): a matrix product with bias, activation
 * and residual in its epilogue, and its backward.  bf16 tensors, dense rows; sums in fp32.
 * Forward:   z = x W + bias,  y = act(z) + residual
 *   x [T,K], W [K,N], bias [N] (may be NULL), residual [T,N] (may be NULL), y [T,N]; z [T,N], which the
 *   backward reads, is written where it is not NULL (never without an activation).  y may be residual
 *   itself and overlaps nothing else.
 * Backward:  dz = dy act'(z),  dx = dz W^T,  dW = x^T dz,  dbias = sum_t dz
 *   dx [T,K], dW [K,N] bf16 and dbias [N] fp32, overwritten; each may be NULL (not all three) and is then
 *   not computed (W is only read for dx, x for dW).  z as the forward left it; NULL without an
 *   activation.  dz enters the products rounded to bf16, dbias as it is.  The residual's gradient is dy itself.
 *   Outputs overlap no input.
 * Activations: relu, silu z / (1 + e^-z), gelu in its tanh form (not the one by erf).  A NaN of z is a NaN of
 * y and of dz.  Sums run in a fixed order: the same call leaves the same bits (the order goes by the sizes and by
 * which of dx and dW are asked for).  0 <= T <= 2^30; K and N multiples of 8, 8 to 65536; T times either below
 * 2^40.  With T == 0 the weight gradients are zeroed.
 * Status word at the start of each scratch. */
typedef enum {
  MOE_ACT_NONE = 0,
  MOE_ACT_RELU = 1,
  MOE_ACT_SILU = 2,
  MOE_ACT_GELU = 3
} moe_act;
typedef struct {
  int32_t T;   /* rows */
  int32_t K;   /* inputs of a row */
  int32_t N;   /* outputs */
  int32_t act; /* moe_act */
} moe_linear_config;
moe_status moe_linear_workspace(const moe_linear_config *cfg, size_t *fwd_scratch, size_t *bwd_scratch);
moe_status moe_linear_forward(const moe_linear_config *cfg, const void *x, const void *W, const void *bias,
                              const void *residual, void *y, void *z, void *scratch, size_t scratch_bytes, void *stream);
moe_status moe_linear_backward(const moe_linear_config *cfg, const void *dy, const void *x, const void *W, const void *z,
                               void *dx, void *dW, float *dbias, void *scratch, size_t scratch_bytes, void *stream);

/* Routing without a caller-provided scratch buffer.  The paper has no
 * counterpart: it exists for callers that cannot allocate device memory --
 * code running while a CUDA graph is captured (cudaMalloc is not allowed
 * there), code inside a framework whose allocator already owns the device
 * memory, or a serving loop that must not allocate on its hot path.
 * Same arguments, results and errors as moe_route, except that the scratch is a
 * fixed 2.5 MiB + 4 KiB array inside this library's device memory (every GPU
 * that loads the library keeps it until the process exits).  It fits every
 * configuration with T <= 32768, and any other whose moe_query_workspace
 * route_scratch is at most that size; for the rest it returns MOE_ERR_WORKSPACE
 * and launches nothing.  Allocates nothing (no cudaMalloc/cudaFree, no
 * allocating library call).
 * device_status: optional device int32 that receives the call's MOE_DEV_* flags
 * (copied on `stream` after the routing kernels); NULL to skip.
 * The first call on a device looks up the array's device address (with that
 * device current) and keeps it for the process; make that first call before
 * any stream capture.  If the lookup fails the call returns MOE_ERR_CUDA with
 * nothing launched and no CUDA error left pending, and the next call on that
 * device looks the address up again.  All calls share the one array and it keeps the last call's
 * contents: calls that overlap on the GPU (for example on two streams) race,
 * so serialise them. */
moe_status moe_route_static_scratch(const moe_config *cfg, const float *logits,
                                    const moe_routing *routing, int32_t *device_status,
                                    void *stream);

/* Diagnostic with no counterpart in the paper: launches one kernel that waits,
 * through the same bounded wait every pipeline stage of the library uses, on
 * an mbarrier nothing arrives at.  The wait gives up after about two seconds
 * of SM clock and the kernel sets MOE_DEV_WAIT_TIMEOUT in *device_status
 * (device int32, 4-byte aligned, zeroed on `stream` first).  It shows that a
 * lost arrival is reported as a status instead of hanging the GPU, and that
 * the context stays usable afterwards.  Returns MOE_ERR_INVALID_ARG for a
 * NULL pointer; asynchronous on `stream`. */
moe_status moe_selftest_wait_timeout(int32_t *device_status, void *stream);

/* Waits for `stream`, then reads the status word at the start of `scratch` (a
 * scratch buffer previously passed to moe_route, moe_forward or moe_backward).
 * *host_code receives the MOE_DEV_* flags; returns MOE_OK when they are zero,
 * MOE_ERR_DEVICE otherwise.  The only call that synchronises. */
moe_status moe_get_device_status(const void *scratch, void *stream, int32_t *host_code);

/* Static description of a status code. */
const char *moe_status_string(moe_status status);

/* Optional per-kernel timing for profiling.  When `events` is non-NULL, every
 * later library call records events[2i] and events[2i+1] (cudaEvent_t as
 * void*) on its stream around the i-th kernel it launches, counting from the
 * attach, up to `capacity` kernels; moe_timing_count returns how many were
 * recorded.  Process-wide, not thread-safe; pass NULL to detach. */
moe_status moe_timing_attach(void *const *events, int32_t capacity);
int32_t moe_timing_count(void);
/* Name of the i-th timed kernel (static string; NULL when out of range). */
const char *moe_timing_label(int32_t i);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_H */
