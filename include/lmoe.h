/*
 * lmoe.h -- C ABI of the LatentMoE feed-forward layer (forward pass) on
 * AMD MI355X (gfx950).
 *
 * The layer (page "Nemotron 3 Ultra 架构深度拆解报告", CH5 §5.6 "7 步数据流",
 * Steps 1-7, router moved onto the latent as the page's summary (CH0) and the
 * page "NVIDIA Nemotron 3 Super 技术解读" §2.2 describe it):
 *
 *   z    = x W1^T                          fc1_latent            [T, R]
 *   l    = z Wg^T, s = sigmoid(l)          fp32 router           [T, E]
 *   I    = top-K of (s + bias), single group, ties to the lower expert id
 *   w    = rho * s[I] / (sum s[I] + 1e-20)  rho = routed_scaling_factor
 *   r    = sum_k w_k relu(z Wup[I_k]^T)^2 Wdn[I_k]^T            [T, R]
 *   y    = r W2^T + relu(x Wsu^T)^2 Wsd^T  fc2_latent + shared   [T, D]
 *
 * Optionally (lmoe_config.fuse) the layer also takes over the two steps of
 * its block on either side (page "Nemotron 3 Ultra 架构深度拆解报告", CH9 §9.3:
 * pre-norm RMSNorm, mixer, residual add); x is then the block's residual
 * stream h:
 *
 *   PRENORM   the layer runs on RMSNorm(h) = r * bf16(gamma * h) with
 *             r = 1 / sqrt(mean(h^2) + norm_eps) per token: the GEMM operand
 *             is the bf16 rounding of gamma * h and r scales the fp32 results
 *             of the latent and shared-up projections (RMSNorm in exact
 *             arithmetic, one bf16 rounding, placed where it can be
 *             reproduced exactly);
 *   RESIDUAL  y = h + (layer output), added in fp32 before the bf16 rounding.
 *
 * Sizes follow the model's config keys (page "Nemotron-3-Labs-Ultra-Math-SFT"
 * article, 核心配置速查表): D = hidden_size, R = moe_latent_size,
 * E = n_routed_experts, K = num_experts_per_tok, F = moe_intermediate_size,
 * S = moe_shared_expert_intermediate_size.
 *
 * Conventions for every entry point:
 *  - bf16 tensors are passed as uint16_t bit patterns; every matrix is
 *    row-major and dense, weights stored out x in (a linear layer's layout),
 *    expert weights as 3-D (expert, out, in) tensors (§5.1 of the page above);
 *  - all tensor pointers are DEVICE pointers, 16-byte aligned, owned by the
 *    caller; the library never allocates or frees device memory;
 *  - `stream` is a hipStream_t (NULL = the null stream); work is enqueued
 *    asynchronously and nothing synchronises the host;
 *  - arguments are checked on the host before any HIP call; on error nothing
 *    is enqueued and the status says why.  Device faults surface at the
 *    caller's next synchronisation.  Inputs must be finite.
 *  - one handle owns one workspace: lmoe_forward and lmoe_route on one
 *    handle use the same workspace (lmoe_route its router-logits part), so
 *    calls on one handle must not overlap: issue them on one stream, or
 *    order them with events.
 *  - lmoe_create creates one auxiliary HIP stream (non-blocking, default
 *    priority) and two events per handle, used to run the shared expert's up
 *    projection concurrently with the latent projection and the router
 *    (forked from `stream` at the start of the forward for small batches,
 *    after the latent projection otherwise, and joined back before the
 *    output projection); lmoe_destroy releases them.  A forward makes no
 *    other HIP object, so any forward (the first included) can be captured
 *    into a HIP graph.
 */
#ifndef LMOE_H
#define LMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LMOE_OK = 0,
  LMOE_ERR_INVALID_ARG = -1,     /* NULL / misaligned / aliased pointer, bad value */
  LMOE_ERR_UNSUPPORTED = -2,     /* a configuration this library does not implement */
  LMOE_ERR_TOO_MANY_TOKENS = -3, /* T > max_tokens of the handle */
  LMOE_ERR_WORKSPACE = -4,       /* workspace missing or smaller than lmoe_workspace_size */
  LMOE_ERR_HIP = -5,             /* a HIP launch or copy returned an error */
  LMOE_ERR_SCRATCH = -6          /* lmoe_forward_noalloc: the forward needs more than
                                    LMOE_NOALLOC_SCRATCH_BYTES of scratch */
} lmoe_status;

/* Path selection for the expert and projection GEMMs.  AUTO picks by token
 * count: weight streaming for small batches, LDS-tiled MFMA otherwise (the
 * projections split over k into fp32 partial sums while T <= 256, to fill
 * the GPU); the other values force one tiling for every GEMM (used by tests;
 * TILED still splits the projections over k when T <= 256).  Results agree
 * across paths to rounding. */
typedef enum { LMOE_PATH_AUTO = 0, LMOE_PATH_STREAM = 1, LMOE_PATH_TILED = 2 } lmoe_path;

/* Storage of the routed experts' weights.  BF16: expert_up / expert_down.
 * MXFP4 (block-scaled FP4 with the E2M1 elements of CH8 §8.1 of the page
 * "Nemotron 3 Ultra 架构深度拆解报告"; block layout: lmoe_quantize_mxfp4):
 * the *_mxfp4 / *_scale fields; the expert GEMMs decode the weights exactly
 * to bf16, streaming them for small batches and, for large ones, copying
 * the FP4 codes into the LDS-tiled GEMM's tiles and decoding them right
 * before the MFMAs (the same lmoe_path choice as bf16 weights; R and F must
 * be multiples of 128).  Everything else stays bf16 / fp32.
 * FP8: the *_fp8 / *_fp8_scale fields, weights as lmoe_quantize_fp8_weight
 * writes them; the expert projections run on 8-bit activations too: the
 * latent (from its fp32 values) and the hidden rows relu(.)^2 (from the
 * unrounded sums) are quantised as by lmoe_quantize_fp8, and the products are
 * summed as by lmoe_fp8_matmul with bf16 y (the up projection's always by the
 * 8-bit matrix instruction).  R and F must be multiples of 128,
 * max_tokens * R below 2^31 (and with LMOE_PATH_STREAM max_tokens * K / 16 *
 * max(F / 128, R / 64) below about 2^24). */
typedef enum {
  LMOE_EXPERTS_BF16 = 0,
  LMOE_EXPERTS_MXFP4 = 1,
  LMOE_EXPERTS_FP8 = 2
} lmoe_expert_format;

/* Block steps fused into the layer (bits of lmoe_config.fuse; CH9 §9.3 of
 * the page "Nemotron 3 Ultra 架构深度拆解报告"): the block's pre-norm RMSNorm
 * (needs lmoe_weights.norm_weight) and its residual add.  See the top of
 * this file for the exact arithmetic. */
typedef enum { LMOE_FUSE_PRENORM = 1, LMOE_FUSE_RESIDUAL = 2 } lmoe_fuse;

typedef struct {
  int32_t hidden_size;                         /* D; multiple of 64 */
  int32_t moe_latent_size;                     /* R; multiple of 64 */
  int32_t n_routed_experts;                    /* E; 1..1024 */
  int32_t num_experts_per_tok;                 /* K; 1..min(E, 64) */
  int32_t moe_intermediate_size;               /* F; multiple of 64 */
  int32_t moe_shared_expert_intermediate_size; /* S; multiple of 64 */
  int32_t n_group;    /* routing groups (§5.5): divides E into groups of >= 2
                         experts (any size when 1); at most 64 */
  int32_t topk_group; /* groups kept per token: 1..n_group, and
                         K <= topk_group * E / n_group */
  float routed_scaling_factor;                 /* rho, finite (5.0 in the model) */
  int32_t max_tokens;                          /* largest T a forward may use; sizes the workspace */
  int32_t path;                                /* lmoe_path */
  int32_t expert_format;                       /* lmoe_expert_format */
  int32_t fuse;                                /* lmoe_fuse bits; 0 = the layer alone */
  float norm_eps;                              /* RMSNorm epsilon, finite, >= 0 (PRENORM) */
} lmoe_config;

/* Device pointers; the handle borrows them and they must outlive it. */
typedef struct {
  const uint16_t *fc1_latent;  /* bf16 [R, D] */
  const float *router;         /* fp32 [E, R]  gate weight */
  const float *router_bias;    /* fp32 [E]     e_score_correction_bias */
  const uint16_t *expert_up;   /* bf16 [E, F, R] */
  const uint16_t *expert_down; /* bf16 [E, R, F] */
  const uint16_t *fc2_latent;  /* bf16 [D, R] */
  const uint16_t *shared_up;   /* bf16 [S, D] */
  const uint16_t *shared_down; /* bf16 [D, S] */
  /* MXFP4 experts (expert_format = LMOE_EXPERTS_MXFP4; else unused): */
  const uint8_t *expert_up_mxfp4;   /* [E, F, R/2] codes, 16-byte aligned */
  const uint8_t *expert_up_scale;   /* [E, F, R/32] block scales */
  const uint8_t *expert_down_mxfp4; /* [E, R, F/2] codes, 16-byte aligned */
  const uint8_t *expert_down_scale; /* [E, R, F/32] block scales */
  /* LMOE_FUSE_PRENORM only (may be NULL otherwise): */
  const uint16_t *norm_weight;      /* bf16 [D] RMSNorm weight gamma */
  /* FP8 experts (expert_format = LMOE_EXPERTS_FP8; else not read), 16-byte
   * aligned: */
  const uint8_t *expert_up_fp8;       /* [E, F, R] e4m3 codes */
  const float *expert_up_fp8_scale;   /* [E, F/128, R/128] block scales */
  const uint8_t *expert_down_fp8;     /* [E, R, F] e4m3 codes */
  const float *expert_down_fp8_scale; /* [E, R/128, F/128] block scales */
} lmoe_weights;

/* Optional device outputs of intermediate values (tests, monitoring).  Any
 * field may be NULL.  Shapes for a forward of T tokens: */
typedef struct {
  float *z_f32;           /* [T, R] fp32 latent (the router's input) */
  int32_t *topk_idx;      /* [T, K] selected experts, ascending id per token */
  float *topk_w;          /* [T, K] routing weights, same order as topk_idx */
  int32_t *expert_counts; /* [E] tokens routed to each expert */
  float *r_latent;        /* [T, R] fp32 weighted sum of expert outputs */
} lmoe_taps;

typedef struct lmoe_handle lmoe_handle;

/* Bytes of device workspace a handle with this configuration needs for
 * forwards of up to cfg->max_tokens tokens: the intermediate tensors of page
 * "Nemotron 3 Ultra 架构深度拆解报告", CH5 §5.6 Steps 1-7 (latent, router
 * logits, top-K, the expert-sorted rows of Step 6's grouping, the experts'
 * hidden and output rows, the weighted sum) plus the shared expert's hidden
 * rows; layout and sizes in the library source.  0 if the configuration is
 * invalid or unsupported.  Pure host function. */
size_t lmoe_workspace_size(const lmoe_config *cfg);

/* Set up one layer (the module of CH5 §5.6 of the page above, bound to its
 * weights): validate `cfg` and `w` (host checks first: on any error nothing
 * is created and *out is NULL), carve `workspace` (device memory of at
 * least lmoe_workspace_size(cfg) bytes, 256-byte aligned, caller-owned; the
 * library never frees it) and return a host-side handle in *out, which
 * borrows `w` and `workspace`.  Its only HIP calls create the handle's
 * auxiliary stream and two events on the current device (LMOE_ERR_HIP if
 * they fail, e.g. with no GPU; nothing is left behind).
 * Debug aid: if the environment variable LMOE_DEBUG is set (and not "0")
 * when the handle is created, lmoe_forward and lmoe_route synchronise the
 * stream (and the handle's auxiliary stream) after every stage and return
 * LMOE_ERR_HIP at the first stage whose launch or execution failed, naming
 * it on stderr.  Same kernels and results; such calls block the host and
 * cannot be captured into a HIP graph. */
lmoe_status lmoe_create(const lmoe_config *cfg, const lmoe_weights *w, void *workspace,
                        size_t workspace_bytes, lmoe_handle **out);

/* y = LatentMoE(x) for T tokens.  x: bf16 [T, D], y: bf16 [T, D] (must not
 * overlap x).  T = 0 is a no-op.  `taps` may be NULL.  Page steps 1-7.
 * With fuse bits set: x is the residual stream h and y = h + LatentMoE(
 * RMSNorm(h)) (or either part alone); taps->z_f32 is then the latent of the
 * normalised input. */
lmoe_status lmoe_forward(lmoe_handle *h, const uint16_t *x, int32_t T, uint16_t *y,
                         void *stream, const lmoe_taps *taps);

/* Router only (page steps 1-4 on a given latent): from z_f32 [T, R] fp32
 * write topk_idx [T, K] (ascending expert id) and topk_w [T, K]. */
lmoe_status lmoe_route(lmoe_handle *h, const float *z_f32, int32_t T, int32_t *topk_idx,
                       float *topk_w, void *stream);

/* MXFP4 quantiser for expert weights: w is bf16 [rows, cols] (row-major,
 * cols a multiple of 32, 16-byte aligned); writes codes [rows, cols/2]
 * (16-byte aligned; element 2i of a row in the low nibble of byte i, code
 * = sign bit 3 | E2M1 magnitude code 0..7 for 0, 0.5, 1, 1.5, 2, 3, 4, 6)
 * and scales [rows, cols/32] (block b of a row holds elements 32b..32b+31
 * and its value is 2^(scale - 127)).  Per block: e = floor(log2 max|w|) - 2
 * clipped to [-127, 127] (-127 for an all-zero block); each element is
 * |w| / 2^e rounded to the nearest E2M1 magnitude, ties to the even code,
 * clamped at 6, signed unless it rounds to 0.  Inputs must be finite.
 * Device pointers; asynchronous on `stream`. */
lmoe_status lmoe_quantize_mxfp4(const uint16_t *w, int64_t rows, int32_t cols, uint8_t *codes,
                                uint8_t *scales, void *stream);

/* Release a handle from lmoe_create: its auxiliary stream, events and any
 * profiling events, and the host-side handle (no device memory is freed:
 * the caller owns all of it).  Work already enqueued on the handle's
 * streams must have finished.  NULL is a no-op. */
void lmoe_destroy(lmoe_handle *h);

/* Static, NUL-terminated text for a status code of this header (not owned
 * by the caller); "unknown status" for any other value.  Pure host function. */
const char *lmoe_status_string(lmoe_status s);

/* ---- allocation-free forward --------------------------------------------
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * forward as lmoe_forward (same kernels, same results bit for bit) without a
 * handle or a workspace.  Its scratch (the workspace a handle for exactly T
 * tokens would need) lives in one static device array of
 * LMOE_NOALLOC_SCRATCH_BYTES that the library holds on every GPU it runs on
 * until the process ends; at the full layer shape (hidden 8192, latent
 * 2048, 512 experts top-22) that covers up to about 90 tokens, e.g. the
 * 32-token decode batch.  Larger forwards return LMOE_ERR_SCRATCH before any
 * launch.  Nothing is allocated and no stream or event is created: the
 * shared expert runs on `stream` after the others.  The first call on a
 * device looks up the array's address there (make it outside graph
 * capture).  `cfg` and `w` are checked as by lmoe_create, x and y as by
 * lmoe_forward; T <= cfg->max_tokens; `stream` must belong to the current
 * device.  Every call on one GPU uses that GPU's one array (it keeps the
 * last call's contents; nothing in it needs clearing): calls that overlap
 * on one GPU, on any streams, race and give wrong results. */
#define LMOE_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
lmoe_status lmoe_forward_noalloc(const lmoe_config *cfg, const lmoe_weights *w,
                                 const uint16_t *x, int32_t T, uint16_t *y, void *stream);

/* ---- operators around the layer -------------------------------------------
 * Each is one call on device arrays, without a handle; the conventions at the
 * top of this file hold (`stream` must belong to the current device; a count
 * of 0 tokens or rows is a no-op).  Arrays are typed by an lmoe_dtype where
 * several types are taken, and need their elements' natural alignment only
 * (16-byte aligned arrays with widths and strides that are multiples of 8 run
 * on wide loads).  Outputs must not overlap inputs or each other. */
typedef enum { LMOE_F32 = 0, LMOE_BF16 = 1 } lmoe_dtype;

/* Routing from given logits (page "Nemotron 3 Ultra 架构深度拆解报告", CH5
 * §5.5 and §5.6 Steps 2-4, with the choices other sparse layers make):
 *   s = sigmoid(l) or softmax(l);  b = s + bias (when one is given)
 *   groups (n_group > 1): a group's score is the sum of its group_score (1 or
 *     2) largest b; the topk_group best groups stay, equal ones: lower index
 *   the top_k experts of the largest b (without a bias: the largest l, which
 *     is the same order) that stay, equal ones: lower id
 *   w = scale s, or scale s / (sum of the selected s + 1e-20) (renormalise)
 * b and the group scores are compared by their values in 64 bits.  A logit of
 * -inf or NaN is an expert that is not available: its score is 0, its b is
 * -inf, and it is selected (with weight 0) only where fewer than top_k
 * others are; +inf counts as the largest finite float. */
typedef enum { LMOE_SCORE_SIGMOID = 0, LMOE_SCORE_SOFTMAX = 1 } lmoe_score;
typedef struct {
  int32_t n_experts;   /* E: 1..1024, any number */
  int32_t top_k;       /* K: 1..min(64, topk_group * E / n_group) */
  int32_t score;       /* lmoe_score */
  int32_t n_group;     /* divides E; at most 64 */
  int32_t topk_group;  /* 1..n_group */
  int32_t group_score; /* 1 or 2 (2 needs groups of >= 2 when n_group > 1) */
  int32_t renormalise; /* 0 or 1 */
  float scale;         /* finite */
} lmoe_router;

/* logits: [T, E] of `logits_type`, rows `logits_stride` (>= E) elements
 * apart; bias: fp32 [E], finite, or NULL; T up to 2^22.  Writes topk_idx
 * [T, K] (ascending ids) and topk_w [T, K]. */
lmoe_status lmoe_route_logits(const lmoe_router *router, const void *logits, int32_t logits_type,
                              int64_t logits_stride, const float *bias, int32_t T,
                              int32_t *topk_idx, float *topk_w, void *stream);

/* The gradient of topk_w in the logits, the selection held fixed: from dw
 * [T, K] (the gradient of topk_w) and the forward's logits and topk_idx,
 * writes dlogits [T, E] (dense, of logits_type; 0 where the logit is not
 * available).  Ids outside [0, E) are ignored, equal ids of a token add up. */
lmoe_status lmoe_route_logits_backward(const lmoe_router *router, const void *logits,
                                       int32_t logits_type, int64_t logits_stride,
                                       const int32_t *topk_idx, const float *dw, int32_t T,
                                       void *dlogits, void *stream);

/* The norms around a block with its gate and residual scale, per token:
 *   n     = post * y / sqrt(mean(y^2) + eps)    (n = y without post_weight)
 *   h_out = res_scale * h + gate * n
 *   x     = pre * h_out / sqrt(mean(h_out^2) + eps)    (if x is wanted)
 * h is the residual stream before the block, y the block's output (NULL: 0,
 * the norm ahead of a first block), x the next block's input.  h_out and x
 * round once from fp32 values (x is computed from the unrounded h_out).
 * Values must be finite, and so must the fp32 sums over a row of y^2 (with
 * post_weight) and of h_out^2. */
typedef enum {
  LMOE_GATE_NONE = 0,    /* 1 */
  LMOE_GATE_CHANNEL = 1, /* [D] */
  LMOE_GATE_TOKEN = 2,   /* [T] */
  LMOE_GATE_FULL = 3     /* [T, D], dense */
} lmoe_gate;
typedef struct {
  const void *h;           /* [T, D], rows h_stride elements apart */
  const void *y;           /* [T, D], rows y_stride elements apart, or NULL */
  int64_t h_stride, y_stride;
  const void *pre_weight;  /* [D] or NULL (1) */
  const void *post_weight; /* [D] or NULL (y is not normalised; NULL if y is) */
  const void *res_scale;   /* [D] or NULL (1) */
  const void *gate;        /* by gate_kind; NULL if LMOE_GATE_NONE */
  int32_t gate_kind;       /* lmoe_gate (LMOE_GATE_NONE if y is NULL) */
  int32_t h_type, y_type;  /* lmoe_dtype: of h, h_out and their gradients; of y, x and theirs */
  int32_t pre_type, post_type, res_scale_type, gate_type; /* lmoe_dtype */
  int32_t T, D;            /* T: 0..2^22 - 1, D: 1..16384 */
  float eps;               /* finite, > 0 */
} lmoe_block_norm_args;

/* h_out [T, D] (h_type), x [T, D] (y_type) or NULL, stats fp32 [T, 2] (the
 * two reciprocal roots, what the backward needs; 1 in place of the first
 * without post_weight and of the second without x) or NULL; all dense. */
lmoe_status lmoe_block_norm(const lmoe_block_norm_args *a, void *h_out, void *x, float *stats,
                            void *stream);

/* Gradients, dense, each in the type of what it belongs to; NULL: not wanted
 * (dy, dpost_weight, dres_scale, dgate must be NULL where their input is).
 * Column sums are added in a fixed order: the same bits every time. */
typedef struct {
  void *dh, *dy;
  void *dpre_weight, *dpost_weight, *dres_scale, *dgate;
} lmoe_block_norm_grads;

/* Bytes of workspace of lmoe_block_norm_backward (partial column sums of the
 * [D] gradients; 0 if none is wanted, or for arguments it refuses).  Pure
 * host function. */
size_t lmoe_block_norm_workspace_size(const lmoe_block_norm_args *a,
                                      const lmoe_block_norm_grads *g);

/* From the forward's arguments and stats, dh_out [T, D] (h_type) and dx
 * [T, D] (y_type; NULL if the forward made no x), either may be NULL (0), the
 * gradients in g.  workspace:
 * 16-byte aligned device memory of the size above; calls that may overlap
 * need one each.  T = 0 writes zeros to the [D] gradients. */
lmoe_status lmoe_block_norm_backward(const lmoe_block_norm_args *a, const float *stats,
                                     const void *dh_out, const void *dx,
                                     const lmoe_block_norm_grads *g, void *workspace,
                                     size_t workspace_bytes, void *stream);

/* 8-bit floating point (e4m3, OCP: one sign, four exponent and three mantissa
 * bits, largest finite value 448) with fp32 scales of blocks of 128 along the
 * last axis: value = code * scale, scale = max(largest magnitude of the block
 * / 448, 2^-126), code = value / scale rounded to the nearest e4m3 number,
 * ties to even (fp32 division, correctly rounded).  Inputs must be finite.
 *
 * Activations: x [rows, cols] (of `x_type`, rows x_stride >= cols elements
 * apart), a scale for each block of a row: codes [rows, cols], scales [rows,
 * ceil(cols / 128)].  Any cols >= 1, fewer than 2^28 blocks. */
lmoe_status lmoe_quantize_fp8(const void *x, int32_t x_type, int64_t rows, int32_t cols,
                              int64_t x_stride, uint8_t *codes, float *scales, void *stream);

/* Weights: `matrices` matrices w [rows, cols], dense, a scale for each block
 * of 128 rows x 128 columns (smaller at the edges): codes like w, scales
 * [matrices, ceil(rows / 128), ceil(cols / 128)], fewer than 2^24 of them. */
lmoe_status lmoe_quantize_fp8_weight(const void *w, int32_t w_type, int64_t matrices, int32_t rows,
                                     int32_t cols, uint8_t *codes, float *scales, void *stream);

/* The product of such activations and weights, y [M, N] = x w^T, rounded once
 * to y_type:
 *   y[m][n] = sum_b xs[r][b] ws[n / 128][b] sum_{k in block b} x[r][k] w[n][k]
 * with r = rows[m], or m when rows is NULL.  The product of two scales is an
 * fp32 number: it must be below 2^128, and keeps fewer bits below 2^-126.  With
 * n_groups >= 1 there are that many weight matrices and row m takes matrix g of
 * the range offsets[g] <= m < offsets[g + 1] (a sparse layer's rows sorted by
 * expert; empty groups are fine); rows of no group are not written.  Offsets are cut to [0, M];
 * they must ascend.  Products whose launch would need 2^32 threads or more are
 * LMOE_ERR_UNSUPPORTED (streamed groups of K above 32768: rows / 16 * N / 64 from
 * 2^24 on).  A row index outside [0, x_rows) gives a row of zeros
 * (if row 0 of x is finite).
 *
 * Sums are fp32 where y is fp32, and where the weights are streamed (M up to 16;
 * groups of up to 4 rows on average, or with K above 32768).  Other bf16 y take the 8-bit matrix
 * instruction: the blocks of k are scaled and added in fp32, but within a block
 * the products of each eight neighbouring k are cut 13 bits below the largest
 * power of two among them before they are added.  Of the sum of the terms'
 * magnitudes that is about 2^-16 on normally distributed values, and 2^-10 was
 * measured where a few values are far larger than the rest; callers who need
 * more take an fp32 y (half the rate). */
typedef struct {
  const uint8_t *x;       /* [x_rows, K] codes, 16-byte aligned */
  const float *x_scales;  /* [x_rows, K / 128] */
  const uint8_t *w;       /* [n_groups or 1, N, K] codes, 16-byte aligned */
  const float *w_scales;  /* [n_groups or 1, ceil(N / 128), K / 128] */
  const int32_t *rows;    /* [M] or NULL (then x_rows >= M) */
  const int32_t *offsets; /* [n_groups + 1], NULL if n_groups is 0 */
  void *y;                /* [M, N], 16-byte aligned */
  int32_t y_type;         /* lmoe_dtype */
  int32_t n_groups;       /* 0 (one matrix, no groups) .. 1024 */
  int32_t M;              /* 0 .. 2^24 */
  int32_t x_rows;         /* >= 1 if M > 0; with rows, x_rows * K < 2^31 */
  int32_t N;              /* a multiple of 16, up to 2^20 */
  int32_t K;              /* a multiple of 128, up to 65536 */
} lmoe_fp8_matmul_args;

/* Bytes of workspace of lmoe_fp8_matmul (the row tiles of each group, or the
 * partial sums of a product split over k; 0 where it needs none, or for
 * arguments it refuses).  Pure host function. */
size_t lmoe_fp8_matmul_workspace_size(const lmoe_fp8_matmul_args *a);

/* workspace: 16-byte aligned device memory of that size; calls that may
 * overlap need one each. */
lmoe_status lmoe_fp8_matmul(const lmoe_fp8_matmul_args *a, void *workspace,
                            size_t workspace_bytes, void *stream);

/* ---- per-kernel timing (HIP events on the forward's stream) ------------ */

/* Number of timed stages of lmoe_forward and the name of stage i.  Stages
 * 0..7 run back to back on the forward's stream (the last one, proj_out,
 * includes the wait for the auxiliary stream; the first, proj_latent,
 * includes the pre-norm kernel when it is fused); stage 8 ("shared_up") is
 * timed on the auxiliary stream and overlaps the stages before proj_out.
 * For T <= 64 (weight-streaming projections) stage 8 also runs the shared
 * expert's down projection and proj_out covers fc2_latent only, adding the
 * shared output before its single rounding. */
int32_t lmoe_num_stages(void);
const char *lmoe_stage_name(int32_t i);

/* Start timing: the next up to `max_forwards` calls of lmoe_forward record
 * a HIP event before and after each stage (events are created here; a
 * hipEventCreate failure returns LMOE_ERR_HIP).  max_forwards <= 4096. */
lmoe_status lmoe_profile_begin(lmoe_handle *h, int32_t max_forwards);

/* Stop timing: wait for the recorded events, write the summed milliseconds
 * of each stage over the recorded forwards into ms[0..n_stages) and the
 * number of recorded forwards into *n_forwards; destroy the events. */
lmoe_status lmoe_profile_end(lmoe_handle *h, float *ms, int32_t n_stages, int32_t *n_forwards);

#ifdef __cplusplus
}
#endif

#endif /* LMOE_H */
