/*
 * beam_moe.h -- C ABI of the MI355X (gfx950) Beam MoE block library.
 *
 * One forward pass of the Mixture-of-Experts block of the Beam model:
 *   router    sigmoid scores over E experts in G contiguous groups, a
 *             per-expert bias that steers selection only, group score = sum
 *             of the group's best two biased scores, keep the best TG
 *             groups, pick the top K experts inside them, normalise the K
 *             unbiased scores to sum 1 and multiply by the routed scale;
 *   experts   K SwiGLU MLPs per token: h = silu(x W_g^T) * (x W_u^T),
 *             y = h W_d^T, no shared expert;
 *   combine   out = sum_k w_k y_k in rank order.
 * Sources: "Hugging Face releases Beam, a 501B-parameter open
 * Mixture-of-Experts model with 1M-token context" (MoE paragraph: 256
 * experts, SwiGLU intermediate 2,560, top 8 of the top 4 of 8 groups of 32);
 * "Reflection Releases Beam: An Open 501B-Parameter MoE Model Under Apache
 * 2.0", section "Where Beam Saves and Where the Memory Bill Comes In" (no
 * shared expert, DeepSeek-V3 group-limited sigmoid router, weights
 * normalised and scaled by 2.5); "Reflection AI Introduces Beam ..." (load
 * balancing by a DeepSeek-V3-style expert bias).  The group-score rule is
 * DeepSeek-V3's (arXiv 2412.19437, section 2.1.2); the pages invoke that
 * scheme without spelling the rule out.
 *
 * Around the block: the gradient of the routing, dense e4m3 products with their
 * quantiser, the step between two blocks with its gradients, the norms and
 * rotation of attention heads with their gradients, attention of new tokens over
 * a paged cache, the cache's page tables, and the scores of tokens with their
 * gradient.
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are device memory owned by the caller.  The
 *     library allocates nothing, frees nothing and keeps no pointer after a
 *     call returns.  Scratch memory is the caller's workspace, sized by
 *     beam_moe_workspace_bytes().
 *   - All work is enqueued on `stream` (a hipStream_t passed as void*; NULL
 *     is the default stream) and is asynchronous: the call returns once the
 *     kernels are launched.  Errors inside kernels surface at the caller's
 *     next synchronisation.
 *   - Argument, shape and workspace errors are detected on the host before
 *     anything is launched (no partial work) and returned as a negative
 *     beam_status.  No exceptions cross the ABI.  T == 0 is a no-op.
 *   - Device pointers must be 16-byte aligned; the workspace 256-byte aligned.
 *   - Layouts are row-major.  Weights use the out x in ("nn.Linear") layout.
 *   - Identical inputs give bitwise identical outputs (no floating-point
 *     atomics).  Calls are reentrant given distinct workspaces.
 *   - Inputs containing NaN or Inf are outside the contract, but where an
 *     entry point says what they give.
 */
#ifndef BEAM_MOE_H
#define BEAM_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BEAM_OK = 0,
  BEAM_ERR_INVALID_ARG = -1, /* null pointer, misalignment, T < 0, bad enum */
  BEAM_ERR_UNSUPPORTED = -2, /* a shape or dtype combination not built here */
  BEAM_ERR_WORKSPACE = -3,   /* workspace missing or smaller than required */
  BEAM_ERR_HIP = -4          /* a HIP launch or runtime call failed */
} beam_status;

typedef enum {
  BEAM_F32 = 0,      /* IEEE binary32 */
  BEAM_BF16 = 1,     /* bfloat16 */
  BEAM_FP8_E4M3 = 2, /* OCP e4m3fn codes with per-128x128-block fp32 scales */
  BEAM_MXFP4 = 3     /* OCP MX FP4: E2M1 codes two per byte (even k in the low
                        nibble), one E8M0 scale byte per 32 k of a row */
} beam_dtype;

/* flags */
#define BEAM_ROUTE_LOGITS_IN (1u << 0) /* route from caller-supplied fp32 logits */
/* Expert path (default: bf16 streams its weights below T*K = E/2 and uses
 * grouped tiles above; MXFP4 and FP8 use grouped tiles; fp32 has one path).
 * Tile height of the grouped path (default: bf16 128 rows below T*K = 96E,
 * 256 above, 160 only on request; MXFP4 64 below 56E when H and I are multiples
 * of 512, else 128 below 32E, 256 above; FP8 128 below 120E, 256 above, an
 * expert's last tile holding up to 288).  Every tile
 * height gives bit-identical outputs; the two paths agree within the layer
 * tolerance (they sum in different orders, and bf16 streaming keeps y in
 * fp32).  The flags exist for measurement and tests; at most one of the
 * BEAM_TILE_* flags, and not both path flags (else BEAM_ERR_INVALID_ARG). */
#define BEAM_PATH_STREAM (1u << 1)     /* force the weight-streaming expert path (bf16, MXFP4) */
#define BEAM_PATH_GROUPED (1u << 2)    /* force the tiled grouped-GEMM expert path */
#define BEAM_TILE_128 (1u << 3)        /* grouped path: force 128-row M tiles */
#define BEAM_TILE_256 (1u << 4)        /* grouped path: force 256-row M tiles (FP8: no 32-row
                                          extension of an expert's last tile) */
#define BEAM_TILE_160 (1u << 5)        /* bf16 grouped path: force 160-row M tiles (MXFP4 and
                                          FP8: the 256-row form) */
#define BEAM_TILE_64 (1u << 6)         /* MXFP4 grouped path: force 64-slot tiles (bf16 and
                                          FP8: the 128-row form) */
/* Router scores and weights (default: sigmoid scores, weights normalised to
 * sum routed_scale).  Both flags work wherever a descriptor routes. */
#define BEAM_ROUTE_SOFTMAX (1u << 7)   /* scores are the softmax over the E logits */
#define BEAM_ROUTE_UNNORMED (1u << 8)  /* weights are score * routed_scale, not normalised */

typedef struct {
  int32_t hidden;           /* H: 5120 for Beam */
  int32_t intermediate;     /* I: 2560 */
  int32_t n_experts;        /* E: 256 */
  int32_t n_groups;         /* G: 8; group g = experts [g*E/G, (g+1)*E/G) */
  int32_t topk_groups;      /* TG: 4 */
  int32_t top_k;            /* K: 8 */
  int32_t group_score_topn; /* 1 or 2 best biased scores summed per group: 2 */
  float routed_scale;       /* 2.5 */
  int32_t act_dtype;        /* dtype of x and out: BEAM_F32 or BEAM_BF16 */
  int32_t weight_dtype;     /* BEAM_F32 (needs act F32), BEAM_BF16, BEAM_FP8_E4M3, BEAM_MXFP4 */
  uint32_t flags;           /* BEAM_* flags above */
} beam_moe_desc;

/* Text for a beam_status value.  Never NULL; static storage. */
const char* beam_status_string(int status);

/* Host-only check of a descriptor and token count: makes no HIP call.
 * Supported: 1 <= E <= 1024, E % G == 0, E/G <= 64, 1 <= TG <= G,
 * 1 <= K <= min(16, TG*E/G), group_score_topn in {1,2} and <= E/G,
 * H % 128 == 0 and I % 128 == 0, routed_scale finite and > 0, T >= 0,
 * T*K*max(H, I) < 2^31 (52,428 tokens for the Beam layer), 2*I*H < 2^31
 * (one expert's gate/up matrix is addressed with 32-bit offsets).  Returns
 * BEAM_OK or the first error found.  beam_moe_route with BEAM_ROUTE_LOGITS_IN
 * and beam_moe_route_backward hold no slots: they take T up to 67,108,860
 * whatever H and I are. */
int beam_moe_validate(const beam_moe_desc* desc, int64_t T);

/* Bytes of workspace beam_moe_forward / beam_moe_route need for T tokens.
 * Writes 0 for T == 0.  Returns beam_moe_validate's status. */
int beam_moe_workspace_bytes(const beam_moe_desc* desc, int64_t T,
                             size_t* bytes);

/* Router only (the steps before the experts): logits x W_r^T, sigmoid
 * scores, the selection bias, group scores, the kept groups, the top K and
 * the normalised, scaled weights.  "Hugging Face releases Beam ..." (MoE
 * paragraph: 8 groups of 32 experts, best 4 groups, top 8); "Reflection
 * Releases Beam ...", section "Where Beam Saves and Where the Memory Bill
 * Comes In" (DeepSeek-V3 group-limited sigmoid router, weights normalised
 * and scaled by 2.5); "Reflection AI Introduces Beam ..." (load-balancing
 * paragraph: the bias steers selection only).
 *   x         device [T, H] act_dtype; unused with BEAM_ROUTE_LOGITS_IN
 *   w_router  device [E, H] fp32; unused with BEAM_ROUTE_LOGITS_IN
 *   bias      device [E] fp32 selection bias, or NULL for zero
 *   logits    device [T, E] fp32: written with the router logits, or read
 *             with BEAM_ROUTE_LOGITS_IN; may be NULL without that flag
 *   topk_idx  device [T, K] int32: expert ids in rank order
 *   topk_w    device [T, K] fp32: routing weights (sum to routed_scale)
 * Given identical fp32 logits the indices and weights are bitwise identical
 * to the routing specification: sigmoid rounded from a fixed binary64
 * evaluation, binary32 sums, ties broken towards the lower index.
 * With BEAM_ROUTE_SOFTMAX the scores are s_e = exp(l_e - max l) / sum exp(l_j
 * - max l) over all E logits, evaluated in binary64 and rounded once to
 * binary32; a logit of -infinity gives the score 0, a row of only those has
 * scores 0, and a NaN or +infinity makes its row's scores and weights NaN (and
 * its chosen experts' gradients), the K experts still different ones.  With BEAM_ROUTE_UNNORMED the weights
 * are s_k * routed_scale.
 * Where the K chosen scores are all 0 (logits so low that binary32 holds no
 * smaller score, or masked ones) the weights are 0.  Keeping every group
 * (topk_groups = n_groups) is plain top-K over the experts. */
int beam_moe_route(const beam_moe_desc* desc, int64_t T, const void* x,
                   const float* w_router, const float* bias, float* logits,
                   int32_t* topk_idx, float* topk_w, void* workspace,
                   size_t ws_bytes, void* stream);

/* Gradient of the routing weights in the logits (the training step's way
 * back through beam_moe_route).  The selection and its bias are constants;
 * with D the sum of the K chosen scores, c = sum_k d_topk_w_k s_k:
 *   sigmoid             d l_k = scale (dw_k - c / D) s_k (1 - s_k) / D
 *   sigmoid, unnormed   d l_k = scale dw_k s_k (1 - s_k)
 *   softmax             d l_k = scale (s_k / D) (dw_k - c / D)
 *   softmax, unnormed   d l_e = scale s_e ([e chosen] dw_e - c), every expert
 * and 0 for the experts not named (in all but the last form).  Scores are
 * recomputed in binary32; a row whose chosen scores are all 0 has gradient 0.
 *   logits    device [T, E] fp32: those the routing was made from
 *   topk_idx  device [T, K] int32; an id outside [0, E) adds nothing, an id
 *             named twice counts as two choices
 *   d_topk_w  device [T, K] fp32: gradient of the weights
 *   d_logits  device [T, E] fp32: output, every element written
 * Follows desc's BEAM_ROUTE_SOFTMAX and BEAM_ROUTE_UNNORMED.  The gradients
 * of x and w_router are the plain products d_logits W_r and d_logits^T x.
 * No workspace. */
int beam_moe_route_backward(const beam_moe_desc* desc, int64_t T, const float* logits,
                            const int32_t* topk_idx, const float* d_topk_w,
                            float* d_logits, void* stream);

/* Token permutation for a given routing (the dispatch between router and
 * experts): a stable counting sort of the T*K assignments by expert.  The
 * pages route each token to 8 of 256 experts ("Hugging Face releases Beam
 * ...", MoE paragraph) and leave the dispatch to the implementation ("Beam
 * Turns Frontier-Scale Openness Into an Infrastructure Decision", section
 * "Sparse compute still requires dense planning": each token's rows have to
 * reach the experts it selected, which this grouping by expert provides).
 *   topk_idx    device [T, K] int32, each row K distinct ids in [0, E)
 *   counts      device [E] int32: assignments per expert
 *   offsets     device [E+1] int32: exclusive prefix sum of counts
 *   slot_token  device [T*K] int32: token of each slot; the slots of expert
 *               e are [offsets[e], offsets[e+1]) in increasing token order
 *   slot_of     device [T*K] int32: slot of assignment (t, k)
 * Uses the workspace (beam_moe_workspace_bytes). */
int beam_moe_permute(const beam_moe_desc* desc, int64_t T,
                     const int32_t* topk_idx, int32_t* counts, int32_t* offsets,
                     int32_t* slot_token, int32_t* slot_of, void* workspace,
                     size_t ws_bytes, void* stream);

/* Per-row, per-128-column dynamic e4m3 quantisation (the FP8 variant's
 * activation recipe): for each block, scale = amax / 448 in binary32 (1 for
 * an all-zero block), code = e4m3(v / scale) with a binary32 division,
 * round to nearest even, saturating to +-448.
 *   v       device [rows, cols] in `dtype` (BEAM_F32 or BEAM_BF16)
 *   q       device [rows, cols] uint8 codes
 *   scales  device [rows, cols/128] fp32
 * cols % 128 == 0.  No workspace. */
int beam_moe_quant_e4m3(int64_t rows, int64_t cols, int32_t dtype,
                        const void* v, uint8_t* q, float* scales, void* stream);

/* Per-row MXFP8 quantisation (the MXFP4 variant's activation recipe, OCP
 * Microscaling layout): for each block of 32 columns, x = the smallest
 * integer with amax / 2^x <= 448, clamped to [-127, 127] (-127 for an
 * all-zero block), code = e4m3(v * 2^-x) (exact scaling, round to nearest
 * even), scale byte x + 127.  (OCP's own rule, floor(log2(amax)) - 8, can
 * saturate the block maximum; this one never does.)
 *   v       device [rows, cols] in `dtype` (BEAM_F32 or BEAM_BF16)
 *   q       device [rows, cols] uint8 codes
 *   scales  device [rows, cols/32] uint8 E8M0
 * cols % 128 == 0.  No workspace. */
int beam_moe_quant_mxfp8(int64_t rows, int64_t cols, int32_t dtype,
                         const void* v, uint8_t* q, uint8_t* scales, void* stream);

/* The whole block: router, K SwiGLU experts per token and the weighted
 * combine ("Hugging Face releases Beam ...", MoE paragraph: SwiGLU
 * intermediate 2,560 on hidden 5,120; "Reflection Releases Beam ...",
 * section "Where Beam Saves and Where the Memory Bill Comes In": no shared
 * expert; "Reflection Beam", section "Where to run it", and the checkpoint
 * paragraph of "Hugging Face releases Beam ...": the FP8 and 4-bit
 * checkpoint forms).
 *   x          device [T, H] act_dtype
 *   w_router   device [E, H] fp32 (unused with BEAM_ROUTE_LOGITS_IN)
 *   bias       device [E] fp32 or NULL
 *   w_gate_up  device [E, 2I, H] weight_dtype: rows 0..I-1 gate, I..2I-1 up
 *              (MXFP4: [E, 2I, H/2] bytes)
 *   s_gate_up  device block scales, NULL for f32/bf16 weights: FP8 fp32
 *              [E, 2I/128, H/128], positive; MXFP4 E8M0 bytes [E, 2I, H/32]
 *   w_down     device [E, H, I] weight_dtype (MXFP4: [E, H, I/2] bytes)
 *   s_down     as s_gate_up: FP8 fp32 [E, H/128, I/128]; MXFP4 bytes [E, H, I/32]
 *   out        device [T, H] act_dtype
 *   topk_idx, topk_w  device [T, K] outputs of the router, or NULL
 *   logits     device [T, E] fp32: output, or input with BEAM_ROUTE_LOGITS_IN;
 *              may be NULL without that flag
 * FP8 weights also quantise x and h per token per 128 channels
 * (beam_moe_quant_e4m3's recipe) and run e4m3 matrix products with binary32
 * accumulation and block scales applied per 128-deep slice.  MXFP4 weights
 * quantise x and h to MXFP8 (beam_moe_quant_mxfp8's recipe) and run E2M1 x
 * E4M3 matrix products whose E8M0 block scales the matrix cores apply, with
 * binary32 accumulation. */
int beam_moe_forward(const beam_moe_desc* desc, int64_t T, const void* x,
                     const float* w_router, const float* bias,
                     const void* w_gate_up, const void* s_gate_up,
                     const void* w_down, const void* s_down, void* out,
                     int32_t* topk_idx, float* topk_w, float* logits,
                     void* workspace, size_t ws_bytes, void* stream);

/* beam_moe_forward for callers that cannot allocate device memory or pass a
 * workspace: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc.  The workspace is instead a device array inside the
 * library, BEAM_NOALLOC_SCRATCH_BYTES bytes, of which every GPU the library
 * runs on holds its own copy until the process ends (looked up once per
 * device, on the first call with that device current).  The call allocates
 * nothing and makes no hipMalloc/hipFree.
 *   Arguments as beam_moe_forward without workspace and ws_bytes; `stream`
 *   must belong to the current device.
 *   BEAM_ERR_WORKSPACE when beam_moe_workspace_bytes(desc, T) exceeds
 *   BEAM_NOALLOC_SCRATCH_BYTES (64 MiB: bf16 Beam-layer batches up to about
 *   500 tokens, FP8 about 580, MXFP4 about 320); nothing is launched then.
 * All calls on one GPU share its array: calls that may overlap on one GPU
 * (on different streams, or from different host threads without ordering)
 * race and give undefined results.  Nothing in the array needs to start
 * cleared: every call writes what it reads.  Results are bitwise identical
 * to beam_moe_forward's. */
#define BEAM_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int beam_moe_forward_noalloc(const beam_moe_desc* desc, int64_t T, const void* x,
                             const float* w_router, const float* bias,
                             const void* w_gate_up, const void* s_gate_up,
                             const void* w_down, const void* s_down, void* out,
                             int32_t* topk_idx, float* topk_w, float* logits,
                             void* stream);

/* beam_moe_forward followed, in the same combine kernel, by the step after
 * the block in a Beam layer stack: the post-sublayer RMSNorm of SandwichNorm
 * and the depth-scaled FP32 residual stream ("Reflection Beam", section
 * "Hybrid Attention and Unusual Residuals": at step k the stream is scaled
 * by sqrt((k-1)/k) and the sublayer output added with weight 1/sqrt(k);
 * SandwichNorm and FP32 residual accumulation from the pretraining paragraph
 * of "Reflection AI Introduces Beam ...").  Per token t, with o the fp32
 * block output before any rounding:
 *   residual[t] = sqrt((k-1)/k) * residual[t]
 *               + (1/sqrt(k)) * o / sqrt(mean(o^2) + eps) * norm_weight
 *   norm_weight  device [H] fp32 (the norm's weights; the pages give none)
 *   eps          >= 0 and finite (not on the pages; 1e-6 is usual)
 *   step         k >= 1 (k = 1 discards the incoming residual)
 *   residual     device [T, H] fp32, read and written in place
 *   out          device [T, H] act_dtype block output, or NULL to skip it
 * Other arguments as beam_moe_forward (routing outputs are not returned).
 * Requires H <= 16384 (the token's fp32 row is held in 64 KiB of LDS;
 * BEAM_ERR_UNSUPPORTED otherwise). */
int beam_moe_forward_residual(const beam_moe_desc* desc, int64_t T, const void* x,
                              const float* w_router, const float* bias,
                              const void* w_gate_up, const void* s_gate_up,
                              const void* w_down, const void* s_down,
                              const float* norm_weight, float eps, int32_t step,
                              float* residual, void* out, void* workspace,
                              size_t ws_bytes, void* stream);

/* ---- dense e4m3 products ---------------------------------------------------
 * y[m,n] = sum_kb sa[m,kb] * sb[.,kb] * sum_{k in block kb} a[m,k] * b[n,k],
 * blocks of 128 along k: the product of beam_moe_quant_e4m3's codes (or
 * beam_moe_norm_residual's) with weights of the FP8 form, for the dense layers
 * around the expert block.  Block sums on the matrix cores, one binary32
 * multiply-add a block with its scales, one rounding to dtype.  With BEAM_F32
 * products and sums are binary32 throughout; with BEAM_BF16 the e4m3 matrix
 * instructions sum, which cut products at 2^-13 of the largest of eight
 * neighbours (1.5e-5 of a result of normal data, against bf16's 2e-3).
 *   a   device [M, K] uint8 e4m3fn codes
 *   sa  device fp32: the scale of row m, block kb at sa[m * sa_row + kb *
 *       sa_block] (beam_moe_quant_e4m3 writes rows: K/128 and 1;
 *       beam_moe_quant_e4m3_2d blocks: 1 and M)
 *   b   device [N, K] uint8 e4m3fn codes (weights out x in)
 *   sb  device fp32: with b_rows 0 a scale for each 128 x 128 block, that of
 *       rows 128 i .. at sb[i * sb_row + kb * sb_block]; with b_rows 1 one for
 *       each row of b, as sa
 *   y   device [M, N] dtype (BEAM_F32 or BEAM_BF16)
 * K % 128 == 0, K <= 2^22, M, N < 2^23 - 127, M * N <= 2^38
 * (BEAM_ERR_UNSUPPORTED otherwise).
 * The two scales of a block are multiplied in binary32 before they meet its
 * sum, so their product has to be 0 or of a size from 2^-126 to below 2^128
 * (smaller ones lose bits, larger ones give infinities and NaN).
 * K == 0 gives zeros.  A NaN code (0x7F, 0xFF) makes its row's or column's
 * results NaN.
 * A linear layer's training step is three of them on what
 * beam_moe_quant_e4m3_2d makes of x [M,K], dy [M,N] and w [N,K]:
 *   y = x w^T    rows of x, blocks of w (straight)
 *   dx = dy w    rows of dy, blocks of w (transposed)
 *   dw = dy^T x  columns of dy, columns of x (both transposed, b_rows 1) */
int beam_moe_matmul_e4m3(int64_t M, int64_t N, int64_t K, const uint8_t* a, const float* sa,
                         int64_t sa_row, int64_t sa_block, const uint8_t* b, const float* sb,
                         int64_t sb_row, int64_t sb_block, int32_t b_rows, int32_t dtype, void* y,
                         void* stream);

/* e4m3 quantisation of a matrix for products along its columns and along its
 * rows, in one reading of it (scale = amax / 448 in binary32, 1 where that is
 * 0; code = e4m3(v / scale), as beam_moe_quant_e4m3).  With R = 128
 * ceil(rows/128) and C = 128 ceil(cols/128), and zeros past the end of v:
 *   v   device [rows, cols] dtype (BEAM_F32 or BEAM_BF16)
 *   q   device [rows, C] uint8 codes, or NULL
 *   s   device fp32, with q: [C/128, rows] with block 0 (a scale for 128
 *       columns of a row, block-major), [R/128, C/128] with block 1 (for 128 x
 *       128 values)
 *   qt  device [cols, R] uint8 codes of v transposed, or NULL (not both)
 *   st  device fp32, with qt: [R/128, cols] with block 0 (a scale for 128 rows
 *       of a column, block-major), [C/128, R/128] with block 1
 * A NaN or an infinity makes codes or a scale that give NaN in every product
 * its block is part of.  At most 2^23 - 1 tiles of 128 x 128
 * (BEAM_ERR_UNSUPPORTED otherwise).  No workspace. */
int beam_moe_quant_e4m3_2d(int64_t rows, int64_t cols, int32_t dtype, int32_t block,
                           const void* v, uint8_t* q, float* s, uint8_t* qt, float* st,
                           void* stream);

/* ---- the step between two blocks -----------------------------------------
 * The norm after a block, its gate, the scaled residual stream and the norm
 * before the next block, per token t:
 *   y  = o / sqrt(mean(o^2) + eps) * post_weight
 *   r' = alpha * residual + beta * sigmoid(gate) * y
 *   x  = r' / sqrt(mean(r'^2) + eps) * pre_weight
 * beam_moe_forward_residual is this step's first half for the block's own
 * output inside its combine; here o is any sublayer's output and the step
 * ends with the next sublayer's input.  Beam's stream at step k has alpha =
 * sqrt((k-1)/k), beta = 1/sqrt(k).
 *   o             device [T, H] dtype, or NULL: r' = residual, post_weight,
 *                 gate, residual_out, alpha and beta are not used
 *   post_weight   device [H] fp32
 *   gate          device [T, gate_cols] dtype before the sigmoid, or NULL with
 *                 gate_cols 0; gate_cols 1 (one gate a token) or H
 *   pre_weight    device [H] fp32, or NULL: x and its codes are not made
 *   residual      device [T, H] fp32
 *   residual_out  device [T, H] fp32: r'; may be residual itself
 *   x             device [T, H] dtype, or NULL
 *   x_codes       device [T, H] uint8, or NULL: x quantised by the recipe of
 *                 beam_moe_quant_e4m3, from x before any rounding
 *   x_scales      device [T, H/128] fp32, with x_codes
 * dtype BEAM_F32 or BEAM_BF16; 1 <= H <= 16384, with x_codes H % 128 == 0
 * (BEAM_ERR_UNSUPPORTED otherwise, and for more tokens than a launch holds:
 * at least 4,194,303, 67 million at H = 128); eps > 0, alpha and beta finite.  A token's
 * sums of squares must be finite in binary32.  No workspace. */
int beam_moe_norm_residual(int64_t T, int64_t H, int32_t dtype, const void* o,
                           const float* post_weight, const void* gate, int64_t gate_cols,
                           const float* pre_weight, float eps, float alpha, float beta,
                           const float* residual, float* residual_out, void* x,
                           uint8_t* x_codes, float* x_scales, void* stream);

/* Bytes of workspace beam_moe_norm_residual_backward needs (0 for T == 0). */
int beam_moe_norm_residual_workspace_bytes(int64_t T, int64_t H, size_t* bytes);

/* Gradients of beam_moe_norm_residual.
 *   residual_out     device [T, H] fp32: the forward's r' (residual where o is
 *                    NULL)
 *   d_residual_out   device [T, H] fp32: gradient of r' from later steps, or
 *                    NULL for zero
 *   d_x              device [T, H] dtype: gradient of x, or NULL with o
 *                    (pre_weight and d_pre_weight are then not used)
 *   d_residual       device [T, H] fp32: output; may be d_residual_out itself
 *   d_o              device [T, H] dtype: output, with o
 *   d_gate           device [T, gate_cols] dtype: output, with gate
 *   d_pre_weight, d_post_weight  device [H] fp32: outputs (sums over the
 *                    tokens, 0 for T == 0), with d_x and with o
 * Other arguments as in the forward.  Identical inputs give bitwise identical
 * outputs. */
int beam_moe_norm_residual_backward(int64_t T, int64_t H, int32_t dtype, const void* o,
                                    const float* post_weight, const void* gate,
                                    int64_t gate_cols, const float* pre_weight, float eps,
                                    float alpha, float beta, const float* residual_out,
                                    const float* d_residual_out, const void* d_x,
                                    float* d_residual, void* d_o, void* d_gate,
                                    float* d_pre_weight, float* d_post_weight,
                                    void* workspace, size_t ws_bytes, void* stream);

/* ---- attention around a paged key-value cache -------------------------------
 * A cache is two arrays of pages, keys and values, each page holding page_size
 * tokens (a power of two) of Hkv heads of D values: value d of head h of token
 * j of page p lies at p * page_stride + j * token_stride + h * head_stride + d,
 * the same strides (in elements, multiples of 8; 4 with BEAM_F32) in both.
 * tables [seqs, table_cols] int32 name the pages of each sequence in order:
 * token i of sequence s lies in page tables[s, i / page_size] at i % page_size.
 * An id outside [0, pages) names no page: nothing is written there, and its
 * tokens take no part in attention.
 * D is a multiple of 8 from 8 to 256, token_stride < 2^25. */

/* Norms of query and key heads and their rotation by position, in one pass,
 * and the keys' and values' way into a paged cache ("Hugging Face releases
 * Beam ..."; "Reflection Releases Beam ...", section "Hybrid Attention and
 * Unusual Residuals": RMSNorm on queries and keys, rotation in the sliding-window
 * layers, none in the global ones, whose queries are scaled by
 * (1 + (pos + 1) / 2048)^0.1).  Per head x of D values of token t:
 *   n = x / sqrt(mean(x^2) + eps) * weight
 *   the pair (n_a, n_b) turned by the angle positions[t] * inv_freq[i], for
 *   i < rot / 2: (a, b) = (i, i + rot / 2), with interleaved (2i, 2i + 1)
 *   queries times (1 + (positions[t] + 1) / temp_length)^temp_exponent
 *   q, k, v     device [T, heads, D] dtype, heads and values contiguous, tokens
 *               q_stride, k_stride, v_stride elements apart (views of one
 *               projection's output; multiples of 8, 4 with BEAM_F32); v only
 *               with a cache
 *   q_weight, k_weight  device [D] fp32
 *   positions   device [T] int32; NULL only with rot 0, temp_length 0 and no cache
 *   inv_freq    device [rot / 2] binary64, radians a position; angles are
 *               reduced in binary64.  rot: 0 or a multiple of 16 up to D
 *   temp_length 0: no temperature; else > 0, positions > -1 - temp_length
 *   q_out       device [T, Hq, D] dtype
 *   k_out       device [T, Hkv, D] dtype, or NULL (with a cache)
 *   k_cache, v_cache  a cache, or both NULL: token t's key (as k_out) and value
 *               go to place positions[t] of sequence rows[t] (rows NULL: of
 *               sequence t).  A token whose position is negative or past the
 *               table, or whose row is outside [0, seqs), is not written.  No two
 *               tokens may name one place.
 * Squares are binary32: a head whose sum of them passes its range gives zeros and no
 * gradients (NaN where a weighted value passes the range as well).
 * Outputs do not overlap inputs.  T * (Hq + 2 Hkv) < 2^31, Hq, Hkv <= 4096, eps >=
 * 2^-126.
 * No workspace. */
int beam_moe_qk_norm_rope(int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype,
                          const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const float* q_weight,
                          const float* k_weight, float eps, const int32_t* positions,
                          const double* inv_freq, int32_t rot, int32_t interleaved,
                          float temp_length, float temp_exponent, void* q_out, void* k_out,
                          void* k_cache, void* v_cache, int64_t page_stride, int64_t token_stride,
                          int64_t head_stride, int64_t pages, int64_t page_size,
                          const int32_t* tables, int64_t seqs, int64_t table_cols,
                          const int32_t* rows, void* stream);

/* Bytes of workspace beam_moe_qk_norm_rope_backward needs (0 for T == 0). */
int beam_moe_qk_norm_rope_workspace_bytes(int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
                                          size_t* bytes);

/* Gradients of beam_moe_qk_norm_rope's q_out and k_out.
 *   d_q_out, d_k_out  device [T, heads, D] dtype, contiguous
 *   d_q, d_k          device [T, heads, D] dtype: outputs, contiguous
 *   d_q_weight, d_k_weight  device [D] fp32: outputs (sums over tokens and heads,
 *                     0 for T == 0)
 * Other arguments as in the forward.  Identical inputs give bitwise identical
 * outputs. */
int beam_moe_qk_norm_rope_backward(int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype,
                                   const void* d_q_out, const void* d_k_out, const void* q,
                                   int64_t q_stride, const void* k, int64_t k_stride,
                                   const float* q_weight, const float* k_weight, float eps,
                                   const int32_t* positions, const double* inv_freq, int32_t rot,
                                   int32_t interleaved, float temp_length, float temp_exponent,
                                   void* d_q, void* d_k, float* d_q_weight, float* d_k_weight,
                                   void* workspace, size_t ws_bytes, void* stream);

/* Bytes of workspace beam_moe_paged_attention needs (0 for seqs == 0). */
int beam_moe_paged_attention_workspace_bytes(int64_t seqs, int32_t Hq, int32_t Hkv, int32_t D,
                                             size_t* bytes);

/* Attention of one new token of every sequence over its cached tokens, the new
 * one's own key and value among them (beam_moe_qk_norm_rope has put them there):
 *   out = softmax(scale q k^T) v [* sigmoid(gate)]
 * over the last `window` of lengths[s] tokens (window 0: all), query head h
 * reading key-value head h / (Hq / Hkv) ("Reflection Releases Beam ...", section
 * "Hybrid Attention and Unusual Residuals": a window of 512 or the whole context, 48
 * query and 8 key-value heads, a sigmoid gate for each head's channels).
 *   q        device [seqs, Hq, D] dtype, contiguous
 *   gate     device [seqs, Hq, D] dtype, contiguous, before the sigmoid, or NULL
 *   lengths  device [seqs] int32: tokens held, the new one among them; a length
 *            past the table counts as the table's, a negative one as 0
 *   out      device [seqs, Hq, D] dtype
 *   lse      device [seqs, Hq] fp32, or NULL: ln sum exp(scale q k^T)
 * A sequence without tokens that take part (length 0, or no page) gives zeros
 * and an lse of -infinity.  What pages hold behind a sequence's length or before
 * its window is not read.  Sums and softmax statistics are binary32, and so are
 * the products with the values; one rounding to dtype.
 * 0 < scale <= 2^127, Hq % Hkv == 0, seqs * Hq < 2^24, table_cols * page_size <=
 * 2^31 - 2^16, seqs times that < 2^36.  Identical inputs give bitwise identical outputs. */
int beam_moe_paged_attention(int64_t seqs, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype,
                             const void* q, const void* gate, const void* k_cache,
                             const void* v_cache, int64_t page_stride, int64_t token_stride,
                             int64_t head_stride, int64_t pages, int64_t page_size,
                             const int32_t* tables, int64_t table_cols, const int32_t* lengths,
                             float scale, int64_t window, void* out, float* lse, void* workspace,
                             size_t ws_bytes, void* stream);

/* The arrays whose pages beam_moe_pages_* copy, up to 8 of them: page p of layer
 * l of array i is `bytes[i]` bytes at base[i] + l * layer_stride[i] + p *
 * page_stride[i] (bytes, multiples of 16), layers <= 65536. */
typedef struct {
  int32_t count;
  int32_t layers;
  void* base[8];
  int64_t bytes[8];
  int64_t layer_stride[8];
  int64_t page_stride[8];
} beam_moe_pools;

/* Copies page src[i] to page dst[i] in every layer of every array, i < n.
 *   src, dst  device [n] int32; a pair with an id outside [0, pages) is left
 *             out.  No page is written twice, none that is written is read.
 * No workspace. */
int beam_moe_pages_copy(const beam_moe_pools* pools, int64_t pages, int64_t n, const int32_t* src,
                        const int32_t* dst, void* stream);

/* Bytes of workspace beam_moe_pages_update and _compact need for a pool of
 * `pages` pages and `rows` rows (of the new batch; any for _compact). */
int beam_moe_pages_workspace_bytes(int64_t pages, int64_t rows, size_t* bytes);

/* The step of a batch's page tables between two decode steps: row i of the new
 * batch goes on from row parents[i] of the old one, or starts anew, and gets
 * room for grow[i] more tokens.  Pages are shared by counting references;
 * a shared last page is copied before its row may write to it; old rows that
 * nobody goes on from give their references up.
 *   tables    device [old_rows, cols] int32; of row s the first ceil(lengths[s] /
 *             page_size) entries count (lengths held to [0, cols * page_size])
 *   lengths   device [old_rows] int32: tokens held
 *   refs      device [pages] int32: references to each page, those of this
 *             batch's rows among them; a page with 0 or fewer is free
 *   parents   device [rows] int32, an id outside [0, old_rows) starts a new
 *             sequence; or NULL: rows == old_rows, each goes on from itself
 *   grow      device [rows] int32 (negative: 0), or NULL: 0 for all
 *   tables_out, lengths_out, refs_out  device [rows, cols], [rows], [pages]
 *             int32: outputs that overlap no input; entries of a table behind its
 *             last page are -1; lengths_out = held + grow, at most cols * page_size
 *   missing   device [1] int32: pages that rows wanted and did not get, for want
 *             of free pages (their entries are -1) or of columns (held to 2^31 - 1)
 * References are first counted for the new rows' held pages.  A page that is the
 * unfilled last page of a row that grows is left to that row if nothing else
 * refers to it, and to the lowest of them if only such rows do; every other such
 * row gets a copy.  Rows in order want a page for their copy, then their new
 * ones in order, and get the free pages in order of their ids, each with one
 * reference.  pools' pages are copied in the same call (count 0: none).
 * Nothing but integers decides anything, and no order of execution.
 * rows, old_rows <= 65536, pages < 2^24, rows * cols and old_rows * cols < 2^31,
 * page_size a power of two, cols * page_size < 2^31. */
int beam_moe_pages_update(int64_t old_rows, int64_t rows, int64_t cols, int64_t pages,
                          int64_t page_size, const int32_t* tables, const int32_t* lengths,
                          const int32_t* refs, const int32_t* parents, const int32_t* grow,
                          int32_t* tables_out, int32_t* lengths_out, int32_t* refs_out,
                          int32_t* missing, const beam_moe_pools* pools, void* workspace,
                          size_t ws_bytes, void* stream);

/* Packs the used pages of a pool to its front: with n used pages, those with
 * ids from n up move, in order of their ids, into the free ones below n, in order.
 *   refs        device [pages] int32 as above
 *   tables, lengths  as above; tables_out device [rows, cols]: the new ids, -1
 *               behind a row's last page and for an id outside [0, pages) or of
 *               a free page; may be tables itself
 *   refs_out    device [pages] int32, not refs itself
 *   new_id      device [pages] int32: where each page is now, -1 for a free one
 *               (for tables kept elsewhere)
 *   live        device [1] int32: n
 * pools' pages are moved in the same call.  Limits as above. */
int beam_moe_pages_compact(int64_t rows, int64_t cols, int64_t pages, int64_t page_size,
                           const int32_t* tables, const int32_t* lengths, const int32_t* refs,
                           int32_t* tables_out, int32_t* refs_out, int32_t* new_id, int32_t* live,
                           const beam_moe_pools* pools, void* workspace, size_t ws_bytes,
                           void* stream);

/* ---- scores of tokens ---------------------------------------------------------
 * Bytes of workspace beam_moe_token_logprobs needs (0 for T == 0). */
int beam_moe_token_logprobs_workspace_bytes(int64_t T, int64_t V, int32_t top, size_t* bytes);

/* Log probabilities of given tokens with the entropy of the distribution and
 * its best alternatives, in one reading of the logits (with alternatives, rows with
 * few unmasked logits or hundreds of equal ones in parts up to `top` times more), per
 * row t:
 *   z = scale * softcap * tanh(l / softcap)   (softcap 0: z = scale * l)
 *   logp = z - ln sum exp(z)
 * ("Reflection Releases Beam ...", section "Hybrid Attention and Unusual
 * Residuals": logits capped by tanh at 30).
 *   logits    device [T, V] dtype, rows row_stride >= V elements apart
 *   targets   device [T] int64, or NULL; one outside [0, V) gives logprob 0
 *   logprobs  device [T] fp32, with targets: logp of the target
 *   entropy   device [T] fp32: -sum p logp
 *   lse       device [T] fp32: ln sum exp(z), held to binary32's range
 *   top_ids, top_logprobs  device [T, top] int32 and fp32, top > 0: the tokens of
 *             the highest logits in order, equal ones by their index
 * A logit of -infinity is masked: it has probability 0, logp -infinity and
 * gradient 0, also under the cap.  A row of only those has lse and logp
 * -infinity and entropy 0.  A mask of the type's lowest value is a logit like any
 * other (a row of only those is uniform, at any scale); a logp past binary32's
 * range is -infinity.  A NaN or +infinity makes its row's results NaN.
 * A capped z is off by at most 16 scale softcap 2^-24 where scale softcap is up to
 * 66, past it by 20 |z| 2^-24.
 * 0 <= top <= min(16, V); softcap >= 0, scale > 0; 3 scale, 3 scale softcap and 3 /
 * softcap in binary32's range; V <= 2^24, T < 2^23. */
int beam_moe_token_logprobs(int64_t T, int64_t V, int32_t dtype, const void* logits,
                            int64_t row_stride, const int64_t* targets, float softcap, float scale,
                            int32_t top, float* logprobs, float* entropy, float* lse,
                            int32_t* top_ids, float* top_logprobs, void* workspace,
                            size_t ws_bytes, void* stream);

/* Gradient of the logits from those of logprobs and entropy (NULL: zero; not
 * both):
 *   d l_j = z'(l_j) (d_logprob ([j = target] - p_j) - d_entropy p_j (logp_j + entropy))
 *   lse, entropy  device [T] fp32: the forward's
 *   d_logits      device [T, V] dtype, rows row_stride elements apart; may be
 *                 logits itself
 * A target outside [0, V) has no gradient of its logprob.  Probabilities come from
 * z and the binary32 lse, off by 2^-18 for its rounding; where |lse| is 128 or more,
 * from the row's largest logit and the sum beside it, formed again by one workgroup a
 * row, so that rows far from 0 have the gradients of rows near it (unless they do not
 * make the given lse, as where the row is a shard of a vocabulary and lse the whole's:
 * then p has lse's rounding).  No workspace. */
int beam_moe_token_logprobs_backward(int64_t T, int64_t V, int32_t dtype, const void* logits,
                                     int64_t row_stride, const int64_t* targets, float softcap,
                                     float scale, const float* lse, const float* entropy,
                                     const float* d_logprobs, const float* d_entropy,
                                     void* d_logits, int64_t d_row_stride, void* stream);

/* Auxiliary-loss-free load balancing step.  The load-balancing paragraph of
 * "Reflection AI Introduces Beam ..." says Beam builds on DeepSeek-V3's
 * bias-update balancing with a cosine decay of the update speed; the rule
 * (arXiv 2412.19437 section 2.1.2) moves each expert's selection bias
 * towards balance after a batch:
 *   load_e = #{(t, k) : topk_idx[t, k] == e}
 *   bias[e] = bias[e] + gamma * sign(T*K/E - load_e)
 * with the sign decided exactly in integers (load_e*E against T*K; sign 0
 * leaves the bias unchanged) and one binary32 addition.
 *   topk_idx  device [T, K] int32 (a routing, e.g. beam_moe_route's);
 *             entries outside [0, E) are not counted
 *   bias      device [E] fp32, updated in place
 * gamma >= 0 and finite (see beam_moe_bias_gamma).  No workspace. */
int beam_moe_bias_update(const beam_moe_desc* desc, int64_t T,
                         const int32_t* topk_idx, float gamma, float* bias,
                         void* stream);

/* Update speed for step t of an n-step cosine schedule from g0 down to g1:
 * g1 + (g0 - g1) * (1 + cos(pi * t / n)) / 2, evaluated in binary64 and
 * rounded to binary32; t is clamped to [0, n].  Host only. */
float beam_moe_bias_gamma(int64_t t, int64_t n, float g0, float g1);

/* ---- measurement support ------------------------------------------------
 * A timer records a HIP event pair around every kernel a timed forward
 * launches, on the stream the kernel runs on, so tools can read per-kernel
 * durations.  It owns its events (created here, destroyed with the timer);
 * it allocates no device memory.  Not thread-safe: one timer per caller. */
typedef struct beam_moe_timer beam_moe_timer;

/* Creates a timer able to hold `capacity` kernel records.  *out is NULL on
 * error. */
int beam_moe_timer_create(int32_t capacity, beam_moe_timer** out);
void beam_moe_timer_destroy(beam_moe_timer* timer);
/* Forgets all records (keeps the events for reuse). */
void beam_moe_timer_reset(beam_moe_timer* timer);
/* Number of kernel records held. */
int32_t beam_moe_timer_count(const beam_moe_timer* timer);
/* Name and duration in milliseconds of record i; waits for its events.
 * *name points to static storage. */
int beam_moe_timer_read(beam_moe_timer* timer, int32_t i, const char** name,
                        float* ms);
/* beam_moe_forward, plus one timer record per launched kernel (records past
 * the timer's capacity are dropped).  timer may be NULL. */
int beam_moe_forward_timed(const beam_moe_desc* desc, int64_t T, const void* x,
                           const float* w_router, const float* bias,
                           const void* w_gate_up, const void* s_gate_up,
                           const void* w_down, const void* s_down, void* out,
                           int32_t* topk_idx, float* topk_w, float* logits,
                           void* workspace, size_t ws_bytes, void* stream,
                           beam_moe_timer* timer);

#ifdef __cplusplus
}
#endif

#endif /* BEAM_MOE_H */
