/*
 * moe.h -- C ABI of the GB300 (sm_103a) MegaMoE expert layer.
 *
 * One call of moe_forward runs, on the caller's CUDA stream, the whole expert
 * layer of a Mixture-of-Experts block on one GPU:
 *
 *   1. dispatch: per-expert counts, exclusive prefix, stable gather map
 *      (MegaMoE SM90 Implementation Design (Final), §9.2; PR357 Green-Context
 *      Split MegaMoE code review, §6.1);
 *   2. L1 grouped GEMM x . W1^T with block scales applied per 128-K block
 *      (design §5.2-§5.3);
 *   3. SwiGLU silu(gate) * up, times the top-k weight (design §10.1 steps 1-3);
 *   4. per-row, per-64-column FP8 E4M3 requantisation, sf = amax / 448
 *      (design §10.1 steps 4-6, §1.1 decision 9);
 *   5. L2 grouped GEMM with the two per-64 activation scales of every
 *      128-K block (design §5.4);
 *   6. BF16 rounding of each (token, slot) output (design §11.1);
 *   7. top-k combine: FP32 sum over active slots in slot order, BF16 y
 *      (design §11.2; PR357 review §6.3 "K3 combine_reduce").
 *
 * Pointers: every buffer argument of moe_create / moe_transform_weights /
 * moe_forward / moe_get_* is DEVICE memory owned by the caller, except the
 * h_* arguments of moe_forward_host, which are HOST memory.  The library never
 * allocates device memory: the caller passes a workspace of
 * moe_workspace_bytes() bytes and a weight store of moe_weight_bytes() bytes,
 * both 256-byte aligned, which must outlive the context.  A moe_ctx holds
 * host state only.
 *
 * Streams: `stream` is a cudaStream_t (NULL = the legacy default stream).
 * Calls are stream-ordered and asynchronous unless stated otherwise; two
 * forwards of one context must not run concurrently (they share the
 * workspace).  Back-to-back forwards need no reset by the caller.
 *
 * Errors: every int-returning call returns MOE_OK (0) or a negative MOE_ERR_*
 * code; nothing is thrown across the ABI.  Argument and shape errors are
 * detected on the host before anything is launched.  Faults found on the
 * device (an expert id outside [-1, E), a pipeline wait that timed out) are
 * recorded in a device error word that moe_device_status() reads.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK 0
#define MOE_ERR_INVALID_ARG (-1)    /* null pointer, bad size, misaligned buffer */
#define MOE_ERR_UNSUPPORTED (-2)    /* shape or format this library does not run */
#define MOE_ERR_CUDA (-3)           /* a CUDA runtime/driver call failed */
#define MOE_ERR_DEVICE_TIMEOUT (-4) /* a bounded device-side wait gave up */
#define MOE_ERR_BAD_EXPERT (-5)     /* topk_idx held an id outside [-1, E) */
#define MOE_ERR_NOT_READY (-6)      /* moe_forward before moe_transform_weights */

typedef struct moe_ctx moe_ctx;

/* Weight formats.
 * MOE_W_FP8_BLK128: W1/W2 FP8 E4M3 with one f32 scale per 128x128 block,
 *   activations x FP8 E4M3 with one f32 scale per 1x128 (recipe (1,1,128),
 *   design §16.1 and §15.2).
 * MOE_W_FP4_E2M1_UE8M0_32: W1/W2 FP4 E2M1 (two codes per byte, low nibble =
 *   even k) with one UE8M0 scale per 1x32; activations FP8 E4M3 with one UE8M0
 *   scale per 1x32; the L2 activations are requantised per 1x32 with UE8M0
 *   scales 2^ceil(log2(amax/448)) (design §2.1, PR357 review §1, §6.1). */
typedef enum { MOE_W_FP8_BLK128 = 0, MOE_W_FP4_E2M1_UE8M0_32 = 1 } moe_wfmt;

typedef struct {
    int max_tokens;   /* T_max: largest num_tokens a forward may pass (>= 1) */
    int hidden;       /* H, multiple of 128 */
    int inter;        /* I (intermediate size per expert), multiple of 128 */
    int num_experts;  /* E, 1..1024 */
    int topk;         /* k, 1..32 */
    int wfmt;         /* moe_wfmt */
    float act_clamp;  /* symmetric clamp of gate and up before SwiGLU; +INFINITY = off
                         (design §10.1 step 3, §1.1 decision 16) */
    int fast_math;    /* SwiGLU exponential: 0 expf (accurate), 1 __expf; the
                         division is the fast one (<= 2 ulp) either way */
} moe_config;

/* Bytes of device workspace for `cfg` (0 if `cfg` is invalid).  The pages
 * size the layer's one buffer with a call of its own (MegaMoE SM90
 * Implementation Design (Final), §16.1 "get_symm_buffer_size_for_sm90_mega_moe";
 * PR357 Green-Context Split MegaMoE code review, §3.1 "Split symmetric
 * buffer"); on one GPU the symmetric buffer is a plain device buffer holding
 * the dispatch tables, the token pool, the L2 activations and their scales,
 * the BF16 pair outputs and the staging of moe_forward_host.  The pages'
 * token-alignment query (design §16.1 "get_token_alignment_for_sm90_mega_moe")
 * has no counterpart: any num_tokens in [0, max_tokens] is accepted. */
MOE_API size_t moe_workspace_bytes(const moe_config *cfg);

/* Bytes of the transformed-weight store for `cfg` (0 if `cfg` is invalid):
 * what moe_transform_weights writes (design §16.1
 * "transform_weights_for_mega_moe_sm90", §15; PR357 review §3.2 "Weight
 * transform"). */
MOE_API size_t moe_weight_bytes(const moe_config *cfg);

/* Create a context bound to the current CUDA device.  The configuration
 * carries the arguments the pages' entry point takes besides its tensors
 * (design §16.1 fp8_mega_moe: num_max_tokens_per_rank, num_experts,
 * num_topk, the (1, 1, 128) recipe, activation_clamp, fast_math), minus the
 * rank and symmetric-buffer arguments.  d_workspace and d_weights are
 * caller-owned device buffers of the sizes above (256-byte aligned).  Writes
 * *out on success. */
MOE_API int moe_create(moe_ctx **out, const moe_config *cfg, void *d_workspace, void *d_weights);

/* Read the canonical weights and write the kernel layout into d_weights
 * (design §15: gate/up rows interleaved in groups of 8 along N).
 * Canonical layouts, all row-major, rows [0, I) of w1 = gate, [I, 2I) = up.
 * MOE_W_FP8_BLK128:
 *   w1    u8 (E4M3) [E, 2I, H],   w1_sf f32 [E, 2I/128, H/128]
 *   w2    u8 (E4M3) [E, H, I],    w2_sf f32 [E, H/128, I/128]
 * MOE_W_FP4_E2M1_UE8M0_32 (32-byte aligned code arrays):
 *   w1    u8 (2 x E2M1) [E, 2I, H/2],  w1_sf u8 (UE8M0) [E, 2I, H/32]
 *   w2    u8 (2 x E2M1) [E, H, I/2],   w2_sf u8 (UE8M0) [E, H, I/32]
 * The inputs may be freed once the stream has passed this call. */
MOE_API int moe_transform_weights(moe_ctx *ctx, const void *w1, const void *w1_sf,
                          const void *w2, const void *w2_sf, void *stream);

/* One forward pass (design §3.3).
 *   num_tokens T, 0 <= T <= max_tokens (T = 0 returns at once)
 *   x             u8 (E4M3) [T, H] row-major, rows 16-byte aligned
 *   x_sf          f32 [T, H/128] (FP8 weights) or u8 UE8M0 [T, H/32] (FP4 weights)
 *   topk_idx      int32 [T, k]; -1 marks an inactive slot
 *   topk_weights  f32 [T, k]
 *   y             bf16 [T, H] (written)
 *   cumulative_expert_counts  int32 [E] or NULL: the per-expert counts of
 *                 this call are added to it (design §16.1
 *                 "cumulative_local_expert_recv_stats")
 * Asynchronous on `stream`.  A call may be captured into a CUDA graph once
 * the same shape has run eagerly on the context (the first call sets kernel
 * attributes, once per process); replays read and write the buffers that
 * were passed at capture, with whatever they hold at replay. */
MOE_API int moe_forward(moe_ctx *ctx, int num_tokens, const void *x, const void *x_sf,
                const int32_t *topk_idx, const float *topk_weights, void *y,
                int32_t *cumulative_expert_counts, void *stream);

/* moe_forward with HOST inputs and output (the pages define no such call:
 * their layer reads inputs already in the symmetric buffer): copies h_x, h_x_sf, h_topk_idx,
 * h_topk_weights into the workspace, runs the forward and copies y back to
 * h_y, then synchronises `stream`.  Host buffers may be pageable or pinned
 * (pinned is faster).  When h_y is page-locked memory the device can
 * address (cudaHostAlloc / cudaHostRegister under unified addressing) and
 * 16-byte aligned, the combine stores y into it directly over the CPU-GPU
 * link and no copy back is made (environment MOE_HOST_DIRECT=0 turns that
 * off). */
MOE_API int moe_forward_host(moe_ctx *ctx, int num_tokens, const void *h_x, const void *h_x_sf,
                     const int32_t *h_topk_idx, const float *h_topk_weights, void *h_y,
                     void *stream);

/* Test export (the pages define no such call): copy the dispatch result of
 * the last forward (T tokens) into caller device
 * buffers: counts int32 [E], offsets int32 [E+1] (exclusive prefix of
 * counts), gather int32 [T*k] whose first offsets[E] entries are the pair ids
 * t*k + j of each expert's pairs in (token, slot) order, experts ascending
 * (later entries unspecified).  Any pointer may be NULL. */
MOE_API int moe_get_dispatch(moe_ctx *ctx, int32_t *counts, int32_t *offsets, int32_t *gather,
                     void *stream);

/* Test export (the pages define no such call): copy intermediates of the
 * last forward (T tokens; row r belongs to pair
 * gather[r], rows r >= offsets[E] unspecified), P = T*k:
 * l2_acts u8 (E4M3) [P, I], l2_sf = the L2 activation scales (f32 [P, I/64]
 * with FP8 weights, u8 UE8M0 [P, I/32] with FP4 weights),
 * l2_out bf16 [P, H] (the rounded L2 outputs).  Any pointer may be NULL.
 * For stage-by-stage tests. */
MOE_API int moe_get_intermediates(moe_ctx *ctx, void *l2_acts, void *l2_sf, void *l2_out,
                          void *stream);

/* Largest problem moe_dispatch_noalloc accepts. */
#define MOE_NOALLOC_MAX_PAIRS 65536   /* num_tokens * topk */
#define MOE_NOALLOC_MAX_EXPERTS 1024

/* The dispatch step alone, for callers that cannot allocate device memory
 * and cannot hand this library a workspace: code that runs inside a host
 * application or serving runtime which plans every device byte itself and
 * offers its plugins no workspace hook, or a path where a cudaMalloc would
 * stall the device or break the runtime's memory budget.  The pages have no
 * counterpart of this entry point.
 *
 * Computes what moe_forward's dispatch computes (counts int32 [E], offsets
 * int32 [E+1], gather int32 [T*k] with the first offsets[E] entries valid)
 * from topk_idx int32 [T,k] (device), into caller device buffers, on
 * `stream`.  It allocates nothing: the kernel's other scratch (pair -> row
 * map, M-block tables, error word) lives in one fixed device array of about
 * 270 KB inside this library, which every GPU that loads the library keeps
 * until the process exits.
 *  - Sizes: returns MOE_ERR_INVALID_ARG, launching nothing, when
 *    num_tokens * topk > MOE_NOALLOC_MAX_PAIRS, num_experts >
 *    MOE_NOALLOC_MAX_EXPERTS, topk outside [1, 32], or a pointer is NULL.
 *  - The first call on a device looks up that array's device address (with
 *    that device current); make this first call before any stream capture.
 *    The address is kept per device and context: after cudaDeviceReset the
 *    next call looks it up again in the new context.
 *  - Every call shares the one array and it keeps the last call's contents;
 *    the call clears what must start at zero.  Calls that overlap on the GPU
 *    (two streams, or two host threads) race on it and must not be issued.
 *  - Expert ids outside [-1, E) are skipped but not reported here. */
MOE_API int moe_dispatch_noalloc(const int32_t *topk_idx, int num_tokens, int topk,
                                 int num_experts, int32_t *counts, int32_t *offsets,
                                 int32_t *gather, void *stream);

/* Measurement plumbing (the pages define no such call).
 * Per-stage timing of the next `max_forwards` forwards: moe_profile_begin
 * creates CUDA events (no device memory) and every following moe_forward
 * records one event before its dispatch and one after each of its four
 * stages (dispatch, L1 GEMM, L2 GEMM, combine) on its stream.
 * moe_profile_end synchronises those events, writes the summed milliseconds
 * of each stage to stage_ms[4] and the number of recorded forwards to
 * *n_forwards, and releases the events. */
MOE_API int moe_profile_begin(moe_ctx *ctx, int max_forwards);
MOE_API int moe_profile_end(moe_ctx *ctx, float *stage_ms, int *n_forwards);

/* Test of the device-side timeout path (the pages have no counterpart; it
 * exists so that failure detection can be tested without faulting a GPU).
 * Arms the next moe_forward of `ctx`: every wait of that forward gives up
 * after `wait_limit_us` microseconds instead of 2 s, and
 *   which = 1 or 2: CTA 0's copy producer in GEMM `which` (1 = L1, 2 = L2)
 *           never fills its first pipeline stage, so the MMA's wait for it
 *           runs out (both weight formats);
 *   which = 3: CTA 0 of the multi-CTA dispatch (batches of 8192 routed pairs
 *           or more) never arrives at the grid-wide barrier, so the other
 *           CTAs' waits run out.
 * A step of a forward that times out makes that forward's later steps skip
 * (they check a per-forward abort word at entry) rather than read tables it
 * left incomplete.  That forward returns MOE_OK; its output is undefined;
 * moe_device_status() then returns MOE_ERR_DEVICE_TIMEOUT, and later forwards
 * run normally whether or not the status was read.  The hook disarms itself
 * after one forward.  Returns MOE_ERR_INVALID_ARG for another `which` or a
 * limit below 1 us. */
MOE_API int moe_test_arm_timeout(moe_ctx *ctx, int which, int wait_limit_us);

/* ABI plumbing (the pages define no such call): synchronise the device,
 * read and clear the device error word: MOE_OK, MOE_ERR_BAD_EXPERT,
 * MOE_ERR_DEVICE_TIMEOUT or MOE_ERR_CUDA. */
MOE_API int moe_device_status(moe_ctx *ctx);

/* ABI plumbing (no counterpart in the pages): static description of an
 * error code. */
MOE_API const char *moe_strerror(int code);

/* ABI plumbing (no counterpart in the pages): free the host state (never
 * the caller's buffers).  NULL is allowed. */
MOE_API void moe_destroy(moe_ctx *ctx);

/* ------------------------------------------------------------------------
 * The MoE block around the expert layer: the norms before and after it, the
 * router with its balance loss, and dense products with FP4 weights for a
 * few tokens (a shared expert at decode).
 *
 * These calls keep no context: the configuration travels with every call,
 * device memory (workspaces, laid-out weights, outputs) is the caller's,
 * calls are stream-ordered and asynchronous, and argument errors are found
 * on the host before anything is launched.  They may be captured into CUDA
 * graphs.  They launch on the calling thread's current device, which must be
 * the one of the stream and the memory.  Row pitches `ld_*` are in elements;
 * rows themselves are contiguous, and any pitch >= the row length and any
 * element-aligned base works (16-byte aligned rows are the fast case).
 * num_tokens = 0 launches nothing that reads tokens: sums over tokens come
 * out zero.
 * ------------------------------------------------------------------------ */

typedef enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_F32 = 1 } moe_dtype;

/* ---- block norms ---- */

typedef enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2 } moe_gate;

/* Input formats of the expert layer that the norm can write itself:
 * MOE_QUANT_FP8_128: E4M3 codes with f32 scales amax/448 per 128 columns
 *   (x, x_sf of MOE_W_FP8_BLK128);
 * MOE_QUANT_UE8M0_32: E4M3 codes with UE8M0 scales 2^ceil(log2(amax/448))
 *   per 32 columns (x, x_sf of MOE_W_FP4_E2M1_UE8M0_32).
 * An all-zero group has scale 0 (UE8M0 code 0) and codes 0. */
typedef enum { MOE_QUANT_NONE = 0, MOE_QUANT_FP8_128 = 1, MOE_QUANT_UE8M0_32 = 2 } moe_quant;

#define MOE_NORM_MAX_HIDDEN 16384

typedef struct {
    int hidden;           /* H, 1..MOE_NORM_MAX_HIDDEN; a multiple of 128 / 32 with the quantised outputs */
    int stream_dtype;     /* moe_dtype of residual, y, h, n and of their gradients */
    int param_dtype;      /* moe_dtype of w_post, w_pre and gate (their gradients are f32) */
    int gate;             /* moe_gate: shape of `gate`, [H] or [T] */
    int quant;            /* moe_quant */
    float eps;            /* > 0 */
    float residual_scale; /* finite */
} moe_norm_config;

/* Forward, per token (all in f32, rounded once per output):
 *   r1 = (mean(y^2) + eps)^-1/2,  u = y r1 w_post      (w_post NULL: u = y)
 *   z  = residual_scale * residual + gate u            (gate NULL: 1)
 *   r2 = (mean(z^2) + eps)^-1/2,  v = z r2 w_pre       (w_pre NULL: none of this)
 * h = z and n = v in the stream's type, codes / sf = v quantised.  Without y
 * the block part is absent: z = residual, and w_post, gate and h must be
 * NULL.  h may be residual itself (same pitch). */
typedef struct {
    const void *residual; int64_t ld_residual;  /* [T, H] */
    const void *y; int64_t ld_y;                /* [T, H] block output, or NULL */
    const void *w_post;                         /* [H] or NULL */
    const void *gate;                           /* [H] / [T] as cfg->gate says, NULL with MOE_GATE_NONE */
    const void *w_pre;                          /* [H] or NULL */
    void *h; int64_t ld_h;                      /* [T, H] out, with y */
    void *n; int64_t ld_n;                      /* [T, H] out or NULL, with w_pre */
    uint8_t *codes;                             /* [T, H] out, with cfg->quant; 16-byte aligned */
    void *sf;                                   /* f32 [T, H/128] or u8 [T, H/32] out, with cfg->quant; 4-byte aligned */
    float *rstd_post, *rstd_pre;                /* [T] out or NULL: r1, r2 for the backward pass */
} moe_norm_io;

MOE_API int moe_norm_forward(const moe_norm_config *cfg, int num_tokens, const moe_norm_io *io, void *stream);

/* Backward of the same.  With a = dn w_pre, zh = h r2, yh = y r1:
 *   D = dh + r2 (a - zh mean(a zh))           dresidual = residual_scale D
 *   b = D gate w_post                         dy = r1 (b - yh mean(b yh))
 *   dw_pre = sum_t dn zh                      dw_post = sum_t D gate yh
 *   dgate  = sum D u over t (channel) or h (token)
 * h stands for z (it is z rounded); the quantiser passes its gradient
 * straight through (add it to dn).  Sums over tokens are taken in a fixed
 * order: the same call gives the same bits.  dh NULL means zero; with dn NULL
 * the pre norm takes no part (w_pre, rstd_pre, dw_pre NULL).  Without y:
 * dresidual = D, and everything of the block is NULL.  dresidual may be dh,
 * dy may be dn (same pitches). */
typedef struct {
    const void *h; int64_t ld_h;                /* [T, H] stream after the block (without y: the residual) */
    const void *y; int64_t ld_y;
    const void *w_post, *gate, *w_pre;
    const float *rstd_post, *rstd_pre;          /* [T], with w_post / w_pre */
    const void *dh; int64_t ld_dh;              /* [T, H] or NULL */
    const void *dn; int64_t ld_dn;              /* [T, H] or NULL */
    void *dresidual; int64_t ld_dresidual;      /* [T, H] out */
    void *dy; int64_t ld_dy;                    /* [T, H] out, with y */
    float *dw_post, *dgate, *dw_pre;            /* f32 out: [H], [H] / [T], [H] */
} moe_norm_grad_io;

/* Bytes of device workspace of moe_norm_backward, 256-byte aligned (0 if
 * `cfg` is invalid or num_tokens < 0); larger batches need no less. */
MOE_API size_t moe_norm_workspace_bytes(const moe_norm_config *cfg, int num_tokens);
MOE_API int moe_norm_backward(const moe_norm_config *cfg, int num_tokens, const moe_norm_grad_io *io,
                              void *d_workspace, void *stream);

/* ---- router and balance loss ---- */

typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

/* What a bias is added to for the choice: the logit, or (MOE_SCORE_SIGMOID
 * only) the score, as routers are trained that balance their experts by such
 * biases.  The two choose differently: of logits 4 and 0 with biases 0 and
 * 0.6, the first by logits, the second by scores. */
typedef enum { MOE_BIAS_LOGIT = 0, MOE_BIAS_SCORE = 1 } moe_bias;

typedef struct {
    int num_experts;      /* E, 1..1024 */
    int topk;             /* k, 1..min(32, E) */
    int score;            /* moe_score of the logits: s = softmax or sigmoid */
    int renormalize;      /* weights = weight_scale * s / (sum of the chosen s), else weight_scale * s */
    int logits_dtype;     /* moe_dtype of logits and d_logits */
    float weight_scale;   /* finite */
    float balance_coef;   /* alpha of the balance loss, finite */
    float z_coef;         /* beta of the z loss, finite; 0 with MOE_SCORE_SIGMOID */
    int bias_on;          /* moe_bias */
} moe_router_config;

/* The choice: the k largest logit + bias, or score + bias (f32 sums, the
 * score within 2^-19 of itself or 2^-40), ties to the lowest expert; without a
 * bias the k largest logits.  A logit of -inf or NaN, or a sum that is, closes
 * its expert for the token; a slot with no open expert left gets topk_idx -1
 * and weight 0 (moe_forward's inactive slot).  +inf counts as the largest
 * finite f32.  The bias takes no part in the weights.  Experts are not limited
 * to groups. */

#define MOE_MAX_SEQS (1 << 20)

/* Losses of a batch of S sequences (token ranges), over the tokens that have
 * an open logit (n_s of sequence s, S' sequences with n_s > 0, N in all), with
 * p the scores scaled to sum 1 and c the chosen slots of each expert:
 *   balance = alpha / S' sum_s sum_e (E c_se / (k n_s)) (sum_t p_te / n_s)
 *   z       = beta / N sum_t logsumexp(logits_t)^2
 * c is a constant for the gradient. */
typedef struct {
    int num_seqs;                  /* S, 1..MOE_MAX_SEQS */
    const int32_t *seq_offsets;    /* [S+1] nondecreasing token offsets within [0, T], or NULL: S = 1, all tokens.
                                      Tokens outside every range are routed but enter no loss */
    float *loss;                   /* [3]: total, balance, z */
    int32_t *counts;               /* [S, E]: c */
    float *prob_mean;              /* [S, E]: sum_t p / n_s (0 for an empty sequence) */
    int32_t *seq_tokens;           /* [S + 2]: n_s of each sequence, then S' and N */
} moe_balance_io;

/* Bytes of device workspace of the calls that compute losses, 256-byte
 * aligned (0 if the arguments are invalid). */
MOE_API size_t moe_router_workspace_bytes(const moe_router_config *cfg, int max_tokens, int max_seqs);

/* topk_idx int32 [T, k] and topk_weights f32 [T, k] (moe_forward's inputs)
 * from logits [T, E]; bias f32 [E] or NULL.  With `loss` (else NULL, and
 * d_workspace unused) the losses of this choice in the same pass. */
MOE_API int moe_router_forward(const moe_router_config *cfg, int num_tokens, const void *logits, int64_t ld_logits,
                               const float *bias, int32_t *topk_idx, float *topk_weights,
                               const moe_balance_io *loss, void *d_workspace, void *stream);

/* The losses of a choice made elsewhere: topk_idx int32 [T, k] is an input,
 * each row's experts distinct (ids outside [0, E) are inactive slots). */
MOE_API int moe_balance_loss(const moe_router_config *cfg, int num_tokens, const void *logits, int64_t ld_logits,
                             const int32_t *topk_idx, const moe_balance_io *loss, void *d_workspace, void *stream);

/* d_logits [T, E] = the gradient through topk_weights (d_weights f32 [T, k],
 * or NULL) plus d_loss (f32 scalar on the device, or NULL) times that of
 * loss[0].  `loss` holds what the forward call wrote (counts and seq_tokens
 * are read; NULL with d_loss NULL).  Closed experts get 0. */
MOE_API int moe_router_backward(const moe_router_config *cfg, int num_tokens, const void *logits, int64_t ld_logits,
                                const int32_t *topk_idx, const float *d_weights, const moe_balance_io *loss,
                                const float *d_loss, void *d_logits, int64_t ld_d_logits, void *stream);

/* ---- FP4 linear for a few tokens ---- */

typedef enum { MOE_ACT_NONE = 0, MOE_ACT_SWIGLU = 1 } moe_act;

#define MOE_FP4_LINEAR_MAX_TOKENS 16
#define MOE_FP4_LINEAR_MAX_IN 24576

typedef struct {
    int in_features;   /* K, a multiple of 32, at most MOE_FP4_LINEAR_MAX_IN */
    int out_features;  /* N rows of the weight; even with MOE_ACT_SWIGLU */
    int act;           /* moe_act; SWIGLU: rows [0, N/2) gate, [N/2, N) up, output silu(gate) * up of N/2 columns */
    int out_dtype;     /* moe_dtype of add and y */
    float act_clamp;   /* symmetric clamp of gate and up before SWIGLU; +INFINITY = off; a NaN stays one */
} moe_fp4_linear_config;

/* Weights in the layer's FP4 format (MOE_W_FP4_E2M1_UE8M0_32): w u8 [N, K/2]
 * (low nibble = even k; 16-byte aligned), w_sf u8 UE8M0 [N, K/32] (code 255
 * is not a number and must not occur; a code 127 or more below its row's
 * largest counts as a scale of 0).  They are laid out once into a store of
 * moe_fp4_linear_weight_bytes() bytes (0 if `cfg` is invalid; 256-byte
 * aligned) and may be freed once the stream has passed that call. */
MOE_API size_t moe_fp4_linear_weight_bytes(const moe_fp4_linear_config *cfg);
MOE_API int moe_fp4_linear_transform_weights(const moe_fp4_linear_config *cfg, const void *w, const void *w_sf,
                                             void *d_weights, void *stream);

/* y [T, N or N/2] = act(x W^T) (+ add), x bf16 [T, K], 0 <= T <=
 * MOE_FP4_LINEAR_MAX_TOKENS, sums in f32.  add may be y itself (same pitch). */
MOE_API int moe_fp4_linear_forward(const moe_fp4_linear_config *cfg, int num_tokens, const void *x, int64_t ld_x,
                                   const void *d_weights, const void *add, int64_t ld_add, void *y, int64_t ld_y,
                                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
