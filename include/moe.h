/*
 * moe.h - C ABI of the MI355X (gfx950) sparse Mixture-of-Experts layer forward.
 *
 * One MoE layer: a router scores every token against n_expert experts, keeps
 * the top-k, renormalises their weights; the token rows are grouped by expert;
 * each selected expert applies a SwiGLU FFN; an always-on shared expert is
 * added; the weighted results return to token order.
 *
 *   logits  l[t,e] = sum_i x[t,i] * Wr[e,i]            (row stride n_expert)
 *   score   s = sigmoid(l)  or  s = sqrt(softplus(l))  or  s = softmax(l)
 *   key     s + bias[e]  (bias optional; it selects, it never weights)
 *   select  top-k keys; equal keys -> lower expert index first; NaN last
 *   weight  w_j = route_scale * s_j / sum over the selected s
 *   FFN_e   Wd[e] . (silu(Wg[e] x) * (Wu[e] x)),  silu(g) = g / (1 + e^-g)
 *   y[t]    FFN_shared(x_t) + sum_j w_j FFN_{e_j}(x_t)
 *
 * Sources: "256 experts, 512 lines" blog post - section "Why GLM-5.2 in an
 * engine built for DeepSeek" (sigmoid routing, top-8, MoE with a shared
 * expert) and section "The constant that always said 256" (sqrt(softplus)
 * scores, top-6, the 1.5 scale, logits addressed with stride n_expert and
 * n_expert a runtime value, a parallel top-k rather than a serial one);
 * NeutronStar README, main branch - Hy3 paragraph (sigmoid scores plus a
 * per-expert bias choosing 8 of 192 experts, and a shared expert); NeutronStar README - "The model"
 * (decision tensors kept at Q8_0/F32), "GLM-5.2 CUDA port" (gate/up and down
 * projection kernels) and the MTP paragraph (only the selected experts' weights
 * are read for small batches; batch kernels address whole [E, rows, cols]
 * expert tensors).
 *
 * Conventions for every entry point
 *  - Pointers are DEVICE pointers owned by the caller; the library never
 *    allocates, frees or synchronises.  `stream` is a hipStream_t (NULL = the
 *    null stream); all work is enqueued on it and the call returns at once.
 *  - Every call validates its arguments first.  On failure it returns a
 *    nonzero moe_status and enqueues nothing.  MOE_ERR_DEVICE reports a launch
 *    error seen right after enqueueing; faults inside kernels surface at the
 *    caller's next synchronisation.
 *  - Activations (x), weight tensors, router weights, slot_out, shared_out,
 *    y and the workspace must be 16-byte aligned; the per-element arrays
 *    (bias, logits, topk_idx, topk_w, offsets, perm_rows, inv_perm) need
 *    4-byte alignment.  Sizes are element counts.
 *  - Layouts are row-major.  Weight tensors are [n, rows, cols] with cols the
 *    reduction dimension.  bf16 and fp16 values are passed as their bit
 *    patterns (uint16).  Q8B32 = int8 quants [n, rows, cols] plus one fp16
 *    scale per 32 consecutive columns [n, rows, cols/32]; weight = scale * q.
 *    F8B128 = e4m3 codes (OCP, largest value 448) [n, rows, cols] plus one
 *    fp32 scale per block of 128 x 128 [n, ceil(rows/128), ceil(cols/128)];
 *    weight = scale * code.
 *    I8CH = int8 codes [n, rows, cols] plus one fp32 scale per row (output
 *    channel) [n, rows]; weight = scale * code.
 *  - Products with F8B128 weights are products of e4m3 operands: activations
 *    are quantised per row and 128 columns as moe_quantize_rows does (x, and
 *    the SwiGLU intermediate from its fp32 values).  Sums are fp32; only
 *    moe_block_matmul to bf16 may take the 8-bit matrix instruction, which cuts
 *    the products of 8 consecutive columns 13 bits below the largest of them
 *    (1.5e-5 of a result on normal operands).  Layers with
 *    F8B128 weights need n_tokens * d_model < 2^32.  Softmax scores are taken
 *    over all n_expert logits of a token.
 *  - Products with I8CH weights are products of int8 operands: activations are
 *    quantised per row as moe_quantize_tokens does (x, and the SwiGLU
 *    intermediate from its fp32 values, over the whole row).  Sums are exact
 *    (int32); d_model, d_ff and d_ff_shared are at most MOE_I8_MAX_K there, and
 *    n_tokens * d_model < 2^32.
 *  - Results: expert indices and the permutation are exact and do not depend
 *    on the path taken; logits and scores are accumulated in fp64 and rounded
 *    once to fp32; the SwiGLU intermediate is rounded to the activation format
 *    (bf16, or fp32 for fp32 layers); y is fp32.
 *  - The workspace (`ws`, `ws_bytes`) is caller-owned scratch of at least
 *    moe_workspace_bytes(cfg) bytes.  It needs no initialisation: every call
 *    writes each workspace word before reading it.  Calls that share a
 *    workspace must not overlap.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H
#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID = 1,     /* NULL/misaligned pointer, value out of range, bad enum */
    MOE_ERR_UNSUPPORTED = 2, /* valid but not provided: dtype pair, d/F not multiples of 64, path */
    MOE_ERR_WORKSPACE = 3,   /* ws_bytes < moe_workspace_bytes(cfg) */
    MOE_ERR_DEVICE = 4       /* the HIP runtime refused a launch */
} moe_status;

typedef enum { MOE_SCORE_SIGMOID = 0, MOE_SCORE_SQRT_SOFTPLUS = 1, MOE_SCORE_SOFTMAX = 2 } moe_score;
typedef enum { MOE_DT_F32 = 0, MOE_DT_BF16 = 1, MOE_DT_Q8B32 = 2, MOE_DT_F8B128 = 3, MOE_DT_I8CH = 4 } moe_dtype;
typedef enum { MOE_PATH_AUTO = 0, MOE_PATH_DECODE = 1, MOE_PATH_PREFILL = 2 } moe_path;

/* Largest token count the decode path accepts (MOE_PATH_AUTO takes it for
 * n_tokens <= MOE_DECODE_MAX_TOKENS). */
#define MOE_DECODE_MAX_TOKENS 8

typedef struct {
    int32_t n_tokens;    /* T >= 1 */
    int32_t d_model;     /* d: multiple of 64 */
    int32_t n_expert;    /* E in [1, 1024], a runtime value */
    int32_t top_k;       /* k in [1, min(E, 32)] */
    int32_t d_ff;        /* F: routed expert hidden size, multiple of 64 */
    int32_t n_shared;    /* 0 or 1 shared expert */
    int32_t d_ff_shared; /* Fs: shared expert hidden size, multiple of 64 (if n_shared) */
    int32_t score;       /* moe_score */
    float route_scale;   /* finite, > 0: 1.5 for the sqrt(softplus) router, 1.0 for sigmoid */
    int32_t act_dtype;   /* moe_dtype of x and of the SwiGLU intermediate: F32 or BF16 */
    int32_t w_dtype;     /* moe_dtype of the expert weights: (F32,F32) (BF16,BF16) (BF16,Q8B32) (BF16,F8B128) (BF16,I8CH) */
    int32_t path;        /* moe_path, used by moe_layer_forward */
} moe_config;

typedef struct {
    const void *q;          /* [n, rows, cols] elements of w_dtype (int8 for Q8B32 and I8CH, e4m3 for F8B128) */
    const uint16_t *scale;  /* Q8B32: fp16 bits [n, rows, cols/32]; F8B128: the address of fp32 [n,
                               ceil(rows/128), ceil(cols/128)], I8CH: of fp32 [n, rows], cast; 4-byte
                               aligned; else ignored */
} moe_mat;

typedef struct {
    const float *w_router;  /* [E, d] fp32 */
    const float *bias;      /* [E] fp32 or NULL */
    moe_mat gate, up;       /* [E, F, d] */
    moe_mat down;           /* [E, d, F] */
    moe_mat s_gate, s_up;   /* [1, Fs, d]   (ignored when n_shared == 0) */
    moe_mat s_down;         /* [1, d, Fs] */
} moe_weights;

/* Stages of moe_layer_forward whose kernels a caller can time: 0 router
 * logits, 1 top-k selection, 2 permutation, 3 gate/up (SwiGLU), 4 down
 * projection, 5 combine.  The decode path (n_tokens <= MOE_DECODE_MAX_TOKENS)
 * builds the permutation inside the selection kernel and the combine inside
 * the down kernel: it launches no kernel for stages 2 and 5 and leaves their
 * events unrecorded.  F8B128 layers have one path: stages 0 to 5 at every
 * n_tokens, but up to 16 tokens stage 1 includes the permutation (stage 2's
 * events stay unrecorded), and the quantisation of x is in stage 1 there and
 * in none beyond.  I8CH layers: the same, stage 3
 * ends with the quantisation of the SwiGLU intermediate, and up to 16 tokens
 * stage 4 includes the combine (stage 5's events stay unrecorded). */
#define MOE_STAGES 6
#define MOE_STAGE_EVENTS (2 * MOE_STAGES)

/* Optional outputs of moe_layer_forward; any field may be NULL. */
typedef struct {
    float *logits;      /* [T, E] */
    int32_t *topk_idx;  /* [T, k] */
    float *topk_w;      /* [T, k] */
    int32_t *offsets;   /* [E+1] */
    int32_t *perm_rows; /* [T*k] */
    int32_t *inv_perm;  /* [T*k] */
    void **stage_events; /* NULL, or MOE_STAGE_EVENTS hipEvent_t created by the caller (entries
                            may be NULL): [2s] receives the start timestamp of stage s's first
                            kernel dispatch, [2s+1] the end timestamp of its last (the dispatch's
                            own timestamps, via hipExtLaunchKernel), so the elapsed time between
                            them is the stage's kernel time without the launch gaps around it */
} moe_debug;

/* Bytes of workspace every entry point below may use for this config
 * (0 if the config is invalid).  Monotone in every size field. */
size_t moe_workspace_bytes(const moe_config *cfg);

/* Router: logits (optional, [T,E]) and the top-k selection.
 * x [T, d] act_dtype; w_router [E, d] fp32; bias [E] or NULL;
 * topk_idx [T, k] int32 in rank order; topk_w [T, k] fp32. */
int moe_route(const moe_config *cfg, const void *x, const float *w_router, const float *bias,
              float *logits, int32_t *topk_idx, float *topk_w, void *ws, size_t ws_bytes,
              void *stream);

/* Selection alone, from given fp32 logits [T, E] (row stride n_expert).
 * n_expert == 256 runs a compile-time 256-expert instantiation of the top-k;
 * cfg->path == MOE_PATH_PREFILL forces the runtime-n_expert kernel instead
 * (both give identical results; the switch exists so that can be checked). */
int moe_select(const moe_config *cfg, const float *logits, const float *bias, int32_t *topk_idx,
               float *topk_w, void *stream);

/* Expert groups of a selection.  The n_expert experts form n_group groups of
 * n_expert / n_group consecutive ones; a group's score is the fp32 sum of its
 * group_top best keys (of all, if it has fewer); the topk_group best groups
 * stay (equal scores: the lower group first; NaN last) and the top-k keys are
 * taken among their experts, with the order of moe_select.
 * 1 <= n_group <= 64 dividing n_expert, 1 <= topk_group <= n_group, group_top
 * 1 or 2, top_k <= topk_group * n_expert / n_group, normalise 0 or 1, else
 * MOE_ERR_INVALID. */
typedef struct {
    int32_t n_group;    /* 1: no groups */
    int32_t topk_group; /* groups that stay */
    int32_t group_top;  /* keys summed into a group's score: 1 or 2 */
    int32_t normalise;  /* 1: w_j = route_scale * s_j / sum of the selected s (0 if that is 0);
                           0: w_j = route_scale * s_j */
} moe_groups;

/* moe_select and moe_route with expert groups; groups == NULL stands for
 * {1, 1, 1, 1}, the selection of moe_select.  Every moe_score, softmax
 * included (as in moe_select, moe_route and the layer calls). */
int moe_select_grouped(const moe_config *cfg, const moe_groups *groups, const float *logits, const float *bias,
                       int32_t *topk_idx, float *topk_w, void *stream);
int moe_route_grouped(const moe_config *cfg, const moe_groups *groups, const void *x, const float *w_router,
                      const float *bias, float *logits, int32_t *topk_idx, float *topk_w, void *ws,
                      size_t ws_bytes, void *stream);

/* Token->expert grouping: a stable counting sort of the flat assignments
 * f = t*k + j by expert.  offsets [E+1] (exclusive prefix sum of the expert
 * counts); perm_rows [T*k]: the f of every assignment, ordered by (expert, f);
 * inv_perm [T*k]: position of f in perm_rows.  Indices outside [0, E) are left
 * out: inv_perm = -1, and the unused tail of perm_rows is -1. */
int moe_permute(const moe_config *cfg, const int32_t *topk_idx, int32_t *offsets,
                int32_t *perm_rows, int32_t *inv_perm, void *ws, size_t ws_bytes, void *stream);

/* Routed and shared experts.  slot_out [T*k, d] fp32: row f = w_f *
 * FFN_{expert of f}(x_t); shared_out [T, d] fp32 = FFN_shared(x_t), or NULL
 * when n_shared == 0.  offsets / perm_rows as produced by moe_permute; topk_w
 * [T, k].  Rows of assignments that perm_rows does not list are not written.
 * Offsets that are not a monotone split of [0, T*k] (checked on the device)
 * leave every slot row unwritten; the shared expert is still computed. */
int moe_expert_ffn(const moe_config *cfg, const void *x, const moe_weights *w,
                   const int32_t *offsets, const int32_t *perm_rows, const float *topk_w,
                   float *slot_out, float *shared_out, void *ws, size_t ws_bytes, void *stream);

/* y [T, d] fp32 = shared_out[t] (if not NULL) + sum_j slot_out[t*k + j]. */
int moe_combine(const moe_config *cfg, const float *slot_out, const float *shared_out, float *y,
                void *stream);

/* The whole layer: route, group, experts, combine.  y [T, d] fp32.
 * cfg->path picks the decode path (GEMV over the selected experts' weights,
 * combine fused; n_tokens <= MOE_DECODE_MAX_TOKENS) or the prefill path
 * (grouped GEMMs, bf16 on MFMA); MOE_PATH_AUTO chooses by n_tokens. */
int moe_layer_forward(const moe_config *cfg, const void *x, const moe_weights *w, float *y,
                      moe_debug *dbg, void *ws, size_t ws_bytes, void *stream);

/* moe_layer_forward with expert groups (NULL: {1, 1, 1, 1}) and a choice of
 * y's type: y_dtype MOE_DT_F32, or MOE_DT_BF16 (the fp32 sum rounded once;
 * F8B128 and I8CH weights only, else MOE_ERR_UNSUPPORTED). */
int moe_layer_forward_grouped(const moe_config *cfg, const moe_groups *groups, const void *x, const moe_weights *w,
                              void *y, int32_t y_dtype, moe_debug *dbg, void *ws, size_t ws_bytes, void *stream);

/* moe_layer_forward for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, results and kernels as moe_layer_forward, but
 * no caller workspace: the library's own static device array of
 * MOE_STATIC_SCRATCH_BYTES serves instead (one per GPU, held from the first
 * call on that GPU until the process ends; the current device's copy is used,
 * so `stream` must belong to the current device).  A config whose
 * moe_workspace_bytes exceeds MOE_STATIC_SCRATCH_BYTES returns
 * MOE_ERR_WORKSPACE and enqueues nothing (64 MiB covers every decode config
 * here and prefill batches of a few hundred tokens at d_model 4096-6144).
 * This call never allocates or frees.  Every call on one GPU shares that GPU's
 * array, which keeps the last call's contents (nothing in it needs to start
 * at zero: each call writes every word before reading it), so calls that
 * overlap on one GPU - on two streams, or from two host threads without
 * ordering - race and must not be issued.  MOE_ERR_DEVICE if the array's
 * device address cannot be obtained.
 * Like moe_layer_forward it takes no expert groups: a grouped layer brings its
 * own workspace (moe_layer_forward_grouped). */
#define MOE_STATIC_SCRATCH_BYTES (64u << 20)
int moe_layer_forward_noalloc(const moe_config *cfg, const void *x, const moe_weights *w, float *y,
                              moe_debug *dbg, void *stream);

/* Top-k over long candidate rows: the sparse attention indexer's selection of
 * the best 512 or 1024 entries of a long score row ("256 experts, 512 lines"
 * blog post, section "The constant that always said 256"), with the order of
 * the expert selection above.  For each of `rows` rows of scores [rows, n]
 * fp32, the k candidates that come first (larger score first, NaN after every
 * number, -0 equal to +0, equal scores by lower candidate index) go to
 * idx [rows, k] int32, listed by ascending candidate index, and their scores,
 * bit for bit, to vals [rows, k] fp32 (vals may be NULL).
 * 1 <= k <= n <= MOE_TOPK_ROWS_MAX_N and rows >= 0 (0 enqueues nothing), else
 * MOE_ERR_INVALID; scores, idx and vals need 4-byte alignment.  No workspace.
 * events: NULL, or 2 hipEvent_t created by the caller (entries may be NULL)
 * that receive the start and end timestamps of the kernel dispatch. */
#define MOE_TOPK_ROWS_MAX_N 65536
int moe_topk_rows(const float *scores, int32_t rows, int32_t n, int32_t k, int32_t *idx, float *vals,
                  void **events, void *stream);

/* Rows to e4m3 codes with one power-of-two scale per 128 columns.  x
 * [rows, cols] of x_dtype (MOE_DT_F32 or MOE_DT_BF16), rows ldx elements
 * apart.  For each row and each block of 128 columns (the last may be
 * shorter) with largest magnitude a, the scale s is the smallest power of two
 * with a <= 448 s, at least 2^-126, and 1 if a = 0; q [rows, cols] = x / s
 * rounded to e4m3 (nearest, ties to even), and scale [rows,
 * MOE_F8_SCALE_LD(cols)] holds s as its e8m0 byte (exponent + 127).  A block
 * with a NaN or an infinity gets the byte 255 (NaN) and NaN codes (0x7F).
 * The bytes of a row past its last block are written as 127.
 * rows >= 0 (0 enqueues nothing), 16 <= cols <= 2^20 a multiple of 16 and
 * ldx >= cols a multiple of 16 bytes, else MOE_ERR_INVALID; x and q 16-byte
 * aligned, scale 4-byte.  q and scale must not overlap x.  No workspace. */
#define MOE_F8_SCALE_LD(cols) (((cols) + 511) / 512 * 4)
int moe_quantize_rows(const void *x, int32_t x_dtype, int32_t rows, int32_t cols, int64_t ldx, uint8_t *q,
                      uint8_t *scale, void *stream);

/* out [m, n] = x [m, k] w[n, k]^T with e4m3 operands:
 *   out[i, j] = sum_b s_x[i, b] * s_w[j / 128, b] * sum_{c in block b} q_x[i, c] * q_w[j, c]
 * (b: the blocks of 128 columns; sums as above; s_x times a block's sum must stay
 * within fp32's range).  x is MOE_DT_F8B128 codes with
 * x_scale [m, MOE_F8_SCALE_LD(k)] as moe_quantize_rows writes them, or
 * MOE_DT_BF16 / MOE_DT_F32 rows, which are quantised that way first (x_scale
 * NULL, workspace needed).  w [n, k] codes, w_scale [ceil(n/128), ceil(k/128)]
 * fp32.  out_dtype MOE_DT_F32, or MOE_DT_BF16 (one rounding).  0 <= m <= 2^20
 * (0 enqueues nothing), 1 <= n <= 2^20, 16 <= k <= 2^20 a multiple of 16,
 * else MOE_ERR_INVALID; x, w, out and ws 16-byte aligned, the scales 4-byte.
 * out must not overlap an input.  The workspace size is 0 for F8B128 rows and
 * for sizes out of range. */
size_t moe_block_matmul_workspace_bytes(int32_t x_dtype, int32_t m, int32_t k);
int moe_block_matmul(const void *x, int32_t x_dtype, const uint8_t *x_scale, const uint8_t *w, const float *w_scale,
                     int32_t m, int32_t n, int32_t k, void *out, int32_t out_dtype, void *ws, size_t ws_bytes,
                     void *stream);

/* Rows to int8 codes with one fp32 scale per row (token).  x [rows, cols] of
 * x_dtype (MOE_DT_F32 or MOE_DT_BF16), rows ldx elements apart.  For each row
 * with largest magnitude a, the scale s is the fp32 value nearest to a / 127, at
 * least 2^-120, and 1 if a = 0; q [rows, cols] is the integer nearest to x / s,
 * ties to even (of the exact quotient).  A row with a NaN or an infinity gets
 * the scale NaN and codes 0.
 * rows >= 0 (0 enqueues nothing), 16 <= cols <= 2^20 a multiple of 16 and
 * ldx >= cols a multiple of 16 bytes, else MOE_ERR_INVALID; x and q 16-byte
 * aligned, scale 4-byte.  q and scale must not overlap x.  No workspace. */
int moe_quantize_tokens(const void *x, int32_t x_dtype, int32_t rows, int32_t cols, int64_t ldx, int8_t *q,
                        float *scale, void *stream);

/* out [m, n] = x [m, k] w[n, k]^T with int8 operands, a scale per token and one
 * per output channel:
 *   out[i, j] = x_scale[i] * w_scale[j] * sum_c x[i, c] * w[j, c]
 * (the sum exact, then rounded to fp32 and multiplied by x_scale and by w_scale:
 * both products must stay within fp32's range).  x is MOE_DT_I8CH codes
 * with x_scale [m], or MOE_DT_BF16 / MOE_DT_F32 rows, which are quantised as
 * moe_quantize_tokens does first (x_scale NULL, workspace needed).  Codes may
 * take every int8 value.  out_dtype MOE_DT_F32, or MOE_DT_BF16 (one rounding
 * more).  0 <= m <= 2^20 (0 enqueues nothing), 1 <= n <= 2^20, 16 <= k <=
 * MOE_I8_MAX_K a multiple of 16, else MOE_ERR_INVALID; x, w, out and ws 16-byte
 * aligned, the scales 4-byte.  out must not overlap an input.  The workspace
 * size is 0 for I8CH rows and for sizes out of range. */
#define MOE_I8_MAX_K 131056
size_t moe_channel_matmul_workspace_bytes(int32_t x_dtype, int32_t m, int32_t k);
int moe_channel_matmul(const void *x, int32_t x_dtype, const float *x_scale, const int8_t *w, const float *w_scale,
                       int32_t m, int32_t n, int32_t k, void *out, int32_t out_dtype, void *ws, size_t ws_bytes,
                       void *stream);

/* How evenly a selection loads the experts, sequence by sequence.  With s the
 * scores of cfg->score, p[t, e] = s[t, e] / sum_e s[t, e]:
 *   counts[q, e]  selections of expert e by the tokens of sequence q
 *   tokens[q]     tokens of sequence q
 *   prob[q, e]    mean of p[t, e] over them (0 if there are none)
 *   loss[q]       sum_e f[q, e] prob[q, e],  f[q, e] = E counts[q, e] / (top_k tokens[q])
 * so f is 1 and the loss 1 where the load is even.  A caller's balance loss is any
 * weighted sum of loss[]; its gradient comes from moe_route_backward.
 * logits [T, E] fp32; topk_idx [T, k] (entries outside [0, E) are not counted);
 * mask [T] bytes or NULL: tokens whose byte is 0 (padding) belong to no
 * sequence, and their logits have no effect; seq_offsets [n_seq + 1] int32, in
 * device memory: sequence q has the tokens seq_offsets[q] <= t < seq_offsets[q +
 * 1] (ascending values in [0, T], else the results are unspecified; empty
 * sequences are allowed and tokens before the first or behind the last offset
 * belong to none), or NULL with n_seq 1: all tokens.  A token whose scores sum
 * to less than 2^-126 has p = 0.  counts [n_seq, E], tokens [n_seq] int32; prob
 * [n_seq, E], loss [n_seq] fp32.  Scores are fp32, their sums over tokens fp32
 * within a workgroup and fp64 beyond, in a fixed order.
 * 1 <= n_seq <= 2^20, else MOE_ERR_INVALID; the workspace has at least
 * moe_balance_workspace_bytes(cfg, n_seq) bytes (0 for invalid arguments; monotone
 * in n_tokens, n_expert and n_seq) and is 16-byte aligned.  Outputs must not
 * overlap inputs. */
size_t moe_balance_workspace_bytes(const moe_config *cfg, int32_t n_seq);
int moe_balance(const moe_config *cfg, const float *logits, const int32_t *topk_idx, const uint8_t *mask,
                const int32_t *seq_offsets, int32_t n_seq, int32_t *counts, int32_t *tokens, float *prob, float *loss,
                void *ws, size_t ws_bytes, void *stream);

/* Gradient of the router's logits: d_logits [T, E] fp32 of
 *   sum_{t, j} d_topk_w[t, j] w[t, j] + sum_q d_loss[q] loss[q]
 * where w are the selection's weights (route_scale * s, divided by the sum of the
 * selected s if groups->normalise; groups == NULL: it is 1) and loss is
 * moe_balance's with its counts as constants, as topk_idx and the expert groups
 * are.  d_topk_w [T, k] and d_loss [n_seq] may be NULL (one of them at most);
 * with d_loss, counts and tokens are moe_balance's outputs.  topk_idx entries
 * outside [0, E) have no weight; an expert listed twice has the sum of both.
 * Renormalised weights whose scores are all 0 as the selection's fp32 scores
 * (below 2^-150) are 0, as there, and have no gradient.
 * Every row is written: rows of tokens that the mask or the offsets leave out are
 * zeros, whatever their logits and d_topk_w hold.  The other arguments as for
 * moe_balance.  No workspace; d_logits must not overlap an input. */
int moe_route_backward(const moe_config *cfg, const moe_groups *groups, const float *logits, const int32_t *topk_idx,
                       const float *d_topk_w, const uint8_t *mask, const int32_t *seq_offsets, int32_t n_seq,
                       const int32_t *counts, const int32_t *tokens, const float *d_loss, float *d_logits,
                       void *stream);

/* Router look-ahead, its read half (NeutronStar fork page, "Cross-layer
 * expert prefetch": the next layer's router runs on this layer's hidden
 * state and the experts it predicts are read while the GPU still computes).
 * The predictions come from moe_route called with the next layer's router
 * weights on this layer's input x; this call then reads the weights of the
 * experts ids [n_ids] int32 (device memory, e.g. that topk_idx; entries
 * outside [0, n_expert) are skipped on the device) of the layer w: bit 0 of
 * `which` selects gate, bit 1 up, bit 2 down (for MOE_DT_Q8B32 the codes
 * and their scales, for MOE_DT_F8B128 and MOE_DT_I8CH the codes), and `rows` > 0 limits the read to the leading rows of
 * each selected matrix (gate and up have d_ff rows, down d_model; 0: all).
 * It writes no memory, so no result of any call changes; the reads leave
 * those weights in the device's memory-side cache (the Infinity Cache),
 * where that layer's expert kernels find them if they run before other
 * traffic evicts them.  Meant for a second stream, beside the work of the
 * current layer: `workgroups` (1 .. MOE_PREFETCH_MAX_WORKGROUPS) fixes the
 * launch's size, so that it takes only part of the chip.
 * 0 <= n_ids <= MOE_PREFETCH_MAX_IDS (0 enqueues nothing), 1 <= which <= 7,
 * rows >= 0, the selected matrices as in moe_weights with their scale
 * arrays (MOE_DT_Q8B32) 16-byte aligned too, else MOE_ERR_INVALID;
 * an expert matrix of more than 2^31 - 1 bytes is MOE_ERR_UNSUPPORTED.  No
 * workspace.  events: NULL, or 2 hipEvent_t created by the caller (entries
 * may be NULL) that receive the start and end timestamps of the dispatch. */
#define MOE_PREFETCH_MAX_IDS 65536
#define MOE_PREFETCH_MAX_WORKGROUPS 4096
int moe_prefetch_experts(const moe_config *cfg, const moe_weights *w, const int32_t *ids, int32_t n_ids,
                         int32_t which, int32_t rows, int32_t workgroups, void **events, void *stream);

/* Human-readable name of a status code (static storage). */
const char *moe_status_str(int status);

#ifdef __cplusplus
}
#endif
#endif
