/*
 * moe_block.h -- the dense operators of an MoE block around its routed experts, and the
 * optimizer step that trains them, for AMD Instinct MI355X (gfx950):
 *
 *   moe_ffn_*    a gated feed-forward block with bf16 weights (shared experts kept dense,
 *                dense layers), with its input and weight gradients;
 *   moe_norm_*   the RMS norms after a block and before the next one, fused with the block's
 *                gate and residual scale, with their gradients;
 *   moe_adamw_*  one AdamW step over many tensors at once, states in fp32 or in 8 bits.
 *
 * Sources: LazyLoRA README, "The engine" (two shared experts beside the routed ones in each MoE
 * layer), "How you know this is real" (rmsnorm among the layer's operators), the training script's
 * AdamW over the adapter with gradient clipping; OCP Microscaling Formats (MX) v1.0 for E4M3.
 *
 * The conventions of moe.h hold: device pointers owned by the caller, calls that only enqueue
 * on the given stream, synchronous argument checks that leave every output untouched, status
 * codes with their text in moe_last_error().  The current device must be the one that holds
 * the buffers.  Outputs overlap no other buffer of a call, but where a call says so (refused
 * otherwise).  One handle may be used from one stream at a time; calls under stream capture
 * are recorded with the pointers and numbers they were given (two graphs that use one handle
 * share its workspace: replay them one after the other).
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ gated feed-forward */

/* y = act(x Wg^T, x Wu^T) Wd^T with bf16 weights Wg, Wu [I][D] and Wd [D][I], the activation a
 * moe_act of moe.h.  Products of bf16 values, fp32 accumulation; the activation is evaluated
 * in fp32.  What the second product reads follows the type asked for its result: for a bf16
 * result h = act(g, u) is rounded once to bf16 (2^-8 relative at most), for an fp32 result h
 * enters as three bf16 terms that hold its 24 bits.  The gradients' dg and du likewise. */
typedef struct {
    int32_t width;       /* D: multiple of 8, at most 2^20 */
    int32_t inter;       /* I: multiple of 8, at most 2^20 */
    int32_t max_tokens;  /* largest T of any call, at most 2^24; sizes the workspace */
    int32_t act;         /* moe_act */
    uint32_t flags;      /* MOE_FFN_* */
} moe_ffn_desc;

enum {
    MOE_FFN_BACKWARD = 1u  /* workspace for moe_ffn_backward */
};

typedef struct moe_ffn moe_ffn;

/* D 3584, I 6144 (the two shared experts of the K3 layer as one block), max_tokens 4096,
 * SwiGLU, with backward. */
void moe_ffn_desc_init(moe_ffn_desc *d);
moe_status moe_ffn_workspace_size(const moe_ffn_desc *d, size_t *bytes);

/* The weights (bf16 bit patterns, 16-byte aligned) and the workspace (256-byte aligned) are
 * borrowed until moe_ffn_destroy(); the weights may be updated between calls. */
moe_status moe_ffn_create(const moe_ffn_desc *d, const uint16_t *w_gate, const uint16_t *w_up, const uint16_t *w_down,
                          void *workspace, size_t ws_bytes, moe_ffn **out);

/* y [T][D] of dtype yt (fp32 or bf16) = ffn(x), or y += ffn(x) with accumulate != 0 (added in
 * fp32, rounded once).  x is [T][D] bf16.  saved_gu, if not NULL, receives the pre-activations
 * [T][2][I] fp32 (gate, up) for moe_ffn_backward().  All 16-byte aligned.  T = 0: no-op. */
moe_status moe_ffn_forward(moe_ffn *f, const uint16_t *x, int32_t T, void *y, int32_t yt, int32_t accumulate,
                           float *saved_gu, void *stream);

/* Gradients of sum_t <dy[t], ffn(x)[t]>: dx [T][D] of dtype dxt (added to what dx holds with
 * accumulate != 0), dw_gate and dw_up [I][D] and dw_down [D][I] of dtype dwt (overwritten).
 * Any of the four may be NULL: it is not computed.  dy is [T][D] bf16; saved_gu from
 * moe_ffn_forward() on the same x, or NULL to recompute it.  The sums run in a fixed order.
 * T = 0 writes zero weight gradients. */
moe_status moe_ffn_backward(moe_ffn *f, const uint16_t *x, const uint16_t *dy, int32_t T, const float *saved_gu,
                            void *dx, int32_t dxt, int32_t accumulate, void *dw_gate, void *dw_up, void *dw_down,
                            int32_t dwt, void *stream);
void moe_ffn_destroy(moe_ffn *f);

/* ------------------------------------------------------------------ block norms */

/* Between two blocks, for each token (all arithmetic in fp32):
 *   n     = y rsqrt(mean(y^2) + eps_post) * w_post      (n = y without MOE_NORM_POST)
 *   r_out = res_scale r + branch_scale gate * n         (rounded to r_dtype)
 *   x     = r_out rsqrt(mean(r_out^2) + eps_next) * w_next  (with MOE_NORM_NEXT; of the stored r_out)
 * With y NULL in the calls the residual passes unchanged (r_out = r, not written) and only x
 * is formed: the norm before a first block. */
typedef enum {
    MOE_GATE_NONE = 0,     /* gate = 1 */
    MOE_GATE_CHANNEL = 1,  /* [D] fp32 */
    MOE_GATE_TOKEN = 2,    /* [T] fp32 */
    MOE_GATE_FULL = 3      /* [T][D] of y_dtype */
} moe_gate;

enum {
    MOE_NORM_POST = 1u,     /* norm of the block's output, weights w_post */
    MOE_NORM_NEXT = 2u,     /* norm before the next block, weights w_next */
    MOE_NORM_BACKWARD = 4u  /* workspace for moe_norm_backward */
};

typedef struct {
    int32_t width;       /* D: 1..16384 */
    int32_t max_tokens;  /* 0..2^30 */
    int32_t r_dtype, y_dtype, x_dtype, w_dtype;  /* moe_dtype: residual, block output, next input, norm weights */
    int32_t gate;        /* moe_gate */
    float eps_post, eps_next;  /* > 0 */
    float res_scale, branch_scale;
    uint32_t flags;
} moe_norm_desc;

typedef struct moe_norm moe_norm;

/* D 3584, max_tokens 4096, fp32 residual, output and weights, bf16 next input, no gate, eps 1e-6, scales 1,
 * both norms with backward. */
void moe_norm_desc_init(moe_norm_desc *d);
moe_status moe_norm_workspace_size(const moe_norm_desc *d, size_t *bytes);

/* w_post and w_next: [D] of w_dtype, borrowed, required exactly when their flag is set (NULL otherwise).
 * The workspace may be NULL when its size is 0. */
moe_status moe_norm_create(const moe_norm_desc *d, const void *w_post, const void *w_next, void *workspace,
                           size_t ws_bytes, moe_norm **out);

/* r, r_out [T][D] of r_dtype, y [T][D] of y_dtype or NULL, gate as the descriptor says (NULL for
 * MOE_GATE_NONE or without y), x [T][D] of x_dtype (NULL without MOE_NORM_NEXT), rstd [2][T] fp32: the
 * two reciprocal roots, for moe_norm_backward (NULL: not kept).  r_out may be r itself.  Buffers must be
 * aligned to their element; 16-byte alignment with D a multiple of 8 takes the wide loads. */
moe_status moe_norm_forward(moe_norm *h, const void *r, const void *y, const void *gate, int32_t T, void *r_out,
                            void *x, float *rstd, void *stream);

/* Gradients for the upstream dr_out [T][D] of r_dtype (NULL: zero) and dx [T][D] of x_dtype (NULL exactly
 * without MOE_NORM_NEXT), given the forward's y, gate, r_out (r itself when y was NULL) and rstd:
 *   dr [T][D] of r_dtype; dy [T][D] of y_dtype (NULL exactly when y is); dgate in the gate's shape, fp32 for
 *   CHANNEL and TOKEN, y_dtype for FULL; dw_post, dw_next [D] of w_dtype (all overwritten).
 * dr may be dr_out itself.  dgate and the two dw may be NULL: not computed.  Sums over tokens run in a fixed order.
 * T = 0 writes zero dw and zero dgate of CHANNEL. */
moe_status moe_norm_backward(moe_norm *h, const void *y, const void *gate, const void *r_out, const float *rstd,
                             const void *dr_out, const void *dx, int32_t T, void *dr, void *dy, void *dgate,
                             void *dw_post, void *dw_next, void *stream);
void moe_norm_destroy(moe_norm *h);

/* ------------------------------------------------------------------ AdamW */

/* One step t = 1, 2, ... for every element of every tensor (fp32 arithmetic):
 *   g' = clip g                     clip = max_norm / max(max_norm, ||all g||), 1 with max_norm = 0
 *   m  = beta1 m + (1 - beta1) g'
 *   v  = beta2 v + (1 - beta2) g'^2
 *   p  = p (1 - lr s wd) - lr s / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * with the tensor's own lr scale s and weight decay wd.  With max_norm > 0 a step whose gradient
 * norm is not finite changes nothing, the step count included; squares are formed in fp32, so a gradient of
 * 2^62 or more in size may count as not finite.
 *
 * MOE_STATE_E4M3 keeps m and sqrt(v) as OCP E4M3 codes, one byte each, with an fp32 scale for each
 * run of 256 consecutive elements of a tensor (the last run may be shorter): scale = max|.| / 448,
 * code = rne(value / scale), value = code * scale.  A run whose scale is below 2^-126 is stored as
 * zeros; a positive sqrt(v) is never stored as code zero (it takes the smallest code), so a decayed
 * moment is not divided by a lost one.  The parameter update uses the unquantized new moments. */
typedef enum { MOE_STATE_F32 = 0, MOE_STATE_E4M3 = 1 } moe_state_fmt;

typedef struct {
    double beta1, beta2;  /* 0 <= beta < 1 */
    double eps;           /* > 0 */
    double max_norm;      /* global gradient-norm clip, 0 = none */
    int32_t state;        /* moe_state_fmt */
    int32_t max_tensors;  /* 1..2^20; sizes the workspace with max_elements */
    int64_t max_elements; /* total over the tensors, at most 2^40 */
} moe_adamw_desc;

/* One tensor of n elements, contiguous.  param is fp32 or bf16 (param_dtype); master, if not NULL, is
 * its fp32 copy: the step updates master and stores its rounding in param (without it a bf16 parameter
 * is updated in fp32 and rounded).  grad is fp32 or bf16.  MOE_STATE_F32: m, v fp32, the scales NULL;
 * MOE_STATE_E4M3: m, v bytes, m_scale and v_scale [ceil(n / 256)] fp32.  Start them at zero.  Pointers
 * aligned to their element. */
typedef struct {
    void *param;
    float *master;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
    int32_t param_dtype, grad_dtype;
    float weight_decay, lr_scale;
} moe_adamw_tensor;

typedef struct moe_adamw moe_adamw;

/* betas 0.9, 0.999, eps 1e-8, no clipping, fp32 states, 1024 tensors, 2^28 elements. */
void moe_adamw_desc_init(moe_adamw_desc *d);
moe_status moe_adamw_workspace_size(const moe_adamw_desc *d, size_t *bytes);
moe_status moe_adamw_create(const moe_adamw_desc *d, void *workspace, size_t ws_bytes, moe_adamw **out);

/* Take these tensors (the array is copied; the buffers are borrowed until the next bind or the destroy),
 * enqueueing their table's upload on the stream.  Nothing that a step writes may overlap another buffer
 * of the set (MOE_ERR_INVALID_ARG), so a tensor named twice is refused.  n = 0 tensors is allowed.
 * A captured step works on the tensors that are bound when it is replayed: replay it only while they are as
 * many and of the sizes it was captured with. */
moe_status moe_adamw_bind(moe_adamw *a, const moe_adamw_tensor *t, int32_t n, void *stream);

/* Set the number of steps taken so far (0 in a new run; kept on the device, so a captured step counts its
 * replays).  Required once before the first step. */
moe_status moe_adamw_set_step(moe_adamw *a, int64_t steps, void *stream);

/* One step with learning rate *lr_dev (a device fp32) or, with lr_dev NULL, lr.  grad_norm, if not NULL,
 * receives the gradients' norm before clipping as a device fp32 (needs max_norm > 0). */
moe_status moe_adamw_step(moe_adamw *a, double lr, const float *lr_dev, float *grad_norm, void *stream);
void moe_adamw_destroy(moe_adamw *a);

#ifdef __cplusplus
}
#endif
#endif /* MOE_BLOCK_H */
