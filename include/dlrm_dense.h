/*
 * dlrm_dense.h -- the dense network around the dot interaction: a dense layer
 * with bias, activation, dropout and residual, its gradient, dropout by itself
 * and a mixture-of-experts layer for a few tokens.
 *
 * "DLRM For PyTorch", §Model architecture: the interaction output is fed to
 * the "top MLP", --top_mlp_sizes 1024,1024,512,256,1.  dlrm_linear_fwd and
 * dlrm_linear_bwd are one layer of it (or of the bottom MLP) in training and
 * in serving; dropout and the mixture have no counterpart on the pages.
 *
 * Shared by every call (next to the conventions of dlrm.h: asynchronous on
 * `stream`, nothing allocated, host errors before anything is enqueued,
 * inputs must not alias outputs, bitwise reproducible results):
 *  - dtype is DLRM_F32, DLRM_F16 or DLRM_BF16 and holds for every void*
 *    tensor of the call.  Sums are held in fp32; each output is rounded once.
 *  - Matrices are row-major with unit column stride; ld* is the distance
 *    between rows in elements (at least the row's width; it is not read when
 *    there is one row).  Any alignment of at least the element's is taken:
 *    16-byte aligned rows are the fast path.
 *  - M may be 0: nothing is written but the gradients that sum over rows,
 *    which become zero.
 *  - Activations a(z): NONE z; RELU z < 0 ? 0 : z (slope 0 at 0); GELU
 *    z Phi(z), Phi the normal distribution function; SILU z / (1 + e^-z).
 *
 * Dropout.  Element (row, col) of an M x N matrix takes 16 bits from
 * Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
 * as 1, 2, 3", SC 2011) with key (rng[0] low, rng[0] high) and counter
 * (col / 8, row, rng[1] low, rng[1] high): half (col % 2, 0 the low one) of
 * output word (col % 8) / 2.  With t = floor(65536 p + 0.5) the element is
 * kept where its number is at least t and then scaled by 65536 / (65536 - t),
 * the inverse of the probability in force, so the expectation is exact;
 * dropped elements are 0 whatever their value.  The mask depends on rng, p and
 * the position alone: a call with the same rng makes the same mask again, so
 * none is stored.  rng is read on the device, so a captured graph can advance
 * it; two calls that share an rng value share their mask.
 */
#ifndef DLRM_GB300_DENSE_H
#define DLRM_GB300_DENSE_H

#include "dlrm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DLRM_ACT_NONE = 0,
    DLRM_ACT_RELU = 1,
    DLRM_ACT_GELU = 2,
    DLRM_ACT_SILU = 3
} dlrm_act;

/*
 * dlrm_dropout_fwd -- y = residual + drop(x).
 *   d_x [M][N]; d_residual [M][N] or NULL; d_y [M][N] (output)
 *   p in [0, 1), 65536 p below 65535.5;  d_rng: device uint64 [2] (may be NULL
 *   when p is 0), 8-byte aligned
 */
dlrm_status dlrm_dropout_fwd(const void* d_x, int64_t ldx, const void* d_residual, int64_t ldr, dlrm_dtype dtype,
                             int M, int N, double p, const uint64_t* d_rng, void* d_y, int64_t ldy, void* stream);

/* dlrm_dropout_bwd -- grad_x = drop(grad_y) with the forward's mask (same p and
 * rng).  The residual's gradient is grad_y itself. */
dlrm_status dlrm_dropout_bwd(const void* d_grad_y, int64_t ldg, dlrm_dtype dtype, int M, int N, double p,
                             const uint64_t* d_rng, void* d_grad_x, int64_t lddx, void* stream);

/*
 * dlrm_linear_fwd -- one dense layer.
 *
 *   z = x W^T + bias;   y = residual + drop(a(z))
 *
 *   d_x [M][K];  d_w [N][K] (PyTorch's Linear layout);  d_bias fp32 [N] or NULL
 *   d_residual [M][N] or NULL;  d_y [M][N] (output)
 *   d_pre [M][N] or NULL: receives z for dlrm_linear_bwd (output).  For RELU
 *     without a residual y itself serves as well (y > 0 exactly where the
 *     gradient passes), and d_pre can be NULL.
 *   p, d_rng: dropout as in dlrm_dropout_fwd; p = 0 for none
 *   d_workspace: dlrm_linear_fwd_workspace_size bytes, 256-byte aligned (may
 *     be NULL when that is 0)
 *   d_status may be NULL; gets DLRM_STATUS_TIMEOUT if a bounded wait gave up.
 * fp32 operands are split into three bf16 parts each, whose six products of
 * weight 2^-16 and more are summed on the tensor cores: the error stays at that
 * of an fp32 sum.  A product of two infinities is a NaN there, and infinite or
 * NaN operands otherwise give what fp32 gives.  Requires N >= 1, K >= 1 and sizes up to
 * 2^31 - 2^20 - 1 (DLRM_ERR_UNSUPPORTED).
 */
dlrm_status dlrm_linear_fwd(const void* d_x, int64_t ldx, const void* d_w, int64_t ldw, const float* d_bias,
                            const void* d_residual, int64_t ldr, dlrm_dtype dtype, int M, int N, int K, dlrm_act act,
                            double p, const uint64_t* d_rng, void* d_y, int64_t ldy, void* d_pre, int64_t ldp,
                            void* d_workspace, size_t workspace_bytes, uint32_t* d_status, void* stream);

/* Workspace bytes of dlrm_linear_fwd for these operands (the addresses and row
 * distances say whether an operand has to be laid out again; nothing is read
 * through them).  0 for invalid sizes too. */
size_t dlrm_linear_fwd_workspace_size(const void* d_x, int64_t ldx, const void* d_w, int64_t ldw, dlrm_dtype dtype,
                                      int M, int N, int K);

/*
 * dlrm_linear_bwd -- gradient of dlrm_linear_fwd.
 *
 *   dZ = a'(pre) * drop(grad_y);  grad_x = dZ W;  grad_w = dZ^T x;
 *   grad_bias[n] = sum over rows of dZ[:, n]
 *
 *   d_grad_y [M][N];  d_x, d_w as in the forward;  d_pre [M][N] (NULL for
 *   DLRM_ACT_NONE);  d_grad_x [M][K], d_grad_w [N][K], d_grad_bias fp32 [N]
 *   (outputs, each may be NULL: that gradient is not computed)
 * The residual's gradient is grad_y itself.  dZ is not rounded to dtype: for NONE
 * and RELU it is grad_y's own values, the dropout's scale being applied to the
 * sums; for GELU and SILU fp16 and bf16 hold it as the sum of two values, which
 * doubles the products' work (an infinite weight or input can then give a NaN
 * where it meets a second value of 0).  fp16: the second value lies on a grid of
 * 2^-24, as grad_y's least values do.
 */
dlrm_status dlrm_linear_bwd(const void* d_grad_y, int64_t ldg, const void* d_x, int64_t ldx, const void* d_w,
                            int64_t ldw, const void* d_pre, int64_t ldp, dlrm_dtype dtype, int M, int N, int K,
                            dlrm_act act, double p, const uint64_t* d_rng, void* d_grad_x, int64_t lddx,
                            void* d_grad_w, int64_t lddw, float* d_grad_bias, void* d_workspace,
                            size_t workspace_bytes, uint32_t* d_status, void* stream);

/* Workspace bytes of dlrm_linear_bwd when all three gradients are asked for
 * (asking for fewer needs no more). */
size_t dlrm_linear_bwd_workspace_size(const void* d_grad_y, int64_t ldg, const void* d_x, int64_t ldx,
                                      const void* d_w, int64_t ldw, dlrm_dtype dtype, int M, int N, int K,
                                      dlrm_act act, double p);

/* The most tokens, experts and experts per token dlrm_moe_fwd takes. */
#define DLRM_MOE_MAX_TOKENS 64
#define DLRM_MOE_MAX_EXPERTS 256
#define DLRM_MOE_MAX_TOP_K 8

/*
 * dlrm_moe_fwd -- a mixture-of-experts layer for a few tokens, in two kernels.
 *
 *   logits[t][e] = x[t] . w_router[e]                       (fp32)
 *   ids[t][0..k): the k experts of the largest logits, largest first, equal
 *     ones by lower index (a NaN counts as largest, -0 equals 0)
 *   probs[t][j] = exp(logits[t][ids[t][j]]) / sum over j of the same
 *   h(t, e) = a(w1[e] x[t])                                 (gated = 0)
 *   h(t, e) = a(w1[e][0..I) x[t]) * (w1[e][I..2I) x[t])     (gated = 1)
 *   y[t] = residual[t] + sum over j of probs[t][j] * w2[ids[t][j]] h(t, ids[t][j])
 *
 *   d_x [T][H];  d_w_router [E][H];  d_w1 [E][I or 2I][H];  d_w2 [E][H][I], the
 *   last three contiguous;  d_residual [T][H] or NULL;  d_y [T][H] (output)
 *   d_ids int32 [T][k] (output);  d_probs fp32 [T][k] (output)
 *   d_workspace: dlrm_moe_fwd_workspace_size bytes, 256-byte aligned
 *   d_status may be NULL; gets DLRM_STATUS_TIMEOUT if a bounded wait gave up.
 * probs * h enters the second product with 21 bits or more: in fp32, as the sum
 * of three bf16 values, or of two fp16 values times a power of two of their own,
 * so its size is not bound by fp16's range.  (Where a second or third value is 0
 * an infinite weight gives a NaN.)
 * Experts that no token chose are not read.  Requires H, I >= 1, 0 <= T <=
 * DLRM_MOE_MAX_TOKENS, 1 <= E <= DLRM_MOE_MAX_EXPERTS and 1 <= k <=
 * min(E, DLRM_MOE_MAX_TOP_K); larger T, E or k, H or I past 2^31 - 2^20 - 1, and
 * 2^31 weight rows (E H, 2 E I) or more are DLRM_ERR_UNSUPPORTED.
 */
dlrm_status dlrm_moe_fwd(const void* d_x, int64_t ldx, const void* d_w_router, const void* d_w1, const void* d_w2,
                         const void* d_residual, int64_t ldr, dlrm_dtype dtype, int T, int H, int I, int E, int k,
                         dlrm_act act, int gated, void* d_y, int64_t ldy, int32_t* d_ids, float* d_probs,
                         void* d_workspace, size_t workspace_bytes, uint32_t* d_status, void* stream);

/* Workspace bytes of dlrm_moe_fwd (0 for invalid sizes and for T = 0). */
size_t dlrm_moe_fwd_workspace_size(dlrm_dtype dtype, int T, int H, int I, int E, int k);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_GB300_DENSE_H */
