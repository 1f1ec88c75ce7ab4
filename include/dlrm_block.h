/*
 * dlrm_block.h -- residual blocks of the dense network: the norms after a block
 * and before the next one with the block's gate and residual scale, the choice
 * of experts and the order of the tokens by expert, the way of the tokens to
 * their experts and back, and activations kept in 8 bits with the gradient of a
 * dense layer that reads them.
 *
 * None of these has a counterpart on the pages; they are what deeper dense
 * networks around the interaction, and mixtures in training, need next to
 * dlrm_dense.h, whose conventions hold here: asynchronous on `stream`, nothing
 * allocated, host errors before anything is enqueued, inputs must not alias
 * outputs (nor outputs one another), bitwise reproducible results, sums in fp32,
 * each output rounded once, row-major matrices with unit column stride and ld*
 * the distance between rows in elements, any alignment of at least the
 * element's (16-byte aligned rows are the fast path), M or T = 0 allowed.
 */
#ifndef DLRM_GB300_BLOCK_H
#define DLRM_GB300_BLOCK_H

#include "dlrm_dense.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DLRM_NORM_RMS = 0,   /* v / sqrt(mean(v^2) + eps) */
    DLRM_NORM_LAYER = 1  /* (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) */
} dlrm_norm;

typedef enum {
    DLRM_GATE_NONE = 0,    /* the gate's own value */
    DLRM_GATE_SIGMOID = 1, /* 1 / (1 + e^-g) */
    DLRM_GATE_SILU = 2     /* g / (1 + e^-g) */
} dlrm_gate;

/* The widest row dlrm_block_norm_fwd and _bwd take, the most experts of the
 * choice and of the sort, and the most experts a token. */
#define DLRM_BLOCK_MAX_WIDTH 8192
#define DLRM_ROUTE_MAX_EXPERTS 256
#define DLRM_ROUTE_MAX_TOP_K 8

/* ------------------------------------------------- norms, gate and residual */
/*
 * dlrm_block_norm_fwd -- the end of one block and the beginning of the next.
 *
 *   u = norm(y) * w_post + b_post
 *   r = residual + scale * gate(g) * u
 *   h = norm(r) * w_pre + b_pre
 *
 *   d_y [M][N]: the block's output, or NULL: r is the residual itself (d_r has
 *     to be NULL then, and d_gate, d_w_post, d_b_post and d_scale too)
 *   d_gate [M][gate_cols] or NULL (1 everywhere); gate_cols is N, or 1: one
 *     value a row
 *   d_residual [M][N] or NULL (0; only with d_y)
 *   d_w_post, d_b_post, d_scale, d_w_pre, d_b_pre: fp32 [N] or NULL (1, 0, 1, 1, 0)
 *   d_r [M][N] (output; has to be given with d_y)
 *   d_h [M][N] (output), or NULL: no norm of r (d_w_pre and d_b_pre NULL then)
 *   d_stats fp32 [M][4], 16-byte aligned (output), or NULL: mean and
 *     1 / sqrt(.. + eps) of y, then those of r, for dlrm_block_norm_bwd; 0 for
 *     means of RMS and for norms that are not taken
 *   eps >= 0 and finite
 * h and r's statistics are taken from r before its rounding to dtype.  A row of
 * zeros with eps = 0 is a row of NaN, as the formula says.  Squares are summed in
 * fp32: where their sum passes its range (values of some 2^63) 1 / sqrt is 0.
 * Requires 1 <= N <= DLRM_BLOCK_MAX_WIDTH (more: DLRM_ERR_UNSUPPORTED).
 */
dlrm_status dlrm_block_norm_fwd(const void* d_y, int64_t ldy, const void* d_gate, int64_t ldg, int gate_cols,
                                const void* d_residual, int64_t ldres, const float* d_w_post, const float* d_b_post,
                                const float* d_scale, const float* d_w_pre, const float* d_b_pre, dlrm_dtype dtype,
                                int M, int N, dlrm_norm norm, dlrm_gate gate_act, double eps, void* d_r, int64_t ldr,
                                void* d_h, int64_t ldh, float* d_stats, void* stream);

/*
 * dlrm_block_norm_bwd -- gradient of dlrm_block_norm_fwd.
 *
 *   dr = grad_r + the gradient through norm(r) of grad_h * w_pre
 *   grad_residual = dr;  du = dr * scale * gate(g)
 *   grad_y = the gradient through norm(y) of du * w_post
 *   grad_gate = gate'(g) * dr * scale * u  (summed over the row where gate_cols is 1)
 *   grad_w_post, grad_b_post, grad_scale, grad_w_pre, grad_b_pre = the sums over
 *     rows of du * norm(y), du, dr * gate(g) * u, grad_h * norm(r), grad_h
 *
 *   d_grad_r [M][N] or NULL (0);  d_grad_h [M][N] or NULL: no norm of r was taken
 *     (d_grad_r and d_y are needed then)
 *   d_y, d_gate, d_w_post, d_b_post, d_scale, d_w_pre as in the forward (d_y NULL:
 *     no block; the outputs of its side have to be NULL then)
 *   d_r [M][N]: the forward's r (its residual where d_y was NULL); NULL without d_grad_h
 *   d_stats: the forward's
 *   d_grad_y, d_grad_gate [M][gate_cols], d_grad_residual (outputs, each may be NULL)
 *   d_grad_w_post .. d_grad_b_pre fp32 [N] (outputs, each may be NULL)
 *   d_workspace: dlrm_block_norm_bwd_workspace_size bytes, 256-byte aligned (may be
 *     NULL when that is 0 or none of the five vectors is asked for)
 * grad_y and the vectors' sums go by dr before its rounding to dtype.
 */
dlrm_status dlrm_block_norm_bwd(const void* d_grad_r, int64_t ldgr, const void* d_grad_h, int64_t ldgh, const void* d_y,
                                int64_t ldy, const void* d_gate, int64_t ldg, int gate_cols, const void* d_r,
                                int64_t ldr, const float* d_stats, const float* d_w_post, const float* d_b_post,
                                const float* d_scale, const float* d_w_pre, dlrm_dtype dtype, int M, int N,
                                dlrm_norm norm, dlrm_gate gate_act, void* d_grad_y, int64_t ldgy, void* d_grad_gate,
                                int64_t ldgg, void* d_grad_residual, int64_t ldgres, float* d_grad_w_post,
                                float* d_grad_b_post, float* d_grad_scale, float* d_grad_w_pre, float* d_grad_b_pre,
                                void* d_workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of dlrm_block_norm_bwd for M rows of N columns (0 for invalid sizes and for M = 0). */
size_t dlrm_block_norm_bwd_workspace_size(int M, int N);

/* --------------------------------------------------------- choice of experts */
/*
 * dlrm_route_fwd -- the k experts of each token and their shares.
 *
 *   ids[t][0..k): the experts of the largest logits, largest first, equal ones by
 *     lower index (a NaN counts as largest, -0 equals 0)
 *   probs[t][j] = exp(logits[t][ids[t][j]]) / sum over j of the same
 * A logit of -infinity closes its expert to the token: it is never chosen.  Where
 * fewer than k are open the last ids are -1 with probs 0 (all of them, where none
 * is).  Where the largest is a NaN or +infinity the probs of the chosen are NaN.
 *   d_logits [T][E];  d_ids int32 [T][k], d_probs fp32 [T][k] (outputs)
 * Requires 1 <= E <= DLRM_ROUTE_MAX_EXPERTS, 1 <= k <= min(E, DLRM_ROUTE_MAX_TOP_K)
 * (larger E or k: DLRM_ERR_UNSUPPORTED).
 */
dlrm_status dlrm_route_fwd(const void* d_logits, int64_t ldl, dlrm_dtype dtype, int T, int E, int k, int32_t* d_ids,
                           float* d_probs, void* stream);

/*
 * dlrm_route_bwd -- gradient of dlrm_route_fwd's probs.
 *
 *   grad_logits[t][ids[t][j]] = probs[t][j] (grad_probs[t][j] - sum over i of grad_probs[t][i] probs[t][i])
 * and 0 for experts that were not chosen.  The choice itself has no gradient.
 *   d_grad_probs fp32 [T][k];  d_ids, d_probs: the forward's;  d_grad_logits [T][E] (output)
 * ids outside [0, E) (-1) take no part.  Of equal ids of a token the last one counts.
 */
dlrm_status dlrm_route_bwd(const float* d_grad_probs, const int32_t* d_ids, const float* d_probs, dlrm_dtype dtype,
                           int T, int E, int k, void* d_grad_logits, int64_t ldgl, void* stream);

/*
 * dlrm_expert_sort -- the order of the tokens' choices by expert.
 *
 * Choice c = t k + j is token t's j-th.  Choices of expert 0 come first, then those
 * of expert 1 and so on, equal experts in the order of c:
 *   offsets[e] .. offsets[e + 1]: the places of expert e's choices
 *   slots[t][j]: the place of a choice, -1 where its id is outside [0, E)
 *   order[place]: the choice at a place, -1 from offsets[E] on
 *   d_ids int32 [T][k];  d_offsets int32 [E + 1], d_slots int32 [T][k] (outputs);
 *   d_order int32 [T k] (output, may be NULL)
 *   d_workspace: dlrm_expert_sort_workspace_size bytes, 256-byte aligned (may be NULL when that is 0)
 *   d_status may be NULL; gets DLRM_STATUS_OOB_INDEX for an id of E or more (negative
 *   ones are choices without an expert)
 * Requires 1 <= E <= DLRM_ROUTE_MAX_EXPERTS, 1 <= k <= DLRM_ROUTE_MAX_TOP_K and T k up to
 * 2^31 - 2^20 - 1 (DLRM_ERR_UNSUPPORTED).
 */
dlrm_status dlrm_expert_sort(const int32_t* d_ids, int T, int k, int E, int32_t* d_offsets, int32_t* d_slots,
                             int32_t* d_order, void* d_workspace, size_t workspace_bytes, uint32_t* d_status,
                             void* stream);

/* Workspace bytes of dlrm_expert_sort (0 for invalid sizes). */
size_t dlrm_expert_sort_workspace_size(int T, int k, int E);

/* ------------------------------------------- tokens to their experts and back */
/*
 * Sorted rows [R][H] hold one row for each place; slots [T][k] says which place
 * is token t's j-th (dlrm_expert_sort).  Slots below 0 have no row and take no part;
 * slots of R or more neither, and set DLRM_STATUS_OOB_INDEX in *d_status (may be NULL).
 * Rows of outputs [R][H] that no slot names stay as they were.  Slots of one output
 * [R][H] are distinct (of equal ones each column is any one's).  1 <= k <= DLRM_ROUTE_MAX_TOP_K,
 * 0 <= R; sizes up to 2^31 - 2^20 - 1.
 *
 *   dlrm_dispatch_fwd   xs[slots[t][j]] = x[t]
 *   dlrm_dispatch_bwd   grad_x[t] = sum over j of grad_xs[slots[t][j]]
 *   dlrm_combine_fwd    y[t] = residual[t] + sum over j of probs[t][j] * ys[slots[t][j]]
 *   dlrm_combine_bwd    grad_ys[slots[t][j]] = probs[t][j] * grad_y[t]
 *                       grad_probs[t][j] = grad_y[t] . ys[slots[t][j]], 0 without a row
 * Sums go by ascending j, the residual last.
 *   d_x, d_y, d_grad_x, d_grad_y [T][H];  d_residual [T][H] or NULL;  d_xs, d_ys,
 *   d_grad_xs, d_grad_ys [R][H];  d_slots int32 [T][k];  d_probs, d_grad_probs fp32
 *   [T][k] contiguous;  d_grad_ys or d_grad_probs may be NULL (not both; d_ys may be
 *   NULL without d_grad_probs, d_probs without d_grad_ys)
 */
dlrm_status dlrm_dispatch_fwd(const void* d_x, int64_t ldx, const int32_t* d_slots, dlrm_dtype dtype, int T, int k,
                              int H, int R, void* d_xs, int64_t ldxs, uint32_t* d_status, void* stream);
dlrm_status dlrm_dispatch_bwd(const void* d_grad_xs, int64_t ldgxs, const int32_t* d_slots, dlrm_dtype dtype, int T,
                              int k, int H, int R, void* d_grad_x, int64_t ldgx, uint32_t* d_status, void* stream);
dlrm_status dlrm_combine_fwd(const void* d_ys, int64_t ldys, const int32_t* d_slots, const float* d_probs,
                             const void* d_residual, int64_t ldres, dlrm_dtype dtype, int T, int k, int H, int R,
                             void* d_y, int64_t ldy, uint32_t* d_status, void* stream);
dlrm_status dlrm_combine_bwd(const void* d_grad_y, int64_t ldgy, const void* d_ys, int64_t ldys, const int32_t* d_slots,
                             const float* d_probs, dlrm_dtype dtype, int T, int k, int H, int R, void* d_grad_ys,
                             int64_t ldgys, float* d_grad_probs, uint32_t* d_status, void* stream);

/* ----------------------------------------------------- activations in 8 bits */
/*
 * A matrix [M][N] in 8 bits: q [M][N], 8-bit floats of 4 exponent and 3 mantissa
 * bits (e4m3: 448 the largest, 2^-9 the least, no infinity), and one byte e for every
 * 32 columns of a row, exps [M][ceil(N / 32)] contiguous: the block's values are q 2^(e - 127).
 * e is the least (0 the least of all) that takes the block's largest finite size to
 * 448 or less, so that all but the smallest values keep 4 significant bits; values are
 * rounded to nearest, ties to even.  Infinities and NaN become NaN.
 * A value read back is at most dtype's largest in size (fp32: bf16's), where rounding
 * took it past that.  (dlrm_pack8 makes no byte e past 247; 255 is not a power of two.)
 *
 *   dlrm_pack8     q, exps = x
 *   dlrm_unpack8   y = q 2^(e - 127)
 * Requires N >= 1 and sizes up to 2^31 - 2^20 - 1.
 */
dlrm_status dlrm_pack8(const void* d_x, int64_t ldx, dlrm_dtype dtype, int M, int N, uint8_t* d_q, int64_t ldq,
                       uint8_t* d_exps, void* stream);
dlrm_status dlrm_unpack8(const uint8_t* d_q, int64_t ldq, const uint8_t* d_exps, dlrm_dtype dtype, int M, int N,
                         void* d_y, int64_t ldy, void* stream);

/*
 * dlrm_linear_bwd8 -- dlrm_linear_bwd with the layer's input and pre-activation in 8 bits.
 *
 *   d_x_q [M][K], d_x_exps: the input (NULL without d_grad_w)
 *   d_pre_q [M][N], d_pre_exps: the pre-activation, or for RELU without a residual
 *     the output (NULL for DLRM_ACT_NONE).  RELU passes no gradient where the value
 *     kept in 8 bits is 0.
 * Everything else is as in dlrm_linear_bwd: the same gradients for the values that
 * the 8 bits stand for, as dlrm_unpack8 reads them.  fp32 layers of more than 16 outputs
 * multiply the input's values as bf16 numbers, which are multiples of 2^-133: values of
 * blocks with e of 0 to 2 are rounded to those.
 */
dlrm_status dlrm_linear_bwd8(const void* d_grad_y, int64_t ldg, const uint8_t* d_x_q, int64_t ldx,
                             const uint8_t* d_x_exps, const void* d_w, int64_t ldw, const uint8_t* d_pre_q, int64_t ldp,
                             const uint8_t* d_pre_exps, dlrm_dtype dtype, int M, int N, int K, dlrm_act act, double p,
                             const uint64_t* d_rng, void* d_grad_x, int64_t lddx, void* d_grad_w, int64_t lddw,
                             float* d_grad_bias, void* d_workspace, size_t workspace_bytes, uint32_t* d_status,
                             void* stream);

/* Workspace bytes of dlrm_linear_bwd8 when all three gradients are asked for. */
size_t dlrm_linear_bwd8_workspace_size(const void* d_grad_y, int64_t ldg, const void* d_w, int64_t ldw,
                                       dlrm_dtype dtype, int M, int N, int K, dlrm_act act, double p);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_GB300_BLOCK_H */
