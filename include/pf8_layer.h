/*
 * pf8_layer.h - C ABI of a decoder layer's steps around its FP8 products (same library, libpf8): the
 * norms of queries and keys for each head with the rotation by positions, the product with bias,
 * activation and residual in its epilogue, and the backward passes of both.
 *
 * The conventions of pf8.h and pf8_train.h hold: device pointers owned by the caller, validation on the
 * host before anything is enqueued, nothing allocated or kept. Pointers that are host pointers say so.
 * Strides and leading dimensions are in elements. "bf16" arrays need 2-byte, float arrays 4-byte, double
 * and 64-bit integer arrays 8-byte alignment, unless stated otherwise; any row pitch is taken.
 */
#ifndef PF8_LAYER_H
#define PF8_LAYER_H

#include "pf8.h"
#include "pf8_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of the inverse frequencies beside PF8_F32 (pf8_dtype). */
#define PF8_F64 2

/* Integer types of positions (pf8_index). */
typedef int pf8_index;
#define PF8_I32 0
#define PF8_I64 1

/* How the rotated pairs are shared out over the position axes (pf8_sections). */
typedef int pf8_sections;
#define PF8_BLOCKED 0 /* the first sections[0] pairs to axis 0, the next sections[1] to axis 1, ... */
#define PF8_CYCLED 1  /* pair i to axis i mod axes while i < axes * sections[i mod axes], else to axis 0 */

/* Limits of the head norm: values of a head, position axes, heads of one tensor. */
#define PF8_HEAD_MAX_DIM 512
#define PF8_HEAD_MAX_AXES 4
#define PF8_HEAD_MAX_HEADS 65536

/* Activations (pf8_activation). */
typedef int pf8_activation;
#define PF8_ACT_NONE 0      /* z */
#define PF8_ACT_RELU 1      /* max(z, 0) */
#define PF8_ACT_RELU2 2     /* max(z, 0)^2 */
#define PF8_ACT_SILU 3      /* z / (1 + exp(-z)) */
#define PF8_ACT_GELU 4      /* z (1 + erf(z / sqrt 2)) / 2 */
#define PF8_ACT_GELU_TANH 5 /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */

/*
 * Norms of queries and keys for each head, and the rotation by positions, in one pass. For each token
 * and each head x of q (and of k, with w_k):
 *
 *   n = x * rsqrt(mean(x^2) + eps) * (w + weight_offset)      n = x without a weight
 *   of each pair (a, b) of the first 2 * pairs values of n, with the angle phi = position * inv_freq[pair]:
 *       a' = rotary_scale * (a cos phi - b sin phi)
 *       b' = rotary_scale * (a sin phi + b cos phi)
 *
 * and the head's further values as they are in n. Pair i holds the values i and pairs + i, or with
 * `interleaved` 2 i and 2 i + 1. The position is that of the token on the pair's axis. FP32, the angle's
 * fraction of a turn from FP64 (off by up to 2^-51.4 of the angle: 2^-11 radians at 2^40, nothing is left of it at
 * 2^52), one rounding to BF16 at the end.
 *
 * q, k: bf16 [tokens, heads, head_dim] with strides _st between tokens and _sh between heads, head
 *   values contiguous. k NULL (with heads_k 0): queries alone. 1 <= head_dim <= 512, tokens * heads < 2^31.
 * w_q, w_k: [head_dim] of wtype (PF8_BF16 or PF8_F32), or NULL: no norm of that tensor.
 * positions: integers of ptype; that of a token on an axis at token * pos_st + axis * pos_sa. NULL (with
 *   pairs 0): no rotation. Positions are not checked.
 * inv_freq: [pairs] of ftype (PF8_F32 or PF8_F64). 0 <= 2 * pairs <= head_dim.
 * axes: 1 to 4. sections: a HOST array of `axes` counts, each at least 1, that sum up to pairs (with
 *   PF8_CYCLED every axis has to find its pairs: a + axes * (sections[a] - 1) < pairs for a > 0); NULL with one axis.
 * q_out, k_out: bf16 results; each may be its input (same address and strides), and otherwise overlaps nothing.
 */
pf8_status pf8_qk_norm_rope(int64_t tokens, int64_t head_dim, const void* q, int64_t heads_q, int64_t q_st, int64_t q_sh,
                            const void* k, int64_t heads_k, int64_t k_st, int64_t k_sh, const void* w_q, const void* w_k,
                            pf8_dtype wtype, float weight_offset, float eps, const void* positions, pf8_index ptype,
                            int64_t pos_st, int64_t pos_sa, const void* inv_freq, pf8_dtype ftype, int64_t pairs,
                            int axes, const int64_t* sections, pf8_sections order, int interleaved, float rotary_scale,
                            void* q_out, int64_t qo_st, int64_t qo_sh, void* k_out, int64_t ko_st, int64_t ko_sh,
                            void* hip_stream);

/*
 * Backward of pf8_qk_norm_rope: the gradients of q, k and the weights from dq, dk, the gradients of q_out
 * and k_out. With d the gradient turned back (the rotation's transpose), r = rsqrt(mean(x^2) + eps), y = x r
 * and t = d * (w + weight_offset):
 *
 *   dx = r * (t - y * mean(t * y))        dx = d without a weight
 *   dw = sum over tokens and heads of d * y
 *
 * dq, dk: bf16, shaped as q and k. q, k are the forward's inputs (read only where there is a weight;
 *   may be NULL otherwise, with their strides ignored).
 * dq_out, dk_out: bf16; NULL: not wanted. Each may be its dq / dk, or its q / k (same address and strides).
 * dw_q, dw_k: float [head_dim], each only with its weight; NULL: not wanted. Overwritten, or with
 *   accumulate = 1 added to. Formed in a fixed order: the same bits each time.
 * workspace: at least pf8_qk_norm_rope_bwd_workspace bytes, 16-byte aligned, where dw_q or dw_k is wanted;
 *   not read before it is written, so calls on one stream may share it.
 */
pf8_status pf8_qk_norm_rope_bwd(int64_t tokens, int64_t head_dim, const void* dq, int64_t dq_st, int64_t dq_sh,
                                const void* dk, int64_t dk_st, int64_t dk_sh, const void* q, int64_t heads_q,
                                int64_t q_st, int64_t q_sh, const void* k, int64_t heads_k, int64_t k_st, int64_t k_sh,
                                const void* w_q, const void* w_k, pf8_dtype wtype, float weight_offset, float eps,
                                const void* positions, pf8_index ptype, int64_t pos_st, int64_t pos_sa,
                                const void* inv_freq, pf8_dtype ftype, int64_t pairs, int axes, const int64_t* sections,
                                pf8_sections order, int interleaved, float rotary_scale,
                                void* dq_out, int64_t dqo_st, int64_t dqo_sh, void* dk_out, int64_t dko_st,
                                int64_t dko_sh, float* dw_q, float* dw_k, int accumulate, void* workspace,
                                int64_t workspace_bytes, void* hip_stream);

/* Bytes of the workspace of pf8_qk_norm_rope_bwd; 0 for sizes that it refuses. Needs no device. */
int64_t pf8_qk_norm_rope_bwd_workspace(int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t head_dim);

/*
 * Backward of an activation (and of the bias before it): from dd, the gradient of d, and z, the value
 * before the activation (bias included):
 *
 *   gated = 0:  d = act(z),       dz = dd * act'(z)                             z, dz [rows, cols]
 *   gated = 1:  d = act(g) * u,   dz = [dd * u * act'(g) | dd * act(g)]         z = [g | u], dz [rows, 2 cols]
 *   dbias = column sums of dz (in FP32, before dz is rounded)
 *
 * dd: bf16 [rows, cols]; z, dz: bf16; pitches at least the columns. act'(0) of PF8_ACT_RELU is 0. z is NULL
 * with PF8_ACT_NONE without a gate (dz = dd), and only then.
 * dz: NULL: not wanted; may be z, or without a gate dd (same address and pitch).
 * dbias: float [cols] or [2 cols]; NULL: not wanted. accumulate as in pf8_qk_norm_rope_bwd, workspace (of
 * pf8_act_bwd_workspace bytes) where dbias is wanted. rows, cols >= 1.
 */
pf8_status pf8_act_bwd(int64_t rows, int64_t cols, const void* dd, int64_t lddd, const void* z, int64_t ldz,
                       pf8_activation activation, int gated, void* dz, int64_t lddz, float* dbias, int accumulate,
                       void* workspace, int64_t workspace_bytes, void* hip_stream);

/* Bytes of the workspace of pf8_act_bwd; 0 for sizes that it refuses. Needs no device. */
int64_t pf8_act_bwd_workspace(int64_t rows, int64_t cols, int gated);

/*
 * pf8_act_bwd with dz as the codes of both groupings, for the data and the weight gradient: exactly
 * pf8_act_bwd (dz rounded to BF16), then pf8_quant_act_dual of that dz, without dz in memory.
 *
 * rows and cols are multiples of 128. dd, z: 16-byte aligned, pitches multiples of 8. With width = cols, or 2 cols
 * with a gate: q_row [rows, width], dscale_row[g * ld_sr + r], q_col [width, rows], dscale_col[g * ld_sc + c], as
 * pf8_quant_act_dual writes them (16-byte aligned codes with pitches of multiples of 16). z NULL with
 * PF8_ACT_NONE: the codes of dd. dbias as in pf8_act_bwd, its sums formed in another fixed order; workspace of
 * pf8_act_bwd_quant_workspace bytes where it is wanted, and with more than 128 rows width < 2^27 there (PF8_ESHAPE).
 */
pf8_status pf8_act_bwd_quant(int64_t rows, int64_t cols, const void* dd, int64_t lddd, const void* z, int64_t ldz,
                             pf8_activation activation, int gated, void* q_row, int64_t ldq_row, float* dscale_row,
                             int64_t ld_sr, void* q_col, int64_t ldq_col, float* dscale_col, int64_t ld_sc,
                             float* dbias, int accumulate, void* workspace, int64_t workspace_bytes, void* hip_stream);

/* Bytes of the workspace of pf8_act_bwd_quant; 0 for sizes that it refuses. Needs no device. */
int64_t pf8_act_bwd_quant_workspace(int64_t rows, int64_t cols, int gated);

/*
 * Block-scaled FP8 product with bias, activation and residual in its epilogue:
 *
 *   z = (the forward product of pf8_block_gemm, PF8_FPROP) + bias       in FP32
 *   d = act(z) + residual                                               gated = 0: d [m, n]
 *   d = act(z[:, :n/2]) * z[:, n/2:] + residual                         gated = 1: d [m, n/2]
 *
 * d and z are each rounded to BF16 once, from FP32.
 *
 * Operands, scales, alignment and limits are those of pf8_block_gemm with PF8_FPROP (m, n >= 1,
 * k % 128 == 0, power-of-two scales; b_dscale[(j / 128) * ld_bs + kb], ld_bs >= k / 128), and its accumulation
 * contract holds for z before its rounding. For few rows the sum over K is formed in parts, joined in a
 * fixed order; the same call gives the same bits each time.
 * gated: 0 or 1; with 1, n is a multiple of 128 and the activation is not PF8_ACT_NONE.
 * bias: [n] of btype (PF8_BF16 or PF8_F32), or NULL.
 * residual: bf16, d's shape, pitch ldr, or NULL. May be d itself (same address and pitch).
 * z: bf16 [m, n], pitch ldz, what pf8_act_bwd takes; or NULL: not wanted. Overlaps nothing.
 * d, z and residual: 16-byte aligned, pitches multiples of 8.
 * Pitches: lda and ldb up to 8388607, ldd, ldr and ldz up to half of that, where there is a single row too.
 */
pf8_status pf8_fprop_act(int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const float* a_dscale,
                         int64_t ld_as, const void* b, int64_t ldb, const float* b_dscale, int64_t ld_bs,
                         const void* bias, pf8_dtype btype, pf8_activation activation, int gated,
                         const void* residual, int64_t ldr, void* z, int64_t ldz, void* d, int64_t ldd,
                         void* hip_stream);

/*
 * Which kernel pf8_fprop_act runs for a size: 65536 * rows + columns of what a workgroup works on. 64, 128 or 256 rows of
 * 64, 128 or 256 rows of W: the tile kernels; 16, 32 or 64 rows of 16 columns of d: the kernel for few tokens. 0
 * for sizes that it refuses. For tests and measurements that mean one of them. Needs no device.
 */
int64_t pf8_fprop_act_tile(int64_t m, int64_t n, int64_t k, int gated);

#ifdef __cplusplus
}
#endif

#endif /* PF8_LAYER_H */
