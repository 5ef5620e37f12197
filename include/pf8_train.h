/*
 * pf8_train.h - C ABI of libpf8's training operators around the FP8 linear layer, for AMD MI355X (gfx950).
 *
 * Between two FP8 projections of a decoder stands the block norm: the branch's result is
 * normalised, gated, scaled and added to the residual stream, and the new stream is normalised
 * into the next projection's input, in BF16 or as the E4M3 codes pf8_block_gemm reads. After the
 * backward pass, an orthogonalising optimiser turns a weight's FP32 main gradient (what
 * pf8_block_gemm_f32 accumulates) into an update by Newton-Schulz products.
 *
 * The conventions of pf8.h hold (device pointers, caller's buffers, asynchronous on `hip_stream`,
 * arguments checked on the host before anything is enqueued, sizes and leading dimensions at most
 * 2^31 - 1, no allocation, no global state, capturable), with these differences:
 *  - BF16 and FP32 arrays of these operators need only their element's alignment, and any leading
 *    dimension >= the row's length; only code arrays keep the 16-byte rule of pf8.h.
 *  - Inputs may hold NaN and infinities: they spread as the formulas say.
 *  - Workspaces are scratch: nothing is kept in them from one call to the next. Two calls that may
 *    run at the same time need two workspaces.
 */
#ifndef PF8_TRAIN_H
#define PF8_TRAIN_H

#include "pf8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of weights and gradients that may be either (pf8_dtype). */
typedef int pf8_dtype;
#define PF8_BF16 0
#define PF8_F32 1

/* Largest row of the block norm. */
#define PF8_NORM_MAX_COLS 16384

/*
 * Block norm, forward. Per row of [rows, cols], everything in FP32, each output rounded once:
 *
 *   u = y * rsqrt(mean(y^2) + eps) * (w_post + weight_offset)      (u = y without w_post)
 *   r = residual_scale * h + branch_scale * gate * u               (no gate: factor 1; r = h without y)
 *   x = r * rsqrt(mean(r^2) + eps) * (w_pre + weight_offset)       (from the unrounded r)
 *
 * h:      bf16 [rows, cols], pitch ldh: the residual stream.
 * y:      bf16 [rows, cols], pitch ldy: the branch's result; NULL: there is none (then w_post, gate
 *         and r are NULL and residual_scale is 1).
 * w_post, w_pre: [cols] of wtype, or NULL (without w_pre there is no x and no q).
 * gate:   NULL, [cols] of wtype (ld_gate = 0), or bf16 [rows, cols] with pitch ld_gate >= cols.
 * r:      bf16 [rows, cols], pitch ldr: the new stream, or NULL.
 * x:      bf16 [rows, cols], pitch ldx, or NULL.
 * q, dscale: E4M3 codes u8 [rows, cols], pitch ldq, and scales f32 [cols/128][rows],
 *         dscale[g * ld_s + row]: bit for bit what pf8_quant_act_1x128(PF8_ALONG_COLS) makes of the
 *         BF16 x; both NULL or both given (then cols is a multiple of 128). x need not be given for it.
 * r and x may be h's or y's own memory (same base, same pitch); no other overlap.
 * rows >= 1, 1 <= cols <= PF8_NORM_MAX_COLS, eps >= 0, scales finite. At least one output.
 */
pf8_status pf8_block_norm(int64_t rows, int64_t cols, const void* h, int64_t ldh, const void* y, int64_t ldy,
                          const void* w_post, const void* gate, int64_t ld_gate, const void* w_pre, pf8_dtype wtype,
                          float residual_scale, float branch_scale, float weight_offset, float eps,
                          void* r, int64_t ldr, void* x, int64_t ldx, void* q, int64_t ldq, float* dscale, int64_t ld_s,
                          void* hip_stream);

/*
 * Block norm, backward: the gradients of h, y, gate and the weights from those of r and x, with the
 * forward's values made again from h and y (in FP32, so that the gradients see no rounded r):
 *
 *   D  = dr + rho_r (t - rn mean(t rn)),   t = dx (w_pre + offset),  rn = r rho_r,  rho_r = rsqrt(mean(r^2) + eps)
 *   dh = residual_scale D,  v = branch_scale D,  dgate = v u,  du = v gate
 *   dy = rho_y (s - yn mean(s yn)),        s = du (w_post + offset), yn = y rho_y   (dy = du without w_post)
 *   dw_pre = sum_rows dx rn,   dw_post = sum_rows du yn
 *
 * dr: bf16, pitch lddr, or NULL (zero).  dx: bf16, pitch lddx, or NULL (zero); one of them is given.
 * h .. eps: as in the forward (w_pre may be NULL only if dx is).
 * dh, dy: bf16 outputs or NULL.
 * dgate: NULL; for a [cols] gate f32 [cols] (ld_dgate = 0); for a [rows, cols] gate bf16, pitch ld_dgate.
 * dw_pre, dw_post: f32 [cols] or NULL.
 * accumulate: 1 adds the f32 [cols] results to what is there, 0 overwrites.
 * workspace: pf8_block_norm_bwd_workspace(rows, cols) bytes, 16-byte aligned; may be NULL if no f32
 *         [cols] result is asked for. The column sums are formed in a fixed order, without atomics:
 *         the same call gives the same bits.
 * dh and dy may be the memory of dr, dx, h or y (same base and pitch); no other overlap.
 */
pf8_status pf8_block_norm_bwd(int64_t rows, int64_t cols, const void* dr, int64_t lddr, const void* dx, int64_t lddx,
                              const void* h, int64_t ldh, const void* y, int64_t ldy, const void* w_post,
                              const void* gate, int64_t ld_gate, const void* w_pre, pf8_dtype wtype,
                              float residual_scale, float branch_scale, float weight_offset, float eps,
                              void* dh, int64_t lddh, void* dy, int64_t lddy, void* dgate, int64_t ld_dgate,
                              float* dw_pre, float* dw_post, int accumulate, void* workspace, int64_t workspace_bytes,
                              void* hip_stream);

/* Bytes of pf8_block_norm_bwd's workspace; 0 for sizes it refuses. */
int64_t pf8_block_norm_bwd_workspace(int64_t rows, int64_t cols);

/* Largest sides of a matrix that pf8_newton_schulz takes: the shorter and the longer one, and the
   largest number of matrices and of steps. */
#define PF8_NS_MAX_SHORT 32768
#define PF8_NS_MAX_LONG 1048576
#define PF8_NS_MAX_BATCH 65535
#define PF8_NS_MAX_STEPS 64

/*
 * Newton-Schulz orthogonalisation of a stack of gradients, as orthogonalising optimisers apply it to
 * a weight matrix's update:
 *
 *   X = G / (|G|_F + eps)
 *   per step (a, b, c):  X <- a X + b (X X^T) X + c (X X^T)^2 X      (X^T X on the right of a tall X)
 *   out = X, rounded to BF16
 *
 * Every singular value s of X becomes a s + b s^3 + c s^5 in each step; the singular vectors stay.
 *
 * g:   `batch` matrices [m, n] of gtype (BF16, or FP32 as a main gradient), row pitch ldg, stride_g
 *      elements from one matrix to the next (not read for batch = 1).
 * out: bf16 [m, n] each, row pitch ldo, stride stride_o; no overlap with g.
 * coefficients: HOST pointer to steps x 3 floats (a, b, c), read before the call returns; finite and at
 *      most 64 in magnitude. They must keep the singular values below 8 between the steps (any
 *      orthogonalising choice keeps them near 1); beyond, FP16 operands overflow to NaN.
 * eps: >= 0. A matrix of zeros gives zeros (NaN with eps = 0); one that holds a NaN or an infinity
 *      gives NaN everywhere.
 *
 * Precision: between the steps X is the sum of two FP16 values, which hold an element to 2^-23 of itself
 * or to 2^-37, whichever is more (X starts with norm 1; FP32 in matrices of at most 64 x 512 or 128 x 256).
 * The diagonals of X X^T and of the polynomial, and every sum, are FP32 or FP64; the matrix products'
 * operands are FP16, scaled by powers of two. Besides the BF16 rounding of the result (1.7e-3 of its 2-norm)
 * five steps of the usual kind leave it off by 0.2e-3 to 1.5e-3 of its 2-norm, up to 2e-3, whatever its rank.
 * Roundings average out less where few elements carry the gradient: up to 4e-3 with under ten rows (or
 * columns), up to 1.5e-2 with under 64 elements, or where all elements have one of a few magnitudes (a
 * constant matrix). What rounding puts outside the space of a gradient of low rank grows by a in every step,
 * as in an FP32 evaluation: rank one is about 3e-3 off after eight steps and 3e-2 after ten. The same call
 * gives the same bits.
 *
 * workspace: pf8_newton_schulz_workspace(batch, m, n) bytes, 256-byte aligned.
 */
pf8_status pf8_newton_schulz(int64_t batch, int64_t m, int64_t n, const void* g, int64_t ldg, int64_t stride_g,
                             pf8_dtype gtype, int steps, const float* coefficients, float eps, void* out, int64_t ldo,
                             int64_t stride_o, void* workspace, int64_t workspace_bytes, void* hip_stream);

/* Bytes of pf8_newton_schulz's workspace; 0 for sizes it refuses. */
int64_t pf8_newton_schulz_workspace(int64_t batch, int64_t m, int64_t n);

#ifdef __cplusplus
}
#endif

#endif /* PF8_TRAIN_H */
