// Host-side launchers of the training operators (called by the C ABI after validation).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pf8 {

constexpr int64_t kNormMaxCols = 16384;

// Operands and scalars that the block norm's forward and backward share.
struct NormArgs {
  int64_t rows;
  int cols;
  const uint16_t* h;
  int64_t ldh;
  const uint16_t* y;  // or null: no branch
  int64_t ldy;
  const void* w_post;  // or null
  const void* gate;    // or null
  int64_t ld_gate;     // 0: [cols] of the weights' type; else bf16 [rows, cols]
  const void* w_pre;   // or null
  int wf32;            // weights (and a [cols] gate) are FP32, else BF16
  float residual_scale, branch_scale, offset, eps;
  float sq, inv_sum;   // squares are summed as (v * sq)^2, sq = 2^-k with 4^k >= cols; inv_sum = 1 / (cols * sq^2)
};

struct NormFwdArgs {
  NormArgs in;
  uint16_t* r;
  int64_t ldr;
  uint16_t* x;
  int64_t ldx;
  uint8_t* q;
  int64_t ldq;
  float* dscale;
  int64_t ld_s;
};

struct NormBwdArgs {
  NormArgs in;
  const uint16_t* dr;
  int64_t lddr;
  const uint16_t* dx;
  int64_t lddx;
  uint16_t* dh;
  int64_t lddh;
  uint16_t* dy;
  int64_t lddy;
  uint16_t* dgate_full;
  int64_t ld_dgate;
  float* sums[3];  // dw_pre, dw_post, dgate of a [cols] gate; null where not asked for
  int accumulate;
  float* partial;  // workspace: [groups][sums asked for][cols]
};

hipError_t launch_norm_fwd(const NormFwdArgs& args, hipStream_t stream);
hipError_t launch_norm_bwd(const NormBwdArgs& args, hipStream_t stream);
// Workgroups of the backward pass, each with one row of partial column sums.
int64_t norm_bwd_groups(int64_t rows, int64_t cols);
// Column sums of partial rows [groups][width], in a fixed order, into outs[c / cols][c % cols]; accumulate: added.
hipError_t launch_column_sums(const float* partial, int groups, int width, int cols, float* const (&outs)[3],
                              int accumulate, hipStream_t stream);

// Newton-Schulz orthogonalisation; the launcher fills in what lies in the workspace.
struct NsArgs {
  int64_t m, n;  // of G
  const void* g;
  int64_t ldg, stride_g;
  int gf32;  // G is FP32, else BF16
  float eps;
  uint16_t* out;
  int64_t ldo, stride_o;
  int64_t pp, qp;   // padded min(m, n) and max(m, n)
  int64_t ldp;       // pitch of FP16 rows of pp values
  int64_t x_elems;   // pp * qp
  _Float16 *rest, *xc[2], *a16, *b16;
  float *da, *db, *part;
  double* norm_part;
};

int64_t ns_workspace(int64_t batch, int64_t m, int64_t n);
// coef: steps x 3 on the host
hipError_t launch_newton_schulz(NsArgs args, int64_t batch, int steps, const float* coef, void* workspace,
                                hipStream_t stream);

}  // namespace pf8
