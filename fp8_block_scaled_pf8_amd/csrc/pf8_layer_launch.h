// Host-side launchers of a decoder layer's steps around its products (called by the C ABI after validation).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pf8 {

constexpr int kHeadMaxDim = 512, kHeadMaxAxes = 4;

// Queries or keys: values (forward) or values and gradients (backward), and the result.
struct HeadTensor {
  const uint16_t* x;
  int64_t x_st, x_sh;
  const uint16_t* d;
  int64_t d_st, d_sh;
  uint16_t* out;  // backward: null where not wanted
  int64_t out_st, out_sh;
  const void* w;  // or null: no norm
  int heads;      // 0: no such tensor
  int sums;       // backward: the weight's gradient is wanted (the launcher fills it in)
};

struct HeadNormArgs {
  HeadTensor t[2];
  int64_t tokens;
  int dim, pairs;
  int wf32;  // weights are FP32, else BF16
  float offset, eps;
  float sq, inv_sum;  // squares are summed as (v * sq)^2, sq = 2^-k with 4^k >= dim; inv_sum = 1 / (dim * sq^2)
  const void* pos;
  int p64;  // positions are 64-bit, else 32-bit integers
  int64_t pos_st, pos_sa;
  const void* freq;
  int f64;  // inverse frequencies are FP64, else FP32
  int axes;
  int share[kHeadMaxAxes];  // blocked: the first pair behind axis a; cycled: axes * sections[a]
  int cycled, interleaved;
  float scale;
  float* partial;  // backward: [blocks][dim]
};

hipError_t launch_head_norm_fwd(const HeadNormArgs& args, hipStream_t stream);
// dw: q's and k's, null where not wanted
hipError_t launch_head_norm_bwd(HeadNormArgs args, float* const (&dw)[2], int accumulate, hipStream_t stream);
// Workgroups of the backward pass, each with one row of partial sums.
int64_t head_norm_bwd_blocks(int64_t tokens, int64_t heads_q, int64_t heads_k);

struct ActBwdArgs {
  int64_t rows;
  int cols;
  const uint16_t* dd;
  int64_t lddd;
  const uint16_t* z;  // null without an activation and a gate
  int64_t ldz;
  int act, gated;
  uint16_t* dz;  // or null
  int64_t lddz;
  float* dbias;    // [cols or 2 cols], or null where no sums are wanted
  int accumulate;
  float* partial;  // [groups][cols or 2 cols]
};

hipError_t launch_act_bwd(const ActBwdArgs& args, hipStream_t stream);
int64_t act_bwd_groups(int64_t rows, int64_t cols);

struct ActQuantArgs {
  int64_t rows, cols;  // of dd: multiples of 128
  const uint16_t* dd;
  int64_t lddd;
  const uint16_t* z;
  int64_t ldz;
  int act, gated;
  uint8_t* q_row;
  int64_t ldq_row;
  float* s_row;
  int64_t ld_sr;
  uint8_t* q_col;
  int64_t ldq_col;
  float* s_col;
  int64_t ld_sc;
  float* dbias;
  int accumulate;
  float* partial;  // [rows / 128][cols or 2 cols]
};

hipError_t launch_act_bwd_quant(const ActQuantArgs& args, hipStream_t stream);

// The forward product with its epilogue; d is [m, gated ? n / 2 : n].
struct FpropActArgs {
  int64_t m, n, k;
  const uint8_t* a;
  int64_t lda;
  const float* a_dscale;
  int64_t ld_as;
  const uint8_t* b;
  int64_t ldb;
  const float* b_dscale;
  int64_t ld_bs;
  const void* bias;  // or null
  int bias_f32;
  int act, gated;
  const uint16_t* residual;  // or null
  int64_t ldr;
  uint16_t* z;  // or null
  int64_t ldz;
  uint16_t* d;
  int64_t ldd;
};

hipError_t launch_fprop_act(const FpropActArgs& args, hipStream_t stream);
// What launch_fprop_act runs for m, n, k and gated: tiles of bm rows and bn rows of W, or for few tokens up to bm of them and
// bn = 16 columns of d a workgroup.
struct FpropActTile {
  int bm, bn;
};
FpropActTile fprop_act_tile(const FpropActArgs& args);
// By tiles of BM rows and BN rows of W.
template <int BM, int BN>
hipError_t launch_fprop_act_tiles(const FpropActArgs& args, hipStream_t stream);

}  // namespace pf8
