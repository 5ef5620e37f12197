// Backward of an activation straight to the codes that the FP8 GEMMs of the backward pass read (gfx950):
// act.hip's dz, rounded to BF16 in registers, then quant.hip's dual quantiser on it. Formulas in
// include/pf8_layer.h.
//
// Bound: HBM. Without a gate 6 bytes a value of dd (dd, z in, two codes out), with one 10; through a BF16 dz in
// memory it would be 10 and 18. 8192 x 6144 with a gate and a bias: 90 us (5.6 TB/s), without a
// gate 59 us, against 176 and 97 us by act.hip and the quantiser after it.
// A workgroup takes a 128 x 128 tile of dd and makes one such tile of dz, or the gate's and the factor's one after
// the other. Column sums over the tile's rows go to one row of partial sums for each 128 rows.
#include "act_device.h"
#include "pf8_layer_launch.h"
#include "pf8_train_launch.h"
#include "quant_device.h"
#include "row_device.h"

namespace pf8 {

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

template <int ACT, bool GATED>
__global__ __launch_bounds__(256) void act_bwd_quant_kernel(ActQuantArgs a) {
  constexpr int PARTS = GATED ? 2 : 1;
  constexpr bool HAS_Z = ACT != PF8_ACT_NONE;
  __shared__ __align__(16) uint32_t red[4][16][4];
  __shared__ __align__(16) uint8_t tile[kGroup * kGroup];
  __shared__ float sh[4][PARTS][kGroup];
  const int64_t gc = blockIdx.x, gr = gridDim.y - 1 - blockIdx.y;  // last rows first, as the quantiser
  const int t = threadIdx.x, rb = t >> 4, cc = t & 15, wave = t >> 6;
  const int64_t r0 = gr * kGroup + 8 * rb, c0 = gc * kGroup + 8 * cc;
  auto load = [&](const uint16_t* p) {  // non-temporal: read once
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
  };
  uint4 v[PARTS][8];
  {
    uint4 dv[8], zv[8], uv[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      dv[p] = load(a.dd + (r0 + p) * a.lddd + c0);
      if constexpr (HAS_Z) zv[p] = load(a.z + (r0 + p) * a.ldz + c0);
      if constexpr (GATED) uv[p] = load(a.z + (r0 + p) * a.ldz + a.cols + c0);
    }
    float sums[PARTS][8] = {};
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      float d[8], z[8], o[8];
      unpack8(dv[p], d);
      if constexpr (HAS_Z) unpack8(zv[p], z);
      if constexpr (GATED) {
        float u[8], up[8];
        unpack8(uv[p], u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float value, slope;
          act_both<ACT>(z[k], value, slope);
          o[k] = d[k] * u[k] * slope;
          up[k] = d[k] * value;
          sums[1][k] += up[k];
        }
        v[PARTS - 1][p] = pack8(up);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float value = 0.0f, slope = 1.0f;
          if constexpr (HAS_Z) act_both<ACT>(z[k], value, slope);
          o[k] = d[k] * slope;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sums[0][k] += o[k];
      v[0][p] = HAS_Z ? pack8(o) : dv[p];
    }
    if (a.dbias) {
#pragma unroll
      for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float s = sums[i][k];
          s += __shfl_xor(s, 16);
          s += __shfl_xor(s, 32);
          if ((t & 63) < 16) sh[wave][i][8 * cc + k] = s;
        }
      __syncthreads();
      float* out = (gridDim.y == 1 ? a.dbias : a.partial + gr * PARTS * a.cols) + gc * kGroup;
      for (int q = t; q < PARTS * kGroup; q += 256) {
        const int i = q / kGroup, c = q % kGroup;
        const float s = (sh[0][i][c] + sh[1][i][c]) + (sh[2][i][c] + sh[3][i][c]);
        float* o = out + i * a.cols + c;
        *o = gridDim.y == 1 && a.accumulate ? *o + s : s;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    if (i) __syncthreads();  // the first part's codes have left the LDS tile
    int p = 0;  // the quantiser asks for this thread's eight rows in order
    quant_dual_values([&](int64_t, int64_t, int) { return v[i][p++]; }, a.q_row, a.ldq_row, a.s_row, a.ld_sr, a.q_col,
                      a.ldq_col, a.s_col, a.ld_sc, gc + i * (a.cols / kGroup), gr, red, tile);
  }
}

}  // namespace

hipError_t launch_act_bwd_quant(const ActQuantArgs& a, hipStream_t stream) {
  const int groups = static_cast<int>(a.rows / kGroup);
  auto go = [&](auto act, auto gated) {
    hipLaunchKernelGGL((act_bwd_quant_kernel<decltype(act)::value, decltype(gated)::value>),
                       dim3(static_cast<uint32_t>(a.cols / kGroup), static_cast<uint32_t>(groups)), dim3(256), 0, stream, a);
    return hipGetLastError();
  };
  const hipError_t e = by_activation(a.act, [&](auto act) {
    if constexpr (decltype(act)::value != PF8_ACT_NONE) {
      if (a.gated) return go(act, std::true_type{});
    }
    return go(act, std::false_type{});
  });
  if (e != hipSuccess || !a.dbias || groups == 1) return e;
  const int width = static_cast<int>(a.gated ? 2 * a.cols : a.cols);
  float* outs[3] = {a.dbias, nullptr, nullptr};
  return launch_column_sums(a.partial, groups, width, width, outs, a.accumulate, stream);
}

}  // namespace pf8
