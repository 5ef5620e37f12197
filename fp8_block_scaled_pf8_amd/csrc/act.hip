// Backward of an activation, gated or not, with the bias's gradient (gfx950). Formulas in include/pf8_layer.h.
//
// Bound: HBM. 6 bytes a value of dd without a gate (dd, z in, dz out), 10 with one: 8192 x 6144 gated 94 us (5.4 TB/s,
// as a large copy). Short batches are bound by one trip through memory and the launches: 1003 x 5407 silu with the bias's
// gradient 12.7 us in two launches, of which the traffic is 6.
// A thread keeps 8 columns and walks rows; a workgroup is as many threads wide as the columns ask for (up
// to 256), the rest of its 256 threads take further rows. Column sums stay in registers over
// a thread's rows, meet in LDS, and a workgroup writes one row of partial sums.
#include "act_device.h"
#include "pf8_layer_launch.h"
#include "pf8_train_launch.h"
#include "row_device.h"

namespace pf8 {

namespace {

// How the last, ragged step of a row is taken: kOdd: the row's last 8 columns, of which the first belong to the
// thread before and are neither counted nor stored; kTiny: rows of under 8 columns, value by value.
enum RowEnd { kEven, kOdd, kTiny };

template <int ACT, bool GATED, RowEnd END>
__global__ __launch_bounds__(256) void act_bwd_kernel(ActBwdArgs a, int wide) {
  const int tx = threadIdx.x & (wide - 1), ty = threadIdx.x / wide, high = 256 / wide;
  const int cols = a.cols;
  const uint32_t c0 = 8 * (blockIdx.x * wide + tx);  // (past 2^31 for the last threads of the widest rows)
  const int n = static_cast<int>(cols - c0);          // columns from here: under 1 for threads behind the row
  int c = static_cast<int>(c0);
  const int first = END == kTiny || n >= 8 ? 0 : n <= 0 ? 8 : 8 - n;
  if (END == kOdd && n < 8) c = cols - 8;
  const bool any = n > 0;
  auto load = [&](const uint16_t* row) {
    return END == kTiny ? load_few(row + c, n) : load8(row + c);
  };
  auto store = [&](uint16_t* row, const float (&f)[8]) {
    const uint4 v = pack8(f);
    uint16_t* p = row + c;
    if constexpr (END == kTiny) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < n) p[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    } else if (END == kEven || first == 0) {
      *reinterpret_cast<u128_a2*>(p) = u128_a2{v.x, v.y, v.z, v.w};
    } else {
      store_last(p, v, 8 - first);
    }
  };
  constexpr int PARTS = GATED ? 2 : 1;
  constexpr bool HAS_Z = ACT != PF8_ACT_NONE;
  float sums[PARTS][8] = {};
  // ROWS rows at a time, all their loads first
  constexpr int ROWS = GATED ? 2 : 4;
  const int64_t step = static_cast<int64_t>(gridDim.y) * high;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * high + ty; any && r0 < a.rows; r0 += ROWS * step) {
    uint4 dv[ROWS], zv[ROWS], uv[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int64_t row = r0 + j * step;
      if (row >= a.rows) break;
      dv[j] = load(a.dd + row * a.lddd);
      if constexpr (HAS_Z) zv[j] = load(a.z + row * a.ldz);
      if constexpr (GATED) uv[j] = load(a.z + row * a.ldz + cols);
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int64_t row = r0 + j * step;
      if (row >= a.rows) break;
      float d[8], z[8], o[8];
      unpack8(dv[j], d);
      if constexpr (HAS_Z) unpack8(zv[j], z);
      if constexpr (GATED) {
        float u[8], up[8];
        unpack8(uv[j], u);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float value, slope;
          act_both<ACT>(z[k], value, slope);
          o[k] = d[k] * u[k] * slope;
          up[k] = d[k] * value;
          sums[1][k] += up[k];
        }
        if (a.dz) store(a.dz + row * a.lddz + cols, up);
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
      if (a.dz) store(a.dz + row * a.lddz, o);
    }
  }
  if (!a.dbias) return;
  __shared__ float sh[256][9];
  const bool alone = gridDim.y == 1;  // the sums themselves, not a row of partial ones
  float* out = alone ? a.dbias : a.partial + static_cast<int64_t>(blockIdx.y) * PARTS * cols;
#pragma unroll
  for (int part = 0; part < PARTS; ++part) {
    if (high > 1) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) sh[threadIdx.x][k] = sums[part][k];
      __syncthreads();
      if (ty == 0) {
        for (int y = 1; y < high; ++y)
#pragma unroll
          for (int k = 0; k < 8; ++k) sums[part][k] += sh[y * wide + tx][k];
      }
    }
    if (ty == 0 && any) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k >= first && c + k < cols) {
          float* o = out + part * cols + c + k;
          *o = alone && a.accumulate ? *o + sums[part][k] : sums[part][k];
        }
    }
  }
}

}  // namespace

// Threads of a workgroup along a row: a power of two, up to `most`. With column sums one wave of them, so that a
// workgroup takes four rows at a time and there are few rows of partial sums to join (1003 x 5407 12.7 us, 16.6 with
// 256 threads along a row; 8192 x 6144 gated 105 and 120).
static int act_bwd_wide(int64_t cols, bool sums) {
  const int most = sums ? 64 : 256;
  int wide = 1;
  while (wide < most && 8 * wide < cols) wide *= 2;
  return wide;
}

// Workgroups along the rows: up to 16 on a CU in all (8192 x 6144 gated 93.9 us, 96.3 with up to 8, 103.8 with 4). With
// column sums 8 rows a thread where that leaves 4 workgroups for each CU (8192 x 2048 21.2 us, with 4 rows 23.2), 4 where it
// leaves one (1024 x 2048 gated 8.8 us, with 8 rows 11.3, with 2 9.1), 2 else (33 x 6144 gated 6.4 us, with 4 rows 7.1).
static int64_t act_bwd_blocks(int64_t rows, int64_t cols, bool sums) {
  const int64_t wide = act_bwd_wide(cols, sums), strips = (cols + 8 * wide - 1) / (8 * wide), high = 256 / wide;
  const int64_t want = (4096 + strips - 1) / strips;
  auto by = [&](int64_t n) { return (rows + n * high - 1) / (n * high); };  // n rows a thread
  int64_t groups = by(sums ? 8 : 1);
  if (sums && groups * strips < 1024) groups = by(4);
  if (sums && groups * strips < 256) groups = by(2);
  return groups < want ? groups : want;
}

int64_t act_bwd_groups(int64_t rows, int64_t cols) { return act_bwd_blocks(rows, cols, true); }

hipError_t launch_act_bwd(const ActBwdArgs& a, hipStream_t stream) {
  const int wide = act_bwd_wide(a.cols, a.dbias != nullptr);
  const int64_t strips = (int64_t{a.cols} + 8 * wide - 1) / (8 * wide), groups = act_bwd_blocks(a.rows, a.cols, a.dbias != nullptr);
  auto go = [&](auto act, auto gated, auto end) {
    hipLaunchKernelGGL((act_bwd_kernel<decltype(act)::value, decltype(gated)::value, decltype(end)::value>),
                       dim3(static_cast<uint32_t>(strips), static_cast<uint32_t>(groups)), dim3(256), 0, stream, a, wide);
    return hipGetLastError();
  };
  auto by_end = [&](auto act, auto gated) {
    if (a.cols < 8) return go(act, gated, std::integral_constant<RowEnd, kTiny>{});
    if (a.cols % 8) return go(act, gated, std::integral_constant<RowEnd, kOdd>{});
    return go(act, gated, std::integral_constant<RowEnd, kEven>{});
  };
  const hipError_t e = by_activation(a.act, [&](auto act) {
    if constexpr (decltype(act)::value != PF8_ACT_NONE) {
      if (a.gated) return by_end(act, std::true_type{});
    }
    return by_end(act, std::false_type{});
  });
  if (e != hipSuccess || !a.dbias || groups == 1) return e;
  const int width = a.gated ? 2 * a.cols : a.cols;
  float* outs[3] = {a.dbias, nullptr, nullptr};
  return launch_column_sums(a.partial, static_cast<int>(groups), width, width, outs, a.accumulate, stream);
}

}  // namespace pf8
