// Block norm for gfx950: post-norm of a branch, gate, residual sum and pre-norm in one pass, with
// its backward pass. Formulas in include/pf8_train.h.
//
// Bound: HBM. Forward 8 bytes an element (h, y in; r, x out), backward 12 (h, y, dr, dx in; dh, dy
// out), one more bf16 each way for a gate per element; a few dozen FP32 operations an element.
// Each row is read once: its values stay in registers between the row sums, 8 consecutive bf16 per
// thread and step. A row belongs to 64, 256 or 1024 threads; sums run over a wave by DPP and, with
// several waves, once through LDS.
#include "pf8_device.h"
#include "pf8_train_launch.h"

namespace pf8 {

namespace {

// 16 bytes at 2-byte alignment: global accesses of any alignment are one instruction on gfx950, so
// odd row pitches take the same path as aligned ones.
typedef uint32_t u128_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f128_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(uint4 p, float (&f)[8]) {
  f[0] = bf_lo(p.x), f[1] = bf_hi(p.x), f[2] = bf_lo(p.y), f[3] = bf_hi(p.y);
  f[4] = bf_lo(p.z), f[5] = bf_hi(p.z), f[6] = bf_lo(p.w), f[7] = bf_hi(p.w);
}

typedef __bf16 nbf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const nbf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// 8 bf16 from p; only the first n are read (n >= 8 except in a row's last step), the rest are zero.
__device__ __forceinline__ uint4 load8(const uint16_t* p, int n) {
  if (n >= 8) {
    const u128_a2 v = *reinterpret_cast<const u128_a2*>(p);
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(uint16_t* p, uint4 v, int n) {
  if (n >= 8) {
    *reinterpret_cast<u128_a2*>(p) = u128_a2{v.x, v.y, v.z, v.w};
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}

// 8 weights (FP32 or BF16) from index c on, plus the offset.
__device__ __forceinline__ void load_w8(const void* w, int wf32, int c, int n, float offset, float (&f)[8]) {
  if (wf32) {
    const float* p = static_cast<const float*>(w) + c;
    if (n >= 8) {
      const f128_a4 a = *reinterpret_cast<const f128_a4*>(p), b = *reinterpret_cast<const f128_a4*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = a[i], f[i + 4] = b[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.0f;
    }
  } else {
    unpack8(load8(static_cast<const uint16_t*>(w) + c, n), f);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] += offset;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// Sums of N values over the L threads of a row. With several waves they meet in `slot`, N floats
// per wave; consecutive reductions take turns between two slots, so one barrier each is enough: a
// slot is written again only after the barrier of the reduction in between, which every thread
// reaches after it has read the slot.
template <int L, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* slot) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (L > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slot[wave * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < L / 64; ++w) s += slot[w * N + i];
      v[i] = s;
    }
  }
}

// 1 / sqrt(mean + eps) from a row's sum of (v * sq)^2. sq is a power of two (exact) near
// 1/sqrt(cols), so that the sum overflows only where the mean does: v up to 2^63 gets its norm.
__device__ __forceinline__ float inv_rms(float sum_sq, const NormArgs& p) {
  return 1.0f / __builtin_sqrtf(__builtin_fmaf(sum_sq, p.inv_sum, p.eps));
}
__device__ __forceinline__ float add_sq(float v, float sq, float s) {
  const float t = v * sq;
  return __builtin_fmaf(t, t, s);
}

// L threads per row, NV steps of 8 values per thread.
template <int L, int NV>
__global__ __launch_bounds__(L < 256 ? 256 : L) void norm_fwd_kernel(NormFwdArgs a) {
  constexpr int THREADS = L < 256 ? 256 : L, RPB = THREADS / L;
  __shared__ float slots[2][L > 64 ? L / 64 : 1];
  const NormArgs& p = a.in;
  const int t = threadIdx.x % L;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / L;
  if (RPB > 1 && row >= p.rows) return;  // whole waves only (one row per wave)
  const int cols = p.cols;

  uint4 hv[NV], yv[NV], gv[NV];
  const bool branch = p.y != nullptr, full_gate = p.gate != nullptr && p.ld_gate != 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (t + i * L), n = cols - c;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    hv[i] = yv[i] = gv[i] = z;
    if (n > 0) {
      hv[i] = load8(p.h + row * p.ldh + c, n);
      if (branch) yv[i] = load8(p.y + row * p.ldy + c, n);
      if (full_gate) gv[i] = load8(static_cast<const uint16_t*>(p.gate) + row * p.ld_gate + c, n);
    }
  }

  float r[NV][8];
  if (branch) {
    float rho_y = 1.0f;
    if (p.w_post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float y[8];
        unpack8(yv[i], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] = add_sq(y[k], p.sq, s[0]);
      }
      row_sum<L, 1>(s, slots[0]);
      rho_y = inv_rms(s[0], p);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (t + i * L), n = cols - c;
      float h[8], y[8];
      unpack8(hv[i], h);
      unpack8(yv[i], y);
      if (p.w_post && n > 0) {
        float w[8];
        load_w8(p.w_post, p.wf32, c, n, p.offset, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = y[k] * rho_y * w[k];
      }
      if (p.gate && n > 0) {
        float g[8];
        if (full_gate) unpack8(gv[i], g);
        else load_w8(p.gate, p.wf32, c, n, 0.0f, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] *= g[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i][k] = p.residual_scale * h[k] + p.branch_scale * y[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack8(hv[i], r[i]);
  }
  if (a.r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (t + i * L), n = cols - c;
      if (n > 0) store8(a.r + row * a.ldr + c, pack8(r[i]), n);
    }
  }
  if (!p.w_pre) return;

  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      // the places behind the row's end hold zeros (times finite scales)
      s[0] = add_sq(r[i][k], p.sq, s[0]);
  row_sum<L, 1>(s, slots[1]);
  const float rho_r = inv_rms(s[0], p);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (t + i * L), n = cols - c;
    if (n <= 0) continue;
    float w[8];
    load_w8(p.w_pre, p.wf32, c, n, p.offset, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = r[i][k] * rho_r * w[k];
    const uint4 v = pack8(w);
    if (a.x) store8(a.x + row * a.ldx + c, v, n);
    if (a.q) {
      // a 1x128 group is 16 consecutive threads; cols is a multiple of 128, so they are all here
      const int e = block_exponent(row16_max(amax8_bits(v)));
      *reinterpret_cast<uint2*>(a.q + row * a.ldq + c) = quant8_scaled(v, pow2f(e));
      if ((t & 15) == 0) a.dscale[static_cast<int64_t>(c >> 7) * a.ld_s + row] = pow2f(e);
    }
  }
}

// Backward: workgroup b takes rows b, b + G, ...; every thread sums its own columns' weight and
// gate gradients over the workgroup's rows in registers and writes one row of partial sums.
template <int L, int NV>
__global__ __launch_bounds__(L) void norm_bwd_kernel(NormBwdArgs a, int n_sums) {
  __shared__ float slots[2][2 * (L / 64)];
  const NormArgs& p = a.in;
  const int t = threadIdx.x, cols = p.cols;
  const bool branch = p.y != nullptr, full_gate = p.gate != nullptr && p.ld_gate != 0;
  const bool pre = a.dx != nullptr, post = p.w_post != nullptr;
  const float inv_n = 1.0f / static_cast<float>(cols);
  float acc[3][NV][8];
#pragma unroll
  for (int j = 0; j < 3; ++j)
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[j][i][k] = 0.0f;
  int turn = 0;

  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    uint4 hv[NV], yv[NV], gv[NV], rv[NV], xv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (t + i * L), n = cols - c;
      hv[i] = yv[i] = gv[i] = rv[i] = xv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (n > 0) {
        if (pre) hv[i] = load8(p.h + row * p.ldh + c, n);
        if (branch) yv[i] = load8(p.y + row * p.ldy + c, n);
        if (full_gate) gv[i] = load8(static_cast<const uint16_t*>(p.gate) + row * p.ld_gate + c, n);
        if (a.dr) rv[i] = load8(a.dr + row * a.lddr + c, n);
        if (pre) xv[i] = load8(a.dx + row * a.lddx + c, n);
      }
    }
    float rho_y = 1.0f;
    if (post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float y[8];
        unpack8(yv[i], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] = add_sq(y[k], p.sq, s[0]);
      }
      row_sum<L, 1>(s, slots[turn]);
      turn ^= 1;
      rho_y = inv_rms(s[0], p);
    }
    // the branch's value u at a step, and the gate's
    auto branch_values = [&](int i, int c, int n, float (&u)[8], float (&g)[8]) {
      unpack8(yv[i], u);
      if (post && n > 0) {
        float w[8];
        load_w8(p.w_post, p.wf32, c, n, p.offset, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = u[k] * rho_y * w[k];
      }
      if (full_gate) {
        unpack8(gv[i], g);
      } else if (p.gate && n > 0) {
        load_w8(p.gate, p.wf32, c, n, 0.0f, g);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = 1.0f;
      }
    };

    float d[NV][8];  // the gradient that reaches r
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack8(rv[i], d[i]);
    if (pre) {
      float s[2] = {0.0f, 0.0f};  // sums of (r sq)^2 and t (r sq)
      float rr[NV][8];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (t + i * L), n = cols - c;
        unpack8(hv[i], rr[i]);
        if (branch) {
          float u[8], g[8];
          branch_values(i, c, n, u, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) rr[i][k] = p.residual_scale * rr[i][k] + p.branch_scale * (u[k] * g[k]);
        }
        if (n > 0) {
          float x[8], w[8];
          unpack8(xv[i], x);
          load_w8(p.w_pre, p.wf32, c, n, p.offset, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float q = rr[i][k] * p.sq;
            s[0] = __builtin_fmaf(q, q, s[0]);
            s[1] = __builtin_fmaf(x[k] * w[k], q, s[1]);
          }
        }
      }
      row_sum<L, 2>(s, slots[turn]);
      turn ^= 1;
      const float rho_r = inv_rms(s[0], p);
      const float m = s[1] * rho_r * (inv_n / p.sq);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (t + i * L), n = cols - c;
        if (n <= 0) continue;
        float x[8], w[8];
        unpack8(xv[i], x);
        load_w8(p.w_pre, p.wf32, c, n, p.offset, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float rn = rr[i][k] * rho_r;
          acc[0][i][k] = __builtin_fmaf(x[k], rn, acc[0][i][k]);
          d[i][k] += rho_r * (x[k] * w[k] - rn * m);
        }
      }
    }
    if (a.dh) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (t + i * L), n = cols - c;
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = p.residual_scale * d[i][k];
        if (n > 0) store8(a.dh + row * a.lddh + c, pack8(o), n);
      }
    }
    if (!branch) continue;
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (t + i * L), n = cols - c;
      if (n <= 0) continue;
      float u[8], g[8];
      branch_values(i, c, n, u, g);
      float o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = p.branch_scale * d[i][k];
        o[k] = v * u[k];
        acc[2][i][k] += o[k];
        d[i][k] = v * g[k];
      }
      if (a.dgate_full) store8(a.dgate_full + row * a.ld_dgate + c, pack8(o), n);
      if (post) {
        float y[8], w[8];
        unpack8(yv[i], y);
        load_w8(p.w_post, p.wf32, c, n, p.offset, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float yn = y[k] * rho_y;
          acc[1][i][k] = __builtin_fmaf(d[i][k], yn, acc[1][i][k]);
          d[i][k] *= w[k];
          s[0] = __builtin_fmaf(d[i][k], yn, s[0]);
        }
      }
    }
    float m2 = 0.0f;
    if (post) {
      row_sum<L, 1>(s, slots[turn]);
      turn ^= 1;
      m2 = s[0] * inv_n;
    }
    if (a.dy) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 8 * (t + i * L), n = cols - c;
        float o[8], y[8];
        unpack8(yv[i], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = post ? rho_y * (d[i][k] - y[k] * rho_y * m2) : d[i][k];
        if (n > 0) store8(a.dy + row * a.lddy + c, pack8(o), n);
      }
    }
  }

  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * n_sums * cols;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    if (!a.sums[j]) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (t + i * L);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < cols) out[c + k] = acc[j][i][k];
    }
    out += cols;
  }
}

// Column sums of the workgroups' partial rows [groups][n_sums * cols], in a fixed order: 8 threads
// per column take every eighth row each, and one adds their eight sums.
constexpr int kSumCols = 32, kSumSlices = 8;
__global__ __launch_bounds__(kSumCols * kSumSlices) void norm_colsum_kernel(const float* partial, int groups, int width,
                                                                            int cols, float* o0, float* o1, float* o2,
                                                                            int accumulate) {
  __shared__ float sh[kSumSlices][kSumCols];
  const int lane = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + lane;
  float s = 0.0f;
  if (c < width) {
#pragma unroll 8
    for (int g = slice; g < groups; g += kSumSlices) s += partial[static_cast<int64_t>(g) * width + c];
  }
  sh[slice][lane] = s;
  __syncthreads();
  if (slice || c >= width) return;
#pragma unroll
  for (int i = 1; i < kSumSlices; ++i) s += sh[i][lane];
  const int j = c / cols, k = c - j * cols;
  float* o = (j == 0 ? o0 : j == 1 ? o1 : o2) + k;
  *o = accumulate ? *o + s : s;
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t stream) {
  const int64_t rows = a.in.rows;
  const int cols = a.in.cols;
  auto wide = [&](auto kern, int threads, int rpb) {
    hipLaunchKernelGGL(kern, dim3(static_cast<uint32_t>((rows + rpb - 1) / rpb)), dim3(threads), 0, stream, a);
    return hipGetLastError();
  };
  if (rows >= 1024 && cols <= 2048) {
    if (cols <= 512) return wide(norm_fwd_kernel<64, 1>, 256, 4);
    if (cols <= 1024) return wide(norm_fwd_kernel<64, 2>, 256, 4);
    return wide(norm_fwd_kernel<64, 4>, 256, 4);
  }
  if (cols <= 512) return wide(norm_fwd_kernel<64, 1>, 256, 4);
  if (cols <= 2048) return wide(norm_fwd_kernel<256, 1>, 256, 1);
  if (cols <= 4096) return wide(norm_fwd_kernel<256, 2>, 256, 1);
  if (cols <= 8192) return wide(norm_fwd_kernel<256, 4>, 256, 1);
  if (cols <= 16384) return wide(norm_fwd_kernel<1024, 2>, 1024, 1);
  return wide(norm_fwd_kernel<1024, 4>, 1024, 1);
}

int64_t norm_bwd_groups(int64_t rows, int64_t cols) {
  (void)cols;
  return rows < 512 ? rows : 512;
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t stream) {
  const int cols = a.in.cols;
  const int groups = static_cast<int>(norm_bwd_groups(a.in.rows, cols));
  float* outs[3] = {nullptr, nullptr, nullptr};
  int n_sums = 0;
  for (float* s : a.sums)
    if (s) outs[n_sums++] = s;
  auto go = [&](auto kern, int threads) {
    hipLaunchKernelGGL(kern, dim3(groups), dim3(threads), 0, stream, a, n_sums);
    return hipGetLastError();
  };
  hipError_t e;
  if (cols <= 512) e = go(norm_bwd_kernel<64, 1>, 64);
  else if (cols <= 2048) e = go(norm_bwd_kernel<256, 1>, 256);
  else if (cols <= 4096) e = go(norm_bwd_kernel<256, 2>, 256);
  else if (cols <= 8192) e = go(norm_bwd_kernel<1024, 1>, 1024);
  else if (cols <= 16384) e = go(norm_bwd_kernel<1024, 2>, 1024);
  else e = go(norm_bwd_kernel<1024, 4>, 1024);
  if (e != hipSuccess || n_sums == 0) return e;
  const int width = n_sums * cols;
  hipLaunchKernelGGL(norm_colsum_kernel, dim3((width + kSumCols - 1) / kSumCols), dim3(kSumCols * kSumSlices), 0, stream,
                     a.partial, groups, width, cols, outs[0], outs[1], outs[2], a.accumulate);
  return hipGetLastError();
}

}  // namespace pf8
