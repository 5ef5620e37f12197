// Block norm for gfx950: post-norm of a branch, gate, residual sum and pre-norm in one pass, with
// its backward pass. Formulas in include/pf8_train.h.
//
// Bound: HBM. Forward 8 bytes an element (h, y in; r, x out), backward 12 (h, y, dr, dx in; dh, dy
// out), one more bf16 each way for a gate per element; a few dozen FP32 operations an element.
// Each row is read once: its values stay in registers between the row sums, 8 consecutive bf16 per
// thread and step. A row belongs to a wave (up to 512 columns forward) or to a workgroup of as many
// waves as it fills; sums run over a wave by DPP and, with several waves, once through LDS.
// 8192 x 2048: forward 25.4 us (5.3 TB/s), backward 52.5 us (3.8 TB/s, of which 5 us are the column
// sums); backward 4096 x 6144 with a gate per element 88 us (4.6 TB/s).
#include "pf8_train_launch.h"
#include "row_device.h"

namespace pf8 {

namespace {

// Sums of N values over the threads of a row: one wave (WAVES = 1), or the whole workgroup of up to WAVES
// waves. With several waves they meet in `slot` (N rows of WAVES values, zero where there is no wave);
// consecutive reductions take turns between two slots, so one barrier each is enough: a slot is written
// again only after the barrier of the reduction in between, which every thread reaches after it has read
// the slot.
template <int WAVES, int N>
struct __align__(16) Slot {
  float v[N][WAVES];
};
template <int WAVES, int N, int M>
__device__ __forceinline__ void row_sum(float (&v)[N], Slot<WAVES, M>& slot) {
  static_assert(N <= M, "room for the values");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (WAVES > 1) {
    static_assert(WAVES % 4 == 0, "four at a time");
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slot.v[i][threadIdx.x >> 6] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; w += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&slot.v[i][w]);
        v[i] += (f.x + f.y) + (f.z + f.w);
      }
    }
  }
}
// Zeros for the waves that a workgroup does not have.
template <int WAVES, int N>
__device__ __forceinline__ void clear(Slot<WAVES, N> (&slots)[2]) {
  if constexpr (WAVES > 1) {
    for (int i = threadIdx.x; i < 2 * N * WAVES; i += blockDim.x) (&slots[0].v[0][0])[i] = 0.0f;
    __syncthreads();
  }
}

// 1 / sqrt(mean + eps) from a row's sum of (v * sq)^2. sq is a power of two (exact) near
// 1/sqrt(cols), so that the sum overflows only where the mean does: v up to 2^63 gets its norm.
__device__ __forceinline__ float inv_rms(float sum_sq, const NormArgs& p) {
  return inv_root(__builtin_fmaf(sum_sq, p.inv_sum, p.eps));
}
__device__ __forceinline__ float add_sq(float v, float sq, float s) {
  const float t = v * sq;
  return __builtin_fmaf(t, t, s);
}

// A thread's part of a row: NV steps of 8 columns, `span` threads apart. In the row's last step, where
// fewer than 8 columns are left, the thread takes the row's last 8 all the same, so that they come by one
// load, and masks those that belong to the thread before it: they count as zeros, and are not stored.
// (Loads put together from pieces would be waited for where they are made, and no longer travel during the
// row before: 8192 x 2047 backward took 143 us, now 54; 2048 columns 47, all from the caches.) kEven: there is
// no such step. kTiny: rows of under 8 columns, loaded value by value, zeros behind.
enum Tail { kEven, kOdd, kTiny };
template <int NV, Tail TAIL>
struct Cols {
  static constexpr bool TINY = TAIL == kTiny;
  int cols;
  int c[NV];      // the first column
  int first[NV];  // the first of the 8 that is the thread's own; 8: none is
  __device__ __forceinline__ Cols(int t, int span, int cols_) : cols(cols_) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = 8 * (t + i * span);
      const int n = cols - c[i];
      first[i] = n >= 8 || (TINY && n > 0) ? 0 : n <= 0 ? 8 : 8 - n;
      if (TAIL == kOdd && n < 8) c[i] = cols - 8;
    }
  }
  __device__ __forceinline__ bool any(int i) const { return first[i] < 8; }
  __device__ __forceinline__ void load(const uint16_t* row, uint4 (&v)[NV]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (any(i)) v[i] = TINY ? load_few(row, cols) : load8(row + c[i]);
    }
  }
  // zeros for the columns that are another thread's
  __device__ __forceinline__ void mask(uint4 (&v)[NV]) const {
    if constexpr (TAIL != kOdd) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (first[i]) {
        auto keep = [&](int w) { return first[i] <= 2 * w ? 0xFFFFFFFFu : first[i] == 2 * w + 1 ? 0xFFFF0000u : 0u; };
        v[i].x &= keep(0), v[i].y &= keep(1), v[i].z &= keep(2), v[i].w &= keep(3);
      }
  }
  __device__ __forceinline__ void store(uint16_t* row, int i, const float (&f)[8]) const { store(row, i, pack8(f)); }
  __device__ __forceinline__ void store(uint16_t* row, int i, uint4 v) const {
    if (!any(i)) return;
    uint16_t* p = row + c[i];
    if constexpr (TINY) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (k < cols) p[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    } else if (TAIL == kEven || first[i] == 0) {
      *reinterpret_cast<u128_a2*>(p) = u128_a2{v.x, v.y, v.z, v.w};
    } else {
      store_last(p, v, 8 - first[i]);
    }
  }
  // the 8 values of a vector of FP32 or BF16, plus the offset
  __device__ __forceinline__ void vector(const void* w, int wf32, int i, float offset, float (&f)[8]) const {
    if (!any(i)) return;
    if constexpr (TINY) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        f[k] = k >= cols ? 0.0f
               : wf32    ? static_cast<const float*>(w)[k]
                         : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(w)[k]) << 16);
    } else if (wf32) {
      const float* p = static_cast<const float*>(w) + c[i];
      const f128_a4 a = *reinterpret_cast<const f128_a4*>(p), b = *reinterpret_cast<const f128_a4*>(p + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = a[k], f[k + 4] = b[k];
    } else {
      unpack8(load8(static_cast<const uint16_t*>(w) + c[i]), f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] += offset;
    // (a zero times another thread's infinity would be a NaN in the row's sums)
    if (TAIL == kOdd && first[i]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = k < first[i] ? 0.0f : f[k];
    }
  }
};

// A [cols] vector's values at a thread's columns: kept in registers over the rows where they are few.
template <int NV, Tail TAIL, bool KEEP>
struct Weights {
  static constexpr bool kKeep = KEEP;
  const void* w;
  int wf32;
  float offset;
  float kept[kKeep ? NV : 1][8];
  __device__ __forceinline__ Weights(const void* w_, int wf32_, float offset_, const Cols<NV, TAIL>& at) : w(w_), wf32(wf32_), offset(offset_) {
    if constexpr (kKeep) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) kept[i][k] = 1.0f;
        if (w) at.vector(w, wf32, i, offset, kept[i]);
      }
    }
  }
  // (1 without a vector)
  __device__ __forceinline__ void get(int i, const Cols<NV, TAIL>& at, float (&f)[8]) const {
    if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = kept[i][k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = 1.0f;
      if (w) at.vector(w, wf32, i, offset, f);
    }
  }
};

// Forward. A row belongs to a wave (SINGLE: four rows a workgroup) or to the workgroup; workgroups walk
// the rows, and (AHEAD) the next row's values are on their way while one is worked on.
template <bool SINGLE, int NV, int THREADS, bool AHEAD, Tail TAIL>
__global__ __launch_bounds__(THREADS) void norm_fwd_kernel(NormFwdArgs a) {
  constexpr int kWaves = SINGLE ? 1 : THREADS / 64;
  __shared__ Slot<kWaves, 1> slots[2];
  clear(slots);
  const NormArgs& p = a.in;
  const int span = SINGLE ? 64 : blockDim.x, t = SINGLE ? threadIdx.x & 63 : threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (SINGLE ? THREADS / 64 : 1);
  const Cols<NV, TAIL> at(t, span, p.cols);
  const bool branch = p.y != nullptr, full_gate = p.gate != nullptr && p.ld_gate != 0, post = p.w_post != nullptr;
  const Weights<NV, TAIL, AHEAD> w_pre(p.w_pre, p.wf32, p.offset, at), w_post(p.w_post, p.wf32, p.offset, at),
      gate(full_gate ? nullptr : p.gate, p.wf32, 0.0f, at);

  uint4 hv[NV], yv[NV], gv[NV], hn[NV], yn[NV], gn[NV];
  auto load_row = [&](int64_t row, uint4 (&h)[NV], uint4 (&y)[NV], uint4 (&g)[NV]) {
    at.load(p.h + row * p.ldh, h);
    if (branch) at.load(p.y + row * p.ldy, y);
    if (full_gate) at.load(static_cast<const uint16_t*>(p.gate) + row * p.ld_gate, g);
  };
  int64_t row = SINGLE ? static_cast<int64_t>(blockIdx.x) * (THREADS / 64) + (threadIdx.x >> 6) : blockIdx.x;
  if (AHEAD && row < p.rows) load_row(row, hn, yn, gn);
  for (; row < p.rows; row += step) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) hv[i] = hn[i], yv[i] = yn[i], gv[i] = gn[i];
      if (row + step < p.rows) load_row(row + step, hn, yn, gn);
    } else {
      load_row(row, hv, yv, gv);
    }
    at.mask(hv);
    at.mask(yv);
    if (full_gate) at.mask(gv);

    float r[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack8(hv[i], r[i]);
    if (branch) {
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
        row_sum<kWaves>(s, slots[0]);
        rho_y = inv_rms(s[0], p);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float y[8], w[8];
        unpack8(yv[i], y);
        if (post) {
          w_post.get(i, at, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = y[k] * rho_y * w[k];
        }
        if (full_gate) unpack8(gv[i], w);
        else gate.get(i, at, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) r[i][k] = p.residual_scale * r[i][k] + p.branch_scale * (w[k] * y[k]);
      }
    }
    if (a.r) {
#pragma unroll
      for (int i = 0; i < NV; ++i) at.store(a.r + row * a.ldr, i, r[i]);
    }
    if (!p.w_pre) {
      if (!SINGLE) __syncthreads();  // slot 0 has been read
      continue;
    }

    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        // places that are not the thread's own hold zeros
        s[0] = add_sq(r[i][k], p.sq, s[0]);
    row_sum<kWaves>(s, slots[1]);
    // without a norm behind the branch, slot 1 alone is used: a barrier before it is written again
    if (!SINGLE && !(branch && post)) __syncthreads();
    const float rho_r = inv_rms(s[0], p);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!at.any(i)) continue;
      float w[8];
      w_pre.get(i, at, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = r[i][k] * rho_r * w[k];
      const uint4 v = pack8(w);
      if (a.x) at.store(a.x + row * a.ldx, i, v);
      if (a.q) {
        // a 1x128 group is 16 consecutive threads; cols is a multiple of 128, so they are all here
        const int e = block_exponent(row16_max(amax8_bits(v)));
        *reinterpret_cast<uint2*>(a.q + row * a.ldq + at.c[i]) = quant8_scaled(v, pow2f(e));
        if ((t & 15) == 0) a.dscale[static_cast<int64_t>(at.c[i] >> 7) * a.ld_s + row] = pow2f(e);
      }
    }
  }
}

// Backward: workgroup b takes rows b, b + G, ... (the next row on its way as above); every thread sums its
// own columns' weight and gate gradients over the workgroup's rows in registers and writes one row of
// partial sums. Where registers are short (over 8192 columns, and over 2048 where a row's odd end takes masks)
// no row is on its way and the two weights' sums lie in LDS, a thread at its own places: 4096 x 16384 in 460 us,
// 635 with the sums in registers, which spilled; 4096 x 5407 in 148 us, 195 with all of it in registers.
template <int NV, int THREADS, bool AHEAD, Tail TAIL>
__global__ __launch_bounds__(THREADS) void norm_bwd_kernel(NormBwdArgs a, int n_sums) {
  __shared__ Slot<THREADS / 64, 2> slots[2];
  clear(slots);
  const NormArgs& p = a.in;
  const int cols = p.cols;
  const Cols<NV, TAIL> at(threadIdx.x, blockDim.x, cols);
  const bool branch = p.y != nullptr, full_gate = p.gate != nullptr && p.ld_gate != 0;
  const bool pre = a.dx != nullptr, post = p.w_post != nullptr;
  const float inv_n = 1.0f / static_cast<float>(cols);
  const Weights<NV, TAIL, AHEAD> w_pre(pre ? p.w_pre : nullptr, p.wf32, p.offset, at), w_post(p.w_post, p.wf32, p.offset, at),
      gate(full_gate ? nullptr : p.gate, p.wf32, 0.0f, at);
  constexpr int kParked = AHEAD ? 0 : 2;  // of the sums for w_pre, w_post and the gate
  __shared__ float4 parked[AHEAD ? 1 : kParked * NV * 2][AHEAD ? 1 : THREADS];
  float acc[3 - kParked][NV][8];
  auto get_sum = [&](auto j, int i, float (&f)[8]) {
    if constexpr (decltype(j)::value < kParked) {
      const float4 a = parked[(decltype(j)::value * NV + i) * 2][threadIdx.x], b = parked[(decltype(j)::value * NV + i) * 2 + 1][threadIdx.x];
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = acc[decltype(j)::value - kParked][i][k];
    }
  };
  auto put_sum = [&](auto j, int i, const float (&f)[8]) {
    if constexpr (decltype(j)::value < kParked) {
      parked[(decltype(j)::value * NV + i) * 2][threadIdx.x] = make_float4(f[0], f[1], f[2], f[3]);
      parked[(decltype(j)::value * NV + i) * 2 + 1][threadIdx.x] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[decltype(j)::value - kParked][i][k] = f[k];
    }
  };
  using Pre = std::integral_constant<int, 0>;
  using Post = std::integral_constant<int, 1>;
  using Gate = std::integral_constant<int, 2>;
  {
    const float none[8] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) put_sum(Pre{}, i, none), put_sum(Post{}, i, none), put_sum(Gate{}, i, none);
  }
  int turn = 0;
  auto sum = [&](auto& s) {
    row_sum<THREADS / 64>(s, slots[turn]);
    turn ^= 1;
  };

  struct Row {
    uint4 h[NV], y[NV], g[NV], dr[NV], dx[NV];
  };
  auto load_row = [&](int64_t row, Row& v) {
    if (pre) {
      at.load(p.h + row * p.ldh, v.h);
      at.load(a.dx + row * a.lddx, v.dx);
    }
    if (branch) at.load(p.y + row * p.ldy, v.y);
    if (full_gate) at.load(static_cast<const uint16_t*>(p.gate) + row * p.ld_gate, v.g);
    if (a.dr) at.load(a.dr + row * a.lddr, v.dr);
  };
  Row cur{}, next{};
  if (AHEAD) load_row(blockIdx.x, next);  // there are no more workgroups than rows
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    if constexpr (AHEAD) {
      cur = next;
      if (row + gridDim.x < p.rows) load_row(row + gridDim.x, next);
    } else {
      asm volatile("" ::: "memory");  // weights are loaded where they are used, not kept
      load_row(row, cur);
    }
    at.mask(cur.y);
    if (full_gate) at.mask(cur.g);
    float rho_y = 1.0f;
    if (post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float y[8];
        unpack8(cur.y[i], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] = add_sq(y[k], p.sq, s[0]);
      }
      sum(s);
      rho_y = inv_rms(s[0], p);
    }
    // the branch's value u at a step, and the gate's
    auto branch_values = [&](int i, float (&u)[8], float (&g)[8]) {
      unpack8(cur.y[i], u);
      if (post) {
        w_post.get(i, at, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = u[k] * rho_y * g[k];
      }
      if (full_gate) unpack8(cur.g[i], g);
      else gate.get(i, at, g);
    };

    at.mask(cur.dr);
    float d[NV][8];  // the gradient that reaches r
    if (pre) {
      at.mask(cur.h);
      at.mask(cur.dx);
      float s[2] = {0.0f, 0.0f};  // sums of (r sq)^2 and t (r sq)
      float rr[NV][8];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack8(cur.h[i], rr[i]);
        if (branch) {
          float u[8], g[8];
          branch_values(i, u, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) rr[i][k] = p.residual_scale * rr[i][k] + p.branch_scale * (u[k] * g[k]);
        }
        float x[8], w[8];
        unpack8(cur.dx[i], x);
        w_pre.get(i, at, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float q = rr[i][k] * p.sq;
          s[0] = __builtin_fmaf(q, q, s[0]);
          s[1] = __builtin_fmaf(x[k] * w[k], q, s[1]);
        }
      }
      sum(s);
      const float rho_r = inv_rms(s[0], p);
      const float m = s[1] * rho_r * (inv_n / p.sq);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[8], w[8], dw[8];
        unpack8(cur.dx[i], x);
        w_pre.get(i, at, w);
        get_sum(Pre{}, i, dw);
        unpack8(cur.dr[i], d[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float rn = rr[i][k] * rho_r;
          dw[k] = __builtin_fmaf(x[k], rn, dw[k]);
          d[i][k] += rho_r * (x[k] * w[k] - rn * m);
        }
        put_sum(Pre{}, i, dw);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack8(cur.dr[i], d[i]);
    }
    if (a.dh) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = p.residual_scale * d[i][k];
        at.store(a.dh + row * a.lddh, i, o);
      }
    }
    if (!branch) continue;
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float u[8], g[8], o[8], dg[8];
      branch_values(i, u, g);
      get_sum(Gate{}, i, dg);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = p.branch_scale * d[i][k];
        o[k] = v * u[k];
        dg[k] += o[k];
        d[i][k] = v * g[k];
      }
      put_sum(Gate{}, i, dg);
      if (a.dgate_full) at.store(a.dgate_full + row * a.ld_dgate, i, o);
      if (post) {
        float y[8], w[8], dw[8];
        unpack8(cur.y[i], y);
        w_post.get(i, at, w);
        get_sum(Post{}, i, dw);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float yn = y[k] * rho_y;
          dw[k] = __builtin_fmaf(d[i][k], yn, dw[k]);
          d[i][k] *= w[k];
          s[0] = __builtin_fmaf(d[i][k], yn, s[0]);
        }
        put_sum(Post{}, i, dw);
      }
    }
    float m2 = 0.0f;
    if (post) {
      sum(s);
      m2 = s[0] * inv_n;
    }
    if (a.dy) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float o[8], y[8];
        unpack8(cur.y[i], y);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = post ? rho_y * (d[i][k] - y[k] * rho_y * m2) : d[i][k];
        at.store(a.dy + row * a.lddy, i, o);
      }
    }
  }

  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * n_sums * cols;
  auto write_sum = [&](auto j) {
    if (!a.sums[decltype(j)::value]) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[8];
      get_sum(j, i, f);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k >= at.first[i] && at.c[i] + k < cols) out[at.c[i] + k] = f[k];
    }
    out += cols;
  };
  write_sum(Pre{}), write_sum(Post{}), write_sum(Gate{});
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

// Workgroups for `units` units of work (rows, or four of them): no more than the card's 256 CUs hold at
// once, and evenly loaded. With inputs in the caches, 8192 x 2048 forward: 22.9 us with 1024 workgroups of 8
// rows, 23.8 with twice as many, 24.4 with one for each row; backward 47.0 us with 512, 51.7 with 745, 57.5
// with 1024 (each writes a row of partial sums).
static int64_t even_groups(int64_t units, int64_t per_cu) {
  const int64_t most = 256 * (per_cu < 1 ? 1 : per_cu), each = (units + most - 1) / most;
  return (units + each - 1) / each;
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t stream) {
  const int64_t rows = a.in.rows;
  const int cols = a.in.cols;
  auto go = [&](auto kern, int64_t groups, int threads) {
    hipLaunchKernelGGL(kern, dim3(static_cast<uint32_t>(groups)), dim3(threads), 0, stream, a);
    return hipGetLastError();
  };
  // A row by one wave, by up to four with the next row on its way (88 registers: 20 waves on a CU), or by up to
  // 16 without (wide rows have enough loads in flight: 4096 x 6144 with a full gate 39.9 us, 40.7 us by half the
  // waves with the next row on its way; 1003 x 5407 12.3 us, 16.9).
  const int threads = (cols + 511) / 512 * 64;  // 8 values each
  if (cols < 8) return go(norm_fwd_kernel<true, 1, 256, true, kTiny>, even_groups((rows + 3) / 4, 5), 256);
  auto by_width = [&](auto tail) {
    constexpr Tail T = decltype(tail)::value;
    if (cols <= 512) return go(norm_fwd_kernel<true, 1, 256, true, T>, even_groups((rows + 3) / 4, 5), 256);
    if (cols <= 2048) return go(norm_fwd_kernel<false, 1, 256, true, T>, even_groups(rows, 1280 / threads), threads);
    if (cols <= 8192) return go(norm_fwd_kernel<false, 1, 1024, false, T>, even_groups(rows, 1536 / threads), threads);
    return go(norm_fwd_kernel<false, 2, 1024, false, T>, even_groups(rows, 1), 1024);
  };
  return cols % 8 ? by_width(std::integral_constant<Tail, kOdd>{}) : by_width(std::integral_constant<Tail, kEven>{});
}

// Threads of a row in the backward pass: whole waves, one or two steps of 8 values each.
static int norm_bwd_threads(int64_t cols) {
  const int64_t steps = cols <= 2048 ? 1 : 2;
  return static_cast<int>((cols + 512 * steps - 1) / (512 * steps) * 64);
}

// Eight waves on a CU: see even_groups. (The kernels' registers would allow more.)
int64_t norm_bwd_groups(int64_t rows, int64_t cols) {
  return even_groups(rows, 512 / norm_bwd_threads(cols));  // (at least one)
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
  const int threads = norm_bwd_threads(cols);
  auto by_width = [&](auto tail) {
    constexpr Tail T = decltype(tail)::value;
    if (cols <= 2048) return go(norm_bwd_kernel<1, 256, true, T>, threads);
    if (cols <= 8192) return go(norm_bwd_kernel<2, 512, T == kEven, T>, threads);
    return go(norm_bwd_kernel<2, 1024, false, T>, threads);
  };
  const hipError_t e = cols < 8   ? go(norm_bwd_kernel<1, 256, true, kTiny>, threads)
                       : cols % 8 ? by_width(std::integral_constant<Tail, kOdd>{})
                                  : by_width(std::integral_constant<Tail, kEven>{});
  if (e != hipSuccess || n_sums == 0) return e;
  return launch_column_sums(a.partial, groups, n_sums * cols, cols, outs, a.accumulate, stream);
}

hipError_t launch_column_sums(const float* partial, int groups, int width, int cols, float* const (&outs)[3],
                              int accumulate, hipStream_t stream) {
  hipLaunchKernelGGL(norm_colsum_kernel, dim3((width + kSumCols - 1) / kSumCols), dim3(kSumCols * kSumSlices), 0, stream,
                     partial, groups, width, cols, outs[0], outs[1], outs[2], accumulate);
  return hipGetLastError();
}

}  // namespace pf8
