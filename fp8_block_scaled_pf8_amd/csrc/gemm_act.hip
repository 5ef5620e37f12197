// Block-scaled FP8 product with bias, activation and residual in its epilogue (gfx950). Formulas in
// include/pf8_layer.h.
#include "act_device.h"
#include "gemm_device.h"
#include "pf8_layer_launch.h"
#include "row_device.h"

namespace pf8 {

namespace {

__device__ __forceinline__ float act_any(int act, float z) {
  switch (act) {
    case PF8_ACT_RELU: return act_value<PF8_ACT_RELU>(z);
    case PF8_ACT_RELU2: return act_value<PF8_ACT_RELU2>(z);
    case PF8_ACT_SILU: return act_value<PF8_ACT_SILU>(z);
    case PF8_ACT_GELU: return act_value<PF8_ACT_GELU>(z);
    case PF8_ACT_GELU_TANH: return act_value<PF8_ACT_GELU_TANH>(z);
    default: return z;
  }
}

// Few tokens. A workgroup of 8 waves owns 16 columns of d (and the 16 or 32 rows of W that make them) for `per`
// tokens, up to 16 MT; its waves take the 128-wide K blocks in turn, each with its own loads straight into registers: no
// row of W is read by two waves, so LDS would only be a detour. One v_mfma_f32_16x16x128_f8f6f4 covers a K block of 16
// rows of W and 16 tokens; its partial is scaled into the wave's FP32 sum. The waves' sums meet in LDS, added in
// the waves' order.
// Bound: what a CU reads, its rows of W and of X, some 30 bytes a nanosecond. On the same operands again (in brackets on
// operands from memory): one token of 12288 x 2048 gated 6.9 us (8.5), 25 MB at 3.6 TB/s (3.0); 33 tokens of 2048 x 6144 with a bias
// onto a residual 10.1 us (12.0), two groups over 256 workgroups, 0.2 MB each. 16 waves, 4
// or 8 rows of W a workgroup, loads of whole cache lines a quarter wave and 3 to 8 K blocks in flight (gated, 6 took
// 8.5 us instead of 6.8) were no faster.
template <int MT, bool GATED>
__global__ __launch_bounds__(512) void fprop_act_few_kernel(FpropActArgs p, int per) {
  constexpr int WAVES = 8, PARTS = GATED ? 2 : 1, U = MT == 4 ? 2 : 4;  // U: K blocks whose loads go out together
  __shared__ v4f red[WAVES][PARTS][MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quarter = lane >> 4;
  const int64_t cols = GATED ? p.n / 2 : p.n;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16, m0 = static_cast<int64_t>(blockIdx.y) * per;
  const int64_t m1 = min64(m0 + per, p.m);  // one behind its tokens
  const int nk = static_cast<int>(p.k / kGroup);
  const uint8_t* w[PARTS];
  const float* sw[PARTS];
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const int64_t first = n0 + i * cols;
    w[i] = p.b + (i * cols + min64(n0 + l16, cols - 1)) * p.ldb + quarter * 32;
    sw[i] = p.b_dscale + (first >> 7) * p.ld_bs;
  }
  const uint8_t* x[MT];
  const float* sx[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t row = min64(m0 + 16 * t + l16, m1 - 1);
    x[t] = p.a + row * p.lda + quarter * 32;
    sx[t] = p.a_dscale + row;
  }
  v4f acc[PARTS][MT];
#pragma unroll
  for (int i = 0; i < PARTS; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[i][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = wave; kb < nk; kb += WAVES * U) {
    v8i fw[U][PARTS], fx[U][MT];
    uint32_t a[U][MT], b[U][PARTS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = kb + u * WAVES;
      if (at >= nk) break;
#pragma unroll
      for (int i = 0; i < PARTS; ++i) {
        fw[u][i] = lds_read32(w[i] + at * kGroup, 0, 16);
        b[u][i] = __float_as_uint(sw[i][at]);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        fx[u][t] = lds_read32(x[t] + at * kGroup, 0, 16);
        a[u][t] = __float_as_uint(sx[t][at * p.ld_as]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + u * WAVES >= nk) break;
#pragma unroll
      for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          // the two powers of two by their exponents: their product may be past FP32's range where the partial times it is not
          const int exponent = static_cast<int>(a[u][t] >> 23) + static_cast<int>(b[u][i] >> 23) - 254;
          const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[u][i], fx[u][t], zero, 0, 0, 0, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][t][r] += __builtin_ldexpf(part[r], exponent);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < PARTS; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) red[wave][i][t][lane] = acc[i][t];
  __syncthreads();
  // a thread takes 4 consecutive columns of a token
  const int t = threadIdx.x >> 6;
  if (t >= MT) return;
  const int64_t m = m0 + 16 * t + l16, n = n0 + 4 * quarter;
  if (m >= m1 || n >= cols) return;
  const int left = static_cast<int>(min64(4, cols - n));
  float v[PARTS][4];
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    v4f s = red[0][i][t][lane];
#pragma unroll
    for (int g = 1; g < WAVES; ++g) s += red[g][i][t][lane];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[i][r] = s[r];
    if (p.bias) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < left) v[i][r] += bias_at(p, i * cols + n + r);
    }
  }
  auto store = [&](uint16_t* out, const float (&f)[4]) {
    const uint32_t w0 = pack2(f[0], f[1]), w1 = pack2(f[2], f[3]);
    if (left == 4) {
      *reinterpret_cast<u64_a2*>(out) = u64_a2{w0, w1};
      return;
    }
    out[0] = static_cast<uint16_t>(w0);
    if (left > 1) out[1] = static_cast<uint16_t>(w0 >> 16);
    if (left > 2) out[2] = static_cast<uint16_t>(w1);
  };
  if (p.z) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) store(p.z + m * p.ldz + i * cols + n, v[i]);
  }
  float d[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    d[r] = act_any(p.act, v[0][r]);
    if constexpr (GATED) d[r] *= v[PARTS - 1][r];
    if (p.residual && r < left) d[r] += bf_lo(p.residual[m * p.ldr + n + r]);
  }
  store(p.d + m * p.ldd + n, d);
}

}  // namespace

// Workgroups along the columns.
static int64_t few_blocks(const FpropActArgs& a) { return ((a.gated ? a.n / 2 : a.n) + 15) / 16; }

// Groups of tokens: as many as there have to be, more where a CU each is left for them, and even ones (33 tokens as 17 and
// 16, not 32 and 1): a workgroup's time goes by the bytes that it reads, its rows of W and of X, which a CU takes at
// some 30 GB/s whatever is in flight. 33 x 2048 x 6144 9.4 us, with 32 and 1 tokens 11.3; 16 x 2048 x 6144 by two
// groups of 8 on 256 workgroups 7.4 us, by one on 128 8.4.
template <int MT>
static int64_t few_groups(const FpropActArgs& a) {
  const int64_t least = (a.m + 16 * MT - 1) / (16 * MT), fill = 256 / few_blocks(a);
  return least > fill ? least : fill < a.m ? fill : a.m;
}

template <int MT>
static hipError_t launch_few(const FpropActArgs& a, hipStream_t stream) {
  const int64_t groups = few_groups<MT>(a), per = (a.m + groups - 1) / groups;
  const dim3 grid(static_cast<uint32_t>(few_blocks(a)), static_cast<uint32_t>((a.m + per - 1) / per)),
      block(512);
  if (a.gated) hipLaunchKernelGGL((fprop_act_few_kernel<MT, true>), grid, block, 0, stream, a, static_cast<int>(per));
  else hipLaunchKernelGGL((fprop_act_few_kernel<MT, false>), grid, block, 0, stream, a, static_cast<int>(per));
  return hipGetLastError();
}

// Modelled times in microseconds, from sweeps of 1 to 8192 rows over weights of 12288 x 2048 (gated and not), 2048 x
// 6144, 2048 x 2048, 4096 x 2048, 1000 x 1536, 512 x 4096 and 6144 x 6144 (gated); what the models choose was within 8 %
// of the best choice, but for a few sizes next to a border. As an example, 64 rows on 2048 x 6144: 11.4 us by the
// kernel for few tokens, 32 of them a workgroup (13.9 by 16, 16.8 by 64), 16.0 by 64 x 64 tiles, 21.9 by 128 x 128.

// Few tokens, 16 MT of them a workgroup: a start, then its K blocks, with its tokens' operands; more workgroups than
// CUs share the memory's rate.
template <int MT>
static double few_cost(const FpropActArgs& a) {
  const int64_t groups = few_groups<MT>(a);
  const double share = static_cast<double>(a.n) / 16 / 256 * static_cast<double>(groups);
  const double tokens = static_cast<double>((a.m + groups - 1) / groups);
  return 3.0 + (share > 1.0 ? share : 1.0) * static_cast<double>(a.k) / 1024 * (0.5 + 0.028 * tokens);
}

// Tiles of one shape: a start, then rounds of one tile on each of 256 CUs, each of them by K and with its own end. A
// round that fills the card takes longer than a tile alone (clock, L2).
struct TileCost {
  int bm, bn;
  double start, alone, full, end;  // alone, full: for 1024 of K
  double operator()(const FpropActArgs& a) const {
    const int64_t out = a.gated ? bn / 2 : bn, cols = a.gated ? a.n / 2 : a.n;
    const int64_t tiles = (a.m + bm - 1) / bm * ((cols + out - 1) / out), rounds = (tiles + 255) / 256;
    const double fill = tiles < 256 ? static_cast<double>(tiles) / 256 : 1.0;
    return start + static_cast<double>(rounds) * ((alone + (full - alone) * fill) * static_cast<double>(a.k) / 1024 + end);
  }
};

FpropActTile fprop_act_tile(const FpropActArgs& a) {
  constexpr TileCost kShapes[] = {{256, 256, 7.0, 8.1, 12.2, 3.0},
                                  {256, 128, 7.0, 4.4, 8.0, 1.0},
                                  {128, 128, 6.0, 2.65, 4.7, 0.0},
                                  {64, 64, 4.0, 2.0, 2.1, 0.1}};
  int best = 0;
  double cost[4];
  for (int i = 0; i < 4; ++i) {
    cost[i] = kShapes[i](a);
    if (cost[i] < cost[best]) best = i;
  }
  const double few[3] = {few_cost<1>(a), few_cost<2>(a), few_cost<4>(a)};
  const int least = few[1] < few[0] ? (few[2] < few[1] ? 2 : 1) : few[2] < few[0] ? 2 : 0;
  if (a.m <= 1024 && few[least] < cost[best]) return {16 << least, 16};  // (the grid is as high as the groups of tokens)
  return {kShapes[best].bm, kShapes[best].bn};
}

hipError_t launch_fprop_act(const FpropActArgs& a, hipStream_t stream) {
  const FpropActTile t = fprop_act_tile(a);
  if (t.bn == 16) return t.bm == 16 ? launch_few<1>(a, stream) : t.bm == 32 ? launch_few<2>(a, stream) : launch_few<4>(a, stream);
  if (t.bn == 256) return launch_fprop_act_tiles<256, 256>(a, stream);
  if (t.bm == 256) return launch_fprop_act_tiles<256, 128>(a, stream);
  return t.bm == 128 ? launch_fprop_act_tiles<128, 128>(a, stream) : launch_fprop_act_tiles<64, 64>(a, stream);
}

}  // namespace pf8
