// Norms of queries and keys for each head with the rotation by positions, and their backward pass
// (gfx950). Formulas in include/pf8_layer.h.
//
// Bound: HBM. Forward 4 bytes a value (in and out), backward 6 (values, gradients, result); some ten FP32
// operations a value, and for each token and pair an angle, its sine and cosine.
// All times in this file are the GPU's alone, of 16 + 8 heads of 128 unless stated, on operands that come from memory
// (sets of over 1 GB in turn); in brackets on the same operands again, of which the caches hold a part. 8192 tokens: forward
// 26.0 us (22.1), 101 MB at 3.9 TB/s; backward 35.0 us (31.0), of which 3.5 are the sums of the weights' gradients, 151 MB at
// 4.8 TB/s without those. Short batches are bound by one trip through memory and its FP64 angles: one token 3.0 us (2.9),
// 1003 tokens of 14 + 2 heads of 80 with three axes 8.3 (7.1).
// A head belongs to a group of lanes of one wave; each lane holds 8 rotated pairs (16 values, two 16-byte
// loads), so that both values of a pair are in the same lane and the sums of a head run over the group by
// DPP. A group takes up to HC heads of one token after another with the same angles; all their loads go out first.
#include "pf8_layer_launch.h"
#include "row_device.h"

namespace pf8 {

namespace {

// Which values a lane holds.
//  kHalves: pair i is (i, pairs + i). A lane has 8 consecutive pairs; what is not rotated counts as pairs too,
//           of its first and second half.
//  kNext:   pair i is (2 i, 2 i + 1). A lane has 16 consecutive values.
//  kSingle: heads that 8 pairs at a time do not cover (odd sizes, under 8 pairs rotated or left over): a whole
//           wave, value by value.
// A last step of fewer than 8 pairs takes the last 8 all the same, so that it comes by the same loads: `first`
// says how many of them are the lane's before. They are left out of sums and stored twice, with the same result.
enum Kind { kHalves, kNext, kSingle };

template <Kind KIND>
struct Lane {
  static constexpr int N = 8;
  struct Raw {
    uint4 u, v;
  };
  int e0, e1, p0, first, rotated;  // values' places, first pair, pairs before it that are another lane's, rotated ones
  __device__ __forceinline__ Lane(int c, const HeadNormArgs& p) {
    const int half = (KIND == kNext ? p.dim : p.dim - 2 * p.pairs) / 2;
    const int steps = KIND == kNext ? 0 : (p.pairs + 7) / 8;
    const bool rot = KIND == kNext || c < steps;
    const int n = rot && KIND == kHalves ? p.pairs : half, at = 8 * (rot ? c : c - steps);
    p0 = min(at, n - 8);
    first = min(at - p0, 8);  // 8: none is left for this lane
    if (first == 8) p0 = 0;
    if (KIND == kNext) {
      e0 = 2 * p0, e1 = e0 + 8;
      rotated = min(max(p.pairs - p0, 0), 8);
    } else {
      e0 = rot ? p0 : 2 * p.pairs + p0;
      e1 = e0 + n;
      rotated = rot ? 8 : 0;
    }
  }
  __device__ __forceinline__ bool any() const { return first < 8; }
  __device__ __forceinline__ bool own(int i) const { return i >= first; }
  __device__ __forceinline__ bool has_b(int) const { return true; }
  __device__ __forceinline__ int pair(int i) const { return p0 + i; }
  __device__ __forceinline__ bool rot(int i) const { return i < rotated; }
  __device__ __forceinline__ int place_a(int i) const { return KIND == kNext ? e0 + 2 * i : e0 + i; }
  __device__ __forceinline__ int place_b(int i) const { return KIND == kNext ? e0 + 2 * i + 1 : e1 + i; }
  __device__ __forceinline__ Raw load(const uint16_t* x) const { return {load8(x + e0), load8(x + e1)}; }
  static __device__ __forceinline__ Raw none() { return {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)}; }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&a)[8], float (&b)[8]) {
    if constexpr (KIND == kNext) {
      const uint32_t w[8] = {r.u.x, r.u.y, r.u.z, r.u.w, r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = bf_lo(w[i]), b[i] = bf_hi(w[i]);
    } else {
      unpack8(r.u, a);
      unpack8(r.v, b);
    }
  }
  __device__ __forceinline__ void store(uint16_t* x, const float (&a)[8], const float (&b)[8]) const {
    uint4 u, v;
    if constexpr (KIND == kNext) {
      u = make_uint4(pack2(a[0], b[0]), pack2(a[1], b[1]), pack2(a[2], b[2]), pack2(a[3], b[3]));
      v = make_uint4(pack2(a[4], b[4]), pack2(a[5], b[5]), pack2(a[6], b[6]), pack2(a[7], b[7]));
    } else {
      u = pack8(a), v = pack8(b);
    }
    // (cached: with non-temporal stores the forward of 8192 tokens takes 20.8 us instead of 26.0, but with a copy of its
    // result after it 45.8 instead of 44.5: whoever reads the result next then reads it from memory)
    *reinterpret_cast<u128_a2*>(x + e0) = u128_a2{u.x, u.y, u.z, u.w};
    *reinterpret_cast<u128_a2*>(x + e1) = u128_a2{v.x, v.y, v.z, v.w};
  }
};

template <>
struct Lane<kSingle> {
  static constexpr int N = 4;  // pairs l, l + 64, ...: up to 256 of them
  struct Raw {
    uint16_t a[4], b[4];
  };
  int l, s, b_off, pairs, dim, next;  // s: pairs, counting what is not rotated
  __device__ __forceinline__ Lane(int c, const HeadNormArgs& p) : l(c), pairs(p.pairs), dim(p.dim), next(p.interleaved) {
    const int rest = (p.dim - 2 * p.pairs + 1) / 2;
    s = p.pairs + rest;
    b_off = rest;
  }
  __device__ __forceinline__ bool any() const { return l < s; }
  __device__ __forceinline__ bool own(int i) const { return pair(i) < s; }
  __device__ __forceinline__ int pair(int i) const { return l + 64 * i; }
  __device__ __forceinline__ bool rot(int i) const { return pair(i) < pairs; }
  __device__ __forceinline__ int place_a(int i) const {
    return next ? 2 * pair(i) : rot(i) ? pair(i) : pairs + pair(i);
  }
  __device__ __forceinline__ int place_b(int i) const {
    return next ? 2 * pair(i) + 1 : rot(i) ? pairs + pair(i) : pairs + pair(i) + b_off;
  }
  __device__ __forceinline__ bool has_b(int i) const { return own(i) && place_b(i) < dim; }
  __device__ __forceinline__ Raw load(const uint16_t* x) const {
    Raw r = none();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (own(i)) r.a[i] = x[place_a(i)];
      if (has_b(i)) r.b[i] = x[place_b(i)];
    }
    return r;
  }
  static __device__ __forceinline__ Raw none() { return {{0, 0, 0, 0}, {0, 0, 0, 0}}; }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&a)[4], float (&b)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = bf_lo(r.a[i]), b[i] = bf_lo(r.b[i]);
  }
  __device__ __forceinline__ void store(uint16_t* x, const float (&a)[4], const float (&b)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = pack2(a[i], b[i]);
      if (own(i)) x[place_a(i)] = static_cast<uint16_t>(w);
      if (has_b(i)) x[place_b(i)] = static_cast<uint16_t>(w >> 16);
    }
  }
};

// Sum over the G consecutive lanes of a group, the same in each of them.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (G == 64) return wave_sum(v);
  auto step = [&](auto ctrl) {
    v += __uint_as_float(static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), decltype(ctrl)::value, 0xF, 0xF, true)));
  };
  // quad_perm [1,0,3,2], quad_perm [2,3,0,1], row_half_mirror, row_mirror
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  if constexpr (G >= 8) step(std::integral_constant<int, 0x141>{});
  if constexpr (G >= 16) step(std::integral_constant<int, 0x140>{});
  if constexpr (G >= 32) v += __shfl_xor(v, 16);
  return v;
}

// Cosines and sines of a lane's pairs at a token. Angles are counted in turns: position * inv_freq / 2 pi in
// FP64 (inv_freq / 2 pi is made once), of which the fraction in (-1/2, 1/2) goes to the FP32 instructions, which take
// turns. An FP32 angle would be off by 2^-24 of itself, 0.06 radians at position 10^6.
template <Kind KIND, bool MULTI>
struct Turns {
  static constexpr int N = Lane<KIND>::N;
  double f[N];
  int axis[MULTI ? N : 1];
  __device__ __forceinline__ Turns(const Lane<KIND>& at, const HeadNormArgs& p) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = 0.0;
    if (!p.freq) return;
    bool whole = false;  // the lane's pairs are all rotated: their frequencies by vector loads
    if constexpr (KIND != kSingle) whole = at.rotated == 8;
    if (whole) {
      if constexpr (KIND != kSingle) {
        if (p.f64) {
          const double* w = static_cast<const double*>(p.freq) + at.p0;
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = w[i];
        } else {
          const float* w = static_cast<const float*>(p.freq) + at.p0;
          const f128_a4 a = *reinterpret_cast<const f128_a4*>(w), b = *reinterpret_cast<const f128_a4*>(w + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = static_cast<double>(a[i]), f[i + 4] = static_cast<double>(b[i]);
        }
      }
    } else if (p.f64) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (at.rot(i)) f[i] = static_cast<const double*>(p.freq)[at.pair(i)];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (at.rot(i)) f[i] = static_cast<double>(static_cast<const float*>(p.freq)[at.pair(i)]);
    }
    const int start = MULTI && p.cycled ? at.pair(0) % p.axes : 0, step = KIND == kSingle ? 64 % p.axes : 1;
    int turn = start;  // the axis whose turn it is
#pragma unroll
    for (int i = 0; i < N; ++i) {
      f[i] *= 0.15915494309189533577;
      if constexpr (MULTI) {
        const int k = at.pair(i);
        if (p.cycled) {
          const int lim = turn == 0 ? p.share[0] : turn == 1 ? p.share[1] : turn == 2 ? p.share[2] : p.share[3];
          axis[i] = k < lim ? turn : 0;
          turn += step;
          if (turn >= p.axes) turn -= p.axes;
        } else {
          axis[i] = (k >= p.share[0]) + (k >= p.share[1]) + (k >= p.share[2]);
        }
      }
    }
  }
  __device__ __forceinline__ void at(int64_t token, const Lane<KIND>& l, const HeadNormArgs& p, float (&c)[N],
                                     float (&s)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = 1.0f, s[i] = 0.0f;
    if (!p.pos) return;
    auto position = [&](int a) {
      if (MULTI && a >= p.axes) return 0.0;
      const int64_t k = token * p.pos_st + a * p.pos_sa;
      // a 64-bit position's low half and high half (or the sign of a 32-bit one)
      const int32_t* q = static_cast<const int32_t*>(p.pos) + (p.p64 ? 2 * k : k);
      const uint32_t low = static_cast<uint32_t>(q[0]);
      const int32_t high = p.p64 ? q[1] : q[0] >> 31;
      return __builtin_fma(static_cast<double>(high), 0x1p32, static_cast<double>(low));
    };
    const double x0 = position(0), x1 = MULTI ? position(1) : 0.0, x2 = MULTI ? position(2) : 0.0,
                 x3 = MULTI ? position(3) : 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!l.rot(i)) continue;
      double x = x0;
      if constexpr (MULTI) x = axis[i] == 0 ? x0 : axis[i] == 1 ? x1 : axis[i] == 2 ? x2 : x3;
      x *= f[i];
      const float t = static_cast<float>(x - __builtin_rint(x));
      c[i] = __builtin_amdgcn_cosf(t) * p.scale;
      s[i] = __builtin_amdgcn_sinf(t) * p.scale;
    }
  }
};

// A head's weight at a lane's values, plus the offset; ones without a weight.
template <Kind KIND>
__device__ __forceinline__ void head_weights(const void* w, const HeadNormArgs& p, const Lane<KIND>& at,
                                             float (&wa)[Lane<KIND>::N], float (&wb)[Lane<KIND>::N]) {
  constexpr int N = Lane<KIND>::N;
#pragma unroll
  for (int i = 0; i < N; ++i) wa[i] = wb[i] = 1.0f;
  if (!w || !at.any()) return;
  if constexpr (KIND == kSingle) {
    auto get = [&](int k) { return p.wf32 ? static_cast<const float*>(w)[k] : bf_lo(static_cast<const uint16_t*>(w)[k]); };
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (at.own(i)) wa[i] = get(at.place_a(i)) + p.offset;
      if (at.has_b(i)) wb[i] = get(at.place_b(i)) + p.offset;
    }
    return;
  } else if (p.wf32) {
    const float* v = static_cast<const float*>(w);
    const f128_a4 q[4] = {*reinterpret_cast<const f128_a4*>(v + at.e0), *reinterpret_cast<const f128_a4*>(v + at.e0 + 4),
                          *reinterpret_cast<const f128_a4*>(v + at.e1), *reinterpret_cast<const f128_a4*>(v + at.e1 + 4)};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      wa[i] = KIND == kNext ? q[i / 2][2 * i % 4] : q[i / 4][i % 4];
      wb[i] = KIND == kNext ? q[i / 2][2 * i % 4 + 1] : q[2 + i / 4][i % 4];
    }
  } else {
    Lane<KIND>::unpack(at.load(static_cast<const uint16_t*>(w)), wa, wb);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) wa[i] += p.offset, wb[i] += p.offset;
}

// A group's items: up to HC consecutive heads of a token.
struct Items {
  int heads, per_token;
  int64_t count;
  __device__ __forceinline__ Items(int64_t tokens, int heads_, int hc)
      : heads(heads_), per_token((heads_ + hc - 1) / hc), count(tokens * per_token) {}
};

template <Kind KIND, int G, int HC, bool MULTI>
__global__ __launch_bounds__(256) void head_norm_fwd_kernel(HeadNormArgs p, unsigned blocks_q) {
  constexpr int N = Lane<KIND>::N;
  const int second = blockIdx.x >= blocks_q;
  const HeadTensor x = second ? p.t[1] : p.t[0];
  const Items items(p.tokens, x.heads, HC);
  const Lane<KIND> at(threadIdx.x % G, p);
  const unsigned block = blockIdx.x - (second ? blocks_q : 0), blocks = second ? gridDim.x - blocks_q : blocks_q;
  // (one item each, but for tensors of more than 2^22 workgroups)
  for (int64_t item = static_cast<int64_t>(block) * (256 / G) + threadIdx.x / G; item < items.count;
       item += static_cast<int64_t>(blocks) * (256 / G)) {
    const uint32_t token = static_cast<uint32_t>(item) / static_cast<uint32_t>(items.per_token);
    const int head = (static_cast<int>(item) - static_cast<int>(token) * items.per_token) * HC;

    typename Lane<KIND>::Raw raw[HC];
    const uint16_t* src = x.x + token * x.x_st + head * x.x_sh;
#pragma unroll
    for (int j = 0; j < HC; ++j) {
      raw[j] = Lane<KIND>::none();
      if (head + j < x.heads && at.any()) raw[j] = at.load(src + j * x.x_sh);
    }
    const Turns<KIND, MULTI> turns(at, p);
    float c[N], s[N], wa[N], wb[N];
    turns.at(token, at, p, c, s);
    head_weights(x.w, p, at, wa, wb);
    uint16_t* dst = x.out + token * x.out_st + head * x.out_sh;
#pragma unroll
    for (int j = 0; j < HC; ++j) {
      if (head + j >= x.heads) break;
      float a[N], b[N];
      Lane<KIND>::unpack(raw[j], a, b);
      if (x.w) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float u = a[i] * p.sq, v = b[i] * p.sq;
          const float both = __builtin_fmaf(u, u, v * v);
          if (at.own(i)) sum += both;
        }
        const float rho = inv_root(__builtin_fmaf(group_sum<G>(sum), p.inv_sum, p.eps));
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = a[i] * rho * wa[i], b[i] = b[i] * rho * wb[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u = a[i] * c[i] - b[i] * s[i], v = a[i] * s[i] + b[i] * c[i];
        a[i] = at.rot(i) ? u : a[i], b[i] = at.rot(i) ? v : b[i];
      }
      if (at.any()) at.store(dst + j * x.out_sh, a, b);
    }
  }
}

// Backward. The first workgroups take q's items, the others k's, in turn; each lane sums the weight's gradient at
// its own values, the groups' sums meet in LDS, and a workgroup writes one row of partial sums. (With both tensors
// in every workgroup a short batch waited for everything twice: 1537 tokens of 7 + 1 heads of 96 with three axes (12.2) us,
// now 11.9 (9.9).)
template <Kind KIND, int G, int HC, bool MULTI>
__global__ __launch_bounds__(256) void head_norm_bwd_kernel(HeadNormArgs p, unsigned blocks_q) {
  constexpr int N = Lane<KIND>::N, GROUPS = 256 / G;
  // a group's sums, in the order of its lanes: [pair of the lane][a or b]
  __shared__ float sums[GROUPS][G][2 * N + 1];
  const int group = threadIdx.x / G, lane = threadIdx.x % G;
  const Lane<KIND> at(lane, p);
  const Turns<KIND, MULTI> turns(at, p);
  const float inv_n = 1.0f / static_cast<float>(p.dim);
  const int second = blockIdx.x >= blocks_q;
  const HeadTensor x = second ? p.t[1] : p.t[0];  // (by an index, the arguments would be copied to scratch memory)
  const Items items(p.tokens, x.heads, HC);
  float wa[N], wb[N], sa[N], sb[N];
  head_weights(x.w, p, at, wa, wb);
#pragma unroll
  for (int i = 0; i < N; ++i) sa[i] = sb[i] = 0.0f;
  const unsigned block = blockIdx.x - (second ? blocks_q : 0), blocks = second ? gridDim.x - blocks_q : blocks_q;
  for (int64_t item = static_cast<int64_t>(block) * GROUPS + group; item < items.count;
       item += static_cast<int64_t>(blocks) * GROUPS) {
    const uint32_t token = static_cast<uint32_t>(item) / static_cast<uint32_t>(items.per_token);
    const int head = (static_cast<int>(item) - static_cast<int>(token) * items.per_token) * HC;
    typename Lane<KIND>::Raw rx[HC], rd[HC];
    const uint16_t* xs = x.x + token * x.x_st + head * x.x_sh;
    const uint16_t* ds = x.d + token * x.d_st + head * x.d_sh;
#pragma unroll
    for (int j = 0; j < HC; ++j) {
      rx[j] = rd[j] = Lane<KIND>::none();
      if (head + j < x.heads && at.any()) {
        if (x.w) rx[j] = at.load(xs + j * x.x_sh);
        rd[j] = at.load(ds + j * x.d_sh);
      }
    }
    float c[N], s[N];
    turns.at(token, at, p, c, s);
    uint16_t* dst = x.out + token * x.out_st + head * x.out_sh;
#pragma unroll
    for (int j = 0; j < HC; ++j) {
      if (head + j >= x.heads) break;
      float a[N], b[N];
      Lane<KIND>::unpack(rd[j], a, b);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u = a[i] * c[i] + b[i] * s[i], v = b[i] * c[i] - a[i] * s[i];
        a[i] = at.rot(i) ? u : a[i], b[i] = at.rot(i) ? v : b[i];
      }
      if (x.w) {
        float ya[N], yb[N], sum = 0.0f, dot = 0.0f;
        Lane<KIND>::unpack(rx[j], ya, yb);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float u = ya[i] * p.sq, v = yb[i] * p.sq;
          const float both = __builtin_fmaf(u, u, v * v), with = __builtin_fmaf(a[i] * wa[i], u, b[i] * wb[i] * v);
          if (at.own(i)) sum += both, dot += with;
        }
        sum = group_sum<G>(sum), dot = group_sum<G>(dot);
        const float rho = inv_root(__builtin_fmaf(sum, p.inv_sum, p.eps));
        const float mean = dot * rho * (inv_n / p.sq);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float u = ya[i] * rho, v = yb[i] * rho;
          sa[i] = __builtin_fmaf(a[i], u, sa[i]), sb[i] = __builtin_fmaf(b[i], v, sb[i]);
          a[i] = rho * (a[i] * wa[i] - u * mean), b[i] = rho * (b[i] * wb[i] - v * mean);
        }
      }
      if (x.out && at.any()) at.store(dst + j * x.out_sh, a, b);
    }
  }
  if (!x.sums) return;
#pragma unroll
  for (int i = 0; i < N; ++i) sums[group][lane][2 * i] = sa[i], sums[group][lane][2 * i + 1] = sb[i];
  __syncthreads();
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.dim;
  for (int q = threadIdx.x; q < G * 2 * N; q += 256) {
    const int l = q / (2 * N), i = q % (2 * N) / 2;
    const Lane<KIND> to(l, p);
    if (!to.any() || !to.own(i) || (q % 2 && !to.has_b(i))) continue;
    float s = 0.0f;
#pragma unroll 4
    for (int g = 0; g < GROUPS; ++g) s += sums[g][l][q % (2 * N)];
    out[q % 2 ? to.place_b(i) : to.place_a(i)] = s;
  }
}

// Sums of the partial rows: q's of the first blocks_q, k's of the others. 32 threads a column take every 32nd row
// each, and one adds their sums.
constexpr int kSumCols = 32, kSumSlices = 32;
__global__ __launch_bounds__(kSumCols * kSumSlices) void head_norm_sums_kernel(const float* partial, int blocks_q, int blocks,
                                                                               int dim, float* dw_q, float* dw_k, int accumulate) {
  __shared__ float sh[kSumSlices][kSumCols];
  const int lane = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols, c = blockIdx.x * kSumCols + lane;
  float* dw = blockIdx.y ? dw_k : dw_q;
  if (!dw) return;
  const int first = blockIdx.y ? blocks_q : 0, end = blockIdx.y ? blocks : blocks_q;
  float s = 0.0f;
  if (c < dim) {
#pragma unroll 8
    for (int g = first + slice; g < end; g += kSumSlices) s += partial[static_cast<int64_t>(g) * dim + c];
  }
  sh[slice][lane] = s;
  __syncthreads();
  if (slice || c >= dim) return;
#pragma unroll
  for (int i = 1; i < kSumSlices; ++i) s += sh[i][lane];
  dw[c] = accumulate ? dw[c] + s : s;
}

}  // namespace

// Groups of lanes of a head: the kernels' kinds and sizes.
struct HeadShape {
  Kind kind;
  int lanes;
};
static HeadShape head_shape(const HeadNormArgs& a) {
  const int rest = a.dim - 2 * a.pairs;
  auto by8 = [](int n) { return n == 0 || n >= 8; };
  int steps = 0;
  if (a.interleaved ? a.dim % 2 == 0 && a.dim >= 16 : rest % 2 == 0 && by8(a.pairs) && by8(rest / 2))
    steps = a.interleaved ? (a.dim / 2 + 7) / 8 : (a.pairs + 7) / 8 + (rest / 2 + 7) / 8;
  if (steps == 0 || steps > 32) return {kSingle, 64};
  return {a.interleaved ? kNext : kHalves, steps <= 4 ? 4 : steps <= 8 ? 8 : steps <= 16 ? 16 : 32};
}

// Calls f with the template arguments as integral constants: kind, lanes of a head, several axes.
template <typename F>
static hipError_t by_shape(const HeadNormArgs& a, F f) {
  const HeadShape s = head_shape(a);
  auto axes = [&](auto kind, auto lanes) {
    return a.axes > 1 ? f(kind, lanes, std::true_type{}) : f(kind, lanes, std::false_type{});
  };
  auto lanes = [&](auto kind) {
    switch (s.lanes) {
      case 4: return axes(kind, std::integral_constant<int, 4>{});
      case 8: return axes(kind, std::integral_constant<int, 8>{});
      case 16: return axes(kind, std::integral_constant<int, 16>{});
      default: return axes(kind, std::integral_constant<int, 32>{});
    }
  };
  if (s.kind == kSingle) return axes(std::integral_constant<Kind, kSingle>{}, std::integral_constant<int, 64>{});
  return s.kind == kNext ? lanes(std::integral_constant<Kind, kNext>{}) : lanes(std::integral_constant<Kind, kHalves>{});
}

hipError_t launch_head_norm_fwd(const HeadNormArgs& a, hipStream_t stream) {
  return by_shape(a, [&](auto kind, auto lanes, auto multi) {
    constexpr int G = decltype(lanes)::value;
    auto go = [&](auto hc) {
      constexpr int HC = decltype(hc)::value;
      auto blocks = [&](int heads) {
        const int64_t all = (a.tokens * ((heads + HC - 1) / HC) + 256 / G - 1) / (256 / G), most = int64_t{1} << 22;
        return all < most ? all : most;  // (a grid has under 2^32 threads)
      };
      const int64_t bq = blocks(a.t[0].heads), bk = blocks(a.t[1].heads);
      hipLaunchKernelGGL((head_norm_fwd_kernel<decltype(kind)::value, G, HC, decltype(multi)::value>),
                         dim3(static_cast<uint32_t>(bq + bk)), dim3(256), 0, stream, a, static_cast<unsigned>(bq));
      return hipGetLastError();
    };
    // Four heads of a token share its angles where there is work enough to fill the card that way: 8192 tokens 26.0 us (22.1)
    // and 26.6 (21.8) head by head, 4096 tokens 15.5 (11.8) and 16.3 (13.4), 2048 tokens 10.4 (8.0) and 10.7 (8.1); 1024
    // tokens, head by head, 6.8 (5.5) and 7.6 (6.0) by fours, 64 tokens 3.8 (3.6) and 5.3 (5.1).
    const int64_t heads = a.tokens * (a.t[0].heads + a.t[1].heads);
    return heads * G >= 5 * 256 * 256 ? go(std::integral_constant<int, 4>{}) : go(std::integral_constant<int, 1>{});
  });
}

// Workgroups of q and k: 768 in all (three on a CU), fewer where there is not as much work, shared out by the heads. More
// of them hide more of the loads and leave more rows of partial sums. With the sums, 8192 tokens by 256, 512, 768 and 1024
// workgroups: 49.6, 37.7, 35.0 and 39.8 us (43.0, 33.2, 31.0 and 33.3), 1536 tokens 19.0, 16.8, 14.2 and 17.1 (15.4, 13.7, 11.6
// and 14.3).
static void bwd_blocks(int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t& q, int64_t& k) {
  const int64_t heads = heads_q + heads_k, work = (tokens * heads + 31) / 32, all = work < 768 ? work : 768;
  q = heads_q ? (all * heads_q + heads - 1) / heads : 0;
  k = heads_k ? (all * heads_k + heads - 1) / heads : 0;
}

int64_t head_norm_bwd_blocks(int64_t tokens, int64_t heads_q, int64_t heads_k) {
  int64_t q, k, most;
  bwd_blocks(tokens, heads_q, heads_k, q, k);
  most = q + k;
  // one of the two alone, where the other's gradients are not wanted
  bwd_blocks(tokens, heads_q, 0, q, k);
  most = most < q ? q : most;
  bwd_blocks(tokens, 0, heads_k, q, k);
  return most < k ? k : most;
}

hipError_t launch_head_norm_bwd(HeadNormArgs a, float* const (&dw)[2], int accumulate, hipStream_t stream) {
  float* out[2];
  for (int k = 0; k < 2; ++k) {
    out[k] = a.t[k].heads ? dw[k] : nullptr;
    a.t[k].sums = out[k] != nullptr;
  }
  int64_t bq, bk;
  bwd_blocks(a.tokens, a.t[0].heads, a.t[1].heads, bq, bk);
  const hipError_t e = by_shape(a, [&](auto kind, auto lanes, auto multi) {
    auto go = [&](auto hc) {
      hipLaunchKernelGGL(
          (head_norm_bwd_kernel<decltype(kind)::value, decltype(lanes)::value, decltype(hc)::value, decltype(multi)::value>),
          dim3(static_cast<uint32_t>(bq + bk)), dim3(256), 0, stream, a, static_cast<unsigned>(bq));
      return hipGetLastError();
    };
    // Two heads of a token share its angles where there is work enough to fill the card that way. With the sums, 8192 tokens
    // 35.0 us (31.0) and 36.5 (31.1) head by head, 1536 tokens 14.2 (11.6) and 14.3 (12.3); 1024 tokens, head by
    // head, 11.4 (9.9) and 12.2 (10.1) by twos, 64 tokens 7.4 (7.1) and 8.1 (7.9).
    const int64_t heads = a.tokens * (a.t[0].heads + a.t[1].heads);
    return heads * decltype(lanes)::value >= 2 * 256 * 512 ? go(std::integral_constant<int, 2>{})
                                                           : go(std::integral_constant<int, 1>{});
  });
  if (e != hipSuccess || (!out[0] && !out[1])) return e;
  hipLaunchKernelGGL(head_norm_sums_kernel, dim3((a.dim + kSumCols - 1) / kSumCols, 2), dim3(kSumCols * kSumSlices), 0, stream,
                     a.partial, static_cast<int>(bq), static_cast<int>(bq + bk), a.dim, out[0], out[1], accumulate);
  return hipGetLastError();
}

}  // namespace pf8
