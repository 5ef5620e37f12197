// Device-side helpers of the kernels that work on rows of BF16 values in FP32 (gfx950 / CDNA4 only).
#pragma once

#include "pf8_device.h"

#include <type_traits>

namespace pf8 {

// 16 bytes at 2-byte alignment: global accesses of any alignment are one instruction on gfx950, so
// odd row pitches take the same path as aligned ones.
typedef uint32_t u128_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u64_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_a2 __attribute__((aligned(2)));
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

__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  const u128_a2 v = *reinterpret_cast<const u128_a2*>(p);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// The first n < 8, zeros behind.
__device__ __forceinline__ uint4 load_few(const uint16_t* p, int n) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The last n < 8 of 8 values whose first belongs at p, in pieces of 1, 2 and 4.
__device__ __forceinline__ void store_last(uint16_t* p, uint4 v, int n) {
  if (n & 1) p[8 - n] = static_cast<uint16_t>((n & 4 ? (n & 2 ? v.x : v.y) : (n & 2 ? v.z : v.w)) >> 16);
  if (n & 2) *reinterpret_cast<u32_a2*>(p + (n & 4 ? 2 : 6)) = n & 4 ? v.y : v.w;
  if (n & 4) *reinterpret_cast<u64_a2*>(p + 4) = u64_a2{v.z, v.w};
}

// Sum over a wave, the same in every lane: four DPP steps within rows of 16 lanes, then the four rows'
// sums by lane reads. (Shuffles through LDS cost some hundred cycles for the six steps, and a row has up to
// three sums that wait for one another.)
__device__ __forceinline__ float wave_sum(float v) {
  auto step = [&](auto ctrl) {
    v += __uint_as_float(static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), decltype(ctrl)::value, 0xF, 0xF, true)));
  };
  // quad_perm [1,0,3,2], quad_perm [2,3,0,1], row_half_mirror, row_mirror
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  step(std::integral_constant<int, 0x141>{});
  step(std::integral_constant<int, 0x140>{});
  const int x = static_cast<int>(__float_as_uint(v));
  auto lane = [&](int l) { return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(x, l))); };
  return (lane(0) + lane(16)) + (lane(32) + lane(48));
}

// 1 / sqrt(a). The instruction's result is off by up to a step; one Newton step v + v (1 - a v v) / 2, with a v in
// two parts, leaves half a step (a square root and a division leave up to one between them, and take longer).
__device__ __forceinline__ float inv_root(float a) {
  if (!(a >= 0x1p-100f && a <= 0x1p100f)) return 1.0f / __builtin_sqrtf(a);  // zeros, subnormals, infinities, NaN too
  const float v = __builtin_amdgcn_rsqf(a);
  const float high = a * v, low = __builtin_fmaf(a, v, -high);
  const float e = __builtin_fmaf(-low, v, __builtin_fmaf(-high, v, 1.0f));
  return __builtin_fmaf(v, 0.5f * e, v);
}

}  // namespace pf8
