// What the block-scaled FP8 GEMM's kernels share: types, operand and output staging helpers, scheduling
// patterns (gfx950 / CDNA4 only).
#pragma once

#include "pf8_device.h"
#include "pf8_launch.h"

#include <atomic>
#include <type_traits>

namespace pf8 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kBufferFlags = 0x00020000;  // raw buffer resource word 3 for gfx9-family (dword data)

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const bf16x2 h = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, h);
}

__device__ __forceinline__ int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

__device__ __forceinline__ int e8m0_of(float s) { return static_cast<int>(__float_as_uint(s) >> 23) & 0xFF; }

__device__ __forceinline__ v8i lds_read32(const uint8_t* base, int off0, int off1) {
  const v4i lo = *reinterpret_cast<const v4i*>(base + off0);
  const v4i hi = *reinterpret_cast<const v4i*>(base + off1);
  return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// First (H = 0) or second (H = 1) 16 bytes of a 32-byte operand fragment, as 8 BF16 values.
template <int H>
__device__ __forceinline__ bf16x8 bf16_half(v8i v) {
  const v4i h = H == 0 ? v4i{v[0], v[1], v[2], v[3]} : v4i{v[4], v[5], v[6], v[7]};
  return __builtin_bit_cast(bf16x8, h);
}

// Scheduling pattern for NM MFMAs: the ND LDS reads and the NV vector-memory reads go out spread
// evenly between them (sched_group_barrier masks: 0x008 MFMA, 0x020 VMEM read, 0x100 DS read).
// Bunching the refill loads behind the last few MFMAs fills the texture unit's queues and stalls
// the wave's instruction stream, matrix instructions included.
// Vector-memory operations of `cnt` consecutive stages whose first is odd (`odd`) or even: D
// direct-to-LDS loads each, plus SS scale loads in each even stage.
constexpr int stage_ops(int cnt, bool odd, int d, int ss) {
  int n = 0;
  for (int i = 0; i < cnt; ++i) n += d + ((odd ? 1 : 0) ^ (i & 1) ? 0 : ss);
  return n;
}

template <int NM, int NV, int ND, int X = 0>
__device__ __forceinline__ void interleave_groups() {
  if constexpr (X < NM) {
    constexpr int d = (ND * (X + 1)) / NM - (ND * X) / NM;
    constexpr int v = (NV * (X + 1)) / NM - (NV * X) / NM;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x020, v, 0);
    interleave_groups<NM, NV, ND, X + 1>();
  }
}

// LDS byte address of a pointer into a __shared__ array.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)p));
}

// The persistent kernel's output staging buffer is written and read back through inline asm. The
// compiler's wait insertion makes an LDS access that aliases none of the direct-to-LDS loads it
// tracks wait for all of them, which here would be the next tile's first stages; the explicit
// lgkmcnt waits and barriers around these accesses order them instead. The read waits for its
// own results inside the asm statement before handing them over.
__device__ __forceinline__ void stg_write8(uint32_t addr, uint32_t w0, uint32_t w1) {
  asm volatile("ds_write_b64 %0, %1" : : "v"(addr), "v"(make_uint2(w0, w1)) : "memory");
}

__device__ __forceinline__ void stg_read8x16(const uint32_t (&addr)[8], v4i (&v)[8]) {
  asm volatile(
      "ds_read_b128 %0, %8\n"
      "ds_read_b128 %1, %9\n"
      "ds_read_b128 %2, %10\n"
      "ds_read_b128 %3, %11\n"
      "ds_read_b128 %4, %12\n"
      "ds_read_b128 %5, %13\n"
      "ds_read_b128 %6, %14\n"
      "ds_read_b128 %7, %15\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
      : "v"(addr[0]), "v"(addr[1]), "v"(addr[2]), "v"(addr[3]), "v"(addr[4]), "v"(addr[5]), "v"(addr[6]), "v"(addr[7])
      : "memory");
}

// CUs of the current device (cached per device).
inline int device_cus() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
  if (dev < 64) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
  if (dev < 64) cache[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

}  // namespace pf8
