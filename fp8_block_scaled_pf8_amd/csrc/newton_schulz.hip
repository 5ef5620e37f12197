// Newton-Schulz orthogonalisation for gfx950: X <- a X + (b A + c A A) X with A = X X^T, from
// X = G / (|G|_F + eps). Contract in include/pf8_train.h.
//
// Bound: the matrix cores. With X [p, q] (p <= q; a tall G is taken transposed) a step is
// p^2 q / 2 multiply-adds for A and p^3 / 2 for A A, both symmetric and formed for their lower tiles
// only, and p^2 q for the update.
//
// Number formats. The products run on FP16 operands with FP32 accumulation; what adds up over the
// steps has more bits:
//  * X itself is kept as the sum of two FP16 values, the operand and its remainder (4 bytes an element and
//    step less to move than FP32 beside the operand: 12288 x 2048 in 1221 us, 1268). That is 22 bits of
//    entries down to 2^-14 (X starts with norm 1); the remainder's steps end at 2^-36, which leaves 18 bits of
//    an entry of 2^-18. All entries of a Gaussian 12288 x 2048 together are off by 4e-8, in FP32 2.5e-8. The
//    update adds a X from both; only the small product B X is formed from X's FP16 rounding. (Rounding X
//    itself would put noise into directions whose singular value is nearly zero, which the iteration
//    multiplies by a in every step: a rank-one G came out 15 % off.)
//  * A and B = b A + c A A are split into their diagonals, kept in FP32, and the rest in FP16:
//    near the end A is close to a multiple of the identity and the diagonal carries nearly all.
//    (A A)_ij = sum A'_ik A'_kj + (d_i + d_j) A'_ij off the diagonal.
//  * FP16 values are scaled by powers of two (X 2^12, A 2^10, B by its step's coefficients: poly_scale), so
//    that entries down to 2^-26 of the norm keep all an operand's bits and singular values up to 8 stay in
//    range.
//  * In every step but the last, the whole of B multiplies one and the same FP16 rounding of X, its
//    diagonal too: B times anything lies in X's column space, so the rounding's part outside of it is
//    gone. With X whole under the diagonal, of some rows or of all, that part would stay, and grow by a
//    in every step behind (a rank-one G came out 4 % off where one row carries most of it). The last
//    step's diagonal takes X whole: nothing grows any more, and of a matrix of full rank, whose diagonals
//    end near 1 - a, the rounding would enter 2.4-fold.
//  * A matrix of at most 64 x 512 or 128 x 256 stays in one workgroup (X in FP32), and its X enters the
//    update as a sum of two FP16 values, diagonal or not: few entries average out little of the
//    rounding noise.
// Against float64, besides the BF16 rounding of the result (1.7e-3 of its 2-norm), five steps are off by
// 1.1e-3 of its 2-norm for Gaussian gradients, up to 2e-3 for others of many rows and up to 1.5e-2 for those of
// a few elements or magnitudes, which round alike; BF16 operands would give eight times that.
//
// Layout. X lives in the workspace, padded to multiples of 128 with zeros that stay zero, so the
// products have no edges: Xc [q][p] (two buffers in turn; the update's operand, and A's by transposing
// reads of LDS: a copy [p][q] for A cost 12288 x 2048 another 49 us of 1144) and the remainders in
// 64x64 regions in the order the update's lanes hold them, so that each lane reads and writes 16
// consecutive bytes. FP16 rows are 128 bytes longer than that: a tile's loads read
// the same columns of many rows, and with a pitch of 4 KiB or a multiple they crowd a few channels.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "pf8_train_launch.h"

namespace pf8 {

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

// The steps' coefficients, by value: the host's array is not read after the call.
struct NsCoef {
  float v[64][5];  // a, b, c, poly_scale(b, c) and its reciprocal
};

constexpr float kSX = 4096.0f, kSA = 1024.0f;  // powers of two that FP16 operands carry
constexpr int kRegion = 64 * 64;
constexpr int64_t kPad = 64;  // values that FP16 rows are longer than padded: see "Layout"

// In a 64x64 region of a product, block (bi, bj) of 32x32 and register 4 g + e of lane l hold the
// element (32 bi + l % 32, 32 bj + 8 g + 4 (l / 32) + e). FP32 sums lie there four registers a lane, the
// remainders of X (FP16) eight, those of two g.
__device__ __forceinline__ int region_offset(int bi, int bj, int g, int lane) {
  return ((bi * 2 + bj) * 4 + g) * 256 + lane * 4;
}
__device__ __forceinline__ int rest_offset(int bi, int bj, int pair, int lane) {
  return ((bi * 2 + bj) * 2 + pair) * 512 + lane * 8;
}

// Up to four stage buffers.
struct Buffers {
  uint8_t *b0, *b1, *b2, *b3;
  template <int I>
  __device__ __forceinline__ uint8_t* at() const {
    if constexpr (I == 0) return b0;
    else if constexpr (I == 1) return b1;
    else if constexpr (I == 2) return b2;
    else return b3;
  }
};

// D[m, n] = sum_k P[m, k] Q[n, k] over an even number of stages of 64 values each: a BM x BN tile by
// (BM/WM)(BN/WN) waves. The operands lie in memory with m and n as rows, or with k as rows (KROWS). Stages
// go straight to LDS (16 bytes a lane) into NST buffers, NST - 1 to NST ahead of use, in rows of 128 bytes or
// more (of 64 bytes, such loads come at half the rate). Their 16-byte chunks change places:
//  * rows of m or n: chunk c of row r sits at c ^ ((r >> 1) & 7), and 16 consecutive rows' reads of one
//    chunk fall into the 16 different 16-byte slots of the 64 banks;
//  * rows of k: transposing reads of 4 rows x 64 bytes by 32 lanes; c ^ 4 (r & 3), with 128-byte rows
//    c ^ 4 (r / 2 & 1), spreads them over all banks.
// One barrier a stage, in its middle, while the matrix cores still have the stage's second half
// to do: behind it every wave's loads of the next stage have landed, and the stage's own buffer, whose
// operands are all in registers, is free to be filled again. The buffers are LDS objects of their own, so that
// the compiler sees that a read of one does not wait for loads into another.
template <int BM, int BN, int WM, int WN, int NST, bool KROWS>
struct Tile {
  static constexpr int kWavesN = BN / WN, kWaves = (BM / WM) * kWavesN, kThreads = 64 * kWaves;
  static constexpr int TM = WM / 32, TN = WN / 32;
  static constexpr int BK = 64, kRow = BK * 2, kStage = (BM + BN) * kRow;
  static constexpr int kLoadsP = BM * kRow / 1024 / kWaves, kLoads = kStage / 1024 / kWaves;  // of 64 lanes x 16 bytes
  static_assert(BM * kRow / 1024 % kWaves == 0 && BN * kRow / 1024 % kWaves == 0, "even loads");
  static_assert(NST >= 2 && NST <= 4, "up to four buffers");
  typedef f16v Acc[TM][TN];

  // what the chunks of an LDS row change places by; ROW: its bytes
  template <int ROW>
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (!KROWS) return (row >> 1) & 7;
    else return ROW == 128 ? (row >> 1 & 1) << 2 : (row & 3) << 2;
  }

  // f(0), f(1), ... with compile-time arguments
  template <typename F, int... V>
  static __device__ __forceinline__ void each(F f, std::integer_sequence<int, V...>) {
    (f(std::integral_constant<int, V>{}), ...);
  }

  static __device__ __forceinline__ void zero(Acc& acc) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  }

  static __device__ __forceinline__ void run(const _Float16* P, int64_t ldp, const _Float16* Q, int64_t ldq, int64_t k0,
                                             int steps, const Buffers& bufs, Acc& acc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    // a wave's loads `from` to `to` of one operand's part of a stage, W values wide (of rows or of columns)
    auto issue_part = [&](auto w_c, const _Float16* X, int64_t ld, uint8_t* buf, int s, auto from, auto to) {
      constexpr int W = decltype(w_c)::value;
      constexpr int kLine = KROWS ? W * 2 : kRow, kLines = KROWS ? BK : W, kChunks = kLine / 16, kSlab = 1024 / kLine;
      const int64_t k = k0 + static_cast<int64_t>(s) * BK;
      const int pitch = static_cast<int>(ld) * 2;
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16*>(X + (KROWS ? k * ld : k)), 0,
                                                                        (kLines - 1) * pitch + kLine, 0x00020000);
      const int line = lane / kChunks;
#pragma unroll
      for (int i = decltype(from)::value; i < decltype(to)::value; ++i) {
        const int slab = wave + i * kWaves;
        const int chunk = (lane % kChunks) ^ swizzle<kLine>(slab * kSlab + line);
        auto* dst = (__attribute__((address_space(3))) void*)(buf + slab * 1024);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, line * pitch + chunk * 16, slab * kSlab * pitch, 0, 0);
      }
    };
    // part 0: P's loads of a stage, 1: Q's
    auto issue = [&](auto part, uint8_t* buf, int s) {
      using Zero = std::integral_constant<int, 0>;
      if constexpr (decltype(part)::value == 0)
        issue_part(std::integral_constant<int, BM>{}, P, ldp, buf, s, Zero{}, std::integral_constant<int, kLoadsP>{});
      else
        issue_part(std::integral_constant<int, BN>{}, Q, ldq, buf + BM * kRow, s, Zero{}, std::integral_constant<int, kLoads - kLoadsP>{});
    };
    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, 1>;
    const int l32 = lane & 31, half = lane >> 5;
    // 8 values along K of each lane's row of P (Q 0) or Q (1). (All that is added to the buffer is added up first:
    // the compiler loses sight of whose LDS a read is in after a few steps of pointer arithmetic.)
    auto frag = [&](auto q_c, const uint8_t* buf, int first, int k) {
      constexpr int W = decltype(q_c)::value ? BN : BM, from = decltype(q_c)::value ? BM * kRow : 0;
      if constexpr (!KROWS) {
        const int row = first + l32;
        return *reinterpret_cast<const h8*>(buf + (from + row * kRow + (((2 * k + half) ^ swizzle<kRow>(row)) << 4)));
      } else {
        // 16 lanes read 4 rows of 16 values and hold their columns
        constexpr int kLine = W * 2;
        const int col = first + (lane & 16) + (lane & 3) * 4;
        h4 v[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = 16 * k + 8 * half + 4 * t + (lane >> 2 & 3);
          const uint8_t* p = buf + (from + row * kLine + (((col >> 3) ^ swizzle<kLine>(row)) << 4) + (col & 4) * 2);
          v[t] = __builtin_bit_cast(h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)(p)));
        }
        return __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
      }
    };
    // operands of the first (0) or second (1) half of a stage's k-steps
    constexpr int kHalf = BK / 32;
    h8 fp[2][kHalf][TM], fq[2][kHalf][TN];
    auto read = [&](auto h_c, const uint8_t* buf) {
      constexpr int h = decltype(h_c)::value;
#pragma unroll
      for (int k = 0; k < kHalf; ++k) {
#pragma unroll
        for (int i = 0; i < TM; ++i) fp[h][k][i] = frag(H0{}, buf, wm * WM + 32 * i, h * kHalf + k);
#pragma unroll
        for (int j = 0; j < TN; ++j) fq[h][k][j] = frag(H1{}, buf, wn * WN + 32 * j, h * kHalf + k);
      }
    };
    auto multiply = [&](auto h_c) {
      constexpr int h = decltype(h_c)::value;
#pragma unroll
      for (int k = 0; k < kHalf; ++k)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fq[h][k][j], fp[h][k][i], acc[i][j], 0, 0, 0);
    };
    // Every wave's loads of a stage have landed and its operand reads are done; `behind` loads after them
    // may still be in flight (loads complete in order).
    auto sync_stage = [&](auto behind) {
      constexpr int fly = decltype(behind)::value;
      static_assert(fly < 64, "the counter's range");
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt((fly & 0xF) | ((fly >> 4) << 14) | (0x7 << 4));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    // The order of a half stage: LDS reads and loads evenly behind the products. (Loads in a row fill the
    // queues of the memory path, and a wave that waits for room there issues no products either.)
    auto spread = [&](auto loads) {
      constexpr int products = kHalf * TM * TN, reads = (KROWS ? 2 : 1) * kHalf * (TM + TN), vm = decltype(loads)::value;
      each(
          [&](auto x_c) {
            constexpr int x = decltype(x_c)::value;
            constexpr int r = reads * (x + 1) / products - reads * x / products, v = vm * (x + 1) / products - vm * x / products;
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
            if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x020, v, 0);
          },
          std::make_integer_sequence<int, products>{});
    };
    using Loads0 = std::integral_constant<int, kLoadsP>;
    using Loads1 = std::integral_constant<int, kLoads - kLoadsP>;
    using None = std::integral_constant<int, 0>;
    // One stage, in buffer U. First half: the second half's operands are read, and the refill of the buffer
    // before (stage s - 1 + NST) gets its second part. The waves meet; then the buffer itself gets the first
    // part of its refill, and the next stage's first operands are read.
    auto stage = [&](auto u_c, int s, auto before, auto refill, auto behind, auto last) {
      constexpr int u = decltype(u_c)::value;
      if constexpr (decltype(before)::value) issue(H1{}, bufs.template at<(u + NST - 1) % NST>(), s - 1 + NST);
      read(H1{}, bufs.template at<u>());
      multiply(H0{});
      if constexpr (decltype(before)::value) spread(Loads1{});
      else spread(None{});
      if constexpr (!decltype(last)::value) {
        sync_stage(behind);
        if constexpr (decltype(refill)::value) issue(H0{}, bufs.template at<u>(), s + NST);
        read(H0{}, bufs.template at<(u + 1) % NST>());
        multiply(H1{});
        if constexpr (decltype(refill)::value) spread(Loads0{});
        else spread(None{});
        __builtin_amdgcn_sched_barrier(0);
      } else {
        multiply(H1{});
      }
    };
    // All waits are exact and known at compile time, which also keeps the compiler from waiting for loads
    // by itself: the last REM stages are a code path of their own.
    auto tail = [&](auto rem_c, int s) {
      constexpr int rem = decltype(rem_c)::value;
      each(
          [&](auto v_c) {
            constexpr int v = decltype(v_c)::value, left = rem - 2 - v;
            stage(std::integral_constant<int, v % NST>{}, s + v, std::bool_constant<(v - 1 + NST < rem)>{},
                  std::bool_constant<(v + NST < rem)>{},
                  std::integral_constant<int, (left < 0 ? 0 : (left < NST - 2 ? left : NST - 2)) * kLoads>{},
                  std::bool_constant<(v + 1 == rem)>{});
          },
          std::make_integer_sequence<int, rem>{});
    };
    // The first N stages go out, and one more's first part (MORE); the first of them is read.
    auto start = [&](auto n_c, auto more) {
      constexpr int n = decltype(n_c)::value;
      each(
          [&](auto u) {
            issue(H0{}, bufs.template at<decltype(u)::value>(), u);
            issue(H1{}, bufs.template at<decltype(u)::value>(), u);
          },
          std::make_integer_sequence<int, n>{});
      if constexpr (decltype(more)::value) issue(H0{}, bufs.template at<n>(), n);
      sync_stage(std::integral_constant<int, (n - 1) * kLoads + (decltype(more)::value ? kLoadsP : 0)>{});
      read(H0{}, bufs.b0);
    };
    // `steps` is even; where NST is too, so is what the main loop leaves
    constexpr int kUnit = NST % 2 == 0 ? 2 : 1;
    if (steps < NST) {
      each(
          [&](auto v_c) {
            constexpr int all = decltype(v_c)::value * kUnit;
            if constexpr (all > 0 && all < NST)
              if (steps == all) {
                start(std::integral_constant<int, all>{}, std::false_type{});
                tail(std::integral_constant<int, all>{}, 0);
              }
          },
          std::make_integer_sequence<int, NST>{});
    } else {
      start(std::integral_constant<int, NST - 1>{}, std::true_type{});
      int s = 0;
      for (; s + 2 * NST <= steps; s += NST)
        each(
            [&](auto u) {
              stage(u, s + decltype(u)::value, std::true_type{}, std::true_type{}, std::integral_constant<int, (NST - 2) * kLoads>{},
                    std::false_type{});
            },
            std::make_integer_sequence<int, NST>{});
      // NST .. 2 NST - 1 stages are left
      each(
          [&](auto v_c) {
            constexpr int rem = decltype(v_c)::value * kUnit;
            if constexpr (rem >= NST && rem < 2 * NST)
              if (steps - s == rem) tail(std::integral_constant<int, rem>{}, s);
          },
          std::make_integer_sequence<int, 2 * NST>{});
    }
    // the buffers may be written by the epilogue once every wave has read its last operands
    sync_stage(std::integral_constant<int, 0>{});
  }
};

// Workgroup ids are dealt over the 8 XCDs, each with an L2 of its own, in turn: this order gives an XCD
// consecutive ones.
__device__ __forceinline__ uint32_t xcd_order(uint32_t id, uint32_t all) {
  const uint32_t xcd = id & 7, q = all >> 3, rem = all & 7;
  return xcd * q + min(xcd, rem) + (id >> 3);
}

// The stage buffers of a kernel, as LDS objects of their own.
#define PF8_NS_BUFFERS(bufs, G, NST)                                                                            \
  __shared__ __align__(16) uint8_t bufs##0 [G::kStage], bufs##1 [G::kStage], bufs##2 [NST > 2 ? G::kStage : 16], \
      bufs##3 [NST > 3 ? G::kStage : 16];                                                                        \
  const Buffers bufs = {bufs##0, bufs##1, bufs##2, bufs##3}

// Tile t of those that cover the lower triangle of a square matrix: BM x BN tiles, numbered by rows (with
// BN = 2 BM by pairs of rows); (ti, tj) in tiles.
template <int BM, int BN>
__device__ __forceinline__ void triangle_tile(int t, int& ti, int& tj) {
  constexpr int kTwo = BM == BN ? 1 : 2;  // pairs of tiles make a square
  static_assert(BM == BN || BN == 2 * BM, "square or twice as wide");
  const int u = t / kTwo;
  int i = static_cast<int>((__builtin_sqrtf(8.0f * static_cast<float>(u) + 1.0f) - 1.0f) * 0.5f);
  while (i * (i + 1) / 2 > u) --i;
  while ((i + 1) * (i + 2) / 2 <= u) ++i;
  const int j = u - i * (i + 1) / 2, odd = t % kTwo;
  ti = BN > BM ? 2 * i + odd : i;
  tj = j;
}

// A finished tile passes through LDS to leave in whole rows, as it is and transposed. Lanes hold four
// consecutive columns of a row; `quad_transpose` exchanges them between four lanes (rows), so that lane
// t of a quad then holds column t of the four. Both go to LDS 8 bytes at a time, 32 lanes to 32 different
// bank pairs:
//  * rows of C columns: 16-byte chunk c of row m sits at c ^ swizzle(m), its 8-byte halves swapped
//    where bit 4 of m is set;
//  * columns (rows of the transposed tile, R long): chunk c of row n sits at c ^ 4 (n & 3), or with
//    128-byte rows (two to a sweep of the banks) at c ^ 4 (n / 2 & 1).
template <int C>
__device__ __forceinline__ int row_swizzle(int m) { return C == 64 ? (m >> 1) & 7 : m & 15; }
template <int R>
__device__ __forceinline__ int col_swizzle(int n) { return R == 64 ? ((n >> 1) & 1) << 2 : (n & 3) << 2; }

template <int C>
__device__ __forceinline__ void put_row(uint8_t* row, int m, int n, h4 v) {
  *reinterpret_cast<h4*>(row + (((n >> 3) ^ row_swizzle<C>(m)) << 4) + ((((n >> 2) ^ (m >> 4)) & 1) << 3)) = v;
}
template <int C>
__device__ __forceinline__ h8 get_row(const uint8_t* row, int m, int chunk) {
  const h8 v = *reinterpret_cast<const h8*>(row + ((chunk ^ row_swizzle<C>(m)) << 4));
  return m & 16 ? __builtin_shufflevector(v, v, 4, 5, 6, 7, 0, 1, 2, 3) : v;
}
__device__ __forceinline__ h4 quad_transpose(h4 v) {
  const uint2 w = __builtin_bit_cast(uint2, v);
  const bool odd = threadIdx.x & 1, upper = threadIdx.x & 2;
  const uint32_t sel = odd ? 0x03020706u : 0x05040100u;
  const int x0 = __builtin_amdgcn_update_dpp(0, static_cast<int>(w.x), 0xB1, 0xF, 0xF, true);
  const int x1 = __builtin_amdgcn_update_dpp(0, static_cast<int>(w.y), 0xB1, 0xF, 0xF, true);
  const uint32_t p0 = __builtin_amdgcn_perm(static_cast<uint32_t>(x0), w.x, sel);
  const uint32_t p1 = __builtin_amdgcn_perm(static_cast<uint32_t>(x1), w.y, sel);
  const uint32_t r = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(upper ? p0 : p1), 0x4E, 0xF, 0xF, true));
  const uint2 o = upper ? make_uint2(r, p1) : make_uint2(p0, r);
  return __builtin_bit_cast(h4, o);
}
// m: the lane's row, n: the column it holds after quad_transpose
template <int R>
__device__ __forceinline__ void put_col(uint8_t* row, int m, int n, h4 v) {
  const int col = m & ~3;
  *reinterpret_cast<h4*>(row + (((col >> 3) ^ col_swizzle<R>(n)) << 4) + ((col >> 2 & 1) << 3)) = quad_transpose(v);
}
template <int R>
__device__ __forceinline__ h8 get_col(const uint8_t* row, int n, int chunk) {
  return *reinterpret_cast<const h8*>(row + ((chunk ^ col_swizzle<R>(n)) << 4));
}

// Row m of a staged tile of R rows with C values: as many rows as fit (a power of two) in each stage buffer.
template <int STAGE, int R, int C, int FIRST>
__device__ __forceinline__ uint8_t* staged(const Buffers& bufs, int m) {
  constexpr int fit = STAGE / (C * 2), per = fit >= R ? R : fit >= 128 ? 128 : fit >= 64 ? 64 : 32, used = R / per;
  static_assert(fit >= 32 && used <= 4, "whole blocks of rows in up to four buffers");
  uint8_t* b = bufs.template at<FIRST>();
  if constexpr (used > 1) b = m / per == 1 ? bufs.template at<FIRST + 1>() : b;
  if constexpr (used > 2) b = m / per == 2 ? bufs.template at<FIRST + 2>() : b;
  if constexpr (used > 2) b = m / per == 3 ? bufs.template at<FIRST + 3>() : b;
  return b + m % per * C * 2;
}

// Writes a staged BM x BN tile (rows from the first buffer on, transposed from buffer COLS on) to rows r0..
// and columns c0.. of a symmetric matrix, and its mirror image: of each 64x64 region on or below the
// diagonal, below it also the image.
template <int STAGE, int BM, int BN, int THREADS, int COLS>
__device__ __forceinline__ void write_symmetric(const Buffers& bufs, _Float16* out, int64_t ld, int64_t r0, int64_t c0) {
#pragma unroll 4
  for (int u = 0; u < BM * BN / 8 / THREADS; ++u) {
    const int c = threadIdx.x + u * THREADS;
    const int row = c / (BN / 8), chunk = c % (BN / 8), n = c / (BM / 8), chunk_m = c % (BM / 8);
    if ((c0 + chunk * 8) / 64 <= (r0 + row) / 64)
      *reinterpret_cast<h8*>(out + (r0 + row) * ld + c0 + chunk * 8) = get_row<BN>(staged<STAGE, BM, BN, 0>(bufs, row), row, chunk);
    if ((c0 + n) / 64 < (r0 + chunk_m * 8) / 64)
      *reinterpret_cast<h8*>(out + (c0 + n) * ld + r0 + chunk_m * 8) = get_col<BM>(staged<STAGE, BN, BM, COLS>(bufs, n), n, chunk_m);
  }
}

// ------------------------------------------------------------------------------ G to X
// Sums of squares of a G, in FP64 (any FP32 value's square is in range): one partial per workgroup.
constexpr int kNormBlocks = 512, kNormThreads = 512;

template <typename T>
__device__ __forceinline__ float value(T v);
template <>
__device__ __forceinline__ float value<float>(float v) { return v; }
template <>
__device__ __forceinline__ float value<uint16_t>(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__device__ __forceinline__ double block_sum(double s, double* sh) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) s += sh[w];
  return s;
}

// 8 values from p, of any alignment.
typedef uint32_t u4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f4_a4 __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ void load_values(const float* p, float (&v)[8]) {
  const f4_a4 x = *reinterpret_cast<const f4_a4*>(p), y = *reinterpret_cast<const f4_a4*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = x[e], v[e + 4] = y[e];
}
__device__ __forceinline__ void load_values(const uint16_t* p, float (&v)[8]) {
  const u4_a2 x = *reinterpret_cast<const u4_a2*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[2 * e] = __uint_as_float(x[e] << 16), v[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
}

template <typename T>
__global__ __launch_bounds__(kNormThreads) void ns_norm_kernel(NsArgs a) {
  __shared__ double sh[kNormThreads / 64];
  const T* g = static_cast<const T*>(a.g) + blockIdx.y * a.stride_g;
  // groups of 8 columns, numbered along the rows, dealt to all threads in turn
  const int64_t per_row = (a.n + 7) / 8, groups = a.m * per_row, all = static_cast<int64_t>(gridDim.x) * kNormThreads;
  double s0 = 0.0, s1 = 0.0;
#pragma unroll 4
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x; u < groups; u += all) {
    const int64_t row = u / per_row, c = (u - row * per_row) * 8;
    const T* src = g + row * a.ldg + c;
    float v[8];
    if (c + 8 <= a.n) {
      load_values(src, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = c + e < a.n ? value<T>(src[e]) : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      s0 = __builtin_fma(static_cast<double>(v[e]), static_cast<double>(v[e]), s0);
      s1 = __builtin_fma(static_cast<double>(v[e + 1]), static_cast<double>(v[e + 1]), s1);
    }
  }
  const double s = block_sum(s0 + s1, sh);
  if (threadIdx.x == 0) a.norm_part[static_cast<int64_t>(blockIdx.y) * kNormBlocks + blockIdx.x] = s;
}

// 1 / (|G| + eps) from the partial sums; NaN if G holds a NaN or an infinity.
__device__ __forceinline__ double inv_norm(const NsArgs& a, int batch, double* sh) {
  double s = 0.0;
  for (int i = threadIdx.x; i < kNormBlocks; i += blockDim.x) s += a.norm_part[static_cast<int64_t>(batch) * kNormBlocks + i];
  s = block_sum(s, sh);
  if (!(s <= 1e300)) return __builtin_nan("");
  return 1.0 / (__builtin_sqrt(s) + static_cast<double>(a.eps));
}

// What FP16 leaves of a value.
__device__ __forceinline__ _Float16 remainder16(float x) {
  return static_cast<_Float16>(x - static_cast<float>(static_cast<_Float16>(x)));
}

// One 64x64 block of X: Xc and the remainders from G, zeros outside.
template <typename T>
__global__ __launch_bounds__(256) void ns_init_kernel(NsArgs a) {
  __shared__ double red[4];
  __shared__ float sh[64][65];  // [i][j]
  const int b = blockIdx.y;
  const int tiles_q = static_cast<int>(a.qp / 64);
  const int64_t i0 = (blockIdx.x / tiles_q) * 64, j0 = (blockIdx.x % tiles_q) * 64;
  const T* g = static_cast<const T*>(a.g) + b * a.stride_g;
  const bool tall = a.m > a.n;
  // read along G's rows: G[row][col] is X[row][col], or X[col][row] of a tall G. (Always a load, of the matrix's
  // last row or column if need be, and all of them before the norm is there.)
  const int64_t r0 = tall ? j0 : i0, c0 = tall ? i0 : j0;
  const int c = threadIdx.x & 63, r = threadIdx.x >> 6;
  const bool col_in = c0 + c < a.n;
  const T* src = g + (col_in ? c0 + c : a.n - 1);
  float v[16];
#pragma unroll
  for (int u = 0; u < 16; ++u) v[u] = value<T>(src[min(r0 + r + 4 * u, a.m - 1) * a.ldg]);
  const double s = inv_norm(a, b, red) * static_cast<double>(kSX);
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int row = r + 4 * u;
    const float x = col_in && r0 + row < a.m ? static_cast<float>(static_cast<double>(v[u]) * s) : 0.0f;
    if (tall) sh[c][row] = x;
    else sh[row][c] = x;
  }
  __syncthreads();
  _Float16* xc = a.xc[0] + b * a.qp * a.ldp;
  for (int t = threadIdx.x; t < kRegion / 8; t += 256) {
    const int r = t >> 3, c = (t & 7) * 8;
    h8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<_Float16>(sh[c + e][r]);
    *reinterpret_cast<h8*>(xc + (j0 + r) * a.ldp + i0 + c) = v;
  }
  _Float16* rest = a.rest + b * a.x_elems + ((j0 / 64) * (a.pp / 64) + i0 / 64) * kRegion;
  for (int t = threadIdx.x; t < kRegion / 8; t += 256) {
    const int lane = t & 63, pair = (t >> 6) & 1, bj = (t >> 7) & 1, bi = t >> 8;
    const int m = 32 * bi + (lane & 31), n = 32 * bj + 16 * pair + 4 * (lane >> 5);
    h8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = remainder16(sh[n + (e & 3) + 2 * (e & 4)][m]);
    *reinterpret_cast<h8*>(rest + rest_offset(bi, bj, pair, lane)) = v;
  }
}

// ------------------------------------------------------------------------------ A = X X^T, B = b A + c A A
// Four elements (m, n..n+3) of a symmetric product's sums -> what is stored of them.
// A: the FP32 diagonal aside, FP16 elsewhere.
__device__ __forceinline__ h4 gram_elements(const NsArgs& a, int b, int64_t m, int64_t n, f4 s) {
  h4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = static_cast<_Float16>(s[e] * (kSA / (kSX * kSX)));
  if (m >= n && m < n + 4) {  // the diagonal
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m == n + e) {
        a.da[b * a.pp + m] = s[e] * (1.0f / (kSX * kSX));
        v[e] = static_cast<_Float16>(0.0f);
      }
  }
  return v;
}
// B, from the sums of A' A' and A'.
__device__ __forceinline__ const h4* poly_a16(const NsArgs& a, int b, int64_t m, int64_t n) {
  return reinterpret_cast<const h4*>(a.a16 + (static_cast<int64_t>(b) * a.pp + m) * a.ldp + n);
}
__device__ __forceinline__ h4 poly_elements(const NsArgs& a, int b, int64_t m, int64_t n, f4 s, h4 av, float cb, float cc, float sb) {
  const float* d = a.da + b * a.pp;
  const float dm = d[m];
  const f4 dn = *reinterpret_cast<const f4*>(d + n);
  const float from = (cb + cc * dm) * (sb / kSA), by = cc * (sb / kSA), squares = cc * (sb / (kSA * kSA));
  h4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = static_cast<_Float16>(__builtin_fmaf(static_cast<float>(av[e]), __builtin_fmaf(by, dn[e], from), squares * s[e]));
  if (m >= n && m < n + 4) {  // the diagonal
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m == n + e) {
        a.db[b * a.pp + m] = cb * dm + cc * (s[e] * (1.0f / (kSA * kSA)) + dm * dm);
        v[e] = static_cast<_Float16>(0.0f);
      }
  }
  return v;
}

// The lower tiles of a symmetric product, K = q of X (POLY = false) or p of A' (true). SPLIT: K is cut into
// gridDim.z parts; each part of a tile leaves as FP32 sums in 64x64 regions, for ns_finish_kernel.
// Otherwise a workgroup makes a whole tile and finishes it. Bound as the update is; 12288 values along K for
// the triangle of 2048 x 2048: 57.5 us (1.0 PFLOP/s on the 128x256 tiles) and 7.6 us for joining three parts.
template <int BM, int BN, int WM, int WN, int NST, bool POLY, bool SPLIT>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void ns_sym_kernel(NsArgs a, int turn, float cb, float cc, float sb) {
  using G = Tile<BM, BN, WM, WN, NST, !POLY>;
  constexpr int TM = G::TM, TN = G::TN;
  PF8_NS_BUFFERS(bufs, G, NST);
  // an XCD's workgroups share the rows of few tiles: 8192 x 8192 in 10.6 ms, dealt in turn 11.5
  const uint32_t grid_xy = gridDim.x * gridDim.y;
  const uint32_t id = xcd_order(blockIdx.x + gridDim.x * blockIdx.y + grid_xy * blockIdx.z, grid_xy * gridDim.z);
  const int z = static_cast<int>(id / grid_xy), b = static_cast<int>(id % grid_xy / gridDim.x), tile = static_cast<int>(id % gridDim.x);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / (BN / WN), wn = wave % (BN / WN);
  const int64_t ld = a.ldp;
  const _Float16* x = POLY ? a.a16 + b * a.pp * ld : a.xc[turn] + b * a.qp * ld;
  int ti, tj;
  triangle_tile<BM, BN>(tile, ti, tj);
  const int64_t r0 = static_cast<int64_t>(ti) * BM, c0 = static_cast<int64_t>(tj) * BN;
  const int units = static_cast<int>((POLY ? a.pp : a.qp) / 128);  // of 128 values, two stages
  const int k0 = SPLIT ? static_cast<int>(static_cast<int64_t>(units) * z / gridDim.z) : 0;
  const int k1 = SPLIT ? static_cast<int>(static_cast<int64_t>(units) * (z + 1) / gridDim.z) : units;
  auto at = [&](int i, int j, int g, int& m, int& n) {
    m = wm * WM + 32 * i + (lane & 31);
    n = wn * WN + 32 * j + 8 * g + 4 * (lane >> 5);
  };
  h4 av[POLY && !SPLIT ? TM : 1][TN][4];  // A', read early
  if constexpr (POLY && !SPLIT) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          int m, n;
          at(i, j, g, m, n);
          av[i][j][g] = *poly_a16(a, b, r0 + m, c0 + n);
        }
  }
  typename G::Acc acc;
  G::zero(acc);
  G::run(x + (POLY ? r0 * ld : r0), ld, x + (POLY ? c0 * ld : c0), ld, k0 * 128, (k1 - k0) * 2, bufs, acc);
  float* out = a.part + ((static_cast<int64_t>(b) * gridDim.z + z) * gridDim.x + tile) * (BM * BN);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f4 v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        int m, n;
        at(i, j, g, m, n);
        if constexpr (SPLIT) {
          const int bm = wm * (WM / 32) + i, bn = wn * (WN / 32) + j;  // the block of 32x32 in the tile
          const int to = (bm / 2 * (BN / 64) + bn / 2) * kRegion + region_offset(bm & 1, bn & 1, g, lane);
          *reinterpret_cast<f4*>(out + to) = v;
        } else {
          h4 h;
          if constexpr (POLY) h = poly_elements(a, b, r0 + m, c0 + n, v, av[i][j][g], cb, cc, sb);
          else h = gram_elements(a, b, r0 + m, c0 + n, v);
          put_row<BN>(staged<G::kStage, BM, BN, 0>(bufs, m), m, n, h);
          put_col<BM>(staged<G::kStage, BN, BM, NST / 2>(bufs, n + (lane & 3)), m, n + (lane & 3), h);
        }
      }
  if constexpr (!SPLIT) {
    __syncthreads();
    write_symmetric<G::kStage, BM, BN, G::kThreads, NST / 2>(bufs, (POLY ? a.b16 : a.a16) + b * a.pp * a.ldp, a.ldp, r0, c0);
  }
}

// Adds the parts of one 64x64 region in their order, and writes what is stored of it.
template <int BM, int BN, bool POLY>
__global__ __launch_bounds__(256) void ns_finish_kernel(NsArgs a, int tiles, int splits, float cb, float cc, float sb) {
  constexpr int kPer = (BM / 64) * (BN / 64);
  __shared__ __align__(16) uint8_t rows[64 * 64 * 2], cols[64 * 64 * 2];
  const Buffers bufs = {rows, cols, rows, rows};
  const int b = blockIdx.y, tile = blockIdx.x / kPer, reg = blockIdx.x % kPer;
  int ti, tj;
  triangle_tile<BM, BN>(tile, ti, tj);
  const int64_t r0 = static_cast<int64_t>(ti) * BM + reg / (BN / 64) * 64, c0 = static_cast<int64_t>(tj) * BN + reg % (BN / 64) * 64;
  if (c0 > r0) return;  // above the diagonal: the mirror image of another region
  const int64_t step = static_cast<int64_t>(tiles) * (BM * BN);
  const float* in = a.part + static_cast<int64_t>(b) * splits * step + static_cast<int64_t>(tile) * (BM * BN) + reg * kRegion;
  f4 s[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) s[u] = *reinterpret_cast<const f4*>(in + (threadIdx.x + 256 * u) * 4);
  for (int k = 1; k < splits; ++k)
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] += *reinterpret_cast<const f4*>(in + k * step + (threadIdx.x + 256 * u) * 4);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = threadIdx.x + 256 * u;
    const int lane = t & 63, g = (t >> 6) & 3, bj = (t >> 8) & 1, bi = t >> 9;
    const int m = 32 * bi + (lane & 31), n = 32 * bj + 8 * g + 4 * (lane >> 5);
    h4 h;
    if constexpr (POLY) h = poly_elements(a, b, r0 + m, c0 + n, s[u], *poly_a16(a, b, r0 + m, c0 + n), cb, cc, sb);
    else h = gram_elements(a, b, r0 + m, c0 + n, s[u]);
    put_row<64>(rows + m * 128, m, n, h);
    put_col<64>(cols + (n + (lane & 3)) * 128, m, n + (lane & 3), h);
  }
  __syncthreads();
  write_symmetric<64 * 64 * 2, 64, 64, 256, 1>(bufs, (POLY ? a.b16 : a.a16) + b * a.pp * a.ldp, a.ldp, r0, c0);
}

// ------------------------------------------------------------------------------ X <- a X + B X
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }

// The first n of 8 BF16 patterns (held as FP16 bits) to a row of any alignment.
__device__ __forceinline__ void store_row(uint16_t* p, h8 v, int64_t n) {
  typedef uint16_t us8 __attribute__((ext_vector_type(8)));
  if (n >= 8) {
    *reinterpret_cast<u4_a2*>(p) = __builtin_bit_cast(u4_a2, v);
    return;
  }
  const us8 w = __builtin_bit_cast(us8, v);
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < n) p[e] = w[e];
}

// Lanes l and l + 32 hold 8 columns each, 8 c .. and 8 (c + 1) ..; afterwards l has the first four of both,
// l + 32 the last four.
__device__ __forceinline__ h8 swap_halves(h8 v) {
  uint4 w = __builtin_bit_cast(uint4, v);
  const auto p = __builtin_amdgcn_permlane32_swap(w.x, w.z, false, false);
  const auto q = __builtin_amdgcn_permlane32_swap(w.y, w.w, false, false);
  w.x = p[0], w.z = p[1], w.y = q[0], w.w = q[1];
  return __builtin_bit_cast(h8, w);
}

// X is read before the product, so that it arrives behind its first stages. Bound by the matrix cores and the
// LDS reads that feed them; among the other kernels 12288 x 2048 takes 125 us (820 TFLOP/s), the last step,
// which writes BF16 only, 120 us.
template <int BM, int BN, int WM, int WN, int NST, bool LAST>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void ns_update_kernel(NsArgs a, float ca, float inv_sb, int turn) {
  using G = Tile<BM, BN, WM, WN, NST, false>;
  constexpr int TM = G::TM, TN = G::TN;
  PF8_NS_BUFFERS(bufs, G, NST);
  const bool tall = a.m > a.n;
  const int b = blockIdx.y;
  const int tiles_p = static_cast<int>(a.pp / BN);
  const int bid = static_cast<int>(xcd_order(blockIdx.x, gridDim.x));
  // strips four tiles wide, so that an XCD's tiles take few rows of both operands through its L2: 8192 x 8192
  // 11.5 ms, 13.5 in rows of all tiles and 12.1 in columns of one
  constexpr int kWide = 4;
  const int tiles_q = static_cast<int>(a.qp / BM);
  const int strip = bid / (kWide * tiles_q), wide = min(kWide, tiles_p - strip * kWide), in = bid - strip * kWide * tiles_q;
  const int64_t j0 = static_cast<int64_t>(in / wide) * BM, i0 = static_cast<int64_t>(strip * kWide + in % wide) * BN;
  const _Float16* xc = a.xc[turn] + b * a.qp * a.ldp;
  const _Float16* B = a.b16 + b * a.pp * a.ldp;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / (BN / WN), wn = wave % (BN / WN);
  // X as it was: a lane reads 8 consecutive columns of X^T, those of its half of the wave's lanes (pair of g) ..
  auto rest_at = [&](int i, int j, int pair) {
    const int m = wm * WM + 32 * i, n = wn * WN + 32 * j;
    const int64_t region = ((j0 + m) / 64) * (a.pp / 64) + (i0 + n) / 64;
    return reinterpret_cast<h8*>(a.rest + b * a.x_elems + region * kRegion + rest_offset((m >> 5) & 1, (n >> 5) & 1, pair, lane));
  };
  h8 xh[TM][TN][2], xl[TM][TN][2];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int pair = 0; pair < 2; ++pair) {
        const int m = wm * WM + 32 * i + (lane & 31), n = wn * WN + 32 * j + 16 * pair + 8 * (lane >> 5);
        xh[i][j][pair] = *reinterpret_cast<const h8*>(xc + (j0 + m) * a.ldp + i0 + n);
        xl[i][j][pair] = *rest_at(i, j, pair);
      }
  typename G::Acc acc;
  G::zero(acc);
  G::run(xc + j0 * a.ldp, a.ldp, B + i0 * a.ldp, a.ldp, 0, static_cast<int>(a.pp / G::BK), bufs, acc);

  const float* d = a.db + b * a.pp + i0;
  h4 v[TM][TN][4];
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {
      f4 dn[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        dn[h] = *reinterpret_cast<const f4*>(d + wn * WN + 32 * j + 8 * (2 * pair + h) + 4 * (lane >> 5));
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        // .. and the halves exchange, so that it has the four columns of each g that its sums belong to
        const h8 hi = swap_halves(xh[i][j][pair]);
        h8 lo = xl[i][j][pair];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int h = k >> 2, e = k & 3, g = 2 * pair + h;
          const float yh = static_cast<float>(hi[k]), x = yh + static_cast<float>(lo[k]);
          const float y = __builtin_fmaf(ca, x, __builtin_fmaf(dn[h][e], LAST ? x : yh, acc[i][j][4 * g + e] * inv_sb));
          if (LAST) {
            v[i][j][g][e] = __builtin_bit_cast(_Float16, bf16_bits(y * (1.0f / kSX)));
          } else {
            v[i][j][g][e] = static_cast<_Float16>(y);
            lo[k] = remainder16(y);
          }
        }
        if (!LAST) *rest_at(i, j, pair) = lo;
      }
    }
  // out through LDS: as rows of X^T, the last step's as rows of G
  auto each_piece = [&](auto f) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) f(wm * WM + 32 * i + (lane & 31), wn * WN + 32 * j + 8 * g + 4 * (lane >> 5), v[i][j][g]);
  };
  constexpr int kPieces = BM * BN / 8 / G::kThreads;
  uint16_t* out = a.out + b * a.stride_o;
  if (!LAST || tall) {
    each_piece([&](int m, int n, h4 w) { put_row<BN>(staged<G::kStage, BM, BN, 0>(bufs, m), m, n, w); });
    __syncthreads();
    _Float16* next = a.xc[turn ^ 1] + b * a.qp * a.ldp;
#pragma unroll 4
    for (int u = 0; u < kPieces; ++u) {
      const int c = threadIdx.x + u * G::kThreads, row = c / (BN / 8), chunk = c % (BN / 8), col = chunk * 8;
      const h8 w = get_row<BN>(staged<G::kStage, BM, BN, 0>(bufs, row), row, chunk);
      if (!LAST) *reinterpret_cast<h8*>(next + (j0 + row) * a.ldp + i0 + col) = w;
      else if (j0 + row < a.m) store_row(out + (j0 + row) * a.ldo + i0 + col, w, a.n - (i0 + col));
    }
  } else {
    each_piece([&](int m, int n, h4 w) {
      const int nt = n + (lane & 3);
      put_col<BM>(staged<G::kStage, BN, BM, 0>(bufs, nt), m, nt, w);
    });
    __syncthreads();
#pragma unroll 4
    for (int u = 0; u < kPieces; ++u) {
      const int c = threadIdx.x + u * G::kThreads, row = c / (BM / 8), chunk = c % (BM / 8), col = chunk * 8;  // row of X
      const h8 w = get_col<BM>(staged<G::kStage, BN, BM, 0>(bufs, row), row, chunk);
      if (i0 + row < a.m) store_row(out + (i0 + row) * a.ldo + j0 + col, w, a.n - (j0 + col));
    }
  }
}

// ------------------------------------------------------------------------------ small matrices
// One matrix of at most P x (NS P) per workgroup, all steps in one launch: the waves hold a WM x 32 part of every
// P x P slab of X^T in registers (FP32); the products' operands go through LDS as FP16, X in the update as value
// and remainder. Bound by the chain of short products, each behind a barrier and 16-wave traffic through LDS:
// 128 x 128, five steps: 26.8 us with 16 waves of 32 x 32, 28.9 with 8 of 64 x 32, for one matrix as for 16.
template <int P, int WM, int NS, typename T>
__global__ __launch_bounds__(64 * (P / WM) * (P / 32)) void ns_small_kernel(NsArgs a, NsCoef coef, int steps) {
  constexpr int TM = WM / 32, TN = 1, kWaves = (P / WM) * (P / 32), PITCH = P + 8;  // 16 rows' 16-byte reads of one column fall into different banks
  __shared__ __align__(16) _Float16 zh[P * PITCH], zl[P * PITCH], ab[P * PITCH];
  __shared__ __align__(16) float da[P], db[P];  // the diagonals of A, and of B plus a
  __shared__ double red[kWaves];
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r0 = wave / (P / 32) * WM, c0 = wave % (P / 32) * 32;
  const bool tall = a.m > a.n;
  const int p = static_cast<int>(tall ? a.n : a.m), q = static_cast<int>(tall ? a.m : a.n);
  const T* g = static_cast<const T*>(a.g) + blockIdx.x * a.stride_g;
  // register r = 4 g + e of block (bi, bj) is element (row(bi), col(bj, r)) of a slab of X^T, of A or of B
  auto row = [&](int bi) { return r0 + 32 * bi + l32; };
  auto col = [&](int bj, int r) { return c0 + 32 * bj + 4 * half + 8 * (r >> 2) + (r & 3); };
  auto blocks = [&](auto f) {
#pragma unroll
    for (int bi = 0; bi < TM; ++bi)
#pragma unroll
      for (int bj = 0; bj < TN; ++bj) f(bi, bj);
  };

  float z[NS][TM][TN][16];
  double sum = 0.0;
#pragma unroll
  for (int s = 0; s < NS; ++s)
    blocks([&](int bi, int bj) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        // (always a load, of the matrix's last row or column if need be: behind a branch each would be waited for)
        const int i = min(col(bj, r), p - 1), j = min(s * P + row(bi), q - 1);
        z[s][bi][bj][r] = value<T>(g[tall ? j * a.ldg + i : i * a.ldg + j]);
      }
    });
#pragma unroll
  for (int s = 0; s < NS; ++s)
    blocks([&](int bi, int bj) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float& v = z[s][bi][bj][r];
        v = col(bj, r) < p && s * P + row(bi) < q ? v : 0.0f;
        sum = __builtin_fma(static_cast<double>(v), static_cast<double>(v), sum);
      }
    });
  sum = block_sum(sum, red);
  const double scale =
      sum <= 1e300 ? static_cast<double>(kSX) / (__builtin_sqrt(sum) + static_cast<double>(a.eps)) : __builtin_nan("");
  // zeros outside the matrix stay zero, or turn NaN with every element inside it
#pragma unroll
  for (int s = 0; s < NS; ++s)
    blocks([&](int bi, int bj) {
#pragma unroll
      for (int r = 0; r < 16; ++r) z[s][bi][bj][r] = static_cast<float>(static_cast<double>(z[s][bi][bj][r]) * scale);
    });

  auto frag = [&](const _Float16* mat, int first, int k) {
    return *reinterpret_cast<const h8*>(mat + (first + l32) * PITCH + 16 * k + 8 * half);
  };
  // four values as FP16 and what that leaves
  auto split = [&](const float (&v)[16], int u, h4& h, h4& l) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[4 * u + e];
      h[e] = static_cast<_Float16>(x);
      l[e] = static_cast<_Float16>(x - static_cast<float>(h[e]));
    }
  };
  f16v acc[TM][TN];
  auto clear = [&] {
    blocks([&](int bi, int bj) {
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[bi][bj][r] = 0.0f;
    });
  };
  for (int step = 0; step < steps; ++step) {
    const float ca = coef.v[step][0], cb = coef.v[step][1], cc = coef.v[step][2], sb = coef.v[step][3], inv_sb = coef.v[step][4];
    clear();
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (s * P >= q) continue;  // uniform
      if (s) __syncthreads();
      blocks([&](int bi, int bj) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          h4 h, l;
          split(z[s][bi][bj], u, h, l);
          *reinterpret_cast<h4*>(zh + (col(bj, 4 * u) + (lane & 3)) * PITCH + (row(bi) & ~3)) = quad_transpose(h);
        }
      });
      __syncthreads();
#pragma unroll
      for (int k = 0; k < P / 16; ++k) {
        h8 fi[TM], fj[TN];
#pragma unroll
        for (int t = 0; t < TM; ++t) fi[t] = frag(zh, r0 + 32 * t, k);
#pragma unroll
        for (int t = 0; t < TN; ++t) fj[t] = frag(zh, c0 + 32 * t, k);
        blocks([&](int bi, int bj) { acc[bi][bj] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fj[bj], fi[bi], acc[bi][bj], 0, 0, 0); });
      }
    }
    // (only the blocks on the diagonal look for it)
    auto diagonal = [&](int bi, int bj) { return r0 + 32 * bi == c0 + 32 * bj; };
    h4 x[TM][TN][4];  // A'
    blocks([&](int bi, int bj) {
      const int m = row(bi);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int n = col(bj, 4 * u);
        h4& v = x[bi][bj][u];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = static_cast<_Float16>(acc[bi][bj][4 * u + e] * (kSA / (kSX * kSX)));
        if (diagonal(bi, bj)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (m == n + e) da[m] = acc[bi][bj][4 * u + e] * (1.0f / (kSX * kSX));
            v[e] = m == n + e ? static_cast<_Float16>(0.0f) : v[e];
          }
        }
        *reinterpret_cast<h4*>(ab + m * PITCH + n) = v;
      }
    });
    __syncthreads();
    clear();
#pragma unroll
    for (int k = 0; k < P / 16; ++k) {
      h8 fi[TM], fj[TN];
#pragma unroll
      for (int t = 0; t < TM; ++t) fi[t] = frag(ab, r0 + 32 * t, k);
#pragma unroll
      for (int t = 0; t < TN; ++t) fj[t] = frag(ab, c0 + 32 * t, k);
      blocks([&](int bi, int bj) { acc[bi][bj] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fj[bj], fi[bi], acc[bi][bj], 0, 0, 0); });
    }
    __syncthreads();  // A' has been read: B' takes its place
    blocks([&](int bi, int bj) {
      const int m = row(bi);
      const float dm = da[m];
      const float from = (cb + cc * dm) * (sb / kSA), by = cc * (sb / kSA), squares = cc * (sb / (kSA * kSA));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int n = col(bj, 4 * u);
        const f4 dn = *reinterpret_cast<const f4*>(da + n);
        h4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = static_cast<_Float16>(__builtin_fmaf(static_cast<float>(x[bi][bj][u][e]), __builtin_fmaf(by, dn[e], from),
                                                      squares * acc[bi][bj][4 * u + e]));
        if (diagonal(bi, bj)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (m == n + e) db[m] = ca + cb * dm + cc * (acc[bi][bj][4 * u + e] * (1.0f / (kSA * kSA)) + dm * dm);
            v[e] = m == n + e ? static_cast<_Float16>(0.0f) : v[e];
          }
        }
        *reinterpret_cast<h4*>(ab + m * PITCH + n) = v;
      }
    });
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (s * P >= q) continue;
      if (s) __syncthreads();
      blocks([&](int bi, int bj) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          h4 h, l;
          split(z[s][bi][bj], u, h, l);
          *reinterpret_cast<h4*>(zh + row(bi) * PITCH + col(bj, 4 * u)) = h;
          *reinterpret_cast<h4*>(zl + row(bi) * PITCH + col(bj, 4 * u)) = l;
        }
      });
      __syncthreads();
      clear();
#pragma unroll
      for (int k = 0; k < P / 16; ++k) {
        h8 fh[TM], fl[TM], fb[TN];
#pragma unroll
        for (int t = 0; t < TM; ++t) fh[t] = frag(zh, r0 + 32 * t, k), fl[t] = frag(zl, r0 + 32 * t, k);
#pragma unroll
        for (int t = 0; t < TN; ++t) fb[t] = frag(ab, c0 + 32 * t, k);
        blocks([&](int bi, int bj) {
          acc[bi][bj] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[bj], fl[bi], acc[bi][bj], 0, 0, 0);
          acc[bi][bj] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[bj], fh[bi], acc[bi][bj], 0, 0, 0);
        });
      }
      blocks([&](int bi, int bj) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          z[s][bi][bj][r] = __builtin_fmaf(db[col(bj, r)], z[s][bi][bj][r], acc[bi][bj][r] * inv_sb);
      });
    }
    __syncthreads();  // the last slab and B' have been read
  }
  uint16_t* out = a.out + blockIdx.x * a.stride_o;
  int pe = p, qe = q;
  asm volatile("" : "+s"(pe), "+s"(qe));  // the comparisons are made again, not kept from the loads
#pragma unroll
  for (int s = 0; s < NS; ++s)
    blocks([&](int bi, int bj) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int i = col(bj, r), j = s * P + row(bi);
        if (i < pe && j < qe) out[tall ? j * a.ldo + i : i * a.ldo + j] = bf16_bits(z[s][bi][bj][r] * (1.0f / kSX));
      }
    });
}

// The power of two that B's FP16 elements carry. Those off the diagonal are at most half as large as B's eigenvalues
// b s^2 + c s^4 lie apart, 32 |b| + 2048 |c| for s up to 8; 60000 leaves the operands' roundings room below FP16's
// 65504. The usual quintic takes 8: elements under 2^-17 lose bits, at most 2^-28 beside the a that B is added to.
float poly_scale(float b, float c) {
  const float most = 32.0f * __builtin_fabsf(b) + 2048.0f * __builtin_fabsf(c);
  float s = 512.0f;
  while (s * most > 60000.0f) s *= 0.5f;
  return s;
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// How a size is run. Tile shapes are chosen by the time that a model of the kernels gives: a card's 256 CUs
// take one workgroup each (two of 64x64), a stage of 64 K values costs a workgroup 0.34 us (128x128), 0.5 us
// (128x256) or 0.3 us (64x64, two on a CU; 0.14 us alone), and a launch with its first loads and its last
// stores the rest. Measured against it, each kernel by itself, for the lower triangle of 2048 x 2048 with
// K = 2048 / 12288: 64x64 21.8 / 122 us, 128x128 18.4 / 73 us, 128x256 with K in three parts 23 / 65 us; of
// 1024 x 1024 with K = 1664: 64x64 7.1 us, 128x128 13.7 us. Update of 2048 x 2048: 128x128 21.6 us, 128x256
// 27.5 us, 64x64 42 us; of 12288 x 2048: 122, 90 and 237 us; of 1664 x 1024: 12.5, 17.6 and 9.5 us.
enum Shape { k64x64, k128x128, k128x256 };
struct Plan {
  int64_t pp, qp;
  Shape gram, poly, update;
  int gram_splits, poly_splits;  // parts of K: with 128x256 tiles, and where 64x64 tiles are few
};

// Tiles of a shape that cover the lower triangle.
int64_t triangle_tiles(Shape s, int64_t pp) {
  const int64_t n = pp / (s == k128x256 ? 256 : s == k64x64 ? 64 : 128);
  return n * (n + 1) / 2 * (s == k128x256 ? 2 : 1);
}

int64_t rounds(int64_t tiles, int64_t slots) { return (tiles + slots - 1) / slots; }

void plan_sym(int64_t pp, int64_t batch, int64_t k, Shape& shape, int& splits) {
  const double stages = static_cast<double>(k / 64);
  const int64_t t64 = batch * triangle_tiles(k64x64, pp), t128 = batch * triangle_tiles(k128x128, pp);
  auto c64 = [&](int64_t parts, double n) {
    return parts <= 256 ? 4.0 + 0.14 * n : 5.0 + 0.3 * n * static_cast<double>(rounds(parts, 512));
  };
  double best = c64(t64, stages);
  shape = k64x64;
  splits = 1;
  // (with no more than pp values along K the parts never come out cheaper)
  for (int s = 2; k > pp && s <= 32 && s <= k / 256; s *= 2) {
    const double c = 4.0 + c64(t64 * s, stages / s) + 0.004 * static_cast<double>(t64 * s);
    if (c < best) best = c, splits = s;
  }
  const double c128 = 8.0 + 0.34 * stages * static_cast<double>(rounds(t128, 256));
  if (c128 < best) best = c128, shape = k128x128, splits = 1;
  if (pp % 256) return;
  for (int s = 1; s <= 8 && s <= k / 512; ++s) {
    const int64_t parts = batch * triangle_tiles(k128x256, pp) * s;
    // the parts are written and read again: 128 KiB each, at 4 TB/s in all
    const double c = 12.0 + 0.5 * stages / s * static_cast<double>(rounds(parts, 256)) + 0.032 * static_cast<double>(parts);
    if (c < best) best = c, shape = k128x256, splits = s;
  }
}

// Values of the split products' partial sums.
int64_t part_elems(Shape shape, int splits, int64_t pp) {
  const int64_t tile = shape == k128x256 ? 128 * 256 : shape == k64x64 && splits > 1 ? 64 * 64 : 0;
  return triangle_tiles(shape, pp) * splits * tile;
}

Plan plan_of(int64_t batch, int64_t m, int64_t n) {
  Plan p;
  const int64_t shorter = m < n ? m : n, longer = m < n ? n : m;
  p.pp = round_up(shorter, shorter > 1024 ? 256 : 128);
  p.qp = round_up(longer, 128);
  const double stages = static_cast<double>(p.pp / 64);
  const int64_t t128 = batch * (p.pp / 128) * (p.qp / 128);
  // the update also reads and writes X: a round of tiles has 8 (14) us of that behind its products
  const double c64 = 5.0 + (0.3 * stages + 6.0) * static_cast<double>(rounds(4 * t128, 512));
  const double c128 = 6.0 + (0.34 * stages + 8.0) * static_cast<double>(rounds(t128, 256));
  const double c256 = 6.0 + (0.5 * stages + 14.0) * static_cast<double>(rounds(t128 / 2, 256));
  p.update = c64 < c128 ? k64x64 : k128x128;
  if (p.pp % 256 == 0 && c256 < std::min(c64, c128)) p.update = k128x256;
  plan_sym(p.pp, batch, p.qp, p.gram, p.gram_splits);
  plan_sym(p.pp, batch, p.pp, p.poly, p.poly_splits);
  return p;
}

// A whole matrix in one workgroup's registers.
bool is_small(int64_t m, int64_t n) {
  const int64_t p = std::min(m, n), q = std::max(m, n);
  return (p <= 64 && q <= 512) || (p <= 128 && q <= 256);
}

template <typename T>
hipError_t launch_small(const NsArgs& a, const NsCoef& coef, int steps, uint32_t batch, hipStream_t stream) {
  const int64_t p = std::min(a.m, a.n), q = std::max(a.m, a.n);
  auto go = [&](auto kern, int threads) {
    hipLaunchKernelGGL(kern, dim3(batch), dim3(threads), 0, stream, a, coef, steps);
    return hipGetLastError();
  };
  if (p <= 64) {
    if (q <= 64) return go(ns_small_kernel<64, 32, 1, T>, 256);
    if (q <= 128) return go(ns_small_kernel<64, 32, 2, T>, 256);
    if (q <= 256) return go(ns_small_kernel<64, 32, 4, T>, 256);
    return go(ns_small_kernel<64, 32, 8, T>, 256);
  }
  if (q <= 128) return go(ns_small_kernel<128, 32, 1, T>, 1024);
  return go(ns_small_kernel<128, 32, 2, T>, 1024);
}

int64_t align256(int64_t v) { return round_up(v, 256); }

}  // namespace

template <bool POLY>
static void launch_sym(const NsArgs& a, Shape shape, int splits, uint32_t batch, int turn, float cb, float cc, float sb,
                       hipStream_t stream) {
  const uint32_t tiles = static_cast<uint32_t>(triangle_tiles(shape, a.pp));
  const dim3 grid(tiles, batch, static_cast<uint32_t>(splits));
  if constexpr (!POLY) {
    if (shape == k64x64 && splits > 1) {
      hipLaunchKernelGGL((ns_sym_kernel<64, 64, 32, 32, 4, false, true>), grid, dim3(256), 0, stream, a, turn, cb, cc, sb);
      hipLaunchKernelGGL((ns_finish_kernel<64, 64, false>), dim3(tiles, batch), dim3(256), 0, stream, a, static_cast<int>(tiles), splits, cb, cc, sb);
      return;
    }
  }
  if (shape == k64x64) {
    hipLaunchKernelGGL((ns_sym_kernel<64, 64, 32, 32, 4, POLY, false>), grid, dim3(256), 0, stream, a, turn, cb, cc, sb);
  } else if (shape == k128x128) {
    hipLaunchKernelGGL((ns_sym_kernel<128, 128, 64, 64, 4, POLY, false>), grid, dim3(256), 0, stream, a, turn, cb, cc, sb);
  } else {
    hipLaunchKernelGGL((ns_sym_kernel<128, 256, 64, 64, 3, POLY, true>), grid, dim3(512), 0, stream, a, turn, cb, cc, sb);
    hipLaunchKernelGGL((ns_finish_kernel<128, 256, POLY>), dim3(tiles * 8, batch), dim3(256), 0, stream, a, static_cast<int>(tiles), splits, cb, cc, sb);
  }
}

template <bool LAST>
static void launch_update(const NsArgs& a, Shape shape, uint32_t batch, float ca, float inv_sb, int turn, hipStream_t stream) {
  const int64_t bm = shape == k64x64 ? 64 : 128, bn = shape == k64x64 ? 64 : shape == k128x128 ? 128 : 256;
  const dim3 grid(static_cast<uint32_t>((a.qp / bm) * (a.pp / bn)), batch);
  if (shape == k64x64) hipLaunchKernelGGL((ns_update_kernel<64, 64, 32, 32, 4, LAST>), grid, dim3(256), 0, stream, a, ca, inv_sb, turn);
  else if (shape == k128x128) hipLaunchKernelGGL((ns_update_kernel<128, 128, 64, 64, 4, LAST>), grid, dim3(256), 0, stream, a, ca, inv_sb, turn);
  else hipLaunchKernelGGL((ns_update_kernel<128, 256, 64, 64, 3, LAST>), grid, dim3(512), 0, stream, a, ca, inv_sb, turn);
}

// Workspace parts, in order: X's remainders, two Xc, A, B, their diagonals, A's partial tiles, norms.
static int64_t ns_layout(int64_t batch, const Plan& p, NsArgs* a, uint8_t* base) {
  const int64_t x = p.pp * p.qp, ldp = p.pp + kPad;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* r = base + at;
    at += align256(bytes);
    return r;
  };
  uint8_t* rest = take(batch * x * 2);
  uint8_t* xc0 = take(batch * p.qp * ldp * 2);
  uint8_t* xc1 = take(batch * p.qp * ldp * 2);
  uint8_t* a16 = take(batch * p.pp * ldp * 2);
  uint8_t* b16 = take(batch * p.pp * ldp * 2);
  uint8_t* da = take(batch * p.pp * 4);
  uint8_t* db = take(batch * p.pp * 4);
  const int64_t gram = part_elems(p.gram, p.gram_splits, p.pp), poly = part_elems(p.poly, p.poly_splits, p.pp);
  uint8_t* part = take(batch * std::max(gram, poly) * 4);
  uint8_t* norm = take(batch * kNormBlocks * 8);
  if (a) {
    a->pp = p.pp, a->qp = p.qp, a->ldp = ldp, a->x_elems = x;
    a->rest = reinterpret_cast<_Float16*>(rest);
    a->xc[0] = reinterpret_cast<_Float16*>(xc0), a->xc[1] = reinterpret_cast<_Float16*>(xc1);
    a->a16 = reinterpret_cast<_Float16*>(a16), a->b16 = reinterpret_cast<_Float16*>(b16);
    a->da = reinterpret_cast<float*>(da), a->db = reinterpret_cast<float*>(db);
    a->part = reinterpret_cast<float*>(part), a->norm_part = reinterpret_cast<double*>(norm);
  }
  return at;
}

int64_t ns_workspace(int64_t batch, int64_t m, int64_t n) {
  if (is_small(m, n)) return 256;
  return ns_layout(batch, plan_of(batch, m, n), nullptr, nullptr);
}

hipError_t launch_newton_schulz(NsArgs a, int64_t batch, int steps, const float* coef, void* workspace, hipStream_t stream) {
  if (is_small(a.m, a.n)) {
    NsCoef c{};
    for (int s = 0; s < steps; ++s) {
      for (int k = 0; k < 3; ++k) c.v[s][k] = coef[3 * s + k];
      c.v[s][3] = poly_scale(coef[3 * s + 1], coef[3 * s + 2]);
      c.v[s][4] = 1.0f / c.v[s][3];
    }
    return a.gf32 ? launch_small<float>(a, c, steps, static_cast<uint32_t>(batch), stream)
                  : launch_small<uint16_t>(a, c, steps, static_cast<uint32_t>(batch), stream);
  }
  const Plan p = plan_of(batch, a.m, a.n);
  ns_layout(batch, p, &a, static_cast<uint8_t*>(workspace));
  const uint32_t nb = static_cast<uint32_t>(batch);
  const dim3 init_grid(static_cast<uint32_t>((p.pp / 64) * (p.qp / 64)), nb);
  if (a.gf32) {
    hipLaunchKernelGGL(ns_norm_kernel<float>, dim3(kNormBlocks, nb), dim3(kNormThreads), 0, stream, a);
    hipLaunchKernelGGL(ns_init_kernel<float>, init_grid, dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL(ns_norm_kernel<uint16_t>, dim3(kNormBlocks, nb), dim3(kNormThreads), 0, stream, a);
    hipLaunchKernelGGL(ns_init_kernel<uint16_t>, init_grid, dim3(256), 0, stream, a);
  }
  if (hipError_t e = hipGetLastError()) return e;
  for (int s = 0; s < steps; ++s) {
    const float ca = coef[3 * s], cb = coef[3 * s + 1], cc = coef[3 * s + 2], sb = poly_scale(cb, cc);
    launch_sym<false>(a, p.gram, p.gram_splits, nb, s & 1, cb, cc, sb, stream);
    launch_sym<true>(a, p.poly, p.poly_splits, nb, s & 1, cb, cc, sb, stream);
    if (s + 1 < steps) launch_update<false>(a, p.update, nb, ca, 1.0f / sb, s & 1, stream);
    else launch_update<true>(a, p.update, nb, ca, 1.0f / sb, s & 1, stream);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace pf8
