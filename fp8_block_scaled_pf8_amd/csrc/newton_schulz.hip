// Newton-Schulz orthogonalisation for gfx950: X <- a X + (b A + c A A) X with A = X X^T, from
// X = G / (|G|_F + eps). Contract in include/pf8_train.h.
//
// Bound: the matrix cores. With X [p, q] (p <= q; a tall G is taken transposed) a step is
// p^2 q multiply-adds for A and p^3 / 2 for A A, both symmetric and formed for their lower tiles
// only, and p^2 q for the update.
//
// Number formats. The products run on FP16 operands with FP32 accumulation; everything that adds
// up over the steps is FP32:
//  * X itself is kept in FP32. The update adds a X from it; only the small product B X is formed
//    from X's FP16 rounding. (Rounding X itself would put noise into directions whose singular
//    value is nearly zero, which the iteration multiplies by a in every step: a rank-one G came
//    out 15 % off.)
//  * A and B = b A + c A A are split into their diagonals, kept in FP32, and the rest in FP16:
//    near the end A is close to a multiple of the identity and the diagonal carries nearly all.
//    (A A)_ij = sum A'_ik A'_kj + (d_i + d_j) A'_ij off the diagonal.
//  * FP16 operands are scaled by powers of two (X 2^12, A 2^10, B 2^9), so that entries down to
//    2^-26 of the norm keep all their bits and singular values up to 8 stay in range.
//  * The diagonal's part of B X takes a row of X in FP32 where the diagonal's element is large, and
//    the row's FP16 rounding elsewhere (kOwnRow). A matrix of full rank ends with diagonals near
//    1 - a, and there the rounding of X would enter 2.4-fold. In a matrix of low rank the diagonal
//    is small, and B' times the rounding alone, without the diagonal's part, would be noise outside
//    of the matrix's column space, which grows by a in every step.
//  * A matrix of at most 64 x 512 or 128 x 256 stays in one workgroup, and its X enters the products as a sum of
//    two FP16 values (22 bits): few entries average out little of the rounding noise.
// Against float64, besides the BF16 rounding of the result (1.7e-3 of its 2-norm), the result is off
// by up to 1.3e-3 of its 2-norm (2.8e-3 where a few entries carry the norm of a larger matrix); BF16
// operands would give 1.4e-2.
//
// Layout. X lives in the workspace, padded to multiples of 128 with zeros that stay zero, so the
// products have no edges: Xr [p][q] (A's operand), Xc [q][p] (the update's operand, two buffers in
// turn) and FP32 in 64x64 regions in the order the update's lanes hold them, so that each lane
// reads and writes 16 consecutive bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pf8_train_launch.h"

namespace pf8 {

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));

// The steps' coefficients, by value: the host's array is not read after the call.
struct NsCoef {
  float v[64][3];
};

constexpr float kSX = 4096.0f, kSA = 1024.0f, kSB = 512.0f;  // powers of two that FP16 operands carry
constexpr int kBK = 64;                                      // K values of one stage (128-byte LDS rows)
constexpr int kRegion = 64 * 64;
// a diagonal element of B over this part of |a - 1| (which a matrix of full rank with singular values
// near one has) multiplies X in FP32
constexpr float kOwnRow = 2.0f / 3.0f;

// In a 64x64 region of a product, block (bi, bj) of 32x32 and register 4 g + e of lane l hold the
// element (32 bi + l % 32, 32 bj + 8 g + 4 (l / 32) + e).
__device__ __forceinline__ int region_offset(int bi, int bj, int g, int lane) {
  return ((bi * 2 + bj) * 4 + g) * 256 + lane * 4;
}

// D[m, n] = sum_k P[m, k] Q[n, k] over `steps` stages of 64: a BM x BN tile by (BM/WM)(BN/WN) waves.
// Stages go straight to LDS (16 bytes a lane), NST - 1 ahead of use. In a 128-byte LDS row, chunk c
// of row r sits at c ^ ((r >> 1) & 7): 16 consecutive rows' reads of one chunk fall into the 16
// different 16-byte slots of the 64 banks. One barrier a stage: behind it every wave's loads of the
// stage have landed and the buffer of the stage before is free to be filled again.
template <int BM, int BN, int WM, int WN, int NST>
struct Tile {
  static constexpr int kWavesN = BN / WN, kWaves = (BM / WM) * kWavesN, kThreads = 64 * kWaves;
  static constexpr int TM = WM / 32, TN = WN / 32;
  static constexpr int kStage = (BM + BN) * 128;
  static constexpr int kLoads = (BM + BN) / 8 / kWaves;  // 1 KiB loads per wave and stage
  static_assert(BM / 8 % kWaves == 0 && BN / 8 % kWaves == 0 && (NST == 2 || NST == 3), "even loads, two or three buffers");
  typedef f16v Acc[TM][TN];

  static __device__ __forceinline__ void zero(Acc& acc) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  }

  static __device__ __forceinline__ void run(const _Float16* P, int64_t ldp, const _Float16* Q, int64_t ldq, int k0,
                                             int steps, uint8_t* b0, uint8_t* b1, uint8_t* b2, Acc& acc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    const int ldpb = static_cast<int>(ldp) * 2, ldqb = static_cast<int>(ldq) * 2;
    const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16*>(P), 0, BM * ldpb, 0x00020000);
    const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<_Float16*>(Q), 0, BN * ldqb, 0x00020000);
    // lane's part of a load: row lane / 8 of 8, and the chunk that belongs at LDS chunk lane % 8.
    // The slab's first row is a multiple of 8, so its part of the swizzle is its bit 3.
    const int lrow = lane >> 3;
    auto issue = [&](uint8_t* buf, int s) {
      const int kofs = (k0 + s * kBK) * 2;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int slab = wave + i * kWaves;
        const int row = slab * 8 + lrow;
        const int chunk = (lane & 7) ^ ((row >> 1) & 7);
        auto* dst = (__attribute__((address_space(3))) void*)(buf + slab * 1024);
        if (i < BM / 8 / kWaves) __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, dst, 16, lrow * ldpb + chunk * 16, slab * 8 * ldpb + kofs, 0, 0);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, dst, 16, lrow * ldqb + chunk * 16, (slab - BM / 8) * 8 * ldqb + kofs, 0, 0);
      }
    };
    const int l32 = lane & 31, half = lane >> 5;
    auto compute = [&](const uint8_t* buf) {
#pragma unroll
      for (int k = 0; k < kBK / 16; ++k) {
        h8 fp[TM], fq[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int row = wm * WM + 32 * i + l32;
          fp[i] = *reinterpret_cast<const h8*>(buf + row * 128 + (((2 * k + half) ^ ((row >> 1) & 7)) << 4));
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int row = BM + wn * WN + 32 * j + l32;
          fq[j] = *reinterpret_cast<const h8*>(buf + row * 128 + (((2 * k + half) ^ ((row >> 1) & 7)) << 4));
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fq[j], fp[i], acc[i][j], 0, 0, 0);
      }
    };
    auto sync_stage = [&](bool more) {
      asm volatile("" ::: "memory");
      // vmcnt(loads of the stages behind this one that may still fly) lgkmcnt(0)
      constexpr int fly = (NST - 2) * kLoads;
      if (more) __builtin_amdgcn_s_waitcnt((fly & 0xF) | ((fly >> 4) << 14) | (0x7 << 4));
      else __builtin_amdgcn_s_waitcnt(0x7 << 4);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    issue(b0, 0);
    if (NST == 3 && steps > 1) issue(b1, 1);
    auto step = [&](uint8_t* use, uint8_t* fill, int s) {
      sync_stage(s + 1 < steps && NST == 3);
      if (s + NST - 1 < steps) issue(fill, s + NST - 1);
      compute(use);
    };
    if constexpr (NST == 3) {
      for (int s = 0; s < steps; s += 3) {
        step(b0, b2, s);
        if (s + 1 < steps) step(b1, b0, s + 1);
        if (s + 2 < steps) step(b2, b1, s + 2);
      }
    } else {
      for (int s = 0; s < steps; s += 2) {
        step(b0, b1, s);
        if (s + 1 < steps) step(b1, b0, s + 1);
      }
    }
    // the buffers may be written by the epilogue once every wave has read its last operands
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x7 << 4);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
};

// Position t of the lower triangle (row by row, diagonal included) -> (row, column).
__device__ __forceinline__ void triangle(int t, int& ti, int& tj) {
  int i = static_cast<int>((__builtin_sqrtf(8.0f * static_cast<float>(t) + 1.0f) - 1.0f) * 0.5f);
  while (i * (i + 1) / 2 > t) --i;
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  ti = i;
  tj = t - i * (i + 1) / 2;
}

// Writes a T x T tile from LDS (FP16, pitch T + 8) to rows r0.. and columns c0.. of a symmetric
// matrix, and its mirror image. In a tile on the diagonal the lower triangle counts.
template <int T, int THREADS>
__device__ __forceinline__ void write_symmetric(const _Float16* sh, _Float16* out, int64_t ld, int64_t r0, int64_t c0) {
  constexpr int PITCH = T + 8;
  const bool diag = r0 == c0;
  for (int c = threadIdx.x; c < T * T / 8; c += THREADS) {
    const int row = c / (T / 8), col = (c % (T / 8)) * 8;
    h8 v = *reinterpret_cast<const h8*>(sh + row * PITCH + col), w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = sh[(col + e) * PITCH + row];
    if (diag) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = col + e <= row ? v[e] : w[e];
    } else {
      *reinterpret_cast<h8*>(out + (c0 + row) * ld + r0 + col) = w;
    }
    *reinterpret_cast<h8*>(out + (r0 + row) * ld + c0 + col) = v;
  }
}

// ------------------------------------------------------------------------------ G to X
// Sums of squares of a G, in FP64 (any FP32 value's square is in range): one partial per workgroup.
constexpr int kNormBlocks = 256, kNormThreads = 512;

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

template <typename T>
__global__ __launch_bounds__(kNormThreads) void ns_norm_kernel(NsArgs a) {
  __shared__ double sh[kNormThreads / 64];
  const T* g = static_cast<const T*>(a.g) + blockIdx.y * a.stride_g;
  // pieces of a row, `kPiece` values each, dealt over the workgroups in turn
  constexpr int kPiece = kNormThreads * 8;
  const int64_t per_row = (a.n + kPiece - 1) / kPiece, pieces = a.m * per_row;
  double s = 0.0;
  for (int64_t p = blockIdx.x; p < pieces; p += gridDim.x) {
    const int64_t row = p / per_row, c0 = (p - row * per_row) * kPiece;
    const T* src = g + row * a.ldg;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = c0 + i * kNormThreads + threadIdx.x;
      const double v = c < a.n ? static_cast<double>(value<T>(src[c])) : 0.0;
      s = __builtin_fma(v, v, s);
    }
  }
  s = block_sum(s, sh);
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

// One 64x64 block of X: FP32 regions, Xr and Xc from G, zeros outside.
template <typename T>
__global__ __launch_bounds__(256) void ns_init_kernel(NsArgs a) {
  __shared__ double red[4];
  __shared__ float sh[64][65];  // [i][j]
  const int b = blockIdx.y;
  const int tiles_q = static_cast<int>(a.qp / 64);
  const int64_t i0 = (blockIdx.x / tiles_q) * 64, j0 = (blockIdx.x % tiles_q) * 64;
  const double s = inv_norm(a, b, red);
  const T* g = static_cast<const T*>(a.g) + b * a.stride_g;
  const bool tall = a.m > a.n;
  // read along G's rows: G[row][col] is X[row][col], or X[col][row] of a tall G
  const int64_t r0 = tall ? j0 : i0, c0 = tall ? i0 : j0;
  for (int t = threadIdx.x; t < kRegion; t += 256) {
    const int r = t >> 6, c = t & 63;
    float v = 0.0f;
    if (r0 + r < a.m && c0 + c < a.n)
      v = static_cast<float>(static_cast<double>(value<T>(g[(r0 + r) * a.ldg + c0 + c])) * s);
    if (tall) sh[c][r] = v;
    else sh[r][c] = v;
  }
  __syncthreads();
  _Float16* xr = a.xr + b * a.x_elems;
  _Float16* xc = a.xc[0] + b * a.x_elems;
  for (int t = threadIdx.x; t < kRegion / 8; t += 256) {
    const int r = t >> 3, c = (t & 7) * 8;
    h8 u, v;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      u[e] = static_cast<_Float16>(sh[r][c + e] * kSX);
      v[e] = static_cast<_Float16>(sh[c + e][r] * kSX);
    }
    *reinterpret_cast<h8*>(xr + (i0 + r) * a.qp + j0 + c) = u;
    *reinterpret_cast<h8*>(xc + (j0 + r) * a.pp + i0 + c) = v;
  }
  float* xf = a.xf + b * a.x_elems + ((j0 / 64) * (a.pp / 64) + i0 / 64) * kRegion;
  for (int t = threadIdx.x; t < kRegion / 4; t += 256) {
    const int lane = t & 63, gq = (t >> 6) & 3, bj = (t >> 8) & 1, bi = t >> 9;
    const int m = 32 * bi + (lane & 31), n = 32 * bj + 8 * gq + 4 * (lane >> 5);
    *reinterpret_cast<f4*>(xf + region_offset(bi, bj, gq, lane)) = f4{sh[n][m], sh[n + 1][m], sh[n + 2][m], sh[n + 3][m]};
  }
}

// ------------------------------------------------------------------------------ A = X X^T
// Lower tiles; K split over blockIdx.z, whose partial tiles go out as 64x64 regions.
template <int T, int W, int NST>
__global__ __launch_bounds__(256) void ns_gram_kernel(NsArgs a, int steps_per_split) {
  using G = Tile<T, T, W, W, NST>;
  __shared__ __align__(16) uint8_t b0[G::kStage], b1[G::kStage], b2[NST == 3 ? G::kStage : 16];
  int ti, tj;
  triangle(blockIdx.x, ti, tj);
  const int b = blockIdx.y, split = blockIdx.z;
  const _Float16* x = a.xr + b * a.x_elems;
  const int all = static_cast<int>(a.qp / kBK), s0 = split * steps_per_split;
  typename G::Acc acc;
  G::zero(acc);
  G::run(x + static_cast<int64_t>(ti) * T * a.qp, a.qp, x + static_cast<int64_t>(tj) * T * a.qp, a.qp, s0 * kBK,
         min(steps_per_split, all - s0), b0, b1, b2, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* out = a.part + ((static_cast<int64_t>(b) * gridDim.x + blockIdx.x) * gridDim.z + split) * (T * T);
  // a wave's W x W part: a whole region, or one block of the tile's only region
#pragma unroll
  for (int i = 0; i < G::TM; ++i)
#pragma unroll
    for (int j = 0; j < G::TN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int at = W == 64 ? wave * kRegion + region_offset(i, j, g, lane) : region_offset(wave >> 1, wave & 1, g, lane);
        *reinterpret_cast<f4*>(out + at) = f4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
      }
}

// Sums the splits of one 64x64 region in order, and writes A' (both triangles) and the diagonal.
template <int T>
__global__ __launch_bounds__(256) void ns_gram_sum_kernel(NsArgs a, int splits) {
  constexpr int PITCH = 72, kPer = (T / 64) * (T / 64);
  __shared__ _Float16 sh[64 * PITCH];
  const int b = blockIdx.y, tile = blockIdx.x / kPer, reg = blockIdx.x % kPer;
  int ti, tj;
  triangle(tile, ti, tj);
  const int64_t r0 = ti * T + (reg / (T / 64)) * 64, c0 = tj * T + (reg % (T / 64)) * 64;
  if (c0 > r0) return;  // in a tile on the diagonal: the mirror image of another region
  const int tiles = gridDim.x / kPer;
  const float* in = a.part + ((static_cast<int64_t>(b) * tiles + tile) * splits) * (T * T) + reg * kRegion;
  float* d = a.da + b * a.pp;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int t = threadIdx.x + 256 * u;
    const int lane = t & 63, g = (t >> 6) & 3, bj = (t >> 8) & 1, bi = t >> 9;
    f4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < splits; ++k) s += *reinterpret_cast<const f4*>(in + static_cast<int64_t>(k) * (T * T) + t * 4);
    const int m = 32 * bi + (lane & 31), n = 32 * bj + 8 * g + 4 * (lane >> 5);
    h4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool on = r0 + m == c0 + n + e;
      if (on) d[r0 + m] = s[e] * (1.0f / (kSX * kSX));
      v[e] = on ? static_cast<_Float16>(0.0f) : static_cast<_Float16>(s[e] * (kSA / (kSX * kSX)));
    }
    *reinterpret_cast<h4*>(sh + m * PITCH + n) = v;
  }
  __syncthreads();
  write_symmetric<64, 256>(sh, a.a16 + static_cast<int64_t>(b) * a.pp * a.pp, a.pp, r0, c0);
}

// ------------------------------------------------------------------------------ B = b A + c A A
template <int T, int W, int NST>
__global__ __launch_bounds__(256) void ns_poly_kernel(NsArgs a, float cb, float cc) {
  using G = Tile<T, T, W, W, NST>;
  __shared__ __align__(16) uint8_t b0[G::kStage], b1[G::kStage], b2[NST == 3 ? G::kStage : 16];
  __shared__ _Float16 sh[T * (T + 8)];
  int ti, tj;
  triangle(blockIdx.x, ti, tj);
  const int b = blockIdx.y;
  const int64_t r0 = static_cast<int64_t>(ti) * T, c0 = static_cast<int64_t>(tj) * T;
  const _Float16* A = a.a16 + static_cast<int64_t>(b) * a.pp * a.pp;
  typename G::Acc acc;
  G::zero(acc);
  G::run(A + r0 * a.pp, a.pp, A + c0 * a.pp, a.pp, 0, static_cast<int>(a.pp / kBK), b0, b1, b2, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / (T / W), wn = wave % (T / W);
  const float* d = a.da + b * a.pp;
#pragma unroll
  for (int i = 0; i < G::TM; ++i) {
    const int m = wm * W + 32 * i + (lane & 31);
    const float dm = d[r0 + m];
#pragma unroll
    for (int j = 0; j < G::TN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = wn * W + 32 * j + 8 * g + 4 * (lane >> 5);
        const f4 dn = *reinterpret_cast<const f4*>(d + c0 + n);
        const h4 av = *reinterpret_cast<const h4*>(A + (r0 + m) * a.pp + c0 + n);
        h4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float aa = acc[i][j][4 * g + e] * (1.0f / (kSA * kSA));
          const float x = static_cast<float>(av[e]) * (1.0f / kSA);
          if (r0 + m == c0 + n + e) {
            a.db[b * a.pp + r0 + m] = cb * dm + cc * (aa + dm * dm);
            v[e] = static_cast<_Float16>(0.0f);
          } else {
            v[e] = static_cast<_Float16>((cb * x + cc * (aa + (dm + dn[e]) * x)) * kSB);
          }
        }
        *reinterpret_cast<h4*>(sh + m * (T + 8) + n) = v;
      }
  }
  __syncthreads();
  write_symmetric<T, 256>(sh, a.b16 + static_cast<int64_t>(b) * a.pp * a.pp, a.pp, r0, c0);
}

// ------------------------------------------------------------------------------ X <- a X + B X
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }

// The first n of 8 BF16 patterns (held as FP16 bits) to a row of any alignment.
typedef uint32_t u4_a2 __attribute__((ext_vector_type(4), aligned(2)));
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

template <int BM, int BN, int W, int NST, bool LAST>
__global__ __launch_bounds__(64 * (BM / W) * (BN / W)) void ns_update_kernel(NsArgs a, float ca, int turn) {
  const float own_from = kOwnRow * __builtin_fabsf(ca - 1.0f);
  using G = Tile<BM, BN, W, W, NST>;
  constexpr int PITCH = BN + 8;
  __shared__ __align__(16) uint8_t b0[G::kStage], b1[G::kStage], b2[NST == 3 ? G::kStage : 16];
  __shared__ _Float16 sh[BM * PITCH];
  const int b = blockIdx.y;
  const int tiles_p = static_cast<int>(a.pp / BN);
  int bid = blockIdx.x;
  {
    // workgroup ids are dealt over the 8 XCDs in turn: give each XCD consecutive tiles
    const int nb = gridDim.x, xcd = bid & 7, q = nb >> 3, rem = nb & 7;
    bid = xcd * q + min(xcd, rem) + (bid >> 3);
  }
  const int64_t j0 = static_cast<int64_t>(bid / tiles_p) * BM, i0 = static_cast<int64_t>(bid % tiles_p) * BN;
  const _Float16* xc = a.xc[turn] + b * a.x_elems;
  const _Float16* B = a.b16 + static_cast<int64_t>(b) * a.pp * a.pp;
  typename G::Acc acc;
  G::zero(acc);
  G::run(xc + j0 * a.pp, a.pp, B + i0 * a.pp, a.pp, 0, static_cast<int>(a.pp / kBK), b0, b1, b2, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / (BN / W), wn = wave % (BN / W);
  const float* d = a.db + b * a.pp;
#pragma unroll
  for (int i = 0; i < G::TM; ++i) {
    const int m = wm * W + 32 * i;  // j0 + m + lane % 32
#pragma unroll
    for (int j = 0; j < G::TN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = wn * W + 32 * j;
        const int64_t region = ((j0 + m) / 64) * (a.pp / 64) + (i0 + n) / 64;
        float* xf = a.xf + b * a.x_elems + region * kRegion + region_offset((m >> 5) & 1, (n >> 5) & 1, g, lane);
        const int nn = n + 8 * g + 4 * (lane >> 5);
        const f4 dn = *reinterpret_cast<const f4*>(d + i0 + nn);
        f4 x = *reinterpret_cast<const f4*>(xf);
        h4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float low = static_cast<float>(static_cast<_Float16>(x[e] * kSX)) * (1.0f / kSX);
          const float xd = __builtin_fabsf(dn[e]) > own_from ? x[e] : low;
          x[e] = ca * x[e] + (dn[e] * xd + acc[i][j][4 * g + e] * (1.0f / (kSX * kSB)));
          if (LAST) v[e] = __builtin_bit_cast(_Float16, bf16_bits(x[e]));
          else v[e] = static_cast<_Float16>(x[e] * kSX);
        }
        if (!LAST) *reinterpret_cast<f4*>(xf) = x;
        *reinterpret_cast<h4*>(sh + (m + (lane & 31)) * PITCH + nn) = v;
      }
  }
  __syncthreads();
  const bool tall = a.m > a.n;
  _Float16* next = a.xc[turn ^ 1] + b * a.x_elems;
  _Float16* xr = a.xr + b * a.x_elems;
  uint16_t* out = a.out + b * a.stride_o;
  if (!LAST || tall) {
    for (int c = threadIdx.x; c < BM * BN / 8; c += G::kThreads) {
      const int row = c / (BN / 8), col = (c % (BN / 8)) * 8;
      const h8 v = *reinterpret_cast<const h8*>(sh + row * PITCH + col);
      if (!LAST) {
        *reinterpret_cast<h8*>(next + (j0 + row) * a.pp + i0 + col) = v;
      } else if (j0 + row < a.m) {
        store_row(out + (j0 + row) * a.ldo + i0 + col, v, a.n - (i0 + col));
      }
    }
  }
  if (!LAST || !tall) {
    for (int c = threadIdx.x; c < BM * BN / 8; c += G::kThreads) {
      const int row = c / (BM / 8), col = (c % (BM / 8)) * 8;  // row of X, columns of X
      h8 v;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = sh[(col + e) * PITCH + row];
      if (!LAST) {
        *reinterpret_cast<h8*>(xr + (i0 + row) * a.qp + j0 + col) = v;
      } else if (i0 + row < a.m) {
        store_row(out + (i0 + row) * a.ldo + j0 + col, v, a.n - (j0 + col));
      }
    }
  }
}

// ------------------------------------------------------------------------------ small matrices
// One matrix of at most P x (NS P) per workgroup, all steps in one launch: (P/32)^2 waves hold one
// 32x32 block of every P x P slab of X^T in registers (FP32); the products' operands go through LDS.
// The slabs enter X X^T and B X as FP16 pairs (value and remainder), A' and B' as FP16.
template <int P, int NS, typename T>
__global__ __launch_bounds__((P / 32) * (P / 32) * 64) void ns_small_kernel(NsArgs a, NsCoef coef, int steps) {
  constexpr int NB = P / 32, PITCH = P + 8;  // 16 rows' 16-byte reads of one column fall into different banks
  __shared__ __align__(16) _Float16 zh[P * PITCH], zl[P * PITCH], ab[P * PITCH];
  __shared__ float da[P], db[P];
  __shared__ double red[NB * NB];
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int bi = wave / NB, bj = wave % NB;
  const bool tall = a.m > a.n;
  const int p = static_cast<int>(tall ? a.n : a.m), q = static_cast<int>(tall ? a.m : a.n);
  const T* g = static_cast<const T*>(a.g) + blockIdx.x * a.stride_g;
  const int m = 32 * bi + l32, n0 = 32 * bj + 4 * half;  // register 4 g + e: X^T[m][n0 + 8 g + e] of a slab

  float z[NS][16];
  double sum = 0.0;
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = n0 + 8 * (r >> 2) + (r & 3), j = s * P + m;
      float v = 0.0f;
      if (i < p && j < q) v = value<T>(tall ? g[j * a.ldg + i] : g[i * a.ldg + j]);
      z[s][r] = v;
      sum = __builtin_fma(static_cast<double>(v), static_cast<double>(v), sum);
    }
  sum = block_sum(sum, red);
  const double scale = sum <= 1e300 ? 1.0 / (__builtin_sqrt(sum) + static_cast<double>(a.eps)) : __builtin_nan("");
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    // zeros outside the matrix stay zero, or turn NaN with every element inside it
    for (int r = 0; r < 16; ++r) z[s][r] = static_cast<float>(static_cast<double>(z[s][r]) * scale);

  auto frag = [&](const _Float16* mat, int row0, int k) {
    return *reinterpret_cast<const h8*>(mat + (row0 + l32) * PITCH + 16 * k + 8 * half);
  };
  for (int step = 0; step < steps; ++step) {
    const float ca = coef.v[step][0], cb = coef.v[step][1], cc = coef.v[step][2];
    f16v acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (s * P >= q) continue;  // uniform
      if (s) __syncthreads();
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int i = n0 + 8 * (r >> 2) + (r & 3);
        const float v = z[s][r] * kSX;
        const _Float16 h = static_cast<_Float16>(v);
        zh[i * PITCH + m] = h;
        zl[i * PITCH + m] = static_cast<_Float16>(v - static_cast<float>(h));
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < P / 16; ++k) {
        const h8 ih = frag(zh, 32 * bi, k), il = frag(zl, 32 * bi, k), jh = frag(zh, 32 * bj, k), jl = frag(zl, 32 * bj, k);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(jl, ih, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(jh, il, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(jh, ih, acc, 0, 0, 0);
      }
    }
    float x[16];  // A' as its FP16 values
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      h4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool on = m == n0 + 2 * r + e;
        if (on) da[m] = acc[r + e] * (1.0f / (kSX * kSX));
        v[e] = on ? static_cast<_Float16>(0.0f) : static_cast<_Float16>(acc[r + e] * (kSA / (kSX * kSX)));
        x[r + e] = static_cast<float>(v[e]) * (1.0f / kSA);
      }
      *reinterpret_cast<h4*>(ab + m * PITCH + n0 + 2 * r) = v;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
#pragma unroll
    for (int k = 0; k < P / 16; ++k)
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(frag(ab, 32 * bj, k), frag(ab, 32 * bi, k), acc, 0, 0, 0);
    __syncthreads();  // A' has been read: B' takes its place
    const float dm = da[m];
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      h4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = n0 + 2 * r + e;
        const float aa = acc[r + e] * (1.0f / (kSA * kSA));
        const float b = m == n ? 0.0f : cb * x[r + e] + cc * (aa + (dm + da[n]) * x[r + e]);
        if (m == n) db[m] = cb * dm + cc * (aa + dm * dm);
        v[e] = static_cast<_Float16>(b * kSB);
      }
      *reinterpret_cast<h4*>(ab + m * PITCH + n0 + 2 * r) = v;
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (s * P >= q) continue;
      if (s) __syncthreads();
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        h4 h, l;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = z[s][r + e] * kSX;
          h[e] = static_cast<_Float16>(v);
          l[e] = static_cast<_Float16>(v - static_cast<float>(h[e]));
        }
        *reinterpret_cast<h4*>(zh + m * PITCH + n0 + 2 * r) = h;
        *reinterpret_cast<h4*>(zl + m * PITCH + n0 + 2 * r) = l;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
#pragma unroll
      for (int k = 0; k < P / 16; ++k) {
        const h8 b = frag(ab, 32 * bj, k);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, frag(zl, 32 * bi, k), acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, frag(zh, 32 * bi, k), acc, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r)
        z[s][r] = (ca + db[n0 + 8 * (r >> 2) + (r & 3)]) * z[s][r] + acc[r] * (1.0f / (kSX * kSB));
    }
    __syncthreads();  // the last slab and B' have been read
  }
  uint16_t* out = a.out + blockIdx.x * a.stride_o;
  int pe = p, qe = q;
  asm volatile("" : "+s"(pe), "+s"(qe));  // the comparisons are made again, not kept from the loads
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = n0 + 8 * (r >> 2) + (r & 3), j = s * P + m;
      if (i < pe && j < qe) out[tall ? j * a.ldo + i : i * a.ldo + j] = bf16_bits(z[s][r]);
    }
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// How a size is run: tile edges of the three products and the splits of A's.
struct Plan {
  int64_t pp, qp;
  int gram_tile, gram_splits, gram_steps, poly_tile, update_tile;
  int64_t gram_tiles() const { return tri(gram_tile); }
  int64_t tri(int t) const { return (pp / t) * (pp / t + 1) / 2; }
};

Plan plan_of(int64_t batch, int64_t m, int64_t n) {
  Plan p;
  p.pp = round_up(m < n ? m : n, 128);
  p.qp = round_up(m < n ? n : m, 128);
  p.update_tile = batch * (p.pp / 128) * (p.qp / 128) >= 256 ? 128 : 64;
  p.poly_tile = batch * p.tri(128) >= 256 ? 128 : 64;
  const int64_t steps = p.qp / kBK;
  p.gram_tile = batch * p.tri(128) >= 64 ? 128 : 64;
  int64_t splits = 512 / (batch * p.tri(p.gram_tile));
  splits = splits < 1 ? 1 : splits;
  if (splits > steps / 4) splits = steps / 4 < 1 ? 1 : steps / 4;
  p.gram_steps = static_cast<int>((steps + splits - 1) / splits);
  p.gram_splits = static_cast<int>((steps + p.gram_steps - 1) / p.gram_steps);
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
    if (q <= 64) return go(ns_small_kernel<64, 1, T>, 256);
    if (q <= 128) return go(ns_small_kernel<64, 2, T>, 256);
    if (q <= 256) return go(ns_small_kernel<64, 4, T>, 256);
    return go(ns_small_kernel<64, 8, T>, 256);
  }
  if (q <= 128) return go(ns_small_kernel<128, 1, T>, 1024);
  return go(ns_small_kernel<128, 2, T>, 1024);
}

int64_t align256(int64_t v) { return round_up(v, 256); }

}  // namespace

// Workspace parts, in order: FP32 X, two Xc, Xr, A, B, their diagonals, A's partial tiles, norms.
static int64_t ns_layout(int64_t batch, const Plan& p, NsArgs* a, uint8_t* base) {
  const int64_t x = p.pp * p.qp, s = p.pp * p.pp;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* r = base + at;
    at += align256(bytes);
    return r;
  };
  uint8_t* xf = take(batch * x * 4);
  uint8_t* xc0 = take(batch * x * 2);
  uint8_t* xc1 = take(batch * x * 2);
  uint8_t* xr = take(batch * x * 2);
  uint8_t* a16 = take(batch * s * 2);
  uint8_t* b16 = take(batch * s * 2);
  uint8_t* da = take(batch * p.pp * 4);
  uint8_t* db = take(batch * p.pp * 4);
  uint8_t* part = take(batch * p.gram_tiles() * p.gram_splits * p.gram_tile * p.gram_tile * 4);
  uint8_t* norm = take(batch * kNormBlocks * 8);
  if (a) {
    a->pp = p.pp, a->qp = p.qp, a->x_elems = x;
    a->xf = reinterpret_cast<float*>(xf);
    a->xc[0] = reinterpret_cast<_Float16*>(xc0), a->xc[1] = reinterpret_cast<_Float16*>(xc1);
    a->xr = reinterpret_cast<_Float16*>(xr);
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
    for (int s = 0; s < steps; ++s)
      for (int k = 0; k < 3; ++k) c.v[s][k] = coef[3 * s + k];
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
    const float ca = coef[3 * s], cb = coef[3 * s + 1], cc = coef[3 * s + 2];
    const dim3 gg(static_cast<uint32_t>(p.gram_tiles()), nb, static_cast<uint32_t>(p.gram_splits));
    if (p.gram_tile == 128) {
      hipLaunchKernelGGL((ns_gram_kernel<128, 64, 2>), gg, dim3(256), 0, stream, a, p.gram_steps);
      hipLaunchKernelGGL((ns_gram_sum_kernel<128>), dim3(gg.x * 4, nb), dim3(256), 0, stream, a, p.gram_splits);
    } else {
      hipLaunchKernelGGL((ns_gram_kernel<64, 32, 3>), gg, dim3(256), 0, stream, a, p.gram_steps);
      hipLaunchKernelGGL((ns_gram_sum_kernel<64>), dim3(gg.x, nb), dim3(256), 0, stream, a, p.gram_splits);
    }
    const dim3 pg(static_cast<uint32_t>(p.tri(p.poly_tile)), nb);
    if (p.poly_tile == 128) hipLaunchKernelGGL((ns_poly_kernel<128, 64, 2>), pg, dim3(256), 0, stream, a, cb, cc);
    else hipLaunchKernelGGL((ns_poly_kernel<64, 32, 3>), pg, dim3(256), 0, stream, a, cb, cc);
    const int64_t t = p.update_tile;
    const dim3 ug(static_cast<uint32_t>((p.qp / t) * (p.pp / t)), nb);
    const int turn = s & 1;
    if (t == 128) {
      if (s + 1 < steps) hipLaunchKernelGGL((ns_update_kernel<128, 128, 64, 2, false>), ug, dim3(256), 0, stream, a, ca, turn);
      else hipLaunchKernelGGL((ns_update_kernel<128, 128, 64, 2, true>), ug, dim3(256), 0, stream, a, ca, turn);
    } else {
      if (s + 1 < steps) hipLaunchKernelGGL((ns_update_kernel<64, 64, 32, 3, false>), ug, dim3(256), 0, stream, a, ca, turn);
      else hipLaunchKernelGGL((ns_update_kernel<64, 64, 32, 3, true>), ug, dim3(256), 0, stream, a, ca, turn);
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace pf8
