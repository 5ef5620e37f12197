// The tile kernel of the block-scaled FP8 product with bias, activation and residual in its epilogue
// (gfx950 / CDNA4 only), and its launcher for one tile shape. Formulas in include/pf8_layer.h.
#pragma once

#include "act_device.h"
#include "gemm_device.h"
#include "pf8_layer_launch.h"
#include "row_device.h"

namespace pf8 {

namespace {

// What a tile kernel is built for: activations that share their instructions.
enum ActClass { kIdentity, kPiecewise, kSigmoid, kNormal };
template <ActClass C>
struct TileAct {
  bool square;
  float c1, c3;
  __device__ __forceinline__ explicit TileAct(int act)
      : square(act == PF8_ACT_RELU2),
        // the sigmoid's argument z (c1 + c3 z^2), times -log2 e
        c1(-1.44269504088896341f * (act == PF8_ACT_SILU ? 1.0f : 2.0f * kTanhScale)),
        c3(act == PF8_ACT_SILU ? 0.0f : -1.44269504088896341f * 2.0f * kTanhScale * kTanhCube) {}
  __device__ __forceinline__ float operator()(float z) const {
    if constexpr (C == kPiecewise) {
      const float y = z <= 0.0f ? 0.0f : z;
      return square ? y * y : y;
    } else if constexpr (C == kIdentity) {
      return z;
    } else if constexpr (C == kSigmoid) {
      // Far out the cube overflows to an infinity of z's sign, and the sigmoid is 0 or 1; the square stays finite, as
      // c3 may be 0.
      const float z2 = fminf(z * z, 3.0e38f);
      return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * __builtin_fmaf(c3, z2, c1)));
    } else {
      return act_value<PF8_ACT_GELU>(z);
    }
  }
};

// Accesses of the staging buffer: inline asm, as in gemm_device.h and for its reason.
__device__ __forceinline__ void stg_write16(uint32_t addr, v4i v) {
  asm volatile("ds_write_b128 %0, %1" : : "v"(addr), "v"(v) : "memory");
}
template <int N>
__device__ __forceinline__ void stg_read16(const uint32_t (&addr)[N], v4i (&v)[N]) {
  if constexpr (N == 8) {
    stg_read8x16(addr, v);
  } else if constexpr (N == 4) {
    asm volatile(
        "ds_read_b128 %0, %4\n"
        "ds_read_b128 %1, %5\n"
        "ds_read_b128 %2, %6\n"
        "ds_read_b128 %3, %7\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(addr[0]), "v"(addr[1]), "v"(addr[2]), "v"(addr[3])
        : "memory");
  } else if constexpr (N == 2) {
    asm volatile(
        "ds_read_b128 %0, %2\n"
        "ds_read_b128 %1, %3\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1])
        : "v"(addr[0]), "v"(addr[1])
        : "memory");
  } else {
    static_assert(N == 1, "1, 2, 4 or 8 chunks");
    asm volatile(
        "ds_read_b128 %0, %1\n"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0])
        : "v"(addr[0])
        : "memory");
  }
}
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void stg_read2x8(uint32_t a0, uint32_t a1, v2u& v0, v2u& v1) {
  asm volatile(
      "ds_read_b64 %0, %2\n"
      "ds_read_b64 %1, %3\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(v0), "=&v"(v1)
      : "v"(a0), "v"(a1)
      : "memory");
}

// Workgroups that a CU holds at once: by their LDS (160 KB), four stages of (BM + BN) x 64 bytes and the slab.
template <int BM, int BN>
constexpr int kTilesPerCu = 160 * 1024 / (4 * (BM + BN) * 64 + 128 * BN);

// The persistent pipeline of gemm_mx_persistent_kernel (the ring of stage buffers that runs on across
// tiles, the explicit waits, the order of tiles and of K) with four differences:
//  * Any sizes: row offsets are in the lanes' offsets, so that the buffer range check turns rows past the edge into
//    zeros (a variant for whole tiles alone was no faster: 8192 x 12288 x 2048 gated 178 against 178 us); K blocks past
//    the end, up to whole bodies of four stages and two bodies, are fetched through a buffer of no size and count as
//    zeros too.
//  * GATED: a tile of BN rows of W is, for each of the two waves of columns, BN / 4 rows that make the gate and the
//    BN / 4 that make what it multiplies, so that a lane holds both values of a column of d.
//  * The epilogue works on the accumulators where they are: bias, rounded z, activation and gate, residual. Every
//    bf16 slab of 64 rows passes through the staging buffer, out (and the residual in) by whole rows.
//  * All workgroups start together: with half of them a third of a tile late, 8192 x 12288 x 2048 gated with z took 199 us
//    instead of 196, without z 179 instead of 174.
// Bound: matrix instructions at the clock that the power allows, and at 256 x 256 the epilogue, which nothing hides: one
// tile's accumulators fill a CU's registers, so the matrix cores wait while its results leave. 8192 x 12288 x 2048 gated:
// 196 us (2.1 PFLOP/s), without z (0.2 GB less to write) 174; the plain product of that size 165. 8192 x 2048 x 6144
// with bias, onto a residual: 89 us (2.3 PFLOP/s) on the same operands again, 102 on operands from memory; the plain
// product 83. Those are one box's; others took up to 206 and 92.
// At 256 x 256 102 to 156 scalar registers are kept in lanes of vector registers (in the plain product's kernel 53 to 70),
// hardly any of them over the K loop; no vector register is spilled.
template <int BM, int BN, bool GATED, bool RES, ActClass ACT>
__global__ __launch_bounds__(256, (kTilesPerCu<BM, BN>)) void fprop_act_tile_kernel(FpropActArgs p, int tiles_m, int tiles_n) {
  constexpr int BK = 64;
  constexpr int WM = BM / 2, WN = BN / 2, TM = WM / 32, TN = WN / 32;
  constexpr int A_ST = BM * BK, ST = (BM + BN) * BK;
  constexpr int A_DMA = BM / 64, B_DMA = BN / 64, D = A_DMA + B_DMA;
  constexpr int SB = GATED && TN > 1 ? 2 : 1;  // scales of W: a wave's rows of a part lie in one 128-row tile
  constexpr int SS = TM + SB;
  constexpr int OUT = GATED ? BN / 2 : BN;     // columns of d
  constexpr int RP = WN * 2, CH = WN / 8;      // a wave's staged row in bytes and 16-byte chunks
  constexpr int CHD = OUT / 16;                // chunks of its row of d
  constexpr int PER_D = 32 * CHD / 64;         // chunks of d per lane and slab
  __shared__ __align__(16) uint8_t buf0[ST];
  __shared__ __align__(16) uint8_t buf1[ST];
  __shared__ __align__(16) uint8_t buf2[ST];
  __shared__ __align__(16) uint8_t buf3[ST];
  __shared__ __align__(512) uint8_t stg[4 * 32 * RP];

  const int t0 = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(t0 >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int nsr = static_cast<int>(p.k / BK);                // stages with operands
  const int ns = max(8, (nsr + 3) & ~3);                     // and in all
  const int64_t cols = GATED ? p.n / 2 : p.n;                // of d

  // ---- this workgroup's tiles ----
  const int nb = tiles_m * tiles_n;
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, slots = gridDim.x >> 3;
  const int q = nb >> 3, rem = nb & 7;
  const int xcd_tiles = q + (xcd < rem ? 1 : 0), xcd_base = xcd * q + min(xcd, rem);
  const int ntiles = slot < xcd_tiles ? (xcd_tiles - slot + slots - 1) / slots : 0;
  if (ntiles == 0) return;
  auto tile_origin = [&](int r, int64_t& m0, int64_t& n0) {
    const int bid = xcd_base + slot + slots * r;
    constexpr int kGroupM = 4;  // (8192 x 2048 x 6144 90 us, with 8 92; 8192 x 12288 x 2048 the same)
    const int per_group = kGroupM * tiles_n;
    const int grp = bid / per_group;
    const int first_m = grp * kGroupM;
    const int gsize = min(tiles_m - first_m, kGroupM);
    const int in_grp = bid - grp * per_group;
    const int tm = __builtin_amdgcn_readfirstlane(first_m + in_grp % gsize);
    const int tn = __builtin_amdgcn_readfirstlane(in_grp / gsize);
    m0 = static_cast<int64_t>(tm) * BM;
    n0 = static_cast<int64_t>(tn) * OUT;
  };
  auto bufs = [&](int u) -> uint8_t* { return u == 0 ? buf0 : u == 1 ? buf1 : u == 2 ? buf2 : buf3; };

  // ---- lane offsets (recomputed per tile) ----
  int t = t0, lane = t0 & 63;
  int lda = static_cast<int>(p.lda), ldb = static_cast<int>(p.ldb);
  int voff_a = 0, voff_b = 0, l32 = 0, half = 0, fo0 = 0, fo1 = 0;
  auto refresh = [&]() {
    asm volatile("" : "+v"(t));
    asm volatile("" : "+s"(lda), "+s"(ldb));
    lane = t & 63;
    const int dma_row = lane >> 2;
    const int dma_chunk = (lane & 3) ^ ((dma_row >> 2) & 3);
    voff_a = dma_row * lda + dma_chunk * 16;
    voff_b = dma_row * ldb + dma_chunk * 16;
    l32 = lane & 31;
    half = lane >> 5;
    const int sw = (l32 >> 2) & 3;
    fo0 = l32 * BK + (((2 * half) ^ sw) << 4);
    fo1 = l32 * BK + (((2 * half + 1) ^ sw) << 4);
  };
  refresh();

  // ---- load state: the tile whose stages the refills fetch ----
  const uint8_t *src_a = nullptr, *src_b[2] = {nullptr, nullptr};
  int size_a = 0, size_b = 0;
  int64_t a_row[TM], b_row[SB];
  int load_rev = 0;  // odd tiles walk K from the end (serpentine)
  auto set_load_tile = [&](int r) {
    load_rev = r & 1;
    int64_t m0, n0;
    tile_origin(r, m0, n0);
    src_a = p.a + m0 * p.lda;
    // gated: 16-row slabs of W alternate between the parts by load (BN = 256) or by wave
    constexpr int PER = WN / 16;
    const int second = GATED && BN < 256 ? wave % PER / (PER > 1 ? PER / 2 : 1) : 0;
    src_b[0] = p.b + (n0 + (second ? cols : 0)) * p.ldb;
    src_b[1] = p.b + (n0 + (GATED ? cols : 0)) * p.ldb;
    size_a = static_cast<int>(min64(BM, p.m - m0)) * lda;
    size_b = static_cast<int>(min64(OUT, cols - n0)) * ldb;
#pragma unroll
    for (int i = 0; i < TM; ++i) a_row[i] = min64(m0 + wm * WM + 32 * i + l32, p.m - 1);
    if constexpr (GATED && TN == 1) {
      b_row[0] = min64(n0 + wn * 16 + (l32 & 15), cols - 1);
      if (l32 >= 16) b_row[0] += cols;
    } else {
      b_row[0] = min64(n0 + wn * (OUT / 2) + l32, cols - 1);
      if constexpr (SB == 2) b_row[1] = b_row[0] + cols;
    }
  };
  // scale registers: one set per even buffer (0 and 2); an odd stage reads the previous buffer's
  uint32_t sc_a[2][TM], sc_b[2][SB];
  auto load_scales = [&](int s, uint32_t (&sa)[TM], uint32_t (&sb)[SB]) {
    // the waits count exactly TM + SB loads here: opaque indices keep the compiler from merging
    // two of them or hoisting one above earlier loads (as in gemm_mx_kernel)
    const int64_t kb = (load_rev ? max(nsr - 1 - s, 0) : min(s, nsr - 1)) >> 1;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      int64_t idx = kb * p.ld_as + a_row[i];
      asm volatile("" : "+v"(idx));
      sa[i] = __float_as_uint(p.a_dscale[idx]);
    }
#pragma unroll
    for (int j = 0; j < SB; ++j) {
      int64_t idx = (b_row[j] >> 7) * p.ld_bs + kb;
      asm volatile("" : "+v"(idx));
      sb[j] = __float_as_uint(p.b_dscale[idx]);
    }
  };
  // loads of the load tile's stage s into buffer u = s mod 4: part 0 = the A operand, part 1 = the
  // scales (even stages) and the B operand
  auto issue_part = [&](auto u_c, int s, auto part_c) {
    constexpr int u = decltype(u_c)::value;
    constexpr int part = decltype(part_c)::value;
    uint8_t* buf = bufs(u);
    if constexpr (part == 1 && (u % 2 == 0)) load_scales(s, sc_a[u / 2], sc_b[u / 2]);
    const bool live = s < nsr;
    const int kofs = live ? (load_rev ? nsr - 1 - s : s) * BK : 0;
    if constexpr (part == 0) {
      const __amdgpu_buffer_rsrc_t rsrc =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(src_a), 0, live ? size_a : 0, kBufferFlags);
#pragma unroll
      for (int j = 0; j < A_DMA; ++j) {
        const int slab = wave + 4 * j;
        auto* dst = (__attribute__((address_space(3))) void*)(buf + slab * 16 * BK);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, dst, 16, voff_a + slab * 16 * lda, kofs, 0, 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < B_DMA; ++j) {
        const int slab = wave + 4 * j;
        // gated: of each wave of columns' slabs the first half makes the gate
        constexpr int PER = WN / 16;
        const int row = GATED ? slab / PER * (WN / 2) + slab % (PER > 1 ? PER / 2 : 1) * 16 : slab * 16;
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(GATED && BN == 256 ? src_b[j & 1] : src_b[0]), 0, live ? size_b : 0, kBufferFlags);
        auto* dst = (__attribute__((address_space(3))) void*)(buf + A_ST + slab * 16 * BK);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, dst, 16, voff_b + row * ldb, kofs, 0, 0);
      }
    }
  };
  using PA = std::integral_constant<int, 0>;
  using PB = std::integral_constant<int, 1>;

  // ---- operand fragments: set f = stage parity ----
  v8i fa[2][TM], fb[2][TN];
  auto read_frags = [&](const uint8_t* buf, v8i (&a)[TM], v8i (&b)[TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = lds_read32(buf, (wm * WM + 32 * i) * BK + fo0, (wm * WM + 32 * i) * BK + fo1);
#pragma unroll
    for (int j = 0; j < TN; ++j)
      b[j] = lds_read32(buf, A_ST + (wn * WN + 32 * j) * BK + fo0, A_ST + (wn * WN + 32 * j) * BK + fo1);
  };

  v16f acc[TM][TN];

#define PF8_WAIT_VM_LGKM0(n0)                                                                  \
  do {                                                                                         \
    constexpr int n_ = (n0) < 63 ? (n0) : 63;                                                  \
    __builtin_amdgcn_s_waitcnt((n_ & 0xF) | ((n_ >> 4) << 14) | (0x7 << 4) | (0x0 << 8));      \
  } while (0)

  // One stage at body position u (tile stage s with s mod 4 = u), as in gemm_mx_persistent_kernel:
  //  PREV: the first half sends the scales and B loads of load-tile stage ps (into buffer u - 1)
  //  REFILL: the second half sends the A loads of load-tile stage rs (into buffer u); EARLYB: and
  //          its B loads too (a tile's last stage; the next tile's first operands are read from LDS behind the
  //          epilogue, which needs their registers)
  //  SWITCH: before the refill the load tile becomes tile `next`
  //  ZERO: the tile's first stage: the MFMAs start from zero
  // The wait leaves in flight what was issued after stage s + 1: stages s + 2 and s + 3. In a tile's first stages the
  // previous tile's stores were issued later still; how many depends on the edges, and they are not counted.
  auto stage = [&](auto u_c, auto prev_c, int ps, auto refill_c, int rs, auto earlyb_c, auto switch_c, int next,
                   auto zero_c) {
    constexpr int u = decltype(u_c)::value;
    constexpr bool prev = decltype(prev_c)::value, refill = decltype(refill_c)::value;
    constexpr bool earlyb = decltype(earlyb_c)::value, sw_tile = decltype(switch_c)::value;
    constexpr bool zero = decltype(zero_c)::value;
    constexpr int f = u & 1, un = (u + 1) & 3, fn = un & 1;
    constexpr bool odd = (u & 1) != 0;
    constexpr int us = u / 2;  // this K block's scale registers (loaded with its even stage)
    int sae[TM], sbe[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      uint32_t v = sc_a[us][i];
      asm volatile("" : "+v"(v));
      sae[i] = static_cast<int>(v >> 23);
    }
    int sbv[SB];
#pragma unroll
    for (int j = 0; j < SB; ++j) {
      uint32_t v = sc_b[us][j];
      asm volatile("" : "+v"(v));
      sbv[j] = static_cast<int>(v >> 23);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) sbe[j] = SB == 2 && j >= TN / 2 ? sbv[SB - 1] : sbv[0];
    auto mfma_rows = [&](int i0, int i1) {
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (i < i0 || i >= i1) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const v16f c = zero ? v16f{} : acc[i][j];
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[f][j], fa[f][i], c, 0, 0, 0, sbe[j], 0, sae[i]);
        }
      }
    };
    // the stage PREV sends lives in buffer u - 1 and has the other parity
    if constexpr (prev) issue_part(std::integral_constant<int, (u + 3) & 3>{}, ps, PB{});
    mfma_rows(0, TM / 2);
    if constexpr (prev) interleave_groups<(TM / 2) * TN, B_DMA + (odd ? SS : 0), 0>();
    __builtin_amdgcn_sched_barrier(0);
    // (one of the two stages is even and carries scales)
    PF8_WAIT_VM_LGKM0(2 * D + SS);
    __builtin_amdgcn_s_barrier();
    if constexpr (sw_tile) set_load_tile(next);
    if constexpr (refill) issue_part(u_c, rs, PA{});
    if constexpr (earlyb) issue_part(u_c, rs, PB{});
    if constexpr (!earlyb) read_frags(bufs(un), fa[fn], fb[fn]);
    mfma_rows(TM / 2, TM);
    interleave_groups<(TM - TM / 2) * TN, (refill ? A_DMA : 0) + (earlyb ? B_DMA : 0), earlyb ? 0 : 2 * (TM + TN)>();
  };

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  using F = std::false_type;
  using T = std::true_type;

  // ---- prologue: tile 0's stages 0..3 ----
  set_load_tile(0);
  issue_part(I0{}, 0, PA{});
  issue_part(I0{}, 0, PB{});
  __builtin_amdgcn_sched_barrier(0);
  issue_part(I1{}, 1, PA{});
  issue_part(I1{}, 1, PB{});
  __builtin_amdgcn_sched_barrier(0);
  issue_part(I2{}, 2, PA{});
  issue_part(I2{}, 2, PB{});
  __builtin_amdgcn_sched_barrier(0);
  issue_part(I3{}, 3, PA{});
  issue_part(I3{}, 3, PB{});
  __builtin_amdgcn_sched_barrier(0);
  PF8_WAIT_VM_LGKM0(D + (D + SS) + D);  // after stage 0: stages 1, 2 and 3
  __builtin_amdgcn_s_barrier();
  read_frags(buf0, fa[0], fb[0]);

  // tile 0's first body (no stores before it)
  stage(I0{}, F{}, 0, T{}, 4, F{}, F{}, 0, T{});
  stage(I1{}, T{}, 4, T{}, 5, F{}, F{}, 0, F{});
  stage(I2{}, T{}, 5, T{}, 6, F{}, F{}, 0, F{});
  stage(I3{}, T{}, 6, T{}, 7, F{}, F{}, 0, F{});
  for (int r = 0;; ++r) {
    refresh();
    int s = 4;
    for (; s < ns - 4; s += 4) {
      stage(I0{}, T{}, s + 3, T{}, s + 4, F{}, F{}, 0, F{});
      stage(I1{}, T{}, s + 4, T{}, s + 5, F{}, F{}, 0, F{});
      stage(I2{}, T{}, s + 5, T{}, s + 6, F{}, F{}, 0, F{});
      stage(I3{}, T{}, s + 6, T{}, s + 7, F{}, F{}, 0, F{});
    }
    // the bias of the rows of W that this lane holds, on its way during the last body (half a wave's: see below)
    int64_t m0, n0;
    tile_origin(r, m0, n0);
    float bias[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      bias[j] = 0.0f;
      if (p.bias && half == 0) {
        const int second = !GATED ? 0 : TN > 1 ? (j >= TN / 2 ? 1 : 0) : l32 >> 4;
        const int64_t c = n0 + wn * (OUT / 2) + (!GATED ? 32 * j + l32 : TN > 1 ? 32 * (j % (TN / 2 ? TN / 2 : 1)) + l32 : l32 & 15);
        if (c < cols) bias[j] = bias_at(p, second * cols + c);
      }
    }
    // The thread's number, opaque: places in the epilogue are made from it there, not kept in registers over the K loop.
    int te = t;
    asm volatile("" : "+v"(te));
    // ---- the residual's rows of a slab, by whole rows as d's; the first slab's are on their way during the last body ----
    const int rows = static_cast<int>(min64(BM, p.m - m0));
    const int first = wn * (OUT / 2);                                  // the wave's first column of d in the tile
    const int left = static_cast<int>(min64(OUT, cols - n0)) - first;  // and its columns from there on
    // byte offset, in the tile's rows of an array of pitch ld, of a lane's first row; and of chunk `it` from there
    auto row_offset = [&](int n, int ld2) { return (wm * WM + te % 64 / n) * ld2; };
    auto step_offset = [&](int n, int i, int it, int ld2) { return (64 / n * it + 32 * i) * ld2; };
    v4i res[RES ? PER_D : 1];
    auto load_residual = [&](int i) {
      const int ld2 = static_cast<int>(p.ldr * 2), c = 8 * (te % CHD), room = left - c;
      const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(p.residual) + m0 * p.ldr + n0, 0, rows * ld2, kBufferFlags);
      const int vo = row_offset(CHD, ld2) + 2 * (first + c);
      if (room >= 8) {
#pragma unroll
        for (int it = 0; it < PER_D; ++it)
          res[it] = __builtin_bit_cast(
              v4i, __builtin_amdgcn_raw_buffer_load_b128(rsrc, vo + step_offset(CHD, i, it, ld2), 0, 0));
      } else {
#pragma unroll
        for (int it = 0; it < PER_D; ++it) {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (e < room)
              w[e / 2] |= static_cast<uint32_t>(static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(
                              rsrc, vo + step_offset(CHD, i, it, ld2) + 2 * e, 0, 0))) << (16 * (e % 2));
          res[it] = v4i{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3])};
        }
      }
    };
    if constexpr (RES) load_residual(0);
    // last body: its refills fetch the next tile's stages 0..3
    const int next = r + 1 < ntiles ? r + 1 : r;
    stage(I0{}, T{}, s + 3, T{}, 0, F{}, T{}, next, F{});
    stage(I1{}, T{}, 0, T{}, 1, F{}, F{}, 0, F{});
    stage(I2{}, T{}, 1, T{}, 2, F{}, F{}, 0, F{});
    stage(I3{}, T{}, 2, T{}, 3, T{}, F{}, 0, F{});

    // ---- epilogue ----
    // The bias is a product of rank one with a row of ones, which leaves it in the accumulators' layout: one
    // v_mfma_f32_32x32x2_f32 a block (K = 2: the lower half wave holds bias and one, the upper half zeros), exact
    // but for the addition. (Through registers it took 64 of them a lane, and spills.)
    if (p.bias) {
      const float one = half == 0 ? 1.0f : 0.0f;
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(bias[j], one, acc[i][j], 0, 0, 0);
    }
    // The accumulators stay where the matrix instructions leave them until a slab takes its own: without this the
    // compiler moves the last body's matrix instructions behind the epilogue's branches, to the slab that uses each, or
    // copies several slabs at once, and spills what it has no registers for.
    auto pin = [&](int i) {
#pragma unroll
      for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(acc[i][j]));
    };
#pragma unroll
    for (int i = 0; i < TM; ++i) pin(i);
    // A lane's accumulator acc[i][j] holds, of row wm WM + 32 i + l32, the 4 columns 8 q4 + 4 half .. +3 of
    // block j for each q4. Gated, the first half of a wave's columns makes the gate. part: which half;
    // place: 8-column chunk of d's tile (less the wave's own offset).
    auto part = [](int j, int q4) { return !GATED ? 0 : TN > 1 ? (j >= TN / 2 ? 1 : 0) : q4 >> 1; };
    auto place = [](int j, int q4) { return !GATED ? 4 * j + q4 : TN > 1 ? 4 * (j % (TN / 2 ? TN / 2 : 1)) + q4 : q4 & 1; };
    // nothing of what follows is computed ahead, for which there are no registers
    auto fence = [&]() { __builtin_amdgcn_sched_barrier(0); };
    const TileAct<ACT> act(p.act);
    // Staging, each wave in a quarter of its own, so that no wave waits for another (LDS accesses of a wave keep their
    // order): slab i's row wm WM + 32 i + r is row r; its chunk c lies at chunk c ^ key(r), which spreads 16 rows over all
    // banks. With a 512-byte aligned buffer a lane's address is one XOR of the chunk's constant bits.
    auto key = [](int r) { return r / (16 / CH) & (CH - 1); };
    const uint32_t base_w = lds_addr(stg) + wave * 32 * RP;
    const uint32_t wbase = (base_w + te % 32 * RP + 8 * (te / 32 % 2)) | (key(te % 32) << 4);
    // Whole rows: lane l takes chunk l mod N of rows l / N + 64 / N it.
    auto row_chunks = [&](auto n_c, uint32_t (&addr)[32 * decltype(n_c)::value / 64]) {
      constexpr int N = decltype(n_c)::value;
#pragma unroll
      for (int it = 0; it < 32 * N / 64; ++it) {
        const int row = te % 64 / N + 64 / N * it;
        addr[it] = base_w + row * RP + ((te % N ^ key(row)) << 4);
      }
    };
    // stores of a thread's chunks of N to an array from its tile's first element on; c: the chunk's first column
    // there, room: the columns left from it. Non-temporal: with d cached 8192 x 12288 x 2048 gated takes 193 us instead of 178,
    // with the quantiser that reads d after it 224 instead of 212 (d of 33 MB, all one round of tiles: 4 us the other way)
    auto store_rows = [&](auto n_c, uint16_t* base, int64_t ld, int c, int room, int i) {
      constexpr int N = decltype(n_c)::value, PER = 32 * N / 64;
      uint32_t addr[PER];
      v4i v[PER];
      row_chunks(n_c, addr);
      stg_read16<PER>(addr, v);
      const int ld2 = static_cast<int>(ld * 2);
      const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(base, 0, rows * ld2, kBufferFlags);
      const int vo = row_offset(N, ld2) + 2 * c;
      if (room >= 8) {
#pragma unroll
        for (int it = 0; it < PER; ++it)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v[it]), rsrc, vo + step_offset(N, i, it, ld2), 0,
                                                 2);  // 2: non-temporal
      } else if (room > 0) {
#pragma unroll
        for (int it = 0; it < PER; ++it)
#pragma unroll
          for (int e = 0; e < 7; ++e)
            if (e < room)
              __builtin_amdgcn_raw_buffer_store_b16(
                  static_cast<uint16_t>(static_cast<uint32_t>(v[it][e / 2]) >> (16 * (e % 2))), rsrc,
                  vo + step_offset(N, i, it, ld2) + 2 * e, 0, 0);
      }
    };
    using NZ = std::integral_constant<int, CH>;
    using ND = std::integral_constant<int, CHD>;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      pin(i);
      if (p.z) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
            stg_write8(wbase ^ ((part(j, q4) * (CH / 2) + place(j, q4)) << 4),
                       pack_bf16x2(acc[i][j][4 * q4], acc[i][j][4 * q4 + 1]),
                       pack_bf16x2(acc[i][j][4 * q4 + 2], acc[i][j][4 * q4 + 3]));
        fence();
        const int c = te % CH, of = GATED ? c % (CH / 2) : c;  // chunk of the part
        const int64_t second = GATED && c >= CH / 2 ? cols : 0;
        store_rows(NZ{}, p.z + m0 * p.ldz + n0, p.ldz, static_cast<int>(second) + first + 8 * of, left - 8 * of, i);
        fence();
      }
      if constexpr (RES) {
        uint32_t addr[PER_D];
        row_chunks(ND{}, addr);
#pragma unroll
        for (int it = 0; it < PER_D; ++it) stg_write16(addr[it], res[it]);
        fence();
        if (i + 1 < TM) load_residual(i + 1);
      }
      // d's values, in the place of the first part's
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q4 = 0; q4 < 4; q4 += 2) {
          if (part(j, q4)) continue;
          float v[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[h][e] = act(acc[i][j][4 * (q4 + h) + e]);
              if constexpr (GATED && TN > 1) v[h][e] *= acc[i][(j + TN / 2) % TN][4 * (q4 + h) + e];
              if constexpr (GATED && TN == 1) v[h][e] *= acc[i][j][(4 * (q4 + h + 2) + e) % 16];
            }
          const uint32_t a0 = wbase ^ (place(j, q4) << 4), a1 = wbase ^ (place(j, q4 + 1) << 4);
          if constexpr (RES) {
            v2u r0, r1;
            stg_read2x8(a0, a1, r0, r1);
            v[0][0] += bf_lo(r0[0]), v[0][1] += bf_hi(r0[0]), v[0][2] += bf_lo(r0[1]), v[0][3] += bf_hi(r0[1]);
            v[1][0] += bf_lo(r1[0]), v[1][1] += bf_hi(r1[0]), v[1][2] += bf_lo(r1[1]), v[1][3] += bf_hi(r1[1]);
          }
          stg_write8(a0, pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]));
          stg_write8(a1, pack_bf16x2(v[1][0], v[1][1]), pack_bf16x2(v[1][2], v[1][3]));
        }
      fence();
      store_rows(ND{}, p.d + m0 * p.ldd + n0, p.ldd, first + 8 * (te % CHD), left - 8 * (te % CHD), i);
      if (i + 1 < TM) fence();
    }
    if (r + 1 == ntiles) break;
    // the next tile's first body: all of its stage 3 came with the last refills (no PREV in
    // stage 0), and this tile's stores follow stages 1..3
    read_frags(buf0, fa[0], fb[0]);
    stage(I0{}, F{}, 0, T{}, 4, F{}, F{}, 0, T{});
    stage(I1{}, T{}, 4, T{}, 5, F{}, F{}, 0, F{});
    stage(I2{}, T{}, 5, T{}, 6, F{}, F{}, 0, F{});
    stage(I3{}, T{}, 6, T{}, 7, F{}, F{}, 0, F{});
  }
  // the last tile's extra fetch writes LDS: it lands before the workgroup ends
  __builtin_amdgcn_s_waitcnt(0);
#undef PF8_WAIT_VM_LGKM0
}

}  // namespace

template <int BM, int BN>
hipError_t launch_fprop_act_tiles(const FpropActArgs& a, hipStream_t stream) {
  const int64_t cols = a.gated ? a.n / 2 : a.n, out = a.gated ? BN / 2 : BN;
  const int64_t tiles_m = (a.m + BM - 1) / BM, tiles_n = (cols + out - 1) / out;
  const int64_t most = static_cast<int64_t>(device_cus()) * kTilesPerCu<BM, BN> / 8 * 8;
  if (most < 8 || tiles_m * tiles_n > 0x7FFFFFFF) return hipErrorInvalidValue;
  const int64_t want = (tiles_m * tiles_n + 7) / 8 * 8;
  const dim3 grid(static_cast<uint32_t>(want < most ? want : most)), block(256);
  auto run = [&](auto gated, auto res, auto act) {
    hipLaunchKernelGGL((fprop_act_tile_kernel<BM, BN, decltype(gated)::value, decltype(res)::value, decltype(act)::value>),
                       grid, block, 0, stream, a, static_cast<int>(tiles_m), static_cast<int>(tiles_n));
    return hipGetLastError();
  };
  auto by_res = [&](auto gated, auto act) {
    return a.residual ? run(gated, std::true_type{}, act) : run(gated, std::false_type{}, act);
  };
  auto by_act = [&](auto gated) {
    if (a.act == PF8_ACT_GELU) return by_res(gated, std::integral_constant<ActClass, kNormal>{});
    if (a.act == PF8_ACT_SILU || a.act == PF8_ACT_GELU_TANH) return by_res(gated, std::integral_constant<ActClass, kSigmoid>{});
    if constexpr (!decltype(gated)::value) {
      if (a.act == PF8_ACT_NONE) return by_res(gated, std::integral_constant<ActClass, kIdentity>{});
    }
    return by_res(gated, std::integral_constant<ActClass, kPiecewise>{});
  };
  return a.gated ? by_act(std::true_type{}) : by_act(std::false_type{});
}

}  // namespace pf8
