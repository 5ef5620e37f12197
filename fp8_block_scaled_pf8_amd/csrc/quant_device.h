// The dual-orientation quantiser of a 128 x 128 tile whose values are in registers (gfx950 / CDNA4 only).
#pragma once

#include "pf8_device.h"

namespace pf8 {

// The LDS tile's layout: see quant.hip.
__device__ __forceinline__ int dual_slot(int c, int s) {
  return (c >> 1) * 256 + 8 * ((s | ((c & 1) << 4)) ^ (((c >> 3) & 7) << 2));
}

// Thread t holds rows 8*(t/16) .. +7, columns 8*(t%16) .. +7 of the tile; load(row, c0, c) gives the 8 packed BF16
// values of a row from column c0 + c on, and is called for the thread's rows in order. gc = column group (row mode),
// gr = row group (col mode). red: [wave][column chunk][packed column pair] words of LDS, tile: kGroup * kGroup bytes.
template <typename LOAD>
__device__ __forceinline__ void quant_dual_values(LOAD load, uint8_t* __restrict__ qr, int64_t ldqr, float* __restrict__ sr,
                                                  int64_t ld_sr, uint8_t* __restrict__ qc, int64_t ldqc,
                                                  float* __restrict__ sc, int64_t ld_sc, int64_t gc, int64_t gr,
                                                  uint32_t (*red)[16][4], uint8_t* tile) {
  const int t = threadIdx.x;
  const int rb = t >> 4;  // rows 8*rb .. 8*rb+7 of the tile
  const int cc = t & 15;  // cols 8*cc .. 8*cc+7 of the tile
  const int wave = t >> 6;
  const int64_t r0 = gr * kGroup, c0 = gc * kGroup;
  uint4 v[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) v[p] = load(r0 + 8 * rb + p, c0, 8 * cc);

  // ---- row mode: 8 rows, one 128-value group each ----
  // (row maxima two at a time: packed 16-bit pairs through the DPP reduction)
  float my_row_scale = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t rm = row16_max_pk(pair_amax(amax8_pk(v[2 * k]), amax8_pk(v[2 * k + 1])));
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int p = 2 * k + hh;
      const float scale = pow2f(block_exponent(hh ? rm >> 16 : rm & 0xFFFFu));
      *reinterpret_cast<uint2*>(qr + (r0 + 8 * rb + p) * ldqr + c0 + 8 * cc) = quant8_scaled(v[p], scale);
      if (cc == p) my_row_scale = scale;
    }
  }
  if (cc < 8) sr[gc * ld_sr + r0 + 8 * rb + cc] = my_row_scale;

  // ---- col mode: per-column maxima, packed as column pairs (2h, 2h+1) in word h ----
  uint32_t m[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) m[h] = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
    for (int h = 0; h < 4; ++h) m[h] = pk_max_u16(m[h], w[h] & 0x7FFF7FFFu);
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    m[h] = pk_max_u16(m[h], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[h]), 16)));
    m[h] = pk_max_u16(m[h], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[h]), 32)));
  }
  if ((t & 63) < 16) *reinterpret_cast<uint4*>(&red[wave][cc][0]) = make_uint4(m[0], m[1], m[2], m[3]);
  __syncthreads();
  float scale[8];
  {
    uint4 a = *reinterpret_cast<const uint4*>(&red[0][cc][0]);
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const uint4 b = *reinterpret_cast<const uint4*>(&red[w][cc][0]);
      a = make_uint4(pk_max_u16(a.x, b.x), pk_max_u16(a.y, b.y), pk_max_u16(a.z, b.z), pk_max_u16(a.w, b.w));
    }
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
    float my_col_scale = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      scale[j] = pow2f(block_exponent((aw[j >> 1] >> (16 * (j & 1))) & 0xFFFFu));
      if (rb == j) my_col_scale = scale[j];
    }
    // thread (rb < 8, cc) writes the scale of column 8*cc + rb
    if (rb < 8) sc[gr * ld_sc + c0 + 8 * cc + rb] = my_col_scale;
  }
  // codes of column j for rows 8*rb .. 8*rb+7: one little-endian 64-bit word; the column's
  // values of rows p, p+1 are paired into one dword (v_perm) and converted together
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int h = j >> 1;
    const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;  // high or low bf16 of each row's word
    uint32_t w[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) w[p] = h == 0 ? v[p].x : h == 1 ? v[p].y : h == 2 ? v[p].z : v[p].w;
    const uint32_t lo = cvt2_bf16_scaled<true>(__builtin_amdgcn_perm(w[3], w[2], sel), scale[j],
                                               cvt2_bf16_scaled<false>(__builtin_amdgcn_perm(w[1], w[0], sel), scale[j], 0u));
    const uint32_t hi = cvt2_bf16_scaled<true>(__builtin_amdgcn_perm(w[7], w[6], sel), scale[j],
                                               cvt2_bf16_scaled<false>(__builtin_amdgcn_perm(w[5], w[4], sel), scale[j], 0u));
    *reinterpret_cast<uint2*>(tile + dual_slot(8 * cc + j, rb)) = make_uint2(lo, hi);
  }
  __syncthreads();
  // 128 transposed rows of 128 bytes: thread t sends chunk (t & 7) of rows (t >> 3) + 32 * i
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = (t >> 3) + 32 * i;
    const int k = t & 7;
    const uint4 val = *reinterpret_cast<const uint4*>(tile + dual_slot(c, 2 * k));
    *reinterpret_cast<uint4*>(qc + (c0 + c) * ldqc + r0 + 16 * k) = val;
  }
}

}  // namespace pf8
