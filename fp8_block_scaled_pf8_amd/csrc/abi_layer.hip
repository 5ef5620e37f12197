// C ABI of a decoder layer's steps around its products (declared in include/pf8_layer.h): host-side
// validation and dispatch. As in abi.hip, every argument is checked before anything is enqueued and the
// checks need no GPU.
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "../../include/pf8_layer.h"
#include "abi_check.h"
#include "pf8_layer_launch.h"

namespace {

using pf8::aligned;
using pf8::any_too_big;
using pf8::device_status;
using pf8::kMaxDim;
using pf8::launch_status;

// Partial column sums are joined by 32 threads a column, and a grid has under 2^32 of them.
constexpr int64_t kMaxSumWidth = int64_t{1} << 27;

// One of the [tokens, heads, head_dim] arrays: its address and strides.
int check_heads(const void* p, int64_t heads, int64_t dim, int64_t st, int64_t sh, int64_t tokens_written = 0) {
  if (!p || st < (tokens_written > 1 ? dim : 0) || (heads > 1 && sh < dim)) return PF8_EINVAL;
  if (any_too_big(st, sh)) return PF8_ESHAPE;
  return aligned(p, 2) ? PF8_OK : PF8_EALIGN;
}

// What both directions check alike: sizes, weights and the rotation.
int check_head_norm(int64_t tokens, int64_t dim, int64_t heads_q, int64_t heads_k, const void* k, const void* w_q,
                    const void* w_k, int wtype, float offset, float eps, const void* positions, int ptype,
                    int64_t pos_st, int64_t pos_sa, const void* inv_freq, int ftype, int64_t pairs, int axes,
                    const int64_t* sections, int order, int interleaved, float scale) {
  if (tokens <= 0 || dim <= 0 || heads_q <= 0 || heads_k < 0 || (!k) != (heads_k == 0) || (w_k && !heads_k))
    return PF8_EINVAL;
  if ((wtype != PF8_BF16 && wtype != PF8_F32) || (interleaved != 0 && interleaved != 1)) return PF8_EINVAL;
  if (!std::isfinite(offset) || !std::isfinite(eps) || eps < 0.0f || !std::isfinite(scale)) return PF8_EINVAL;
  if (pairs < 0 || 2 * std::min(pairs, kMaxDim) > dim || (!positions) != (pairs == 0) || (!inv_freq) != (pairs == 0))
    return PF8_EINVAL;
  if (!positions && !w_q && !w_k) return PF8_EINVAL;  // nothing to do
  if (dim > PF8_HEAD_MAX_DIM || heads_q > PF8_HEAD_MAX_HEADS || heads_k > PF8_HEAD_MAX_HEADS) return PF8_ESHAPE;
  if (tokens > kMaxDim / std::max(heads_q, heads_k)) return PF8_ESHAPE;
  if (positions) {
    if ((ptype != PF8_I32 && ptype != PF8_I64) || (ftype != PF8_F32 && ftype != PF8_F64)) return PF8_EINVAL;
    if (axes < 1 || axes > PF8_HEAD_MAX_AXES || (order != PF8_BLOCKED && order != PF8_CYCLED)) return PF8_EINVAL;
    if (pos_st < 0 || pos_sa < 0) return PF8_EINVAL;
    if (any_too_big(pos_st, pos_sa)) return PF8_ESHAPE;
    if (axes > 1) {
      if (!sections) return PF8_EINVAL;
      int64_t sum = 0;
      for (int a = 0; a < axes; ++a) {
        if (sections[a] < 1 || sections[a] > pairs) return PF8_EINVAL;
        if (order == PF8_CYCLED && a > 0 && a + axes * (sections[a] - 1) >= pairs) return PF8_EINVAL;
        sum += sections[a];
      }
      if (sum != pairs) return PF8_EINVAL;
    }
  }
  const uintptr_t wb = wtype == PF8_F32 ? 4 : 2;
  if (!aligned(w_q, wb) || !aligned(w_k, wb) || !aligned(positions, ptype == PF8_I64 ? 8 : 4) ||
      !aligned(inv_freq, ftype == PF8_F64 ? 8 : 4))
    return PF8_EALIGN;
  return PF8_OK;
}

pf8::HeadNormArgs head_norm_args(int64_t tokens, int64_t dim, int wtype, float offset, float eps, const void* positions,
                                 int ptype, int64_t pos_st, int64_t pos_sa, const void* inv_freq, int ftype,
                                 int64_t pairs, int axes, const int64_t* sections, int order, int interleaved,
                                 float scale) {
  int k = 0;
  while ((int64_t{1} << (2 * k)) < dim) ++k;
  pf8::HeadNormArgs a{};
  a.tokens = tokens, a.dim = static_cast<int>(dim), a.pairs = static_cast<int>(pairs);
  a.wf32 = wtype == PF8_F32, a.offset = offset, a.eps = eps, a.sq = std::ldexp(1.0f, -k);
  a.inv_sum = static_cast<float>(static_cast<double>(int64_t{1} << (2 * k)) / static_cast<double>(dim));
  a.pos = positions, a.p64 = ptype == PF8_I64, a.pos_st = pos_st, a.pos_sa = pos_sa;
  a.freq = inv_freq, a.f64 = ftype == PF8_F64, a.interleaved = interleaved, a.scale = scale;
  a.axes = positions ? axes : 1, a.cycled = order == PF8_CYCLED;
  int64_t end = 0;
  for (int i = 0; i < pf8::kHeadMaxAxes; ++i) {
    const int64_t n = a.axes > 1 && i < axes ? sections[i] : 0;
    end = a.axes > 1 && i < axes ? end + n : pairs;
    a.share[i] = static_cast<int>(a.cycled ? axes * n : end);
  }
  return a;
}

}  // namespace

static_assert(PF8_HEAD_MAX_DIM == pf8::kHeadMaxDim && PF8_HEAD_MAX_AXES == pf8::kHeadMaxAxes,
              "the header's limits are the kernels'");

extern "C" {

pf8_status pf8_qk_norm_rope(int64_t tokens, int64_t head_dim, const void* q, int64_t heads_q, int64_t q_st, int64_t q_sh,
                            const void* k, int64_t heads_k, int64_t k_st, int64_t k_sh, const void* w_q, const void* w_k,
                            pf8_dtype wtype, float weight_offset, float eps, const void* positions, pf8_index ptype,
                            int64_t pos_st, int64_t pos_sa, const void* inv_freq, pf8_dtype ftype, int64_t pairs,
                            int axes, const int64_t* sections, pf8_sections order, int interleaved, float rotary_scale,
                            void* q_out, int64_t qo_st, int64_t qo_sh, void* k_out, int64_t ko_st, int64_t ko_sh,
                            void* hip_stream) {
  if (int e = check_head_norm(tokens, head_dim, heads_q, heads_k, k, w_q, w_k, wtype, weight_offset, eps, positions,
                              ptype, pos_st, pos_sa, inv_freq, ftype, pairs, axes, sections, order, interleaved,
                              rotary_scale))
    return e;
  if (int e = check_heads(q, heads_q, head_dim, q_st, q_sh)) return e;
  if (int e = check_heads(q_out, heads_q, head_dim, qo_st, qo_sh, tokens)) return e;
  if (k) {
    if (int e = check_heads(k, heads_k, head_dim, k_st, k_sh)) return e;
    if (int e = check_heads(k_out, heads_k, head_dim, ko_st, ko_sh, tokens)) return e;
  } else if (k_out) {
    return PF8_EINVAL;
  }
  if (int e = device_status()) return e;
  pf8::HeadNormArgs a = head_norm_args(tokens, head_dim, wtype, weight_offset, eps, positions, ptype, pos_st, pos_sa,
                                       inv_freq, ftype, pairs, axes, sections, order, interleaved, rotary_scale);
  a.t[0] = {static_cast<const uint16_t*>(q), q_st, q_sh, nullptr, 0, 0, static_cast<uint16_t*>(q_out), qo_st, qo_sh, w_q,
            static_cast<int>(heads_q), 0};
  a.t[1] = {static_cast<const uint16_t*>(k), k_st, k_sh, nullptr, 0, 0, static_cast<uint16_t*>(k_out), ko_st, ko_sh, w_k,
            static_cast<int>(heads_k), 0};
  return launch_status(pf8::launch_head_norm_fwd(a, static_cast<hipStream_t>(hip_stream)));
}

int64_t pf8_qk_norm_rope_bwd_workspace(int64_t tokens, int64_t heads_q, int64_t heads_k, int64_t head_dim) {
  if (tokens <= 0 || heads_q <= 0 || heads_k < 0 || head_dim <= 0 || head_dim > PF8_HEAD_MAX_DIM ||
      heads_q > PF8_HEAD_MAX_HEADS || heads_k > PF8_HEAD_MAX_HEADS || tokens > kMaxDim / std::max(heads_q, heads_k))
    return 0;
  return pf8::head_norm_bwd_blocks(tokens, heads_q, heads_k) * head_dim * 4;
}

pf8_status pf8_qk_norm_rope_bwd(int64_t tokens, int64_t head_dim, const void* dq, int64_t dq_st, int64_t dq_sh,
                                const void* dk, int64_t dk_st, int64_t dk_sh, const void* q, int64_t heads_q,
                                int64_t q_st, int64_t q_sh, const void* k, int64_t heads_k, int64_t k_st, int64_t k_sh,
                                const void* w_q, const void* w_k, pf8_dtype wtype, float weight_offset, float eps,
                                const void* positions, pf8_index ptype, int64_t pos_st, int64_t pos_sa,
                                const void* inv_freq, pf8_dtype ftype, int64_t pairs, int axes, const int64_t* sections,
                                pf8_sections order, int interleaved, float rotary_scale,
                                void* dq_out, int64_t dqo_st, int64_t dqo_sh, void* dk_out, int64_t dko_st,
                                int64_t dko_sh, float* dw_q, float* dw_k, int accumulate, void* workspace,
                                int64_t workspace_bytes, void* hip_stream) {
  if (int e = check_head_norm(tokens, head_dim, heads_q, heads_k, dk, w_q, w_k, wtype, weight_offset, eps, positions,
                              ptype, pos_st, pos_sa, inv_freq, ftype, pairs, axes, sections, order, interleaved,
                              rotary_scale))
    return e;
  if ((dw_q && !w_q) || (dw_k && !w_k) || (dk_out && !dk) || (accumulate != 0 && accumulate != 1)) return PF8_EINVAL;
  if (!dq_out && !dk_out && !dw_q && !dw_k) return PF8_EINVAL;
  if (int e = check_heads(dq, heads_q, head_dim, dq_st, dq_sh)) return e;
  if (w_q)
    if (int e = check_heads(q, heads_q, head_dim, q_st, q_sh)) return e;
  if (dq_out)
    if (int e = check_heads(dq_out, heads_q, head_dim, dqo_st, dqo_sh, tokens)) return e;
  if (dk)
    if (int e = check_heads(dk, heads_k, head_dim, dk_st, dk_sh)) return e;
  if (w_k)
    if (int e = check_heads(k, heads_k, head_dim, k_st, k_sh)) return e;
  if (dk_out)
    if (int e = check_heads(dk_out, heads_k, head_dim, dko_st, dko_sh, tokens)) return e;
  const bool sums = dw_q || dw_k;
  if (sums && (!workspace ||
               workspace_bytes < pf8_qk_norm_rope_bwd_workspace(tokens, heads_q, heads_k, head_dim)))
    return PF8_EINVAL;
  if (!aligned(dw_q, 4) || !aligned(dw_k, 4) || (sums && !aligned(workspace, 16))) return PF8_EALIGN;
  if (int e = device_status()) return e;
  pf8::HeadNormArgs a = head_norm_args(tokens, head_dim, wtype, weight_offset, eps, positions, ptype, pos_st, pos_sa,
                                       inv_freq, ftype, pairs, axes, sections, order, interleaved, rotary_scale);
  a.t[0] = {static_cast<const uint16_t*>(q), q_st, q_sh, static_cast<const uint16_t*>(dq), dq_st, dq_sh,
            static_cast<uint16_t*>(dq_out), dqo_st, dqo_sh, w_q, dq_out || dw_q ? static_cast<int>(heads_q) : 0, 0};
  a.t[1] = {static_cast<const uint16_t*>(k), k_st, k_sh, static_cast<const uint16_t*>(dk), dk_st, dk_sh,
            static_cast<uint16_t*>(dk_out), dko_st, dko_sh, w_k, dk_out || dw_k ? static_cast<int>(heads_k) : 0, 0};
  a.partial = static_cast<float*>(workspace);
  return launch_status(pf8::launch_head_norm_bwd(a, {dw_q, dw_k}, accumulate, static_cast<hipStream_t>(hip_stream)));
}

int64_t pf8_act_bwd_workspace(int64_t rows, int64_t cols, int gated) {
  if (rows <= 0 || cols <= 0 || (gated != 0 && gated != 1) || any_too_big(rows, cols) ||
      any_too_big((gated ? 2 : 1) * cols))
    return 0;
  return pf8::act_bwd_groups(rows, cols) * (gated ? 2 : 1) * cols * 4;
}

pf8_status pf8_act_bwd(int64_t rows, int64_t cols, const void* dd, int64_t lddd, const void* z, int64_t ldz,
                       pf8_activation activation, int gated, void* dz, int64_t lddz, float* dbias, int accumulate,
                       void* workspace, int64_t workspace_bytes, void* hip_stream) {
  if (!dd || rows <= 0 || cols <= 0 || (gated != 0 && gated != 1) || (accumulate != 0 && accumulate != 1))
    return PF8_EINVAL;
  if (activation < PF8_ACT_NONE || activation > PF8_ACT_GELU_TANH || (gated && activation == PF8_ACT_NONE))
    return PF8_EINVAL;
  if ((!z) != (activation == PF8_ACT_NONE) || (!dz && !dbias)) return PF8_EINVAL;
  if (any_too_big(rows, cols, lddd, z ? ldz : 0, dz ? lddz : 0)) return PF8_ESHAPE;
  const int64_t width = gated ? 2 * cols : cols;
  if (lddd < cols || (z && ldz < width) || (dz && lddz < width)) return PF8_EINVAL;
  if (width > kMaxDim) return PF8_ESHAPE;
  if (dbias && (!workspace || workspace_bytes < pf8_act_bwd_workspace(rows, cols, gated))) return PF8_EINVAL;
  if (!aligned(dd, 2) || !aligned(z, 2) || !aligned(dz, 2) || !aligned(dbias, 4) || (dbias && !aligned(workspace, 16)))
    return PF8_EALIGN;
  if (int e = device_status()) return e;
  const pf8::ActBwdArgs a{rows, static_cast<int>(cols), static_cast<const uint16_t*>(dd), lddd,
                          static_cast<const uint16_t*>(z), ldz, activation, gated, static_cast<uint16_t*>(dz), lddz,
                          dbias, accumulate, static_cast<float*>(workspace)};
  return launch_status(pf8::launch_act_bwd(a, static_cast<hipStream_t>(hip_stream)));
}

int64_t pf8_act_bwd_quant_workspace(int64_t rows, int64_t cols, int gated) {
  if (rows <= 0 || cols <= 0 || (gated != 0 && gated != 1) || any_too_big(rows, cols) ||
      any_too_big((gated ? 2 : 1) * cols) || rows % 128 || cols % 128 || rows / 128 > 65535)
    return 0;
  return rows / 128 * (gated ? 2 : 1) * cols * 4;
}

pf8_status pf8_act_bwd_quant(int64_t rows, int64_t cols, const void* dd, int64_t lddd, const void* z, int64_t ldz,
                             pf8_activation activation, int gated, void* q_row, int64_t ldq_row, float* dscale_row,
                             int64_t ld_sr, void* q_col, int64_t ldq_col, float* dscale_col, int64_t ld_sc,
                             float* dbias, int accumulate, void* workspace, int64_t workspace_bytes, void* hip_stream) {
  if (!dd || !q_row || !dscale_row || !q_col || !dscale_col || rows <= 0 || cols <= 0) return PF8_EINVAL;
  if ((gated != 0 && gated != 1) || (accumulate != 0 && accumulate != 1)) return PF8_EINVAL;
  if (activation < PF8_ACT_NONE || activation > PF8_ACT_GELU_TANH || (gated && activation == PF8_ACT_NONE) ||
      (!z) != (activation == PF8_ACT_NONE))
    return PF8_EINVAL;
  if (any_too_big(rows, cols, lddd, z ? ldz : 0, ldq_row, ld_sr, ldq_col, ld_sc)) return PF8_ESHAPE;
  const int64_t width = gated ? 2 * cols : cols;
  if (lddd < cols || (z && ldz < width) || ldq_row < width || ld_sr < rows || ldq_col < rows || ld_sc < width)
    return PF8_EINVAL;
  if (rows % 128 || cols % 128 || rows / 128 > 65535 || width > kMaxDim) return PF8_ESHAPE;
  if (dbias && rows > 128 && width >= kMaxSumWidth) return PF8_ESHAPE;
  if (dbias && (!workspace || workspace_bytes < pf8_act_bwd_quant_workspace(rows, cols, gated))) return PF8_EINVAL;
  if (!aligned(dd, 16) || lddd % 8 || !aligned(z, 16) || (z && ldz % 8) || !aligned(q_row, 16) || ldq_row % 16 ||
      !aligned(q_col, 16) || ldq_col % 16 || !aligned(dscale_row, 4) || !aligned(dscale_col, 4) || !aligned(dbias, 4) ||
      (dbias && !aligned(workspace, 16)))
    return PF8_EALIGN;
  if (int e = device_status()) return e;
  const pf8::ActQuantArgs a{rows, cols, static_cast<const uint16_t*>(dd), lddd, static_cast<const uint16_t*>(z), ldz,
                            activation, gated, static_cast<uint8_t*>(q_row), ldq_row, dscale_row, ld_sr,
                            static_cast<uint8_t*>(q_col), ldq_col, dscale_col, ld_sc, dbias, accumulate,
                            static_cast<float*>(workspace)};
  return launch_status(pf8::launch_act_bwd_quant(a, static_cast<hipStream_t>(hip_stream)));
}

pf8_status pf8_fprop_act(int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const float* a_dscale,
                         int64_t ld_as, const void* b, int64_t ldb, const float* b_dscale, int64_t ld_bs,
                         const void* bias, pf8_dtype btype, pf8_activation activation, int gated,
                         const void* residual, int64_t ldr, void* z, int64_t ldz, void* d, int64_t ldd,
                         void* hip_stream) {
  if (!a || !a_dscale || !b || !b_dscale || !d || m <= 0 || n <= 0 || k <= 0) return PF8_EINVAL;
  if ((btype != PF8_BF16 && btype != PF8_F32) || (gated != 0 && gated != 1)) return PF8_EINVAL;
  if (activation < PF8_ACT_NONE || activation > PF8_ACT_GELU_TANH || (gated && activation == PF8_ACT_NONE))
    return PF8_EINVAL;
  if (any_too_big(m, n, k, lda, ld_as, ldb, ld_bs, residual ? ldr : 0, z ? ldz : 0, ldd)) return PF8_ESHAPE;
  if (k % 128 != 0 || (gated && n % 128 != 0)) return PF8_ESHAPE;
  const int64_t cols = gated ? n / 2 : n;
  if (lda < k || ldb < k || ld_as < m || ld_bs < k / 128 || ldd < cols || (residual && ldr < cols) || (z && ldz < n))
    return PF8_EINVAL;
  if (lda > pf8::kMaxTilePitch || ldb > pf8::kMaxTilePitch || ldd > pf8::kMaxTilePitch / 2 ||
      (residual && ldr > pf8::kMaxTilePitch / 2) || (z && ldz > pf8::kMaxTilePitch / 2))
    return PF8_ESHAPE;
  if ((m + 63) / 64 > 65535 * int64_t{64}) return PF8_ESHAPE;
  if (!aligned(a, 16) || !aligned(b, 16) || lda % 16 || ldb % 16 || !aligned(a_dscale, 4) || !aligned(b_dscale, 4) ||
      !aligned(bias, btype == PF8_F32 ? 4 : 2) || !aligned(d, 16) || ldd % 8 || !aligned(residual, 16) ||
      (residual && ldr % 8) || !aligned(z, 16) || (z && ldz % 8))
    return PF8_EALIGN;
  if (int e = device_status()) return e;
  const pf8::FpropActArgs args{m, n, k, static_cast<const uint8_t*>(a), lda, a_dscale, ld_as,
                               static_cast<const uint8_t*>(b), ldb, b_dscale, ld_bs, bias, btype == PF8_F32, activation,
                               gated, static_cast<const uint16_t*>(residual), ldr, static_cast<uint16_t*>(z), ldz,
                               static_cast<uint16_t*>(d), ldd};
  return launch_status(pf8::launch_fprop_act(args, static_cast<hipStream_t>(hip_stream)));
}

int64_t pf8_fprop_act_tile(int64_t m, int64_t n, int64_t k, int gated) {
  if (m <= 0 || n <= 0 || k <= 0 || (gated != 0 && gated != 1) || any_too_big(m, n, k) || k % 128 != 0 ||
      (gated && n % 128 != 0) || (m + 63) / 64 > 65535 * int64_t{64})
    return 0;
  pf8::FpropActArgs args{};
  args.m = m, args.n = n, args.k = k, args.gated = gated;
  const pf8::FpropActTile t = pf8::fprop_act_tile(args);
  return int64_t{t.bm} * 65536 + t.bn;
}

}  // extern "C"
