// C ABI of the training operators (declared in include/pf8_train.h): host-side validation and
// dispatch. As in abi.hip, every argument is checked before anything is enqueued and the checks
// need no GPU.
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "../../include/pf8_train.h"
#include "abi_check.h"
#include "pf8_train_launch.h"

namespace {

using pf8::aligned;
using pf8::any_too_big;
using pf8::device_status;
using pf8::kMaxDim;
using pf8::launch_status;

// What the block norm's two directions check alike.
int check_norm_inputs(int64_t rows, int64_t cols, const void* h, int64_t ldh, const void* y, int64_t ldy,
                      const void* w_post, const void* gate, int64_t ld_gate, const void* w_pre, int wtype,
                      float residual_scale, float branch_scale, float weight_offset, float eps) {
  if (!h || rows <= 0 || cols <= 0 || (wtype != PF8_BF16 && wtype != PF8_F32)) return PF8_EINVAL;
  if (!std::isfinite(residual_scale) || !std::isfinite(branch_scale) || !std::isfinite(weight_offset) ||
      !std::isfinite(eps) || eps < 0.0f)
    return PF8_EINVAL;
  if (ldh < cols || (y && ldy < cols)) return PF8_EINVAL;
  if (!y && (w_post || gate || residual_scale != 1.0f)) return PF8_EINVAL;
  if (gate && ld_gate != 0 && ld_gate < cols) return PF8_EINVAL;
  if (cols > PF8_NORM_MAX_COLS || any_too_big(rows, ldh, y ? ldy : 0, gate ? ld_gate : 0)) return PF8_ESHAPE;
  const uintptr_t wb = wtype == PF8_F32 ? 4 : 2;
  if (!aligned(h, 2) || !aligned(y, 2) || !aligned(w_post, wb) || !aligned(w_pre, wb) ||
      !aligned(gate, ld_gate ? 2 : wb))
    return PF8_EALIGN;
  return PF8_OK;
}

pf8::NormArgs norm_args(int64_t rows, int64_t cols, const void* h, int64_t ldh, const void* y, int64_t ldy,
                        const void* w_post, const void* gate, int64_t ld_gate, const void* w_pre, int wtype,
                        float residual_scale, float branch_scale, float weight_offset, float eps) {
  int k = 0;
  while ((int64_t{1} << (2 * k)) < cols) ++k;
  const double four_k = static_cast<double>(int64_t{1} << (2 * k));
  return {rows, static_cast<int>(cols), static_cast<const uint16_t*>(h), ldh, static_cast<const uint16_t*>(y), ldy,
          w_post, gate, ld_gate, w_pre, wtype == PF8_F32, residual_scale, branch_scale, weight_offset, eps,
          std::ldexp(1.0f, -k), static_cast<float>(four_k / static_cast<double>(cols))};
}

}  // namespace

static_assert(PF8_NORM_MAX_COLS == pf8::kNormMaxCols, "the header's limit is the kernels'");

extern "C" {

pf8_status pf8_block_norm(int64_t rows, int64_t cols, const void* h, int64_t ldh, const void* y, int64_t ldy,
                          const void* w_post, const void* gate, int64_t ld_gate, const void* w_pre, pf8_dtype wtype,
                          float residual_scale, float branch_scale, float weight_offset, float eps,
                          void* r, int64_t ldr, void* x, int64_t ldx, void* q, int64_t ldq, float* dscale, int64_t ld_s,
                          void* hip_stream) {
  if (int e = check_norm_inputs(rows, cols, h, ldh, y, ldy, w_post, gate, ld_gate, w_pre, wtype, residual_scale,
                                branch_scale, weight_offset, eps))
    return e;
  if ((!r && !x && !q) || (r && !y) || ((x || q) && !w_pre) || (!q) != (!dscale)) return PF8_EINVAL;
  if ((r && ldr < cols) || (x && ldx < cols) || (q && (ldq < cols || ld_s < rows))) return PF8_EINVAL;
  if (q && cols % 128) return PF8_ESHAPE;
  if (any_too_big(r ? ldr : 0, x ? ldx : 0, q ? ldq : 0, q ? ld_s : 0)) return PF8_ESHAPE;
  if (!aligned(r, 2) || !aligned(x, 2) || !aligned(q, 16) || !aligned(dscale, 4) || (q && ldq % 16)) return PF8_EALIGN;
  if (int e = device_status()) return e;
  pf8::NormFwdArgs a{norm_args(rows, cols, h, ldh, y, ldy, w_post, gate, ld_gate, x || q ? w_pre : nullptr, wtype,
                               residual_scale, branch_scale, weight_offset, eps),
                     static_cast<uint16_t*>(r), ldr, static_cast<uint16_t*>(x), ldx, static_cast<uint8_t*>(q), ldq,
                     dscale, ld_s};
  return launch_status(pf8::launch_norm_fwd(a, static_cast<hipStream_t>(hip_stream)));
}

int64_t pf8_block_norm_bwd_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols > PF8_NORM_MAX_COLS || rows > kMaxDim) return 0;
  return pf8::norm_bwd_groups(rows, cols) * 3 * cols * 4;
}

pf8_status pf8_block_norm_bwd(int64_t rows, int64_t cols, const void* dr, int64_t lddr, const void* dx, int64_t lddx,
                              const void* h, int64_t ldh, const void* y, int64_t ldy, const void* w_post,
                              const void* gate, int64_t ld_gate, const void* w_pre, pf8_dtype wtype,
                              float residual_scale, float branch_scale, float weight_offset, float eps,
                              void* dh, int64_t lddh, void* dy, int64_t lddy, void* dgate, int64_t ld_dgate,
                              float* dw_pre, float* dw_post, int accumulate, void* workspace, int64_t workspace_bytes,
                              void* hip_stream) {
  if (int e = check_norm_inputs(rows, cols, h, ldh, y, ldy, w_post, gate, ld_gate, w_pre, wtype, residual_scale,
                                branch_scale, weight_offset, eps))
    return e;
  const bool full = gate && ld_gate != 0;
  if ((!dr && !dx) || (dx && !w_pre) || (accumulate != 0 && accumulate != 1)) return PF8_EINVAL;
  if (!dh && !dy && !dgate && !dw_pre && !dw_post) return PF8_EINVAL;
  if ((dy && !y) || (dgate && !gate) || (dw_pre && !dx) || (dw_post && !w_post)) return PF8_EINVAL;
  if ((dr && lddr < cols) || (dx && lddx < cols) || (dh && lddh < cols) || (dy && lddy < cols)) return PF8_EINVAL;
  if (dgate && (full ? ld_dgate < cols : ld_dgate != 0)) return PF8_EINVAL;
  if (any_too_big(dr ? lddr : 0, dx ? lddx : 0, dh ? lddh : 0, dy ? lddy : 0, dgate ? ld_dgate : 0)) return PF8_ESHAPE;
  const bool sums = dw_pre || dw_post || (dgate && !full);
  if (sums && (!workspace || workspace_bytes < pf8_block_norm_bwd_workspace(rows, cols))) return PF8_EINVAL;
  if (!aligned(dr, 2) || !aligned(dx, 2) || !aligned(dh, 2) || !aligned(dy, 2) || !aligned(dgate, full ? 2 : 4) ||
      !aligned(dw_pre, 4) || !aligned(dw_post, 4) || (sums && !aligned(workspace, 16)))
    return PF8_EALIGN;
  if (int e = device_status()) return e;
  pf8::NormBwdArgs a{norm_args(rows, cols, h, ldh, y, ldy, w_post, gate, ld_gate, w_pre, wtype, residual_scale,
                               branch_scale, weight_offset, eps),
                     static_cast<const uint16_t*>(dr), lddr, static_cast<const uint16_t*>(dx), lddx,
                     static_cast<uint16_t*>(dh), lddh, static_cast<uint16_t*>(dy), lddy,
                     full ? static_cast<uint16_t*>(dgate) : nullptr, ld_dgate,
                     {dw_pre, dw_post, full ? nullptr : static_cast<float*>(dgate)}, accumulate,
                     static_cast<float*>(workspace)};
  return launch_status(pf8::launch_norm_bwd(a, static_cast<hipStream_t>(hip_stream)));
}

int64_t pf8_newton_schulz_workspace(int64_t batch, int64_t m, int64_t n) {
  if (batch <= 0 || m <= 0 || n <= 0 || batch > PF8_NS_MAX_BATCH || std::min(m, n) > PF8_NS_MAX_SHORT ||
      std::max(m, n) > PF8_NS_MAX_LONG)
    return 0;
  return pf8::ns_workspace(batch, m, n);
}

pf8_status pf8_newton_schulz(int64_t batch, int64_t m, int64_t n, const void* g, int64_t ldg, int64_t stride_g,
                             pf8_dtype gtype, int steps, const float* coefficients, float eps, void* out, int64_t ldo,
                             int64_t stride_o, void* workspace, int64_t workspace_bytes, void* hip_stream) {
  if (!g || !out || !coefficients || !workspace || batch <= 0 || m <= 0 || n <= 0) return PF8_EINVAL;
  if ((gtype != PF8_BF16 && gtype != PF8_F32) || steps <= 0 || steps > PF8_NS_MAX_STEPS) return PF8_EINVAL;
  if (!std::isfinite(eps) || eps < 0.0f || ldg < n || ldo < n) return PF8_EINVAL;
  for (int i = 0; i < 3 * steps; ++i)
    if (!(std::fabs(coefficients[i]) <= 64.0f)) return PF8_EINVAL;
  if (batch > PF8_NS_MAX_BATCH || std::min(m, n) > PF8_NS_MAX_SHORT || std::max(m, n) > PF8_NS_MAX_LONG ||
      any_too_big(ldg, ldo))
    return PF8_ESHAPE;
  // a matrix spans less than 2^51 elements here, and strides up to 2^46 times the batch stay in range
  if (batch > 1 && (stride_g < (m - 1) * ldg + n || stride_o < (m - 1) * ldo + n)) return PF8_EINVAL;
  if (batch > 1 && (stride_g > (int64_t{1} << 46) || stride_o > (int64_t{1} << 46))) return PF8_ESHAPE;
  if (workspace_bytes < pf8_newton_schulz_workspace(batch, m, n)) return PF8_EINVAL;
  if (!aligned(g, gtype == PF8_F32 ? 4 : 2) || !aligned(out, 2) || !aligned(workspace, 256)) return PF8_EALIGN;
  if (int e = device_status()) return e;
  pf8::NsArgs a{};
  a.m = m, a.n = n, a.g = g, a.ldg = ldg, a.stride_g = batch > 1 ? stride_g : 0, a.gf32 = gtype == PF8_F32, a.eps = eps;
  a.out = static_cast<uint16_t*>(out), a.ldo = ldo, a.stride_o = batch > 1 ? stride_o : 0;
  return launch_status(pf8::launch_newton_schulz(a, batch, steps, coefficients, workspace,
                                                 static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
