"""Block-scaled FP8 (E4M3) linear-layer quantisers and GEMM for AMD MI355X (gfx950), with the
training operators around the layer (block norm, Newton-Schulz orthogonalisation) and a decoder layer's steps around
its products (head norms with rotation, products with bias, activation and residual in their epilogue).

The computation lives in libpf8.so (HIP kernels behind a C ABI: include/pf8.h, include/pf8_train.h and
include/pf8_layer.h); this package is its Python binding. Importing it fails when the library has not been built.
"""
from . import _lib
from ._lib import (
    PF8_ALONG_COLS,
    PF8_ALONG_ROWS,
    PF8_BF16,
    PF8_DGRAD,
    PF8_F32,
    PF8_FPROP,
    PF8_GEMM_AUTO,
    PF8_GEMM_MX_SCALED,
    PF8_GEMM_PROMOTE,
    PF8_WGRAD,
    pf8_abi_version,
    pf8_act_bwd,
    pf8_act_bwd_quant,
    pf8_act_bwd_quant_workspace,
    pf8_act_bwd_workspace,
    pf8_block_gemm,
    pf8_block_gemm_f32,
    pf8_block_gemm_variant,
    pf8_block_norm,
    pf8_block_norm_bwd,
    pf8_block_norm_bwd_workspace,
    pf8_fprop_act,
    pf8_fprop_act_tile,
    pf8_gemm_bf16,
    pf8_newton_schulz,
    pf8_newton_schulz_workspace,
    pf8_qk_norm_rope,
    pf8_qk_norm_rope_bwd,
    pf8_qk_norm_rope_bwd_workspace,
    pf8_quant_act_1x128,
    pf8_quant_act_dual,
    pf8_quant_fwd,
    pf8_quant_w_128x128,
    pf8_strerror,
)
from .epilogue import ActGrads, ActQuantGrads, act_backward, act_backward_quant, fprop_act
from .heads import (QKNormRope, QKNormRopeFunction, QKNormRopeGrads, fp8_qk_norm_rope, qk_norm_rope,
                    qk_norm_rope_backward)
from .linear import Fp8Linear, Fp8LinearActFunction, Fp8LinearFunction, fp8_linear, fp8_linear_act
from .norm import (BlockNorm, BlockNormFunction, BlockNormGrads, block_norm, block_norm_backward, block_norm_quant,
                   fp8_block_norm)
from .orthogonal import newton_schulz
from .ops import (LinearStep, block_gemm, block_gemm_f32, dgrad, fprop, gemm_bf16, quant_act_1x128, quant_act_dual,
                  quant_w_128x128, wgrad, wgrad_f32)

__all__ = [
    "PF8_ALONG_COLS", "PF8_ALONG_ROWS", "PF8_FPROP", "PF8_DGRAD", "PF8_WGRAD",
    "PF8_GEMM_AUTO", "PF8_GEMM_MX_SCALED", "PF8_GEMM_PROMOTE",
    "pf8_abi_version", "pf8_block_gemm", "pf8_block_gemm_f32", "pf8_block_gemm_variant", "pf8_gemm_bf16", "pf8_quant_act_1x128", "pf8_quant_act_dual",
    "pf8_quant_fwd", "pf8_quant_w_128x128", "pf8_strerror",
    "LinearStep", "block_gemm", "block_gemm_f32", "dgrad", "fprop", "gemm_bf16", "quant_act_1x128", "quant_act_dual",
    "quant_w_128x128", "wgrad", "wgrad_f32", "Fp8Linear", "Fp8LinearActFunction", "Fp8LinearFunction", "fp8_linear", "fp8_linear_act",
    "PF8_BF16", "PF8_F32", "pf8_block_norm", "pf8_block_norm_bwd", "pf8_block_norm_bwd_workspace",
    "BlockNorm", "BlockNormFunction", "BlockNormGrads", "block_norm", "block_norm_backward", "block_norm_quant",
    "fp8_block_norm", "pf8_newton_schulz", "pf8_newton_schulz_workspace", "newton_schulz",
    "pf8_qk_norm_rope", "pf8_qk_norm_rope_bwd", "pf8_qk_norm_rope_bwd_workspace", "pf8_act_bwd", "pf8_act_bwd_workspace",
    "QKNormRope", "QKNormRopeFunction", "QKNormRopeGrads", "fp8_qk_norm_rope", "qk_norm_rope", "qk_norm_rope_backward",
    "pf8_fprop_act", "pf8_fprop_act_tile", "pf8_act_bwd_quant", "pf8_act_bwd_quant_workspace",
    "ActGrads", "ActQuantGrads", "act_backward", "act_backward_quant", "fprop_act",
]
