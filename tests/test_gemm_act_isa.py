"""The tile kernels of the product with its epilogue wait for counted vector-memory loads, as the plain product's do.
This test compiles them for gfx950 (device code only, no GPU needed) and checks in the assembly that the compiler
issues the loads those counts assume: each four-stage trip of a K loop holds 4 (A_DMA + B_DMA) direct-to-LDS loads
and two sets of TM + SB scale loads, and no stores; the whole kernel 20 A_DMA + 19 B_DMA and ten sets (the prologue's
four stages, the first, inner, last and next tile's first body). A scale load merged or dropped would make the waits too
permissive."""
import os
import re
import shutil
import subprocess

import pytest

from tests.test_gemm_isa import _functions, _inner_loops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_block_scaled_pf8_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
KERNEL = re.compile(r"_ZN3pf8.*fprop_act_tile_kernelILi(\d+)ELi(\d+)ELb(\d)ELb(\d)E")


@pytest.mark.parametrize("source,kernels", [("gemm_act_256.hip", 14), ("gemm_act_128.hip", 42)])
def test_tile_kernel_load_counts(tmp_path, source, kernels):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path / "k.s"
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "--cuda-device-only", "-S", "-o", str(out), os.path.join(CSRC, source)]
    subprocess.run(cmd, check=True, capture_output=True, timeout=900)
    checked = 0
    is_lds = lambda ln: ln.strip().startswith("buffer_load_dword") and " lds" in ln  # noqa: E731
    for name, body in _functions(out.read_text()).items():
        m = KERNEL.match(name)
        if not m:
            continue
        bm, bn, gated, _ = (int(x) for x in m.groups())
        a_dma, b_dma, tm, tn = bm // 64, bn // 64, bm // 64, bn // 64
        ss = tm + (2 if gated and tn > 1 else 1)
        assert sum(map(is_lds, body)) == 20 * a_dma + 19 * b_dma, name
        loops = [lp for lp in _inner_loops(body) if any(ln.strip().startswith("v_mfma_scale") for ln in lp)]
        assert loops, name
        for lp in loops:
            n_sc = sum(1 for ln in lp if ln.strip().startswith("global_load_dword "))
            n_st = sum(1 for ln in lp if ln.strip().startswith(("global_store", "buffer_store", "scratch_")))
            assert (sum(map(is_lds, lp)), n_sc, n_st) == (4 * (a_dma + b_dma), 2 * ss, 0), name
        # the bias adds up to 2 TN loads of a dword to the scales'
        total = sum(1 for ln in body if ln.strip().startswith("global_load_dword "))
        assert 10 * ss <= total <= 10 * ss + 2 * tn, f"{name}: {total} dword loads for {10 * ss} scales"
        checked += 1
    assert checked == kernels, checked
