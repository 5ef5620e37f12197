"""Build libpf8.so (HIP kernels + C ABI) in-tree for gfx950 with hipcc.

    python fp8_block_scaled_pf8_amd/build.py [--asm DIR]

(run as a file: importing the package first would load the library being rebuilt)

--asm DIR additionally writes the gfx950 assembly of every source into DIR.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
SOURCES = ["quant.hip", "gemm.hip", "norm.hip", "newton_schulz.hip", "head_norm.hip", "act.hip", "act_quant.hip", "gemm_act.hip",
           "gemm_act_256.hip", "gemm_act_128.hip", "abi.hip", "abi_train.hip", "abi_layer.hip"]
LIB_NAME = "libpf8.so"
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # keep hipcc from forming packed fp32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libpf8)")


def lib_path() -> str:
    return os.path.join(PKG_DIR, LIB_NAME)


def _jobs() -> int:
    """Compilers at once: MAX_JOBS where it is set, else the CPUs of this process, 16 at most."""
    if os.environ.get("MAX_JOBS", "").isdigit():
        return max(1, int(os.environ["MAX_JOBS"]))
    return min(16, len(os.sched_getaffinity(0)))


def build(asm_dir: "str | None" = None, verbose: bool = False) -> str:
    """Compile every source for gfx950, side by side, and link libpf8.so next to this file. Returns its path."""
    cc = hipcc()
    out = lib_path()
    tmp = out + ".tmp"
    if asm_dir:
        os.makedirs(asm_dir, exist_ok=True)

    def run(args):
        cmd = [cc, *HIPCC_FLAGS, *args]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        errs = [ln for ln in (res.stderr or "").splitlines() if "packed-fp32-ops" not in ln]
        if res.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + "\n".join(errs))
        if verbose and errs:
            print("\n".join(errs), file=sys.stderr)

    with tempfile.TemporaryDirectory() as objs, ThreadPoolExecutor(_jobs()) as pool:
        objects, work = [], []
        for source in SOURCES:
            src, base = os.path.join(CSRC, source), os.path.splitext(source)[0]
            objects.append(os.path.join(objs, base + ".o"))
            work.append(["-c", "-o", objects[-1], src])
            if asm_dir:
                work.append(["--cuda-device-only", "-S", "-o", os.path.join(asm_dir, base + ".s"), src])
        list(pool.map(run, work))
        run(["-shared", "-o", tmp, *objects])
    os.replace(tmp, out)
    return out


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--asm", default=None, help="also write gfx950 assembly into this directory")
    args = ap.parse_args()
    print(build(args.asm, verbose=True))


if __name__ == "__main__":
    main()
