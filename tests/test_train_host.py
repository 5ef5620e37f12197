"""The training operators' C ABI and wrappers on the host (no GPU needed): declared symbols, statuses
of bad arguments, workspace sizes."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pf8_train.h")

L = pytest.importorskip("fp8_block_scaled_pf8_amd._lib", reason="libpf8.so not built (run __graft_entry__.build())")

P = [0x10000 * i for i in range(1, 16)]  # fake, aligned device addresses: validation never dereferences them


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int64_t|pf8_status)\s+(pf8_\w+)\s*\(", text, flags=re.M))
    assert names == set(L.TRAIN_SIGNATURES)
    lib = ctypes.CDLL(L.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)
    defs = dict(re.findall(r"#define\s+(PF8_\w+)\s+(\d+)", text))
    for name in ("PF8_BF16", "PF8_F32", "PF8_NORM_MAX_COLS", "PF8_NS_MAX_SHORT", "PF8_NS_MAX_LONG", "PF8_NS_MAX_BATCH",
                 "PF8_NS_MAX_STEPS"):
        assert int(defs[name]) == getattr(L, name)


_IN = dict(h=P[0], ldh=512, y=P[1], ldy=512, w_post=P[2], gate=P[3], ld_gate=0, w_pre=P[4], wtype=0,
           residual_scale=1.0, branch_scale=1.0, weight_offset=0.0, eps=1e-6)


def _fwd(**kw):
    a = dict(rows=4, cols=512, **_IN, r=P[5], ldr=512, x=P[6], ldx=512, q=P[7], ldq=512, dscale=P[8], ld_s=4)
    a.update(kw)
    return L.pf8_block_norm(*a.values(), 0)


def _bwd(**kw):
    a = dict(rows=4, cols=512, dr=P[9], lddr=512, dx=P[10], lddx=512, **_IN, dh=P[5], lddh=512, dy=P[6], lddy=512,
             dgate=P[7], ld_dgate=0, dw_pre=P[11], dw_post=P[12], accumulate=0, workspace=P[13],
             workspace_bytes=L.pf8_block_norm_bwd_workspace(4, 512))
    a.update(kw)
    return L.pf8_block_norm_bwd(*a.values(), 0)


# argument sets that both directions refuse
SHARED = [
    (dict(h=0), "EINVAL"), (dict(rows=0), "EINVAL"), (dict(rows=-1), "EINVAL"), (dict(cols=0), "EINVAL"),
    (dict(ldh=511), "EINVAL"), (dict(ldy=511), "EINVAL"), (dict(ld_gate=511), "EINVAL"), (dict(ld_gate=-1), "EINVAL"),
    (dict(wtype=2), "EINVAL"), (dict(wtype=-1), "EINVAL"), (dict(eps=-1e-6), "EINVAL"),
    (dict(eps=float("nan")), "EINVAL"), (dict(eps=float("inf")), "EINVAL"), (dict(branch_scale=float("nan")), "EINVAL"),
    (dict(residual_scale=float("inf")), "EINVAL"), (dict(weight_offset=float("nan")), "EINVAL"),
    (dict(rows=1 << 31, ld_s=1 << 31), "ESHAPE"), (dict(ldh=1 << 31), "ESHAPE"), (dict(ldy=1 << 31), "ESHAPE"),
    (dict(ld_gate=1 << 31), "ESHAPE"),
    (dict(h=P[0] + 1), "EALIGN"), (dict(y=P[1] + 1), "EALIGN"), (dict(gate=P[3] + 1), "EALIGN"),
    (dict(gate=P[3] + 2, wtype=1), "EALIGN"), (dict(w_pre=P[4] + 2, wtype=1), "EALIGN"), (dict(w_post=P[2] + 1), "EALIGN"),
]


@pytest.mark.parametrize("kw,status", SHARED)
def test_block_norm_inputs_are_checked(kw, status):
    want = getattr(L, "PF8_" + status)
    assert _fwd(**kw) == want
    kw = {k: v for k, v in kw.items() if k != "ld_s"}
    if "rows" in kw and kw["rows"] == 1 << 31:
        kw["workspace_bytes"] = 1 << 40
    if "ld_gate" in kw:
        kw["ld_dgate"] = 512
    assert _bwd(**kw) == want


WIDE = {k: 40000 for k in ("cols", "ldh", "ldy", "ldr", "ldx")}


@pytest.mark.parametrize("kw,status", [
    (dict(r=0, x=0, q=0, dscale=0), "EINVAL"), (dict(y=0, w_post=0, gate=0), "EINVAL"), (dict(w_pre=0), "EINVAL"),
    (dict(y=0, r=0), "EINVAL"), (dict(y=0, r=0, w_post=0, gate=0, residual_scale=0.5), "EINVAL"),
    (dict(q=0), "EINVAL"), (dict(dscale=0), "EINVAL"), (dict(ldr=511), "EINVAL"), (dict(ldx=511), "EINVAL"),
    (dict(ldq=511), "EINVAL"), (dict(ld_s=3), "EINVAL"), (dict(cols=500), "ESHAPE"),
    (dict(WIDE, q=0, dscale=0), "ESHAPE"), (dict(ldr=1 << 31), "ESHAPE"), (dict(ldq=1 << 31), "ESHAPE"),
    (dict(r=P[5] + 1), "EALIGN"), (dict(q=P[7] + 8), "EALIGN"), (dict(ldq=520), "EALIGN"), (dict(dscale=P[8] + 2), "EALIGN"),
])
def test_block_norm_outputs_are_checked(kw, status):
    assert _fwd(**kw) == getattr(L, "PF8_" + status)


@pytest.mark.parametrize("kw,status", [
    (dict(dr=0, dx=0), "EINVAL"), (dict(w_pre=0), "EINVAL"), (dict(accumulate=2), "EINVAL"),
    (dict(dh=0, dy=0, dgate=0, dw_pre=0, dw_post=0), "EINVAL"), (dict(gate=0), "EINVAL"), (dict(w_post=0), "EINVAL"),
    (dict(dx=0), "EINVAL"), (dict(lddr=511), "EINVAL"), (dict(lddx=511), "EINVAL"), (dict(lddh=511), "EINVAL"),
    (dict(lddy=511), "EINVAL"), (dict(ld_dgate=512), "EINVAL"), (dict(ld_gate=512, ld_dgate=511), "EINVAL"),
    (dict(y=0, w_post=0, gate=0, dgate=0, dw_post=0), "EINVAL"),
    (dict(workspace=0), "EINVAL"), (dict(workspace_bytes=4 * 3 * 512 * 4 - 1), "EINVAL"), (dict(workspace=P[13] + 8), "EALIGN"),
    (dict(dw_pre=P[11] + 2), "EALIGN"), (dict(dgate=P[7] + 2), "EALIGN"), (dict(dx=P[10] + 1), "EALIGN"),
    (dict(lddy=1 << 31), "ESHAPE"),
])
def test_block_norm_backward_is_checked(kw, status):
    assert _bwd(**kw) == getattr(L, "PF8_" + status)


def test_block_norm_workspace():
    size = L.pf8_block_norm_bwd_workspace
    assert size(0, 512) == size(4, 0) == size(4, 40000) == size(1 << 31, 512) == size(-1, 5) == 0
    assert size(1, 1) >= 12 and size(8192, 2048) >= 3 * 2048 * 4
    assert size((1 << 31) - 1, 16384) < 1 << 30


def _ns(**kw):
    a = dict(batch=2, m=100, n=200, g=P[0], ldg=200, stride_g=20000, gtype=1, steps=1,
             coefficients=(ctypes.c_float * 3)(1.5, -0.5, 0.0), eps=1e-7, out=P[1], ldo=200, stride_o=20000,
             workspace=P[2], workspace_bytes=L.pf8_newton_schulz_workspace(2, 100, 200))
    a.update(kw)
    return L.pf8_newton_schulz(*a.values(), 0)


@pytest.mark.parametrize("kw,status", [
    (dict(g=0), "EINVAL"), (dict(out=0), "EINVAL"), (dict(workspace=0), "EINVAL"), (dict(coefficients=None), "EINVAL"),
    (dict(batch=0), "EINVAL"), (dict(m=0), "EINVAL"), (dict(n=-1), "EINVAL"), (dict(gtype=2), "EINVAL"),
    (dict(steps=0), "EINVAL"), (dict(steps=65), "EINVAL"), (dict(eps=-1.0), "EINVAL"), (dict(eps=float("nan")), "EINVAL"),
    (dict(ldg=199), "EINVAL"), (dict(ldo=199), "EINVAL"), (dict(stride_g=19999), "EINVAL"), (dict(stride_o=0), "EINVAL"),
    (dict(coefficients=(ctypes.c_float * 3)(64.5, 0.0, 0.0)), "EINVAL"),
    (dict(coefficients=(ctypes.c_float * 3)(1.0, float("nan"), 0.0)), "EINVAL"),
    (dict(batch=65536), "ESHAPE"), (dict(m=32769, n=32769, ldg=32769, ldo=32769), "ESHAPE"),
    (dict(n=1048577, ldg=1048577, ldo=1048577), "ESHAPE"), (dict(ldg=1 << 31), "ESHAPE"),
    (dict(stride_g=(1 << 46) + 1), "ESHAPE"),
    (dict(workspace_bytes=L.pf8_newton_schulz_workspace(2, 100, 200) - 1), "EINVAL"),
    (dict(g=P[0] + 2), "EALIGN"), (dict(out=P[1] + 1), "EALIGN"), (dict(workspace=P[2] + 128), "EALIGN"),
])
def test_newton_schulz_is_checked(kw, status):
    assert _ns(**kw) == getattr(L, "PF8_" + status)


def test_newton_schulz_workspace():
    size = L.pf8_newton_schulz_workspace
    assert size(0, 5, 5) == size(1, 0, 5) == size(1, 5, -1) == size(1, 32769, 32769) == size(1, 5, 1048577) == 0
    assert size(65536, 5, 5) == 0 and size(1, 1, 1) > 0
    # an element is kept as a transposed FP16 operand in two buffers and an FP16 remainder: 6 bytes
    assert size(1, 2048, 512) == size(1, 512, 2048) >= 2048 * 512 * 6


def test_rows_that_share_memory_are_found():
    """Against the sets of bytes: never missed, and exact where the pitches are one or a side is a single row."""
    import itertools

    from fp8_block_scaled_pf8_amd.norm import _rows_meet

    def rows(first, count, width, pitch):
        at = {first + r * pitch + b for r in range(count) for b in range(width)}
        return at, (first, max(at) + 1, width, pitch if count > 1 else 0)

    for (f, n, w, p), (k, v, q) in itertools.product(
            itertools.product(range(0, 30), (1, 3), (1, 3, 5), (5, 8)), itertools.product((1, 2, 4), (2, 5), (5, 8))):
        a, at_a = rows(f, n, w, p)
        b, at_b = rows(12, k, v, q)
        shared, found = bool(a & b), _rows_meet(at_a, at_b)
        assert found == _rows_meet(at_b, at_a)
        assert found if shared else True
        if n > 1 and k > 1 and p == q and not shared:
            # (rows beyond one side's end count as its own: they lie within the other's extent)
            assert not found or not rows(f, 20, w, p)[0].isdisjoint(rows(12, 20, v, q)[0] | rows(12 - 10 * q, 20, v, q)[0])
