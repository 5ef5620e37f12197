"""The C ABI and wrappers of the layer's steps on the host (no GPU needed): declared symbols, statuses of bad
arguments, workspace sizes."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pf8_layer.h")

L = pytest.importorskip("fp8_block_scaled_pf8_amd._lib", reason="libpf8.so not built (run __graft_entry__.build())")

P = [0x10000 * i for i in range(1, 16)]  # fake, aligned device addresses: validation never dereferences them
NAN, INF = float("nan"), float("inf")
BIG = 1 << 31


def _status(name):
    return getattr(L, "PF8_" + name)


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int64_t|pf8_status)\s+(pf8_\w+)\s*\(", text, flags=re.M))
    assert names == set(L.LAYER_SIGNATURES)
    lib = ctypes.CDLL(L.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)
    defs = dict(re.findall(r"#define\s+(PF8_\w+)\s+(\d+)", text))
    defs.pop("PF8_LAYER_H", None)
    assert len(defs) >= 14
    for name, value in defs.items():
        assert int(value) == getattr(L, name), name


def _sec(*v):
    return (ctypes.c_int64 * len(v))(*v)


_ROT = dict(w_q=P[2], w_k=P[3], wtype=0, offset=0.0, eps=1e-6, pos=P[4], ptype=1, pos_st=1, pos_sa=0, freq=P[5], ftype=1,
            pairs=64, axes=1, sections=None, order=0, interleaved=0, scale=1.0)


def _fwd(**kw):
    a = dict(tokens=4, dim=128, q=P[0], hq=16, q_st=2048, q_sh=128, k=P[1], hk=8, k_st=1024, k_sh=128, **_ROT, qo=P[6],
             qo_st=2048, qo_sh=128, ko=P[7], ko_st=1024, ko_sh=128)
    a.update(kw)
    return L.pf8_qk_norm_rope(*a.values(), 0)


def _bwd(**kw):
    a = dict(tokens=4, dim=128, dq=P[8], dq_st=2048, dq_sh=128, dk=P[9], dk_st=1024, dk_sh=128, q=P[0], hq=16, q_st=2048,
             q_sh=128, k=P[1], hk=8, k_st=1024, k_sh=128, **_ROT, qo=P[6], qo_st=2048, qo_sh=128, ko=P[7], ko_st=1024,
             ko_sh=128, dw_q=P[10], dw_k=P[11], accumulate=0, ws=P[12],
             ws_bytes=L.pf8_qk_norm_rope_bwd_workspace(4, 16, 8, 128))
    a.update(kw)
    return L.pf8_qk_norm_rope_bwd(*a.values(), 0)


SHARED = [
    (dict(tokens=0), "EINVAL"), (dict(tokens=-1), "EINVAL"), (dict(dim=0), "EINVAL"), (dict(hq=0), "EINVAL"),
    (dict(hk=0), "EINVAL"), (dict(hk=-1), "EINVAL"), (dict(wtype=2), "EINVAL"), (dict(interleaved=2), "EINVAL"),
    (dict(offset=NAN), "EINVAL"), (dict(eps=-1.0), "EINVAL"), (dict(eps=NAN), "EINVAL"), (dict(scale=INF), "EINVAL"),
    (dict(pairs=0), "EINVAL"), (dict(pairs=65), "EINVAL"), (dict(pairs=-1), "EINVAL"), (dict(pairs=1 << 62), "EINVAL"),
    (dict(pos=0), "EINVAL"), (dict(freq=0), "EINVAL"), (dict(pos=0, freq=0, pairs=0, w_q=0, w_k=0), "EINVAL"),
    (dict(ptype=2), "EINVAL"), (dict(ftype=0), "EINVAL"), (dict(axes=0), "EINVAL"), (dict(axes=5), "EINVAL"),
    (dict(order=2), "EINVAL"), (dict(pos_st=-1), "EINVAL"), (dict(pos_sa=-1), "EINVAL"), (dict(pos_st=BIG), "ESHAPE"),
    (dict(axes=2), "EINVAL"), (dict(axes=2, sections=_sec(32, 31)), "EINVAL"), (dict(axes=2, sections=_sec(64, 0)), "EINVAL"),
    (dict(axes=2, sections=_sec(-1, 65)), "EINVAL"), (dict(axes=2, sections=_sec(16, 48), order=1), "EINVAL"),
    (dict(dim=513), "ESHAPE"), (dict(hq=65537), "ESHAPE"), (dict(hk=65537), "ESHAPE"), (dict(tokens=1 << 28), "ESHAPE"),
    (dict(tokens=1 << 62), "ESHAPE"), (dict(w_q=P[2] + 1), "EALIGN"), (dict(w_k=P[3] + 2, wtype=1), "EALIGN"),
    (dict(pos=P[4] + 4), "EALIGN"), (dict(pos=P[4] + 2, ptype=0), "EALIGN"), (dict(freq=P[5] + 4, ftype=2), "EALIGN"),
    (dict(q=0), "EINVAL"), (dict(q_sh=127), "EINVAL"), (dict(q_st=-1), "EINVAL"), (dict(q_st=BIG), "ESHAPE"),
    (dict(q=P[0] + 1), "EALIGN"), (dict(k_sh=127), "EINVAL"), (dict(k=P[1] + 1), "EALIGN"), (dict(k_sh=BIG), "ESHAPE"),
    (dict(qo_st=0), "EINVAL"), (dict(qo_sh=100), "EINVAL"), (dict(qo=P[6] + 1), "EALIGN"), (dict(ko_st=127), "EINVAL"),
]


@pytest.mark.parametrize("kw,want", SHARED)
@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_head_norm_refuses(kw, want, call):
    assert call(**kw) == _status(want)


def test_head_norm_other_statuses():
    ok = L.PF8_ENODEV if not _gpu() else None
    if ok is not None:  # on a GPU machine these would be launched
        for call in (_fwd, _bwd):
            assert call() == ok
            assert call(axes=3, sections=_sec(24, 20, 20), order=1, pos_sa=4) == ok
            assert call(pos=0, freq=0, pairs=0) == ok
            assert call(w_q=0, dw_q=0) == ok if call is _bwd else call(w_q=0) == ok
        assert _fwd(k=0, hk=0, w_k=0, ko=0) == ok
        assert _bwd(dk=0, hk=0, w_k=0, ko=0, dw_k=0) == ok
        assert _bwd(w_q=0, w_k=0, dw_q=0, dw_k=0, q=0, k=0, ws=0, ws_bytes=0) == ok
    for kw in (dict(qo=0), dict(ko=0), dict(k=0, w_k=0, hk=0)):
        assert _fwd(**kw) == L.PF8_EINVAL
    for kw in (dict(w_q=0), dict(accumulate=2), dict(qo=0, ko=0, dw_q=0, dw_k=0), dict(ws=0), dict(ws_bytes=8), dict(dq=0),
               dict(dk=0)):
        assert _bwd(**kw) == L.PF8_EINVAL
    for kw in (dict(dw_q=P[10] + 2), dict(ws=P[12] + 8), dict(dq=P[8] + 1)):
        assert _bwd(**kw) == L.PF8_EALIGN


def _gpu():
    import torch

    return torch.cuda.is_available()


def test_head_norm_workspace():
    f = L.pf8_qk_norm_rope_bwd_workspace
    assert f(1, 1, 0, 64) > 0 and f(8192, 16, 8, 128) % (4 * 128) == 0
    for bad in ((0, 1, 1, 64), (1, 0, 1, 64), (1, 1, -1, 64), (1, 1, 1, 513), (1, 65537, 1, 64), (BIG, 1, 1, 64), (1, 1, 1, 0)):
        assert f(*bad) == 0


def _act(**kw):
    a = dict(rows=8, cols=64, dd=P[0], lddd=64, z=P[1], ldz=128, act=3, gated=1, dz=P[2], lddz=128, dbias=P[3], accumulate=0,
             ws=P[4], ws_bytes=L.pf8_act_bwd_workspace(8, 64, 1))
    a.update(kw)
    return L.pf8_act_bwd(*a.values(), 0)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(cols=-1), "EINVAL"), (dict(dd=0), "EINVAL"), (dict(z=0), "EINVAL"),
    (dict(act=-1), "EINVAL"), (dict(act=6), "EINVAL"), (dict(act=0), "EINVAL"), (dict(act=0, gated=0), "EINVAL"),
    (dict(gated=2), "EINVAL"), (dict(accumulate=2), "EINVAL"), (dict(dz=0, dbias=0), "EINVAL"), (dict(lddd=63), "EINVAL"),
    (dict(ldz=127), "EINVAL"), (dict(lddz=127), "EINVAL"), (dict(ws=0), "EINVAL"), (dict(ws_bytes=16), "EINVAL"),
    (dict(rows=BIG), "ESHAPE"), (dict(cols=BIG, lddd=BIG, ldz=2 * BIG, lddz=2 * BIG), "ESHAPE"), (dict(ldz=BIG), "ESHAPE"),
    (dict(cols=BIG // 2, lddd=BIG // 2, ldz=BIG - 1, lddz=BIG - 1), "EINVAL"),
    (dict(dd=P[0] + 1), "EALIGN"), (dict(z=P[1] + 1), "EALIGN"), (dict(dz=P[2] + 1), "EALIGN"), (dict(dbias=P[3] + 2), "EALIGN"),
    (dict(ws=P[4] + 8), "EALIGN"),
])
def test_act_refuses(kw, want):
    assert _act(**kw) == _status(want)


def test_act_workspace():
    f = L.pf8_act_bwd_workspace
    assert f(1, 1, 0) > 0 and f(100, 64, 1) == 2 * f(100, 64, 0)
    for bad in ((0, 1, 0), (1, 0, 0), (1, 1, 2), (BIG, 1, 0), (1, BIG, 0), (1, BIG // 2, 1)):
        assert f(*bad) == 0
    if not _gpu():
        assert _act() == L.PF8_ENODEV
        assert _act(z=0, act=0, gated=0, dz=0) == L.PF8_ENODEV


def _act_quant(**kw):
    a = dict(rows=256, cols=128, dd=P[0], lddd=128, z=P[1], ldz=256, act=3, gated=1, qr=P[2], ldqr=256, sr=P[3], ld_sr=256,
             qc=P[4], ldqc=256, sc=P[5], ld_sc=256, dbias=P[6], accumulate=0, ws=P[7],
             ws_bytes=L.pf8_act_bwd_quant_workspace(256, 128, 1))
    a.update(kw)
    return L.pf8_act_bwd_quant(*a.values(), 0)


@pytest.mark.parametrize("kw,want", [
    *((dict([(p, 0)]), "EINVAL") for p in ("dd", "z", "qr", "sr", "qc", "sc", "rows", "cols", "ws")),
    (dict(rows=-128), "EINVAL"), (dict(act=6), "EINVAL"), (dict(act=-1), "EINVAL"), (dict(act=0), "EINVAL"),
    (dict(act=0, gated=0), "EINVAL"), (dict(z=0, act=3, gated=0), "EINVAL"), (dict(gated=2), "EINVAL"),
    (dict(accumulate=2), "EINVAL"), (dict(lddd=127), "EINVAL"), (dict(ldz=255), "EINVAL"), (dict(ldqr=255), "EINVAL"),
    (dict(ld_sr=255), "EINVAL"), (dict(ldqc=255), "EINVAL"), (dict(ld_sc=255), "EINVAL"), (dict(ws_bytes=16), "EINVAL"),
    (dict(rows=192), "ESHAPE"), (dict(cols=64), "ESHAPE"), (dict(rows=BIG, ld_sr=BIG, ldqc=BIG), "ESHAPE"),
    (dict(ldz=BIG), "ESHAPE"), (dict(rows=65536 * 128, ld_sr=65536 * 128, ldqc=65536 * 128), "ESHAPE"),
    (dict(cols=BIG // 2, lddd=BIG // 2, ldz=BIG - 1, ldqr=BIG - 1, ld_sc=BIG - 1), "EINVAL"),
    (dict(dd=P[0] + 2), "EALIGN"), (dict(z=P[1] + 8), "EALIGN"), (dict(lddd=132), "EALIGN"), (dict(ldz=260), "EALIGN"),
    (dict(qr=P[2] + 8), "EALIGN"), (dict(qc=P[4] + 8), "EALIGN"), (dict(ldqr=264), "EALIGN"), (dict(ldqc=264), "EALIGN"),
    (dict(sr=P[3] + 2), "EALIGN"), (dict(sc=P[5] + 2), "EALIGN"), (dict(dbias=P[6] + 2), "EALIGN"), (dict(ws=P[7] + 8), "EALIGN"),
])
def test_act_quant_refuses(kw, want):
    assert _act_quant(**kw) == _status(want)


def test_act_quant_workspace():
    f = L.pf8_act_bwd_quant_workspace
    assert f(256, 128, 0) == 2 * 128 * 4 and f(256, 128, 1) == 2 * f(256, 128, 0)
    for bad in ((0, 128, 0), (128, 0, 0), (128, 128, 2), (64, 128, 0), (128, 64, 0), (BIG, 128, 0), (128, BIG // 2, 1),
                (65536 * 128, 128, 0)):
        assert f(*bad) == 0
    if not _gpu():
        assert _act_quant() == L.PF8_ENODEV
        assert _act_quant(dbias=0, ws=0) == L.PF8_ENODEV
        assert _act_quant(z=0, act=0, gated=0) == L.PF8_ENODEV


def _prod(**kw):
    a = dict(m=8, n=256, k=256, a=P[0], lda=256, a_ds=P[1], ld_as=8, b=P[2], ldb=256, b_ds=P[3], ld_bs=2, bias=P[4], btype=0,
             act=3, gated=1, residual=P[5], ldr=128, z=P[6], ldz=256, d=P[7], ldd=128)
    a.update(kw)
    return L.pf8_fprop_act(*a.values(), 0)


@pytest.mark.parametrize("kw,want", [
    (dict(m=0), "EINVAL"), (dict(n=-1), "EINVAL"), (dict(k=0), "EINVAL"), (dict(a=0), "EINVAL"), (dict(a_ds=0), "EINVAL"),
    (dict(b=0), "EINVAL"), (dict(b_ds=0), "EINVAL"), (dict(d=0), "EINVAL"), (dict(btype=2), "EINVAL"), (dict(gated=2), "EINVAL"),
    (dict(act=-1), "EINVAL"), (dict(act=6), "EINVAL"), (dict(act=0), "EINVAL"), (dict(lda=255), "EINVAL"),
    (dict(ldb=255), "EINVAL"), (dict(ld_as=7), "EINVAL"), (dict(ld_bs=1), "EINVAL"), (dict(ldd=127), "EINVAL"),
    (dict(ldr=127), "EINVAL"), (dict(ldz=255), "EINVAL"), (dict(gated=0), "EINVAL"), (dict(k=192), "ESHAPE"),
    (dict(n=192), "ESHAPE"), (dict(m=BIG, ld_as=BIG), "ESHAPE"), (dict(lda=1 << 24), "ESHAPE"), (dict(ldd=1 << 23), "ESHAPE"),
    (dict(ldz=1 << 23), "ESHAPE"), (dict(ldr=1 << 23), "ESHAPE"), (dict(ldz=BIG), "ESHAPE"),
    (dict(a=P[0] + 8), "EALIGN"), (dict(b=P[2] + 8), "EALIGN"), (dict(lda=264), "EALIGN"), (dict(ldb=264), "EALIGN"),
    (dict(a_ds=P[1] + 2), "EALIGN"), (dict(b_ds=P[3] + 2), "EALIGN"), (dict(bias=P[4] + 1), "EALIGN"),
    (dict(bias=P[4] + 2, btype=1), "EALIGN"), (dict(d=P[7] + 8), "EALIGN"), (dict(ldd=132), "EALIGN"),
    (dict(residual=P[5] + 8), "EALIGN"), (dict(ldr=132), "EALIGN"), (dict(z=P[6] + 8), "EALIGN"), (dict(ldz=260), "EALIGN"),
])
def test_product_refuses(kw, want):
    assert _prod(**kw) == _status(want)


def test_product_takes():
    if not _gpu():
        for kw in (dict(), dict(bias=0), dict(residual=0, ldr=0), dict(z=0, ldz=0), dict(act=0, gated=0, n=128, ldz=128),
                   dict(residual=P[7])):
            assert _prod(**kw) == L.PF8_ENODEV
