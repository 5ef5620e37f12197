"""The FP8 product with bias, activation and residual in its epilogue, on the GPU against the float64 oracle.

Tolerances, fixed before the first run. z before its rounding is within the accumulation contract of
pf8_block_gemm (window and FP32 terms, oracle.contract_allowance less its rounding), plus 2^-22 of |z| + |bias| for
the bias's addition and the parts of a sum over K. An activation turns an error e of z into at most L e, L = 1.2
(the largest slope of the five is 1.13; relu2: 2 |z| + e), and is itself held to 2^-18 max(1, |z|)^2; a gate's
product into |u| e_g + |g| e_u + e_g e_u; a residual adds a rounding of 2^-23 of the terms. Last, d and z are rounded
once: 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
import oracle
from oracle import layer
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ACTS = ["relu", "relu2", "silu", "gelu", "gelu_tanh"]


def _rand(shape, seed, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


def _np(t):
    return t.detach().cpu().double().numpy()


def _codes(n, k, seed, rows, scale=1.0, pitch=None):
    """Random E4M3 codes (of normal values) and power-of-two scales around `scale`, made on the host."""
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(n, k, generator=g) * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    e = torch.randint(-1, 2, (-(-n // rows), k // 128), generator=g)
    s = torch.ldexp(torch.full(e.shape, 2.0 ** round(np.log2(scale / 64))), e)
    if rows == 1:
        s = s.t().contiguous()
    if pitch is None:
        return q.to(DEV), s.to(DEV)
    buf = torch.full((n, pitch), 0x7F, dtype=torch.uint8, device=DEV)  # NaN codes beside the rows
    buf[:, :k] = q.to(DEV)
    return buf[:, :k], s.to(DEV)


def _operands(m, n, k, seed=0, pitch=None):
    qx, sx = _codes(m, k, seed + 1, 1, pitch=pitch)
    qw, sw = _codes(n, k, seed + 2, 128, 1.5 / k ** 0.5, pitch=pitch)
    return qx, sx, qw, sw


def _reference(op, bias, act, gated, residual):
    """(d, its allowance, z, its allowance), allowances without the last rounding."""
    qx, sx, qw, sw = (t.cpu().numpy() for t in op)
    n = qw.shape[0]
    x = oracle.dequant_act_groups(qx, sx)
    w = oracle.decode_e4m3(qw) * np.repeat(np.repeat(sw.astype(np.float64), 128, 0)[:n], 128, 1)
    p = x @ w.T
    e = oracle.contract_allowance(x, w, np.zeros_like(p))
    b = np.zeros(n) if bias is None else _np(bias)
    z = p + b
    e = e + 2.0 ** -22 * (np.abs(z) + np.abs(b))

    def value(v, err):
        slope = 2 * np.abs(v) + err if act == "relu2" else 1.2
        loose = 0.0 if act is None else 2.0 ** -18 * np.maximum(1, np.abs(v)) ** 2
        return layer.act(v, act)[0], slope * err + loose

    if gated:
        h = n // 2
        g, eg = value(z[:, :h], e[:, :h])
        u, eu = z[:, h:], e[:, h:]
        d, ed = g * u, np.abs(u) * eg + np.abs(g) * eu + eg * eu
    else:
        d, ed = value(z, e)
    if residual is not None:
        ed = ed + 2.0 ** -23 * (np.abs(d) + np.abs(_np(residual)))
        d = d + _np(residual)
    return d, ed + 2.0 ** -22 * np.abs(d), z, e


def _near(got, ref, allow, what):
    got = _np(got)
    assert got.shape == ref.shape, what
    tol = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * allow + 2.0 ** -134
    off = np.abs(got - ref)
    assert (off <= tol).all(), f"{what}: {np.max(off / tol)} of the tolerance, {np.count_nonzero(~(off <= tol))} outside"


def _check(m, n, k, act=None, gated=False, bias=None, residual=False, seed=0, pitch=None):
    op = _operands(m, n, k, seed, pitch)
    b = None if bias is None else _rand((n,), seed + 3, 0.5, bias)
    r = _rand((m, -(-(n // 2 if gated else n) // 8) * 8), seed + 4, 2.0)[:, :n // 2 if gated else n] if residual else None
    d, ed, z, ez = _reference(op, b, act, gated, r)
    got, gz = pf8.fprop_act(*op, bias=b, activation=act, gated=gated, residual=r, save_z=True)
    _near(gz, z, ez, "z")
    _near(got, d, ed, "d")
    alone = pf8.fprop_act(*op, bias=b, activation=act, gated=gated, residual=r)
    assert torch.equal(alone, got)


# tokens up to 64 stream the weights, more go by tiles; sizes at and off every tile edge
MS = [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 130, 257, 300]


@pytest.mark.parametrize("m", MS)
@pytest.mark.parametrize("n,k", [(16, 128), (250, 384), (257, 640), (512, 256), (1, 128), (129, 1024)])
def test_sizes(m, n, k):
    _check(m, n, k, "silu" if n % 2 else None, bias=torch.float32, residual=m % 2 == 1)


@pytest.mark.parametrize("m", [1, 31, 64, 128, 200, 256, 300])
@pytest.mark.parametrize("n,k", [(128, 128), (256, 384), (384, 512), (512, 1024), (640, 256)])
def test_gated_sizes(m, n, k):
    _check(m, n, k, "silu", gated=True, bias=BF, residual=m % 2 == 0)


@pytest.mark.parametrize("m", [5, 140])
@pytest.mark.parametrize("act", [None, *ACTS])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bias", [None, BF, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_epilogues(m, act, gated, bias, residual):
    if gated and act is None:
        return
    _check(m, 384, 256, act, gated, bias, residual, seed=7, pitch=400)


@pytest.mark.parametrize("m,n,k", [(40, 200, 3840), (700, 1000, 512), (1024, 768, 768), (520, 1536, 1152)])
@pytest.mark.parametrize("gated", [False, True])
def test_larger(m, n, k, gated):
    if gated:
        n = -(-n // 128) * 128
    _check(m, n, k, "gelu_tanh", gated, BF, True)


def test_many_tiles_match_the_plain_product():
    """More tiles than CUs, whole and ragged: z is the same product as fprop's, each within the contract."""
    for m, n, k in ((4096, 8192, 512), (5000, 8200, 384)):
        op = _operands(m, n, k)
        _, z = pf8.fprop_act(*op, activation="silu", save_z=True)
        d = pf8.fprop_act(*op)
        y = pf8.fprop(*op).float()
        rms = y.square().mean().sqrt()
        # two sums over K of the same truncated products, rounded to bf16: 2 * 2^-8 |y|, and twice the window
        tol = 2.0 ** -7 * y.abs() + 2.0 ** -9 * rms
        for t in (z, d):
            assert ((t.float() - y).abs() <= tol).all()
        g = _rand((m, n), 1)
        got = pf8.fprop_act(*op, residual=g).float()
        # one more rounding of the sum
        assert ((got - (y + g.float())).abs() <= tol + 2.0 ** -8 * (y + g.float()).abs() + 2.0 ** -8 * y.abs()).all()


def test_gated_many_tiles_match_the_plain_product():
    for m, n, k in ((4096, 8192, 512), (5000, 8320, 384)):
        op = _operands(m, n, k)
        d, z = pf8.fprop_act(*op, activation="silu", gated=True, save_z=True)
        y = pf8.fprop(*op).float()
        rms = y.square().mean().sqrt()
        assert ((z.float() - y).abs() <= 2.0 ** -7 * y.abs() + 2.0 ** -9 * rms).all()
        g, u = z[:, :n // 2].float(), z[:, n // 2:].float()
        want = torch.nn.functional.silu(g) * u
        # from rounded g and u: each 2^-8 off, and the result's rounding
        assert ((d.float() - want).abs() <= 2.0 ** -6 * (g.abs() * u.abs()) + 2.0 ** -8 * want.abs() + 1e-6).all()


@pytest.mark.parametrize("m", [3, 150])
def test_places_in_wider_buffers_and_in_place(m):
    n, k = 200, 256
    op = _operands(m, n, k)
    res = _rand((m, 208), 5)
    want, wz = pf8.fprop_act(*op, activation="gelu", residual=res[:, :n], save_z=True)
    buf = torch.full((m, 512), 7.0, dtype=BF, device=DEV)
    zbuf = torch.full((m, 512), 7.0, dtype=BF, device=DEV)
    got, z = pf8.fprop_act(*op, activation="gelu", residual=res[:, :n], out=buf[:, 64:64 + n], z_out=zbuf[:, 8:8 + n])
    assert torch.equal(got, want) and torch.equal(z, wz)
    assert (buf[:, :64] == 7).all() and (buf[:, 64 + n:] == 7).all() and (zbuf[:, :8] == 7).all() and (zbuf[:, 8 + n:] == 7).all()
    tail = res[:, n:].clone()
    assert torch.equal(pf8.fprop_act(*op, activation="gelu", residual=res[:, :n], out=res[:, :n]), want)
    assert torch.equal(res[:, n:], tail)


@pytest.mark.parametrize("m", [1, 48, 200])
def test_repeats_and_replays(m):
    op = list(_operands(m, 512, 768))
    b = _rand((512,), 3)
    a = pf8.fprop_act(*op, bias=b, activation="silu", gated=True)
    assert torch.equal(a, pf8.fprop_act(*op, bias=b, activation="silu", gated=True))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g, gz = pf8.fprop_act(*op, bias=b, activation="silu", gated=True, save_z=True)
    for i in range(3):
        op[0].copy_(_codes(m, 768, 30 + i, 1)[0])
        graph.replay()
        e, ez = pf8.fprop_act(*op, bias=b, activation="silu", gated=True, save_z=True)
        torch.cuda.synchronize()
        assert torch.equal(g, e) and torch.equal(gz, ez)


@pytest.mark.parametrize("m", [2, 100])
def test_infinities_and_not_a_number_stay_in_their_rows(m):
    op = list(_operands(m, 256, 256))
    want = pf8.fprop_act(*op, activation="silu")
    res = torch.zeros((m, 256), dtype=BF, device=DEV)
    res[1, 5], res[0, 7] = float("inf"), float("nan")
    got = pf8.fprop_act(*op, activation="silu", residual=res)
    assert got[1, 5] == float("inf") and got[0, 7].isnan()
    got[1, 5], got[0, 7] = want[1, 5], want[0, 7]
    assert torch.equal(got, want)
    op[0] = op[0].clone()
    op[0][0, 3] = 0x7F
    got = pf8.fprop_act(*op, activation="silu")
    assert got[0].isnan().all() and torch.equal(got[1:], want[1:])


@pytest.mark.parametrize("act", ACTS + [None])
@pytest.mark.parametrize("m", [3, 300, 2100])
def test_infinite_bias(m, act):
    """An activation of an infinite value is its limit, and the other columns are as without one."""
    op = _operands(m, 512, 256)
    bias = _rand((512,), 3, 0.5)
    far = bias.clone()
    far[[1, 40, 300]] = float("inf")
    got, want = (pf8.fprop_act(*op, bias=b, activation=act) for b in (far, bias))
    assert (got[:, [1, 40, 300]] == float("inf")).all()
    if act == "relu":
        far[7] = -float("inf")
        assert (pf8.fprop_act(*op, bias=far, activation=act)[:, 7] == 0).all()
    got[:, [1, 40, 300]] = want[:, [1, 40, 300]]
    assert torch.equal(got, want)
    if act:
        got, want = (pf8.fprop_act(*op, bias=b, activation=act, gated=True) for b in (far, bias))
        assert got[:, [1, 40]].isinf().all()  # (of the factor's sign)
        assert act != "silu" or got[:, 300 - 256].isinf().all()  # (other gates vanish far below zero: 0 times infinity)
        keep = [c for c in range(256) if c not in (1, 7, 40, 44)]
        assert torch.equal(got[:, keep], want[:, keep])


def test_no_tokens_and_refusals():
    op = _operands(4, 256, 256)
    qx, sx, qw, sw = op
    assert pf8.fprop_act(qx[:0], sx[:, :0], qw, sw).shape == (0, 256)
    d, z = pf8.fprop_act(qx[:0], sx[:, :0], qw, sw, activation="relu", gated=True, save_z=True)
    assert d.shape == (0, 128) and z.shape == (0, 256)
    res = _rand((4, 256), 1)
    for bad in (dict(activation="swish"), dict(gated=True), dict(bias=res[0, :255]), dict(bias=res[0].half()),
                dict(residual=res[:3]), dict(residual=res.float()), dict(residual=res[:, 1:]), dict(out=res[:, :255]),
                dict(residual=res, activation="silu", gated=True), dict(qx=qx[:, :128]), dict(sx=sx[:1]), dict(sx=sx[:, :3]),
                dict(sw=sw[:1]), dict(sw=sw.double()), dict(qx=qx.cpu()), dict(qx=qx.float()), dict(sx=sx.cpu()),
                dict(qx=qx[:, :100], qw=qw[:, :100])):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            pf8.fprop_act(**{**dict(qx=qx, sx=sx, qw=qw, sw=sw), **bad})
    odd = _operands(4, 192, 256)
    with pytest.raises(ValueError):
        pf8.fprop_act(*odd, activation="silu", gated=True)
    buf = torch.zeros((4, 1024), dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        pf8.fprop_act(*op, residual=buf[:, :256], out=buf[:, 128:384])
    with pytest.raises(ValueError, match="overlap"):
        pf8.fprop_act(*op, out=buf[:, :256], z_out=buf[:, 248:504])
    pf8.fprop_act(*op, out=buf[:, :256], z_out=buf[:, 256:512])


def test_another_stream():
    op = _operands(2000, 1024, 512)
    want = pf8.fprop_act(*op, activation="relu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = op[0] | 0
        got = pf8.fprop_act(x, *op[1:], activation="relu")
    s.synchronize()
    assert torch.equal(got, want)


def test_drawn_sizes():
    rng = np.random.default_rng(5)
    for i in range(40):
        gated = bool(rng.integers(2))
        n = 128 * int(rng.integers(1, 5)) if gated else int(rng.integers(1, 600))
        act = [None, *ACTS][int(rng.integers(1 if gated else 0, 6))]
        _check(int(rng.integers(1, 400)), n, 128 * int(rng.integers(1, 7)), act, gated,
               [None, BF, torch.float32][int(rng.integers(3))], bool(rng.integers(2)), seed=100 * i)
