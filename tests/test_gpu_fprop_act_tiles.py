"""The tile kernels of the product with its epilogue on the GPU, each by sizes that run it.

``CASES`` names the tile of each size; a host test checks the names, and that every tile is among them. Sizes: K of two
to 32 stages of 64 (the pipeline pads to whole bodies of four and to eight at least), ragged rows and columns, gates that end
inside a scale's 128 columns, fewer tiles than the card holds at once and more (tiles of odd rounds walk K backwards).

Compared with a float64 product on the GPU, with the tolerances of the tests of small sizes: z before its rounding within the
accumulation contract of pf8_block_gemm (7 * 2^-13 of the largest product of each 8, and K / 4 FP32 roundings of the sum of
magnitudes), plus 2^-22 of |z| + |bias| for the bias's addition. An activation turns an error e of z into at most 1.2 e (the
largest slope is 1.13; relu2: (2 |z| + e) e), and is itself held to 2^-18 max(1, |z|)^2; a gate's product into
|u| e_g + |g| e_u + e_g e_u; a residual adds 2^-23 of the terms, the arithmetic of d 2^-22 of it. Last, d and z are rounded
once: 2^-8 of the value."""
import math

import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ACTS = [None, "relu", "relu2", "silu", "gelu", "gelu_tanh"]

# (rows, columns of W) of a tile, gated, m, n, k; the first size of each runs every epilogue
CASES = [
    ((64, 64), False, 1035, 132, 640), ((64, 64), False, 1041, 250, 128), ((64, 64), False, 1067, 131, 384),
    ((64, 64), False, 453, 8209, 512), ((64, 64), False, 903, 8705, 128), ((64, 64), False, 1055, 129, 2048),
    ((64, 64), True, 1027, 384, 640), ((64, 64), True, 1025, 128, 256), ((64, 64), True, 1100, 640, 128),
    ((64, 64), True, 523, 7296, 384), ((64, 64), True, 965, 8320, 128), ((64, 64), True, 1030, 128, 2048),
    ((128, 128), False, 195, 8211, 768), ((128, 128), False, 605, 9798, 256), ((128, 128), False, 265, 9918, 512),
    ((128, 128), False, 65, 8675, 2048), ((128, 128), False, 7817, 1285, 128), ((128, 128), False, 1549, 10019, 512),
    ((128, 128), True, 199, 8576, 768), ((128, 128), True, 583, 9856, 256), ((128, 128), True, 259, 9856, 512),
    ((128, 128), True, 65, 8576, 2048), ((128, 128), True, 1287, 7808, 128), ((128, 128), True, 1541, 10112, 768),
    ((256, 128), False, 385, 8611, 2048), ((256, 128), False, 8261, 593, 768), ((256, 128), False, 6519, 2311, 1152),
    ((256, 128), False, 4225, 4767, 1152),
    ((256, 128), True, 385, 8576, 2048), ((256, 128), True, 1487, 3456, 768), ((256, 128), True, 2341, 6528, 1152),
    ((256, 128), True, 2313, 8832, 1152),
    ((256, 256), False, 775, 9434, 1152), ((256, 256), False, 1177, 9805, 640), ((256, 256), False, 5637, 5003, 640),
    ((256, 256), False, 4519, 10034, 640), ((256, 256), False, 777, 9347, 2048),
    ((256, 256), True, 795, 9600, 1152), ((256, 256), True, 1159, 9856, 640), ((256, 256), True, 3229, 8832, 640),
    ((256, 256), True, 5035, 9088, 640), ((256, 256), True, 771, 9600, 2048),
]
FIRST = [c for i, c in enumerate(CASES) if c[:2] not in [d[:2] for d in CASES[:i]]]


def _rand(shape, seed, scale=1.0, dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _operands(m, n, k, seed=0):
    """Normal values times 64 as codes in rows with NaN codes behind them, power-of-two scales about 1 / 64 and
    1.5 / (64 sqrt k)."""
    def codes(rows, per, scale, seed):
        buf = torch.full((rows, k + 16), 0x7F, dtype=torch.uint8, device=DEV)
        buf[:, :k] = _rand((rows, k), seed, 64.0, F32).to(torch.float8_e4m3fn).view(torch.uint8)
        g = torch.Generator(device=DEV).manual_seed(seed + 1)
        e = torch.randint(-1, 2, (-(-rows // per), k // 128), generator=g, device=DEV)
        return buf[:, :k], torch.ldexp(torch.full(e.shape, 2.0 ** round(math.log2(scale / 64)), device=DEV), e)

    qx, sx = codes(m, 1, 1.0, 10 * seed + 1)
    qw, sw = codes(n, 128, 1.5 / k ** 0.5, 10 * seed + 5)
    return qx, sx.t().contiguous(), qw, sw


def _values(q, s, per):
    n, k = q.shape
    s = s.double().repeat_interleave(per, 0)[:n].repeat_interleave(128, 1)
    return q.contiguous().view(torch.float8_e4m3fn).float().double() * s


def _product(op):
    """X W^T in float64 and what the contract allows for it before its rounding."""
    qx, sx, qw, sw = op
    x, w = _values(qx, sx.t(), 1), _values(qw, sw, 128)
    p = x @ w.t()
    x, w = x.abs(), w.abs()
    e = (x.shape[1] // 4) * 2.0 ** -24 * (x @ w.t())
    group, one = torch.empty_like(p), torch.empty_like(p)
    for g in range(0, x.shape[1], 8):
        group.zero_()
        for k in range(g, g + 8):
            torch.mul(x[:, k, None], w[:, k], out=one)
            torch.maximum(group, one, out=group)
        e += 7 * 2.0 ** -13 * group
    return p, e


def _act(v, name):
    if name == "relu":
        return v.clamp(min=0)
    if name == "relu2":
        return v.clamp(min=0) ** 2
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def _reference(p, e, bias, act, gated, residual):
    b = 0.0 if bias is None else bias.double()
    z = p + b
    e = e + 2.0 ** -22 * (z.abs() + (0.0 if bias is None else b.abs()))

    def value(v, err):
        slope = 2 * v.abs() + err if act == "relu2" else 1.2
        loose = 0.0 if act is None else 2.0 ** -18 * v.abs().clamp(min=1) ** 2
        return _act(v, act), slope * err + loose

    if gated:
        h = z.shape[1] // 2
        (g, eg), u, eu = value(z[:, :h], e[:, :h]), z[:, h:], e[:, h:]
        d, ed = g * u, u.abs() * eg + g.abs() * eu + eg * eu
    else:
        d, ed = value(z, e)
    if residual is not None:
        ed = ed + 2.0 ** -23 * (d.abs() + residual.double().abs())
        d = d + residual.double()
    return d, ed + 2.0 ** -22 * d.abs(), z, e


def _near(got, ref, allow, what):
    assert got.shape == ref.shape, what
    tol = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * allow + 2.0 ** -134
    off = (got.double() - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {float((off / tol).max())} of the tolerance, {int(bad.sum())} outside, first {bad.nonzero()[0].tolist()}"


def _wide(m, n, before, value=7.0):
    """A bf16 [m, n] view with other values beside it, 16-byte aligned rows."""
    buf = torch.full((m, before + -(-n // 8) * 8 + 24), value, dtype=BF, device=DEV)
    return buf, buf[:, before:before + n]


def _claim(tile, gated, m, n, k):
    assert pf8.pf8_fprop_act_tile(m, n, k, int(gated)) == tile[0] * 65536 + tile[1]


def _run(op, pe, act, gated, bias, residual, save_z, what):
    m, n = op[0].shape[0], op[2].shape[0]
    cols = n // 2 if gated else n
    b = None if bias is None else _rand((n,), 3, 0.5, bias)
    r = None
    if residual:
        r = _wide(m, cols, 16)[1]
        r.copy_(_rand((m, cols), 4, 2.0))
    dbuf, d = _wide(m, cols, 8)
    zbuf, z = _wide(m, n, 24)
    pf8.fprop_act(*op, bias=b, activation=act, gated=gated, residual=r, out=d, z_out=z if save_z else None)
    rd, ed, rz, ez = _reference(*pe, b, act, gated, r)
    _near(d, rd, ed, f"{what}: d")
    assert (dbuf[:, :8] == 7).all() and (dbuf[:, 8 + cols:] == 7).all(), what
    if save_z:
        _near(z, rz, ez, f"{what}: z")
        assert (zbuf[:, :24] == 7).all() and (zbuf[:, 24 + n:] == 7).all(), what
    else:
        assert (zbuf == 7).all()


@pytest.mark.parametrize("tile,gated,m,n,k", FIRST)
def test_every_epilogue(tile, gated, m, n, k):
    _claim(tile, gated, m, n, k)
    op = _operands(m, n, k)
    pe = _product(op)
    for act in ACTS[1:] if gated else ACTS:
        for bias in (None, BF, F32):
            for residual in (False, True):
                for save_z in (False, True):
                    _run(op, pe, act, gated, bias, residual, save_z, f"{act} bias {bias} residual {residual} z {save_z}")


@pytest.mark.parametrize("tile,gated,m,n,k", CASES)
def test_sizes(tile, gated, m, n, k):
    _claim(tile, gated, m, n, k)
    op = _operands(m, n, k, seed=1)
    pe = _product(op)
    _run(op, pe, "silu", gated, F32, True, True, "silu, all")
    _run(op, pe, "gelu" if gated else None, gated, None, False, False, "nothing beside")


@pytest.mark.parametrize("tile,gated,m,n,k", FIRST)
def test_in_place_repeats_and_replays(tile, gated, m, n, k):
    """The residual's place may be the result's; the same call gives the same bits, and so do replays with other inputs,
    z kept or not."""
    _claim(tile, gated, m, n, k)
    op = _operands(m, n, k, seed=2)
    op = (op[0].clone(), *op[1:])
    cols = n // 2 if gated else n
    bias = _rand((n,), 3, 0.5, F32)
    rbuf, r = _wide(m, cols, 16)
    r.copy_(_rand((m, cols), 4, 2.0))
    args = dict(bias=bias, activation="silu", gated=gated)
    want, z = pf8.fprop_act(*op, residual=r, save_z=True, **args)
    assert torch.equal(pf8.fprop_act(*op, residual=r, **args), want)
    kept = rbuf.clone()
    assert pf8.fprop_act(*op, residual=r, out=r, **args) is r and torch.equal(r, want)
    kept[:, 16:16 + cols] = want
    assert torch.equal(rbuf, kept)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gd, gz = pf8.fprop_act(*op, residual=r, save_z=True, **args)
    for i in range(3):
        op[0].copy_(_operands(m, 128, k, seed=5 + i)[0])
        r.copy_(_rand((m, cols), 40 + i, 2.0))
        graph.replay()
        ed, ez = pf8.fprop_act(*op, residual=r, save_z=True, **args)
        torch.cuda.synchronize()
        assert torch.equal(gd, ed) and torch.equal(gz, ez) and not torch.equal(gz, z)


@pytest.mark.parametrize("tile,gated,m,n,k", FIRST)
def test_infinities_and_not_a_number_stay_in_their_places(tile, gated, m, n, k):
    _claim(tile, gated, m, n, k)
    qx, sx, qw, sw = _operands(m, n, k, seed=3)
    cols = n // 2 if gated else n
    args = dict(activation="gelu", gated=gated, save_z=True)
    want, wz = pf8.fprop_act(qx, sx, qw, sw, residual=torch.zeros((m, -(-cols // 8) * 8), dtype=BF, device=DEV)[:, :cols], **args)
    res = torch.zeros((m, -(-cols // 8) * 8), dtype=BF, device=DEV)[:, :cols]
    res[1, 5], res[0, cols - 1], res[m - 1, 7] = float("inf"), float("nan"), -float("inf")
    x, w = qx.clone(), qw.clone()
    x[m // 2, 3] = 0x7F   # a token
    w[n - 2, k - 1] = 0x7F  # a column of z, and of d (its factor's)
    got, gz = pf8.fprop_act(x, sx, w, sw, residual=res, **args)
    lost = (n - 2) - (cols if gated else 0)
    assert got[m // 2].isnan().all() and got[:, lost].isnan().all() and gz[m // 2].isnan().all() and gz[:, n - 2].isnan().all()
    assert got[1, 5] == float("inf") and got[0, cols - 1].isnan() and got[m - 1, 7] == -float("inf")
    for t, ref in ((got, want), (gz, wz)):
        t[m // 2] = ref[m // 2]
    got[:, lost], gz[:, n - 2] = want[:, lost], wz[:, n - 2]
    got[1, 5], got[0, cols - 1], got[m - 1, 7] = want[1, 5], want[0, cols - 1], want[m - 1, 7]
    assert torch.equal(got, want) and torch.equal(gz, wz)


@pytest.mark.parametrize("tile,gated,m,n,k", FIRST)
def test_another_stream(tile, gated, m, n, k):
    _claim(tile, gated, m, n, k)
    op = _operands(m, n, k, seed=4)
    want = pf8.fprop_act(*op, activation="relu", gated=gated)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = op[0] | 0
        got = pf8.fprop_act(x, *op[1:], activation="relu", gated=gated)
    s.synchronize()
    assert torch.equal(got, want)
