"""The block norm on the GPU against the float64 oracle.

Tolerances, fixed before the first run. A bf16 output is rounded once: half a step, 2^-8 of the
value, plus 2^-134 below bf16's smallest step. The FP32 work before it: no value passes more than
2^10 roundings of 2^-24 of the magnitudes it is made of (row sums: at most 32 products a thread,
10 levels of a tree and 16 waves; three such sums follow one another, each with under 16 roundings
around it; a sum's relative error counts for the stream's cancellation at most four-fold, as the
data's |beta h| + |alpha g u| stays within 4 |r| in the root mean square), so 2^-14 of the
oracle's "size" of the output. FP32 column sums add at most one rounding per row of the workgroup and
of the partial sums, which the same 2^-14 covers up to 8000 rows of one workgroup.
"""
import numpy as np
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from oracle import train
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed, scale=1.0, dtype=BF, pitch=None):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(shape, generator=g) * scale).to(dtype)
    if pitch is None:
        return x.to(DEV)
    buf = torch.full((shape[0], pitch), 7.0, dtype=dtype, device=DEV)
    buf[:, :shape[1]] = x.to(DEV)
    return buf[:, :shape[1]]


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _case(rows, cols, post=True, pre=True, gate="vector", wdt=BF, seed=0, pitch=None, branch=True, offset=False):
    base = 0.0 if offset else 1.0
    w = lambda s: (base + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(s))).to(wdt).to(DEV)  # noqa: E731
    k = dict(h=_rand((rows, cols), seed + 1, 2.0, pitch=pitch),
             y=_rand((rows, cols), seed + 2, pitch=pitch) if branch else None,
             w_pre=w(seed + 3) if pre else None, w_post=w(seed + 4) if post and branch else None, gate=None)
    if branch and gate == "vector":
        k["gate"] = w(seed + 5)
    elif branch and gate == "full":
        k["gate"] = _rand((rows, cols), seed + 6, pitch=pitch)
    return k


def _oracle_kw(k, sc):
    return dict({n: _np(t) for n, t in k.items()}, beta=sc.get("residual_scale", 1.0), alpha=sc.get("branch_scale", 1.0),
                eps=float(np.float32(sc.get("eps", 1e-6))), offset=1.0 if sc.get("unit_offset") else 0.0)


def _close(got, ref, size, what):
    """Within the module's tolerance, NaN and infinities in the same places."""
    low = got.dtype == BF
    got = _np(got)
    assert got.shape == ref.shape, what
    fine = np.isfinite(ref)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=what)
    np.testing.assert_array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)], err_msg=what)
    tol = (2.0 ** -8 * np.abs(ref[fine]) if low else 0.0) + 2.0 ** -14 * size[fine] + 2.0 ** -134
    off = np.abs(got[fine] - ref[fine])
    assert (off <= tol).all(), f"{what}: {np.max(off / tol)} of the tolerance"


def _check_forward(k, sc, out):
    r, x = out
    R, X, rs, xs = train.block_norm(**_oracle_kw(k, sc))
    if k["y"] is None:
        assert r is k["h"]
    else:
        _close(r, R, rs, "r")
    if X is None:
        assert x is None
    else:
        _close(x, X, xs, "x")


def _check_backward(k, sc, dr, dx, g):
    v, s = train.block_norm_grads(_np(dr), _np(dx), **_oracle_kw(k, sc))
    for n in ("dh", "dy", "dgate", "dw_pre", "dw_post"):
        got, ref = getattr(g, n), getattr(v, n)
        assert (got is None) == (ref is None), n
        if ref is not None:
            _close(got, ref, getattr(s, n), n)


SIZES = [(1, 1), (1, 2048), (3, 7), (5, 64), (2, 511), (4, 512), (3, 513), (1030, 520), (1025, 1000), (1100, 2048),
         (7, 1536), (6, 2047), (2600, 2047), (1300, 4099), (600, 9001), (9000, 5), (8000, 13), (3000, 8), (2500, 999), (5, 2056), (9, 4096), (2, 4100), (3, 5407), (2, 6144), (4, 8192), (2, 8193), (3, 16384),
         (2, 16383), (2, 12000)]


@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(rows, cols):
    k = _case(rows, cols, seed=cols)
    sc = dict(residual_scale=0.75, branch_scale=0.5, eps=1e-5)
    _check_forward(k, sc, pf8.block_norm(**k, **sc))
    dr, dx = _rand((rows, cols), 11, 1e-3), _rand((rows, cols), 12, 1e-3)
    _check_backward(k, sc, dr, dx, pf8.block_norm_backward(dr, dx, **k, **sc))


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", ["none", "vector", "full"])
@pytest.mark.parametrize("wdt", [BF, torch.float32])
@pytest.mark.parametrize("offset", [False, True])
def test_parts(post, pre, gate, wdt, offset):
    rows, cols = 37, 777
    k = _case(rows, cols, post, pre, gate, wdt, seed=3, offset=offset)
    sc = dict(unit_offset=offset, branch_scale=0.25)
    _check_forward(k, sc, pf8.block_norm(**k, **sc))
    dr, dx = _rand((rows, cols), 21), _rand((rows, cols), 22) if pre else None
    for a, b in ((dr, dx), (None, dx), (dr, None)):
        if a is not None or b is not None:
            _check_backward(k, sc, a, b, pf8.block_norm_backward(a, b, **k, **sc))


@pytest.mark.parametrize("wdt", [BF, torch.float32])
def test_without_a_branch(wdt):
    k = _case(65, 1024, branch=False, wdt=wdt)
    _check_forward(k, {}, pf8.block_norm(**k))
    dr, dx = _rand((65, 1024), 1), _rand((65, 1024), 2)
    _check_backward(k, {}, dr, dx, pf8.block_norm_backward(dr, dx, **k))
    _check_backward(k, {}, None, dx, pf8.block_norm_backward(None, dx, **k))


@pytest.mark.parametrize("rows,cols", [(1, 128), (5, 384), (1030, 512), (1100, 2048), (3, 4096), (2, 12288), (2, 16384)])
def test_codes_are_the_quantisers_of_the_same_x(rows, cols):
    k = _case(rows, cols, gate="full", seed=9)
    k["h"][0, :min(cols, 256)] = 0
    k["y"][0, :min(cols, 256)] = 0  # a group of zeros: scale 1
    r, x = pf8.block_norm(**k)
    r2, q, s = pf8.block_norm_quant(**k)
    q1, s1 = pf8.quant_act_1x128(x)
    assert torch.equal(r, r2) and torch.equal(q, q1) and torch.equal(s, s1)


def test_padded_odd_pitches_and_untouched_surroundings():
    rows, cols, pitch = 19, 1001, 1111
    k = _case(rows, cols, gate="full", pitch=pitch)
    bufs = [torch.full((rows + 2, pitch), 5.0, dtype=BF, device=DEV) for _ in range(2)]
    r, x = (b[1:-1, 3:3 + cols] for b in bufs)
    out = pf8.block_norm(**k, r_out=r, x_out=x)
    assert out[0] is r and out[1] is x
    _check_forward(k, {}, out)
    for b, o in zip(bufs, (r, x)):
        o.fill_(5.0)
        assert (b == 5.0).all()
    dr, dx = _rand((rows, cols), 1, pitch=pitch + 1), _rand((rows, cols), 2, pitch=pitch + 2)
    _check_backward(k, {}, dr, dx, pf8.block_norm_backward(dr, dx, **k))


def test_outputs_in_the_inputs_place():
    k = _case(1200, 1536)
    want = pf8.block_norm(**k)
    h, y = k["h"].clone(), k["y"].clone()
    r, x = pf8.block_norm(**{**k, "h": h, "y": y}, r_out=h, x_out=y)
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    h, y = k["h"].clone(), k["y"].clone()
    pf8.block_norm(**{**k, "h": h, "y": y}, r_out=y, x_out=h)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("cols", [3, 509, 1003, 2047, 4099, 9001])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (False, False)])
def test_outputs_in_the_inputs_place_with_odd_rows(cols, post, pre):
    """The last threads of a row read columns that others have already overwritten."""
    k = _case(1500, cols, post, pre, gate="full", seed=cols)
    want = pf8.block_norm(**k)
    for swap in (False, True):
        h, y = k["h"].clone(), k["y"].clone()
        r, x = (y, h) if swap else (h, y)
        pf8.block_norm(**{**k, "h": h, "y": y}, r_out=r, x_out=x if pre else None)
        assert torch.equal(r, want[0]) and (not pre or torch.equal(x, want[1]))


@pytest.mark.parametrize("cols", [5, 512, 777, 2048, 5407, 8192, 9001])
def test_gradients_in_the_inputs_place(cols):
    """What the C interface allows: dh and dy in the memory of dr, dx, h or y."""
    from fp8_block_scaled_pf8_amd import _lib as L
    rows = 700
    k = _case(rows, cols, seed=cols)
    dr, dx = _rand((rows, cols), 31), _rand((rows, cols), 32)
    want = pf8.block_norm_backward(dr, dx, **k)
    ws = torch.empty(L.pf8_block_norm_bwd_workspace(rows, cols), dtype=torch.uint8, device=DEV)
    for i, j in ((0, 3), (1, 2), (2, 3), (3, 1)):
        t = [v.clone() for v in (dr, dx, k["h"], k["y"])]
        sums = torch.empty((3, cols), device=DEV)
        L.check(L.pf8_block_norm_bwd(
            rows, cols, t[0].data_ptr(), cols, t[1].data_ptr(), cols, t[2].data_ptr(), cols, t[3].data_ptr(), cols,
            k["w_post"].data_ptr(), k["gate"].data_ptr(), 0, k["w_pre"].data_ptr(), L.PF8_BF16, 1.0, 1.0, 0.0, 1e-6,
            t[i].data_ptr(), cols, t[j].data_ptr(), cols, sums[2].data_ptr(), 0, sums[0].data_ptr(), sums[1].data_ptr(), 0,
            ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream))
        assert torch.equal(t[i], want.dh) and torch.equal(t[j], want.dy)
        assert all(torch.equal(a, b) for a, b in zip(sums, (want.dw_pre, want.dw_post, want.dgate)))


def test_special_values_stay_in_their_rows():
    k = _case(8, 640, gate="none")
    k["h"][1, 5] = float("nan")
    k["y"][2, 600] = float("inf")
    k["h"][3, 0] = float("-inf")
    k["h"][4], k["y"][4] = 0, 0
    k["h"][5] *= 2.0 ** 60      # squares near the top of FP32's range
    k["y"][6] *= 2.0 ** -60     # squares that vanish beside eps
    for sc in ({}, {"eps": 0.0}):
        if sc:
            k["y"][6] = k["y"][7]  # without eps such squares have no FP32 value
        _check_forward(k, sc, pf8.block_norm(**k, **sc))
    dr, dx = _rand((8, 640), 1), _rand((8, 640), 2)
    g = pf8.block_norm_backward(dr, dx, **k)
    for row in (0, 4, 5, 6, 7):
        assert torch.isfinite(g.dh[row]).all() and torch.isfinite(g.dy[row]).all()
    keep = [0, 4, 7]
    sub = {n: t[keep].contiguous() if t is not None and t.dim() == 2 else t for n, t in k.items()}
    h = pf8.block_norm_backward(dr[keep].contiguous(), dx[keep].contiguous(), **sub)
    assert torch.equal(g.dh[keep], h.dh) and torch.equal(g.dy[keep], h.dy)
    assert torch.isnan(g.dw_pre).any()


@pytest.mark.parametrize("what", ["w_pre", "w_post", "gate", "full gate"])
@pytest.mark.parametrize("cols", [5, 511, 777, 2047, 2041, 4099, 9001])
def test_infinite_weights_near_the_odd_end_of_a_row(cols, what):
    """The last threads of a row read columns that are not theirs: what stands there counts once."""
    k = _case(3, cols, gate="full" if what == "full gate" else "vector", seed=cols)
    at = max(cols - 8, 0)
    if what == "full gate":
        k["gate"][1, at] = float("inf")
    else:
        k[what][at] = float("-inf")
    _check_forward(k, {}, pf8.block_norm(**k))
    dr, dx = _rand((3, cols), 41), _rand((3, cols), 42)
    _check_backward(k, {}, dr, dx, pf8.block_norm_backward(dr, dx, **k))


def test_gradient_against_differences_of_the_kernel():
    """dh and dy against differences of the kernel's own forward, in the direction of each gradient."""
    rows, cols = 4, 256
    k = _case(rows, cols, gate="vector", wdt=torch.float32)
    dr, dx = _rand((rows, cols), 31), _rand((rows, cols), 32)
    g = pf8.block_norm_backward(dr, dx, **k)

    def loss(kk):
        r, x = pf8.block_norm(**kk)
        return float((r.double() * dr.double()).sum() + (x.double() * dx.double()).sum())

    # outputs carry a bf16 rounding of up to 2^-8 |value| each, independent: the loss is off by about
    # 2^-8 / sqrt(3) * sqrt(sum (r dr)^2 + (x dx)^2) < 0.3 on either side (values of order 2, 2048 of them),
    # against a difference of 2 * step * |grad|^2 (|grad|^2 > 500, step 0.1: over 100); curvature: step^2 / 10
    for n, d in (("h", g.dh), ("y", g.dy)):
        lo, hi = dict(k), dict(k)
        step = 0.1
        lo[n], hi[n] = (k[n].float() - step * d.float()).to(BF), (k[n].float() + step * d.float()).to(BF)
        moved = ((hi[n].double() - lo[n].double()) * d.double()).sum().item()
        assert abs((loss(hi) - loss(lo)) / moved - 1) < 0.05, n


def test_accumulate_adds_to_the_buffers():
    k = _case(300, 520, wdt=torch.float32)
    dr, dx = _rand((300, 520), 1), _rand((300, 520), 2)
    one = pf8.block_norm_backward(dr, dx, **k)
    bufs = dict(dw_pre_out=torch.ones(520, device=DEV), dw_post_out=torch.full((520,), 2.0, device=DEV),
                dgate_out=torch.full((520,), 3.0, device=DEV))
    pf8.block_norm_backward(dr, dx, **k, **bufs, accumulate=True)
    for b, o, base in zip(bufs.values(), (one.dw_pre, one.dw_post, one.dgate), (1, 2, 3)):
        assert torch.equal(b, o + base)
    over = pf8.block_norm_backward(dr, dx, **k, **bufs)
    assert torch.equal(over.dw_pre, one.dw_pre) and over.dw_pre is bufs["dw_pre_out"]


def test_same_call_same_bits():
    k = _case(5000, 768, gate="full")
    dr, dx = _rand((5000, 768), 1), _rand((5000, 768), 2)
    a, b = (pf8.block_norm_backward(dr, dx, **k) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_no_tokens():
    k = _case(3, 256)
    k = {n: t[:0] if t.dim() == 2 else t for n, t in k.items()}
    r, x = pf8.block_norm(**k)
    assert r.shape == x.shape == (0, 256)
    r, q, s = pf8.block_norm_quant(**k)
    assert q.shape == (0, 256) and s.shape == (2, 0)
    e = torch.zeros((0, 256), dtype=BF, device=DEV)
    g = pf8.block_norm_backward(e, e, **k)
    assert g.dh.shape == (0, 256) and not g.dw_pre.any() and not g.dgate.any()
    keep = torch.ones(256, device=DEV)
    pf8.block_norm_backward(e, e, **{**k, "w_post": None, "gate": None}, dw_pre_out=keep, accumulate=True)
    assert (keep == 1).all()


def test_past_two_to_the_31_elements():
    rows, cols = (1 << 31) // 4096 + 3, 4096
    g = torch.Generator(device=DEV).manual_seed(1)
    h = torch.empty((rows, cols), dtype=BF, device=DEV).normal_(generator=g)
    w = torch.ones(cols, dtype=BF, device=DEV)
    r, x = pf8.block_norm(h, h, w, w)
    at = [0, rows // 2, rows - 2, rows - 1]
    k = dict(h=h[at].contiguous(), y=h[at].contiguous(), w_pre=w, w_post=w, gate=None)
    _check_forward(k, {}, (r[at].contiguous(), x[at].contiguous()))
    d = pf8.block_norm_backward(x, None, h, h, None, w)
    v, s = train.block_norm_grads(_np(x[at]), None, **_oracle_kw({**k, "w_pre": None}, {}))
    _close(d.dy[at], v.dy, s.dy, "dy")


def test_another_stream():
    k = _case(2000, 2048)
    want = pf8.block_norm(**k)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kk = {n: t.clone() for n, t in k.items()}
        r, x = pf8.block_norm(**kk)
    side.synchronize()
    assert torch.equal(r, want[0]) and torch.equal(x, want[1])


def test_captured_forward_and_backward_replay():
    k = _case(700, 1536)
    dr, dx = _rand((700, 1536), 1), _rand((700, 1536), 2)
    acc = torch.zeros(1536, device=DEV)
    pf8.block_norm(**k), pf8.block_norm_backward(dr, dx, **k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, x = pf8.block_norm(**k)
        g = pf8.block_norm_backward(dr, dx, **k)
    for i in range(4):
        k["h"].copy_(_rand((700, 1536), 50 + i, 2.0))
        dx.copy_(_rand((700, 1536), 60 + i))
        graph.replay()
        got = [t.clone() for t in (r, x, *g)]
        want = [*pf8.block_norm(**k), *pf8.block_norm_backward(dr, dx, **k)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    del acc


# ------------------------------------------------------------------------------ autograd and module
@pytest.mark.parametrize("gate", ["none", "vector", "full"])
def test_autograd_gives_the_functional_gradients(gate):
    k = _case(2 * 64, 512, gate=gate)
    lead = (2, 64, 512)
    leaf = {n: (t.reshape(lead) if t.dim() == 2 else t).clone().requires_grad_(True) for n, t in k.items() if t is not None}
    r, x = pf8.fp8_block_norm(**leaf, branch_scale=0.5)
    dr, dx = _rand((128, 512), 1), _rand((128, 512), 2)
    torch.autograd.backward([r, x], [dr.reshape(lead), dx.reshape(lead)])
    g = pf8.block_norm_backward(dr, dx, **k, branch_scale=0.5)
    assert torch.equal(leaf["h"].grad.reshape(128, 512), g.dh) and torch.equal(leaf["y"].grad.reshape(128, 512), g.dy)
    assert torch.equal(leaf["w_pre"].grad, g.dw_pre.to(BF)) and torch.equal(leaf["w_post"].grad, g.dw_post.to(BF))
    if gate == "vector":
        assert torch.equal(leaf["gate"].grad, g.dgate.to(BF))
    elif gate == "full":
        assert torch.equal(leaf["gate"].grad.reshape(128, 512), g.dgate)


def test_autograd_with_one_output_used_and_views():
    k = _case(96, 256, gate="none")
    h, y = (k[n].t().contiguous().t().requires_grad_(True) for n in ("h", "y"))  # columns first in memory
    w = k["w_pre"].clone().requires_grad_(True)
    r, x = pf8.fp8_block_norm(h, y, w)
    r.sum().backward()  # the gradient is an expanded scalar
    assert (h.grad == 1).all() and (y.grad == 1).all() and w.grad is None
    r, x = pf8.fp8_block_norm(k["h"], None, w)
    assert r is k["h"]
    x.backward(torch.ones_like(x))
    g = pf8.block_norm_backward(None, torch.ones((96, 256), dtype=BF, device=DEV), k["h"], None, k["w_pre"])
    assert torch.equal(w.grad, g.dw_pre.to(BF))


def test_module_around_fp8_linear_trains_its_main_grads():
    """norm -> FP8 layer -> norm, two micro-batches, against the functional calls on the same values."""
    tokens, cols = 256, 512
    lin = pf8.Fp8Linear(cols, cols, device=DEV, fp32_main_grad=True)
    first = pf8.BlockNorm(cols, post=False, device=DEV, fp32_main_grad=True)
    second = pf8.BlockNorm(cols, gate=True, gate_init=0.5, branch_scale=0.5, device=DEV, fp32_main_grad=True)
    want = [torch.zeros(cols, device=DEV) for _ in range(4)]
    for mb in range(2):
        h = _rand((2, tokens // 2, cols), 70 + mb, 2.0).requires_grad_(True)
        s, x = first(h)
        y = lin(x)
        y.retain_grad(), x.retain_grad()
        r, z = second(s, y)
        dr, dz = _rand(r.shape, 80 + mb, 1e-2), _rand(r.shape, 90 + mb, 1e-2)
        torch.autograd.backward([r, z], [dr, dz])
        f = lambda t: t.detach().reshape(tokens, cols)  # noqa: E731
        g = pf8.block_norm_backward(f(dr), f(dz), f(h), f(y), second.w_pre.detach(), second.w_post.detach(),
                                    second.gate.detach(), branch_scale=0.5)
        assert torch.equal(f(y.grad), g.dy)
        p = pf8.block_norm_backward(None, f(x.grad), f(h), None, first.w_pre.detach())
        assert torch.equal(h.grad.reshape(tokens, cols), (p.dh.float() + g.dh.float()).to(BF))
        for w, d in zip(want, (p.dw_pre, g.dw_pre, g.dw_post, g.dgate)):
            w += d
    for w, par in zip(want, (first.w_pre, second.w_pre, second.w_post, second.gate)):
        assert par.grad is None and torch.equal(par.main_grad, w)
    assert lin.weight.main_grad.abs().sum() > 0


def test_module_codes_feed_the_fp8_gemm():
    norm = pf8.BlockNorm(1024, device=DEV)
    k = _case(200, 1024)
    qw, _, sw = pf8.quant_w_128x128(_rand((512, 1024), 5, 0.02))
    with torch.no_grad():
        r, x = norm(k["h"], k["y"])
    r2, q, s = norm.quantised(k["h"], k["y"])
    assert torch.equal(r, r2)
    assert torch.equal(pf8.fprop(q, s, qw, sw), pf8.fprop(*pf8.quant_act_1x128(x), qw, sw))


def test_a_captured_backward_refuses_leaf_gradients():
    k = _case(64, 256, gate="none")
    w = k["w_pre"].clone().requires_grad_(True)
    main = torch.zeros(256, device=DEV)
    h0 = k["h"].clone().requires_grad_(True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, x = pf8.fp8_block_norm(k["h"], None, w)
        with pytest.raises(RuntimeError, match="captured backward"):
            x.backward(torch.ones_like(x))
        _, x = pf8.fp8_block_norm(k["h"], None, w, main_grads=(main, None, None))
        x.backward(torch.ones_like(x))
    assert h0.grad is None
    main.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    g = pf8.block_norm_backward(None, torch.ones((64, 256), dtype=BF, device=DEV), k["h"], None, k["w_pre"])
    one = g.dw_pre
    assert torch.equal(main, one + one + one) and w.grad is None


def test_wrappers_refuse_before_any_launch():
    k = _case(8, 256, gate="full")
    bad = [
        (dict(h=k["h"].float()), TypeError), (dict(y=k["y"][:4]), ValueError), (dict(w_pre=k["w_pre"][:8]), ValueError),
        (dict(w_pre=k["w_pre"].half()), TypeError), (dict(w_post=k["w_post"].float()), TypeError),
        (dict(gate=k["gate"][:1].expand(8, 256)), ValueError), (dict(h=k["h"].t()), ValueError),
        (dict(y=None), ValueError), (dict(w_pre=k["w_pre"].cpu()), ValueError), (dict(eps=-1.0), RuntimeError),
        (dict(eps=float("nan")), RuntimeError), (dict(branch_scale=float("inf")), RuntimeError),
        (dict(r_out=k["gate"]), ValueError), (dict(x_out=k["h"], r_out=k["h"]), ValueError),
        (dict(x_out=k["h"][:, :255]), ValueError),
    ]
    for change, err in bad:
        with pytest.raises(err):
            pf8.block_norm(**{**k, **change})
    wide = torch.zeros(9 * 256, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        pf8.block_norm(wide[:2048].view(8, 256), k["y"], r_out=wide[256:].view(8, 256))
    with pytest.raises(ValueError, match="128"):
        pf8.block_norm_quant(k["h"][:, :100], None, k["w_pre"][:100])
    with pytest.raises(ValueError):
        pf8.block_norm_backward(None, None, **k)
    with pytest.raises(ValueError, match="accumulate needs"):
        pf8.block_norm_backward(k["h"], k["h"], **k, accumulate=True)
    with pytest.raises(ValueError):
        pf8.block_norm(torch.zeros((2, 40000), dtype=BF, device=DEV), None, torch.zeros(40000, dtype=BF, device=DEV))
