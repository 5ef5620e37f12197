"""The layer's steps together, as a decoder layer runs them: the FP8 linear layer with its epilogue under autograd,
and a whole layer around attention, forward, backward and for single tokens.

The linear layer's gradients are compared with the same steps made one by one from entry points that are tested by
themselves: equal bit for bit. The whole layer is compared with the same layer from plain torch operations in
float64 whose products take the same FP8 rounding of their operands (dequantised codes); tolerances at each test."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_pf8_amd as pf8
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed, scale=1.0, dtype=BF):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


@pytest.mark.parametrize("activation,gated", [(None, False), ("gelu", False), ("relu2", False), ("silu", True), ("gelu_tanh", True)])
@pytest.mark.parametrize("bias", [None, BF, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_linear_layer_is_its_steps(activation, gated, bias, residual):
    m, k, n = 256, 384, 512
    cols = n // 2 if gated else n
    x, w = _rand((2, 128, k), 1).requires_grad_(), _rand((n, k), 2, 0.05).requires_grad_()
    b = None if bias is None else _rand((n,), 3, 0.3, bias).requires_grad_()
    r = _rand((2, 128, cols), 4).requires_grad_() if residual else None
    d = pf8.fp8_linear_act(x, w, b, activation, gated, r)
    dd = _rand(d.shape, 5, 1e-2)
    d.backward(dd)
    qx, sx, qxt, sxt = pf8.quant_act_dual(x.detach().reshape(m, k))
    qw, qwt, sw = pf8.quant_w_128x128(w.detach())
    want, z = pf8.fprop_act(qx, sx, qw, sw, None if b is None else b.detach(), activation, gated,
                            None if r is None else r.detach().reshape(m, cols), save_z=True)
    assert torch.equal(d.reshape(m, cols), want)
    dz, dbias = dd.reshape(m, cols), None
    if activation is not None or b is not None:
        z = z if activation else None
        if b is not None:
            dbias = pf8.act_backward_quant(dz, z, activation, gated, bias_grad=True).dbias
        dz = pf8.act_backward(dz, z, activation, gated, bias_grad=b is not None).dz
    q, s, qt, st = pf8.quant_act_dual(dz)
    assert torch.equal(x.grad.reshape(m, k), pf8.dgrad(q, s, qwt, sw))
    assert torch.equal(w.grad, pf8.wgrad(qt, st, qxt, sxt))
    if b is not None:
        assert torch.equal(b.grad, dbias.to(bias))
    if r is not None:
        assert torch.equal(r.grad, dd)


@pytest.mark.parametrize("n", [128, 384])
def test_gate_over_half_a_group(n):
    """A gate's half may end inside a scale's 128 columns; the layer still is its steps."""
    m, k = 128, 256
    x, w, b = _rand((m, k), 1).requires_grad_(), _rand((n, k), 2, 0.05).requires_grad_(), _rand((n,), 3).requires_grad_()
    dd = _rand((m, n // 2), 5, 1e-2)
    pf8.fp8_linear_act(x, w, b, "silu", True).backward(dd)
    qx, sx, qxt, sxt = pf8.quant_act_dual(x.detach())
    qw, qwt, sw = pf8.quant_w_128x128(w.detach())
    z = pf8.fprop_act(qx, sx, qw, sw, b.detach(), "silu", True, save_z=True)[1]
    dz, dbias = pf8.act_backward(dd, z, "silu", True, bias_grad=True)
    q, s, qt, st = pf8.quant_act_dual(dz)
    assert torch.equal(x.grad, pf8.dgrad(q, s, qwt, sw)) and torch.equal(w.grad, pf8.wgrad(qt, st, qxt, sxt))
    assert torch.equal(b.grad, dbias.to(BF))


def test_gradients_of_a_subset():
    """Only the asked-for gradients are made, each the same as among all of them."""
    m, k, n = 128, 256, 512
    w, x, b, r = _rand((n, k), 2, 0.05), _rand((m, k), 1), _rand((n,), 3), _rand((m, n // 2), 4)
    dd = _rand((1, n // 2), 5, 1e-2).expand(m, n // 2)  # broadcast: one row for all tokens
    def grads(flags):
        ts = [t.clone().requires_grad_(f) for t, f in zip((x, w, b, r), flags)]
        pf8.fp8_linear_act(ts[0], ts[1], ts[2], "silu", True, ts[3]).backward(dd)
        return [t.grad for t in ts]
    every = grads((True,) * 4)
    for i in range(4):
        got = grads(tuple(j == i for j in range(4)))
        assert torch.equal(got[i], every[i]) and all(g is None for j, g in enumerate(got) if j != i)


def test_linear_layer_main_grads_and_inference():
    m, k, n = 128, 256, 512
    lin = pf8.Fp8Linear(k, n, device=DEV, fp32_main_grad=True, bias=True, activation="silu", gated=True)
    plain = pf8.Fp8Linear(k, n, device=DEV, weight=lin.weight.detach().clone(), bias=True, activation="silu", gated=True)
    with torch.no_grad():
        lin.bias.copy_(_rand((n,), 1))
        plain.bias.copy_(lin.bias)
    x, res, dd = _rand((m, k), 2), _rand((m, n // 2), 3), _rand((m, n // 2), 4, 1e-2)
    for layer in (lin, plain):
        for _ in range(2):
            layer(x, res).backward(dd)
    assert lin.weight.grad is None and lin.bias.grad is None
    # 2 g in FP32 against the sum of two bf16 gradients
    for a, b in ((lin.weight.main_grad, plain.weight.grad), (lin.bias.main_grad, plain.bias.grad)):
        assert ((a - b.float()).abs() <= 2.0 ** -8 * a.abs() + 1e-30).all()
    want = lin(x, res).detach()
    assert torch.equal(lin.infer(x, res), want)
    assert torch.equal(lin.infer(pf8.quant_act_1x128(x), res), want)
    for t in (1, 3, 17, 65, 100):  # any number of tokens: z differs in the order of its sum over K alone
        got = lin.infer(x[:t].reshape(1, t, k), res[:t].reshape(1, t, -1))
        assert got.shape == (1, t, n // 2)
        assert ((got[0].float() - want[:t].float()).abs() <= 2.0 ** -6 * want[:t].float().abs() + 2.0 ** -8).all()
    assert lin.infer(x[:0]).shape == (0, n // 2)
    with pytest.raises(ValueError):
        lin.infer(x, res[:5])
    with pytest.raises(ValueError):
        pf8.Fp8Linear(k, n, device=DEV, gated=True)
    with pytest.raises(ValueError):
        lin(x[:100], res[:100])  # training needs whole groups of 128 tokens


def test_no_tokens():
    lin = pf8.Fp8Linear(256, 512, device=DEV, bias=True, activation="relu")
    x = _rand((0, 256), 1).requires_grad_()
    lin(x, _rand((0, 512), 2)).sum().backward()
    assert x.grad.shape == x.shape and (lin.weight.grad == 0).all() and (lin.bias.grad == 0).all()


def test_captured_backward():
    """Main gradients are added to inside a graph; a gradient for a leaf is refused."""
    lin = pf8.Fp8Linear(256, 512, device=DEV, fp32_main_grad=True, bias=True, activation="silu", gated=True)
    x, dd = _rand((128, 256), 1), _rand((128, 256), 2, 1e-2)
    lin(x).backward(dd)
    one = (lin.weight.main_grad.clone(), lin.bias.main_grad.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin(x).backward(dd)
    for i in range(3):
        lin.weight.main_grad.zero_(), lin.bias.main_grad.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lin.weight.main_grad, one[0]) and torch.equal(lin.bias.main_grad, one[1])
    leaf = x.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="leaf"):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lin(leaf).backward(dd)


class Layer(torch.nn.Module):
    """A decoder layer: norm, q/k/v product, head norms and rotation, attention, output product onto the stream,
    norm, gated product, down product onto the stream."""

    def __init__(self, hidden, heads, kv, dim, ffn):
        super().__init__()
        self.h, self.kv, self.d = heads, kv, dim
        self.norm1, self.norm2 = pf8.BlockNorm(hidden, post=False, device=DEV), pf8.BlockNorm(hidden, post=False, device=DEV)
        self.qkv = pf8.Fp8Linear(hidden, (heads + 2 * kv) * dim, device=DEV, bias=True)
        self.rope = pf8.QKNormRope(dim, base=1e4, device=DEV)
        self.out = pf8.Fp8Linear(heads * dim, hidden, device=DEV)
        self.up = pf8.Fp8Linear(hidden, 2 * ffn, device=DEV, activation="silu", gated=True)
        self.down = pf8.Fp8Linear(ffn, hidden, device=DEV)

    def split(self, qkv):
        return [t.unflatten(-1, (-1, self.d)) for t in qkv.split([self.h * self.d, self.kv * self.d, self.kv * self.d], -1)]

    def attend(self, q, k, v, mask):
        """Causal attention in the values' own type, written out."""
        g = self.h // self.kv
        k, v = k.repeat_interleave(g, -2).transpose(-2, -3), v.repeat_interleave(g, -2).transpose(-2, -3)
        s = torch.matmul(q.transpose(-2, -3).contiguous(), k.transpose(-1, -2).contiguous()) / self.d ** 0.5
        p = torch.softmax(s.masked_fill(~mask, float("-inf")), -1)
        return torch.matmul(p, v.contiguous()).transpose(-2, -3).flatten(-2)

    def forward(self, x, pos):
        q, k, v = self.split(self.qkv(self.norm1(x)[1]))
        q, k = self.rope(q, k, pos)
        mask = torch.ones(x.shape[-2], x.shape[-2], dtype=torch.bool, device=x.device).tril()
        a = self.attend(q.float(), k.float(), v.float(), mask).to(BF)
        x = self.out(a, x)
        return self.down(self.up(self.norm2(x)[1]), x)

    def plain(self, x, pos):
        """The same from plain operations in float64, on the codes' values; gradients pass the rounding to codes."""
        def fp8(t, rows):
            with torch.no_grad():
                v = t.detach().float().reshape(-1, t.shape[-1])
                w = v.view(-1, rows, v.shape[1] // 128, 128)
                man, ex = torch.frexp(w.abs().amax((1, 3), keepdim=True))
                sc = torch.ldexp(torch.ones_like(man), ex - 9 + (man > 0.875).int())
                back = ((w / sc).to(torch.float8_e4m3fn).float() * sc).view(v.shape).reshape(t.shape)
            return t + (back.double() - t.detach())

        low = lambda t: t + (t.detach().to(BF).double() - t.detach())  # noqa: E731 (rounding to bf16)
        prod = lambda t, lin: fp8(t, 1) @ fp8(lin.weight.double(), 128).t()  # noqa: E731
        norm = lambda t, w: low(t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w.double())  # noqa: E731
        qkv = low(prod(norm(x, self.norm1.w_pre), self.qkv) + self.qkv.bias.double())
        q, k, v = self.split(qkv)
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV), pos[:, None].double() * self.rope.inv_freq.double())[:, None]

        def head(t, w):
            n = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            c = torch.complex(n[..., :self.d // 2], n[..., self.d // 2:]) * turn
            return low(torch.cat([c.real, c.imag], -1))

        q, k = head(q, self.rope.w_q), head(k, self.rope.w_k)
        mask = torch.ones(x.shape[-2], x.shape[-2], dtype=torch.bool, device=x.device).tril()
        a = low(self.attend(q, k, v, mask))
        x = low(prod(a, self.out) + x)
        z = prod(norm(x, self.norm2.w_pre), self.up)
        n = z.shape[-1] // 2
        y = low(torch.nn.functional.silu(z[..., :n]) * z[..., n:])
        return low(prod(y, self.down) + x)


def _layer():
    torch.manual_seed(1)
    m = Layer(256, 4, 2, 64, 384)
    with torch.no_grad():
        m.qkv.bias.copy_(_rand(m.qkv.bias.shape, 1, 0.2))
        for w in (m.rope.w_q, m.rope.w_k, m.norm1.w_pre, m.norm2.w_pre):
            w.copy_(1 + _rand(w.shape, 2, 0.2))
    return m


def test_whole_layer_forward_backward():
    """Against the float64 layer on the same rounded operands: what differs are roundings that fall to the other side. A
    bf16 value next to a code's border gives a code one step (2^-3 of its value at most) off, for under one in 2^4
    of the values that are themselves off by a bf16 step (under one in 2^3): root mean squares of the result within
    2^-3 * sqrt(2^-7) = 1.1 % of one product; three follow one another: 2 % asked. Gradients also round their own operands
    to codes, which the plain layer does not: 2^-4 at most and about 2.6 % in the root mean square for each of up
    to four products in a row: 8 % asked."""
    m = _layer()
    x = _rand((128, 256), 3).requires_grad_()
    pos = torch.arange(128, device=DEV) + 1000
    y = m(x, pos)
    dy = _rand(y.shape, 4)
    y.backward(dy)
    got = {"x": x.grad, **{n: p.grad.clone() for n, p in m.named_parameters()}}
    m.zero_grad()
    xd = x.detach().double().requires_grad_()
    yd = m.plain(xd, pos)
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(y, yd) <= 0.02
    yd.backward(dy.double())
    want = {"x": xd.grad, **{n: p.grad for n, p in m.named_parameters()}}
    off = {n: rel(got[n], want[n].double()) for n in want}
    assert max(off.values()) <= 0.08, off


def test_single_tokens_follow_the_whole_layer():
    """Token by token with a cache of keys and values, by the forms without gradients: the last token's result as the
    whole layer has it. Products sum over K in another order and round to the other side of a border as above: 2 %."""
    m = _layer()
    x = _rand((128, 256), 3)
    pos = torch.arange(128, device=DEV) + 1000
    with torch.no_grad():
        want = m(x, pos)
        _, qs, ss = m.norm1.quantised(x[:127])
        q, k, v = m.split(m.qkv.infer((qs, ss)))
        _, k = pf8.qk_norm_rope(q, k, pos[:127], m.rope.inv_freq, m.rope.w_q, m.rope.w_k)
        one = x[127:]
        _, qs, ss = m.norm1.quantised(one)
        q1, k1, v1 = m.split(m.qkv.infer((qs, ss)))
        pf8.qk_norm_rope(q1, k1, pos[127:], m.rope.inv_freq, m.rope.w_q, m.rope.w_k, q_out=q1, k_out=k1)
        k, v = torch.cat([k, k1]), torch.cat([v, v1])
        a = m.attend(q1.float(), k.float(), v.float(), torch.ones(1, 128, dtype=torch.bool, device=DEV)).to(BF)
        h = m.out.infer(a, one)
        _, qs, ss = m.norm2.quantised(h)
        y = m.down.infer(m.up.infer((qs, ss)), h)
    assert float((y.double() - want[127:].double()).norm() / want[127:].double().norm()) <= 0.02
