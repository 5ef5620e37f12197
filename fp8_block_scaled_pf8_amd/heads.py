"""Norms of queries and keys for each head with the rotation by positions: functional forms, autograd, a module.

Per token and head x (include/pf8_layer.h has the details):

    n = x * rsqrt(mean(x^2) + eps) * w            (n = x without a weight)
    of each rotated pair (a, b) of n, with phi = position * inv_freq:
        (a, b) -> rotary_scale * (a cos phi - b sin phi, a sin phi + b cos phi)

in one kernel for queries and keys, read where the projection left them, and backward in one kernel plus the
sums of the weights' gradients. Pair i is (i, pairs + i), or (2 i, 2 i + 1) with ``interleaved``; values
behind the pairs are not rotated. With several position axes (time, height, width) ``sections`` says how many
pairs turn by each: runs of pairs ("blocked"), or the axes in turn ("cycled": pair i to axis i mod axes until
that axis has its share, the rest to the first). With ``unit_offset`` the weights stand for 1 + w.

Functional forms take [tokens, heads, head_dim] tensors and know nothing of autograd; ``fp8_qk_norm_rope``
and the module ``QKNormRope`` take any leading dimensions and are differentiable.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib as L
from .norm import _call, _rows_meet, _vector

Tensor = torch.Tensor


class QKNormRopeGrads(NamedTuple):
    """Gradients of the head norm: bf16 dq and dk (in the inputs' shapes); float32 [head_dim] weights."""
    dq: Tensor
    dk: Optional[Tensor]
    dw_q: Optional[Tensor]
    dw_k: Optional[Tensor]


def _like(t: Tensor, name: str, shape, device) -> Tuple[int, int, int]:
    """``_heads`` of a tensor that has to have another one's shape and device."""
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return _heads(t, name, shape)


def _heads(t: Tensor, name: str, shape) -> Tuple[int, int, int]:
    """(address, stride of tokens, stride of heads) of a bf16 [tokens, heads, head_dim] tensor after its checks."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    tokens, heads, dim = shape
    st, sh, sd = t.stride()
    if tokens == 0:
        return 0, 0, 0
    if sd != 1 and dim != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    if sh < dim and heads > 1:
        raise ValueError(f"the heads of {name} overlap (stride {sh} for {dim} values)")
    return t.data_ptr(), st, sh


def _bytes_at(t: Tensor) -> Tuple[int, int, int, int]:
    """norm._rows_meet's view of a [tokens, heads, head_dim] tensor (at least one value) or of a vector: its tokens
    as rows where the heads of a token lie within its stride, else all of it as one."""
    first = t.data_ptr()
    if t.dim() != 3:
        size = t.numel() * t.element_size()
        return first, first + size, size, 0
    (n, h, d), (st, sh, _) = t.shape, t.stride()
    width = (h - 1) * sh + d
    if n == 1 or st >= width:
        return first, first + 2 * ((n - 1) * st + width), 2 * width, 2 * st if n > 1 else 0
    whole = 2 * ((n - 1) * st + width)
    return first, first + whole, whole, 0


def _may_write(out: Tensor, name: str, others) -> None:
    """Raise if `out` shares memory with itself, or with another operand without being the very same values of it."""
    (n, h, d), (st, sh, _) = out.shape, out.stride()
    if n > 1 and not (st >= (h - 1) * sh + d or (st >= d and (h == 1 or sh >= (n - 1) * st + d))):
        raise ValueError(f"the tokens of {name} overlap")
    a = _bytes_at(out)
    for o, same_ok in others:
        if o is None or o.device != out.device or not o.numel():
            continue
        if _rows_meet(a, _bytes_at(o)) and not (same_ok and o.data_ptr() == a[0] and o.stride() == out.stride()):
            raise ValueError(f"{name} overlaps another operand")


@functools.lru_cache(maxsize=256)
def _sections(sections: Tuple[int, ...], pairs: int, order: str):
    """The host array of an axis split after its checks."""
    if any(not isinstance(s, int) or isinstance(s, bool) or s < 1 for s in sections) or sum(sections) != pairs:
        raise ValueError(f"sections must be positive whole numbers that sum up to the {pairs} rotated pairs, got {sections}")
    n = len(sections)
    if not 1 <= n <= L.PF8_HEAD_MAX_AXES:
        raise ValueError(f"1 to {L.PF8_HEAD_MAX_AXES} position axes, got {n}")
    if order == "cycled" and any(a + n * (s - 1) >= pairs for a, s in enumerate(sections) if a):
        raise ValueError(f"cycled sections {sections} ask for more pairs of an axis than there are in turn")
    return (ctypes.c_int64 * n)(*sections)


_ORDERS = {"blocked": L.PF8_BLOCKED, "cycled": L.PF8_CYCLED}
_FREQ = {torch.float32: L.PF8_F32, torch.float64: L.PF8_F64}
_INDEX = {torch.int32: L.PF8_I32, torch.int64: L.PF8_I64}


def _common(q, k, dims, positions, inv_freq, w_q, w_k, sections, section_order, interleaved, rotary_scale, eps,
            unit_offset):
    """Checks what both directions take; the C call's arguments w_q .. rotary_scale."""
    tokens, dim, dev = dims
    if not 1 <= dim <= L.PF8_HEAD_MAX_DIM:
        raise ValueError(f"heads of 1 to {L.PF8_HEAD_MAX_DIM} values, got {dim}")
    if k is None and w_k is not None:
        raise ValueError("w_k without k")
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq come together")
    wt = w_q if w_q is not None else w_k
    wdt = torch.bfloat16 if wt is None else wt.dtype
    if wdt not in (torch.bfloat16, torch.float32):
        raise TypeError(f"weights must be bfloat16 or float32, got {wdt}")
    pwq = 0 if w_q is None else _vector(w_q, "w_q", dim, wdt, dev)
    pwk = 0 if w_k is None else _vector(w_k, "w_k", dim, wdt, dev)
    wtype, offset = L.PF8_F32 if wdt == torch.float32 else L.PF8_BF16, 1.0 if unit_offset else 0.0
    if positions is None:
        if wt is None:
            raise ValueError("nothing to do: neither positions nor a weight")
        if sections is not None or interleaved or rotary_scale != 1.0:
            raise ValueError("without positions there are no sections, no interleaved pairs and no rotary_scale")
        return pwq, pwk, wtype, offset, eps, 0, 0, 0, 0, 0, 0, 0, 1, None, 0, 0, 1.0
    order = _ORDERS.get(section_order)
    if order is None:
        raise ValueError(f"section_order must be 'blocked' or 'cycled', got {section_order!r}")
    ftype, ptype = _FREQ.get(inv_freq.dtype), _INDEX.get(positions.dtype)
    if ftype is None:
        raise TypeError(f"inv_freq must be float32 or float64, got {inv_freq.dtype}")
    if ptype is None:
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    freqs = inv_freq.shape
    if len(freqs) != 1 or not inv_freq.is_contiguous() or not 1 <= freqs[0] <= dim // 2:
        raise ValueError(f"inv_freq must be a contiguous vector of 1 to {dim // 2} pairs, got {tuple(freqs)}")
    if inv_freq.device != dev or positions.device != dev:
        raise ValueError(f"positions and inv_freq must be on {dev}")
    pairs = freqs[0]
    if sections is None:
        axes, array, want = 1, None, (tokens,)
    else:
        array = _sections(tuple(sections), pairs, section_order)
        axes = len(array)
        want = (axes, tokens)
    if positions.shape != want and not (axes == 1 and positions.shape == (1, tokens)):
        raise ValueError(f"positions must have the shape {want}, got {tuple(positions.shape)}")
    ps = positions.stride()
    return (pwq, pwk, wtype, offset, eps, positions.data_ptr(), ptype, ps[-1], ps[0] if axes > 1 else 0,
            inv_freq.data_ptr(), ftype, pairs, axes, array, order, 1 if interleaved else 0, rotary_scale)


def _shape(t: Tensor, name: str):
    shape = t.shape if isinstance(t, Tensor) else ()
    if len(shape) != 3:
        raise ValueError(f"{name} must be a [tokens, heads, head_dim] tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a HIP device")
    if not 1 <= shape[1] <= L.PF8_HEAD_MAX_HEADS:
        raise ValueError(f"{name} must have 1 to {L.PF8_HEAD_MAX_HEADS} heads, got {shape[1]}")
    return shape


def _k_shape(k: Optional[Tensor], name: str, qs, device):
    if k is None:
        return None
    ks = _shape(k, name)
    if k.device != device:
        raise ValueError(f"{name} must be on {device}, got {k.device}")
    if ks[0] != qs[0] or ks[2] != qs[2]:
        raise ValueError(f"queries {tuple(qs)} and keys {tuple(ks)} differ in tokens or head_dim")
    return ks


def _result(out: Optional[Tensor], name: str, shape, like: Tensor) -> Tuple[Tensor, int, int, int]:
    if out is not None:
        return (out, *_like(out, name, shape, like.device))
    out = torch.empty_like(like, memory_format=torch.contiguous_format)  # (half of what torch.empty takes)
    return out, out.data_ptr(), shape[1] * shape[2], shape[2]


def qk_norm_rope(q: Tensor, k: Optional[Tensor] = None, positions: Optional[Tensor] = None,
                 inv_freq: Optional[Tensor] = None, w_q: Optional[Tensor] = None, w_k: Optional[Tensor] = None,
                 sections: Optional[Sequence[int]] = None, section_order: str = "blocked", interleaved: bool = False,
                 rotary_scale: float = 1.0, eps: float = 1e-6, unit_offset: bool = False,
                 q_out: Optional[Tensor] = None, k_out: Optional[Tensor] = None) -> Tuple[Tensor, Optional[Tensor]]:
    """Norm and rotation of bf16 q [tokens, heads, head_dim] and k [tokens, other heads, head_dim]; returns both.

    Any strides between tokens and heads are taken (views of a packed projection's result). positions are
    int32 or int64 [tokens], or [axes, tokens] with ``sections``; inv_freq is float32 or float64, one for each
    rotated pair, up to head_dim / 2. Weights are bf16 or float32 [head_dim], both of one type; a tensor without
    one is only rotated, and without positions only the norms are taken. q_out and k_out may be q and k
    themselves. No tokens: empty results.
    """
    qs = _shape(q, "q")
    dev, tokens, dim = q.device, qs[0], qs[2]
    ks = _k_shape(k, "k", qs, dev)
    args = _common(q, k, (tokens, dim, dev), positions, inv_freq, w_q, w_k, sections, section_order, interleaved,
                   rotary_scale, eps, unit_offset)
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    aq = _heads(q, "q", qs)
    ak = (0, 0, 0) if k is None else _heads(k, "k", ks)
    oq, *pq = _result(q_out, "q_out", qs, q)
    ok, *pk = (None, 0, 0, 0) if k is None else _result(k_out, "k_out", ks, k)
    if tokens == 0:
        return oq, ok
    if q_out is not None or k_out is not None:
        rest = [(w_q, False), (w_k, False)]
        if q_out is not None:
            _may_write(q_out, "q_out", [(q, True), (k, False), (k_out, False), *rest])
        if k_out is not None:
            _may_write(k_out, "k_out", [(k, True), (q, False), *rest])
    _call(L.pf8_qk_norm_rope, dev, tokens, dim, aq[0], qs[1], aq[1], aq[2], ak[0], 0 if k is None else ks[1], ak[1],
          ak[2], *args, *pq, *pk)
    return oq, ok


def qk_norm_rope_backward(dq: Tensor, dk: Optional[Tensor], q: Optional[Tensor], k: Optional[Tensor] = None,
                          positions: Optional[Tensor] = None, inv_freq: Optional[Tensor] = None,
                          w_q: Optional[Tensor] = None, w_k: Optional[Tensor] = None,
                          sections: Optional[Sequence[int]] = None, section_order: str = "blocked",
                          interleaved: bool = False, rotary_scale: float = 1.0, eps: float = 1e-6,
                          unit_offset: bool = False, dq_out: Optional[Tensor] = None, dk_out: Optional[Tensor] = None,
                          dw_q_out: Optional[Tensor] = None, dw_k_out: Optional[Tensor] = None,
                          accumulate: bool = False) -> QKNormRopeGrads:
    """Gradients of ``qk_norm_rope`` from those of its results.

    q and k are the forward's inputs; a tensor without a weight does not need its own (None). dq_out and
    dk_out may be views of one packed gradient, or dq and dk themselves. dw_q and dw_k are float32 sums over
    tokens and heads, formed in a fixed order; given the ``_out`` buffers (float32 [head_dim]) they are written
    there, or with ``accumulate`` added to what is there.
    """
    qs = _shape(dq, "dq")
    dev, tokens, dim = dq.device, qs[0], qs[2]
    ks = _k_shape(dk, "dk", qs, dev)
    args = _common(dq, dk, (tokens, dim, dev), positions, inv_freq, w_q, w_k, sections, section_order, interleaved,
                   rotary_scale, eps, unit_offset)
    if dk is None and (k is not None or dk_out is not None):
        raise ValueError("k or dk_out without dk")

    def values(t, name, w, shape):
        if w is None:
            return (0, 0, 0)
        if t is None:
            raise ValueError(f"the weight's gradient needs {name}")
        return _like(t, name, shape, dev)

    aq, ak = values(q, "q", w_q, qs), values(k, "k", w_k, ks)
    gq = _heads(dq, "dq", qs)
    gk = (0, 0, 0) if dk is None else _heads(dk, "dk", ks)

    def vector(out, name, w):
        if w is None:
            if out is not None:
                raise ValueError(f"{name} is given, but there is no such weight")
            return None, 0
        if out is None:
            if accumulate:
                raise ValueError(f"accumulate needs {name}")
            out = torch.empty(dim, dtype=torch.float32, device=dev)
            return out, out.data_ptr()
        return out, _vector(out, name, dim, torch.float32, dev)

    dw_q, pwq = vector(dw_q_out, "dw_q_out", w_q)
    dw_k, pwk = vector(dw_k_out, "dw_k_out", w_k)
    oq, *pq = _result(dq_out, "dq_out", qs, dq)
    ok, *pk = (None, 0, 0, 0) if dk is None else _result(dk_out, "dk_out", ks, dk)
    sums = [t for t in (dw_q, dw_k) if t is not None]
    if tokens == 0:
        if not accumulate:
            for t in sums:
                t.zero_()
        return QKNormRopeGrads(oq, ok, dw_q, dw_k)
    if dq_out is not None or dk_out is not None or dw_q_out is not None or dw_k_out is not None:
        vectors = [(t, False) for t in (w_q, w_k, *sums)]
        if dq_out is not None:
            _may_write(dq_out, "dq_out", [(dq, True), (q, True), (dk, False), (k, False), (dk_out, False), *vectors])
        if dk_out is not None:
            _may_write(dk_out, "dk_out", [(dk, True), (k, True), (dq, False), (q, False), *vectors])
        operands = [t for t in (dq, dk, q, k, w_q, w_k) if t is not None and t.numel()]
        for i, t in enumerate(sums):
            if any(_rows_meet(_bytes_at(t), _bytes_at(o)) for o in operands + sums[:i]):
                raise ValueError("a gradient buffer overlaps another operand")
    ws, nws = None, 0
    if sums:
        nws = L.pf8_qk_norm_rope_bwd_workspace(tokens, qs[1], 0 if dk is None else ks[1], dim)
        ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    _call(L.pf8_qk_norm_rope_bwd, dev, tokens, dim, *gq, *gk, aq[0], qs[1], aq[1], aq[2], ak[0],
          0 if dk is None else ks[1], ak[1], ak[2], *args, *pq, *pk, pwq, pwk, int(accumulate),
          0 if ws is None else ws.data_ptr(), nws)
    return QKNormRopeGrads(oq, ok, dw_q, dw_k)


def _as_heads(t: Optional[Tensor]) -> Optional[Tensor]:
    """[..., heads, head_dim] as [tokens, heads, head_dim] that the kernels take, copied only where it has to be."""
    if t is None:
        return None
    t = t.reshape(-1, *t.shape[-2:])
    if t.shape[2] > 1 and t.stride(2) != 1 or t.shape[1] > 1 and t.stride(1) < t.shape[2]:
        t = t.contiguous()
    return t


class QKNormRopeFunction(torch.autograd.Function):
    """Autograd function of the head norm; saves its inputs only (the backward makes the rest again)."""

    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, w_q, w_k, options, main_grads):
        ctx.set_materialize_grads(False)
        q3, k3 = _as_heads(q), _as_heads(k)
        ctx.save_for_backward(q3 if w_q is not None else None, k3 if w_k is not None else None, positions, inv_freq, w_q,
                              w_k)
        ctx.options, ctx.main_grads = options, main_grads
        ctx.shapes = (q.shape, None if k is None else k.shape)
        ctx.leaves = [t is not None and t.requires_grad and t.is_leaf for t in (q, k, w_q, w_k)]
        oq, ok = qk_norm_rope(q3, k3, positions, inv_freq, w_q, w_k, **options)
        return oq.reshape(q.shape), None if k is None else ok.reshape(k.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        q, k, positions, inv_freq, w_q, w_k = ctx.saved_tensors
        need = [ctx.needs_input_grad[i] for i in (0, 1, 4, 5)]
        main = (None, None) if ctx.main_grads is None else ctx.main_grads
        if torch.cuda.is_current_stream_capturing():
            # autograd's accumulator of a leaf belongs to the stream of the first graph that used the
            # leaf; from inside a capture it may wait on that stream, which breaks the capture
            if any(leaf and n and m is None for leaf, n, m in zip(ctx.leaves, need, (None, None, *main))):
                raise RuntimeError("a captured backward cannot hand gradients to leaf tensors: capture "
                                   "qk_norm_rope_backward, or give the weights a main_grad")
        none = (None,) * 8
        if dq is None and dk is None:
            return none

        def one(d, x, w, m, wanted):
            """(dx, dw) of one tensor, as a call for queries alone."""
            if d is None:
                return None, None
            if w is None and positions is None:  # neither normalised nor rotated: a copy
                return d.to(torch.bfloat16), None
            d3 = _as_heads(d.to(torch.bfloat16))
            add = w is not None and m is not None and wanted
            g = qk_norm_rope_backward(d3, None, x, None, positions, inv_freq, w, None, **ctx.options,
                                      dw_q_out=m if add else None, accumulate=add)
            return g.dq, None if add or w is None or not wanted else g.dw_q.to(w.dtype)

        adds = [w is not None and m is not None and n for w, m, n in zip((w_q, w_k), main, need[2:])]
        shared = all(adds) and main[0].data_ptr() == main[1].data_ptr()  # of one weight for both: one after the other
        if dq is None or dk is None or adds[0] != adds[1] or shared:
            gq, gwq = one(dq, q, w_q, main[0], need[2])
            gk, gwk = one(dk, k, w_k, main[1], need[3])
        else:
            g = qk_norm_rope_backward(_as_heads(dq.to(torch.bfloat16)), _as_heads(dk.to(torch.bfloat16)), q, k, positions,
                                      inv_freq, w_q, w_k, **ctx.options, dw_q_out=main[0] if adds[0] else None,
                                      dw_k_out=main[1] if adds[1] else None, accumulate=adds[0])
            gq, gk = g.dq, g.dk
            gwq = g.dw_q.to(w_q.dtype) if w_q is not None and need[2] and not adds[0] else None
            gwk = g.dw_k.to(w_k.dtype) if w_k is not None and need[3] and not adds[1] else None
        return (gq.reshape(ctx.shapes[0]) if gq is not None and need[0] else None,
                gk.reshape(ctx.shapes[1]) if gk is not None and need[1] else None, None, None, gwq, gwk, None, None)


def fp8_qk_norm_rope(q: Tensor, k: Optional[Tensor] = None, positions: Optional[Tensor] = None,
                     inv_freq: Optional[Tensor] = None, w_q: Optional[Tensor] = None, w_k: Optional[Tensor] = None,
                     sections: Optional[Sequence[int]] = None, section_order: str = "blocked", interleaved: bool = False,
                     rotary_scale: float = 1.0, eps: float = 1e-6, unit_offset: bool = False, main_grads=None
                     ) -> Tuple[Tensor, Optional[Tensor]]:
    """The head norm under autograd, for q [..., heads, head_dim] and k [..., other heads, head_dim].

    positions have the leading shape, or one that broadcasts to it ([seq] for [batch, seq]), behind an axis
    dimension with ``sections``. Weights' gradients come in the weights' type, or, where ``main_grads`` = (of
    w_q, of w_k) holds a float32 buffer, are added to it while autograd receives none. A backward pass that is
    being captured into a graph hands no gradient to leaf tensors: it raises, unless they go to ``main_grads``.
    """
    if not isinstance(q, Tensor) or q.dim() < 2 or (k is not None and (k.dim() < 2 or k.shape[:-2] != q.shape[:-2])):
        raise ValueError("q and k must be [..., heads, head_dim] tensors of the same leading shape")
    lead = q.shape[:-2]
    if positions is not None:
        axis = () if sections is None else (positions.shape[0],)
        rest = positions.shape[len(axis):]
        ones = (1,) * (len(lead) - len(rest))  # dimensions that the leading shape has more, behind the axes
        positions = positions.reshape(*axis, *ones, *rest).expand(*axis, *lead).reshape(*axis, -1)
    if main_grads is not None:
        for m, w in zip(main_grads, (w_q, w_k)):
            if m is not None and (w is None or m.dtype != torch.float32 or m.shape != w.shape):
                raise ValueError("a main_grad must be a float32 tensor of its weight's shape")
    options = dict(sections=None if sections is None else tuple(sections), section_order=section_order,
                   interleaved=bool(interleaved), rotary_scale=float(rotary_scale), eps=float(eps),
                   unit_offset=bool(unit_offset))
    return QKNormRopeFunction.apply(q, k, positions, inv_freq, w_q, w_k, options,
                                    None if main_grads is None else tuple(main_grads))


class QKNormRope(torch.nn.Module):
    """Head norms and rotation between the query/key/value projection and attention: ``q, k = m(q, k, positions)``.

    Rotates the first ``rotary_dim`` values of a head (all by default) with frequencies base^(-2 i / rotary_dim)
    for pair i, or with the given ``inv_freq``. ``norm`` False: rotation alone. Weights are kept in ``dtype``; with
    ``fp32_main_grad`` each carries a float32 ``main_grad`` that every backward pass adds to, and its ``grad``
    stays None. The frequencies stay float32 whatever type the module is cast to.
    """

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, base: float = 1e6,
                 sections: Optional[Sequence[int]] = None, section_order: str = "blocked", interleaved: bool = False,
                 rotary_scale: float = 1.0, norm: bool = True, eps: float = 1e-6, unit_offset: bool = False,
                 dtype: torch.dtype = torch.bfloat16, device=None, fp32_main_grad: bool = False, inv_freq=None):
        super().__init__()
        if not 2 <= head_dim <= L.PF8_HEAD_MAX_DIM:
            raise ValueError(f"heads of 2 to {L.PF8_HEAD_MAX_DIM} values, got {head_dim}")
        if inv_freq is None:
            rotary_dim = head_dim // 2 * 2 if rotary_dim is None else rotary_dim
            if rotary_dim % 2 or not 2 <= rotary_dim <= head_dim:
                raise ValueError(f"rotary_dim must be even, from 2 to head_dim, got {rotary_dim}")
            inv_freq = (float(base) ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim))
        elif rotary_dim is not None:
            raise ValueError("rotary_dim and inv_freq exclude one another")
        self._freq = torch.as_tensor(inv_freq, dtype=torch.float32, device="cpu").clone()
        if self._freq.dim() != 1 or not 1 <= self._freq.numel() <= head_dim // 2:
            raise ValueError(f"inv_freq must be a vector of 1 to {head_dim // 2} pairs")
        self.sections = None if sections is None else tuple(sections)
        if section_order not in _ORDERS:
            raise ValueError(f"section_order must be 'blocked' or 'cycled', got {section_order!r}")
        if self.sections is not None:
            _sections(self.sections, self._freq.numel(), section_order)
        self.section_order, self.interleaved, self.rotary_scale = section_order, interleaved, rotary_scale
        self.eps, self.unit_offset = eps, unit_offset

        def weight():
            if not norm:
                return None
            w = torch.nn.Parameter(torch.full((head_dim,), 0.0 if unit_offset else 1.0, dtype=dtype, device=device))
            if fp32_main_grad:
                w.main_grad = torch.zeros(head_dim, dtype=torch.float32, device=w.device)
            return w

        self.w_q, self.w_k = weight(), weight()
        self.register_buffer("inv_freq", self._freq.to(device) if device is not None else self._freq.clone(), persistent=False)

    def _apply(self, fn, recurse=True):
        super()._apply(fn, recurse)
        self.inv_freq = self._freq.to(self.inv_freq.device)  # a cast of the module is not one of its frequencies
        return self

    def forward(self, q: Tensor, k: Optional[Tensor], positions: Tensor) -> Tuple[Tensor, Optional[Tensor]]:
        w_k = self.w_k if k is not None else None
        main = (getattr(self.w_q, "main_grad", None), getattr(w_k, "main_grad", None))
        return fp8_qk_norm_rope(q, k, positions, self.inv_freq, self.w_q, w_k, self.sections, self.section_order,
                                self.interleaved, self.rotary_scale, self.eps, self.unit_offset,
                                None if main == (None, None) else main)
