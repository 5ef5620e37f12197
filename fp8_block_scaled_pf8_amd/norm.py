"""The block norm between two FP8 projections: functional forms, autograd and a module.

Per token of the residual stream h, with a branch's result y (include/pf8_train.h has the details):

    u = y * rsqrt(mean(y^2) + eps) * w_post          norm after the block (u = y without w_post)
    r = residual_scale * h + branch_scale * gate * u  gate and residual sum
    x = r * rsqrt(mean(r^2) + eps) * w_pre            norm before the next block

in one kernel, and backward in one kernel plus the column sums of the weights' gradients. With
``block_norm_quant`` x leaves as E4M3 codes and 1x128 scales, which ``fprop`` takes as they are.
With ``unit_offset`` the weights stand for 1 + w.

Functional forms take 2-D tensors and know nothing of autograd; ``fp8_block_norm`` and the module
``BlockNorm`` take any leading dimensions and are differentiable.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib as L
from .ops import GROUP, _call, code_buffer

Tensor = torch.Tensor


class BlockNormGrads(NamedTuple):
    """Gradients of a block norm: bf16 dh, dy (and dgate of a [tokens, cols] gate); float32 [cols] weights."""
    dh: Optional[Tensor]
    dy: Optional[Tensor]
    dgate: Optional[Tensor]
    dw_pre: Optional[Tensor]
    dw_post: Optional[Tensor]


def _rows(t: Tensor, name: str, shape, device) -> Tuple[int, int]:
    """(address, pitch) of a bf16 [rows, cols] tensor after its checks."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    if shape[0] <= 1:
        return t.data_ptr(), max(s0, shape[1])
    if s0 < shape[1]:
        raise ValueError(f"the rows of {name} overlap (stride {s0} for {shape[1]} columns)")
    return t.data_ptr(), s0


def _vector(t: Tensor, name: str, cols: int, dtype, device) -> int:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (weights and a [cols] gate share one type), got {t.dtype}")
    if t.shape != (cols,):
        raise ValueError(f"{name} must have the shape ({cols},), got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _inputs(h: Tensor, y: Optional[Tensor], w_pre, w_post, gate, residual_scale, branch_scale, eps, unit_offset):
    """Checks what both directions take; (rows, cols, the C call's arguments h .. eps)."""
    if not isinstance(h, Tensor) or h.dim() != 2:
        raise ValueError("h must be a 2-D tensor")
    if not h.is_cuda:
        raise ValueError("h must be on a HIP device")
    shape, dev = h.shape, h.device
    rows, cols = shape
    if not 1 <= cols <= L.PF8_NORM_MAX_COLS:
        raise ValueError(f"the block norm takes 1 to {L.PF8_NORM_MAX_COLS} columns, got {cols}")
    ph, ldh = _rows(h, "h", shape, dev)
    py = ldy = pg = ldg = pn = pp = 0
    full = False
    if y is not None:
        py, ldy = _rows(y, "y", shape, dev)
        if gate is not None:
            full = gate.dim() == 2
            if full:
                pg, ldg = _rows(gate, "gate", shape, dev)
    elif w_post is not None or gate is not None or residual_scale != 1.0:
        raise ValueError("without a branch y there is no w_post, no gate and no residual_scale")
    wt = w_pre if w_pre is not None else w_post if w_post is not None else gate if gate is not None and not full else None
    wdt = torch.bfloat16 if wt is None else wt.dtype
    if wdt not in (torch.bfloat16, torch.float32):
        raise TypeError(f"weights must be bfloat16 or float32, got {wdt}")
    if w_pre is not None:
        pn = _vector(w_pre, "w_pre", cols, wdt, dev)
    if w_post is not None:
        pp = _vector(w_post, "w_post", cols, wdt, dev)
    if gate is not None and not full:
        pg = _vector(gate, "gate", cols, wdt, dev)
    args = (ph, ldh, py, ldy, pp, pg, ldg, pn, L.PF8_F32 if wdt == torch.float32 else L.PF8_BF16,
            residual_scale, branch_scale, 1.0 if unit_offset else 0.0, eps)
    return rows, cols, full, args


def _output(out: Optional[Tensor], name: str, like: Tensor) -> Tuple[Tensor, int, int]:
    """A bf16 result of like's shape: the one given, after its checks, or a new one."""
    if out is not None:
        return (out, *_rows(out, name, like.shape, like.device))
    out = torch.empty_like(like, memory_format=torch.contiguous_format)
    return out, out.data_ptr(), like.shape[1]


def _rows_meet(a: Tuple[int, int, int, int], b: Tuple[int, int, int, int]) -> bool:
    """Whether two sets of rows share memory; each (first byte, byte behind the last, bytes of a row, pitch or 0 of
    a single row). Rows of one pitch may lie between one another's; rows of different pitches count as
    shared where their extents meet."""
    (a0, a1, wa, pa), (b0, b1, wb, pb) = a, b
    if a1 <= b0 or b1 <= a0:
        return False
    pitch = pa or pb
    if not pitch or (pb or pitch) != pitch:
        return True
    ahead = (b0 - a0) % pitch
    return ahead < wa or ahead + wb > pitch


def _rows_at(t: Tensor) -> Tuple[int, int, int, int]:
    """_rows_meet's view of a 1-D or 2-D tensor with at least one element and contiguous rows."""
    first, size = t.data_ptr(), t.element_size()
    width = t.shape[-1] * size
    pitch = t.stride(0) * size if t.dim() == 2 and t.shape[0] > 1 else 0
    return first, first + (t.shape[0] - 1) * pitch + width, width, pitch


def _may_write(out: Tensor, name: str, others) -> None:
    """Raise if `out` shares memory with another operand without being the very same rows of it."""
    a = _rows_at(out)
    for o, same_ok in others:
        if o is None or o.device != out.device:
            continue
        b = _rows_at(o)
        if _rows_meet(a, b) and not (same_ok and a[0] == b[0] and a[3] == b[3]):
            raise ValueError(f"{name} overlaps another operand")


def _forward(h, y, w_pre, w_post, gate, residual_scale, branch_scale, eps, unit_offset, r_out, x_out, codes):
    rows, cols, _, args = _inputs(h, y, w_pre, w_post, gate, residual_scale, branch_scale, eps, unit_offset)
    dev = h.device
    if y is None and r_out is not None:
        raise ValueError("without a branch y the stream is h itself: there is no r_out")
    if x_out is not None and w_pre is None:
        raise ValueError("without w_pre there is no x")
    if codes and (w_pre is None or cols % GROUP):
        raise ValueError("block_norm_quant needs w_pre and a multiple of 128 columns")
    if y is None and w_pre is None:
        raise ValueError("nothing to do: neither a branch y nor w_pre")
    r = x = q = s = None
    pr = ldr = px = ldx = pq = ldq = ps = lds = 0
    if y is not None:
        r, pr, ldr = _output(r_out, "r_out", h)
    if w_pre is not None and not codes:
        x, px, ldx = _output(x_out, "x_out", h)
    if codes:
        q = code_buffer(rows, cols, dev)
        s = torch.empty((cols // GROUP, rows), dtype=torch.float32, device=dev)
        pq, ldq, ps, lds = q.data_ptr(), q.stride(0), s.data_ptr(), rows
    if rows and (r_out is not None or x_out is not None):
        rest = [(w_pre, False), (w_post, False), (gate, False)]
        if r_out is not None:
            _may_write(r_out, "r_out", [(h, True), (y, True), *rest, (x_out, False)])
        if x_out is not None:
            _may_write(x_out, "x_out", [(h, True), (y, True), *rest])
    if rows:
        _call(L.pf8_block_norm, dev, rows, cols, *args, pr, ldr, px, ldx, pq, ldq, ps, lds)
    return (h if r is None else r), x, q, s


def block_norm(h: Tensor, y: Optional[Tensor] = None, w_pre: Optional[Tensor] = None, w_post: Optional[Tensor] = None,
               gate: Optional[Tensor] = None, residual_scale: float = 1.0, branch_scale: float = 1.0,
               eps: float = 1e-6, unit_offset: bool = False, r_out: Optional[Tensor] = None,
               x_out: Optional[Tensor] = None) -> Tuple[Tensor, Optional[Tensor]]:
    """The block norm of bf16 h, y [tokens, cols]; returns (r, x).

    r is the new residual stream (h itself without a branch y), x the next block's normalised input
    (None without w_pre). Weights and a [cols] gate are bf16 or float32, all of one type; a
    [tokens, cols] gate is bf16. r_out and x_out may be h or y themselves. No tokens: empty results.
    """
    r, x, _, _ = _forward(h, y, w_pre, w_post, gate, residual_scale, branch_scale, eps, unit_offset, r_out, x_out, False)
    return r, x


def block_norm_quant(h: Tensor, y: Optional[Tensor] = None, w_pre: Optional[Tensor] = None,
                     w_post: Optional[Tensor] = None, gate: Optional[Tensor] = None, residual_scale: float = 1.0,
                     branch_scale: float = 1.0, eps: float = 1e-6, unit_offset: bool = False,
                     r_out: Optional[Tensor] = None) -> Tuple[Tensor, Tensor, Tensor]:
    """The block norm with x as E4M3 codes; returns (r, q uint8 [tokens, cols], s float32 [cols/128, tokens]).

    q and s are bit for bit what ``quant_act_1x128(x)`` makes of ``block_norm``'s x: ``fprop``'s first
    operand, without the BF16 x ever being written. For passes that keep no transposed codes, i.e.
    without a weight gradient.
    """
    r, _, q, s = _forward(h, y, w_pre, w_post, gate, residual_scale, branch_scale, eps, unit_offset, r_out, None, True)
    return r, q, s


def block_norm_backward(dr: Optional[Tensor], dx: Optional[Tensor], h: Tensor, y: Optional[Tensor] = None,
                        w_pre: Optional[Tensor] = None, w_post: Optional[Tensor] = None, gate: Optional[Tensor] = None,
                        residual_scale: float = 1.0, branch_scale: float = 1.0, eps: float = 1e-6,
                        unit_offset: bool = False, dw_pre_out: Optional[Tensor] = None,
                        dw_post_out: Optional[Tensor] = None, dgate_out: Optional[Tensor] = None,
                        accumulate: bool = False) -> BlockNormGrads:
    """Gradients of ``block_norm`` from those of r and x (either may be None: zero).

    The forward's values are made again from its inputs. dw_pre, dw_post and the gradient of a [cols]
    gate are float32 sums over the tokens, formed in a fixed order; given the ``_out`` buffers
    (float32 [cols]) they are written there, or with ``accumulate`` added to what is there.
    """
    rows, cols, full, args = _inputs(h, y, w_pre, w_post, gate, residual_scale, branch_scale, eps, unit_offset)
    dev, shape = h.device, h.shape
    if dr is None and dx is None:
        raise ValueError("one of dr and dx is needed")
    if dx is not None and w_pre is None:
        raise ValueError("dx without w_pre: the forward has no x")
    pdr = ldr = pdx = ldx = 0
    if dr is not None:
        pdr, ldr = _rows(dr, "dr", shape, dev)
    if dx is not None:
        pdx, ldx = _rows(dx, "dx", shape, dev)

    def column(out, name, wanted):
        if not wanted:
            if out is not None:
                raise ValueError(f"{name} is given, but there is no such gradient")
            return None, 0
        if out is None:
            if accumulate:
                raise ValueError(f"accumulate needs {name}")
            out = torch.empty(cols, dtype=torch.float32, device=dev)
            return out, out.data_ptr()
        return out, _vector(out, name, cols, torch.float32, dev)

    dw_pre, p_pre = column(dw_pre_out, "dw_pre_out", dx is not None)
    dw_post, p_post = column(dw_post_out, "dw_post_out", w_post is not None)
    dgate, p_gate = column(dgate_out, "dgate_out", gate is not None and not full)
    sums = [t for t in (dw_pre, dw_post, dgate) if t is not None]
    ld_dg = 0
    if full:
        dgate, p_gate, ld_dg = _output(None, "", h)
    dh, p_dh, _ = _output(None, "", h)
    dy, p_dy, _ = (None, 0, 0) if y is None else _output(None, "", h)
    if accumulate or dw_pre_out is not None or dw_post_out is not None or dgate_out is not None:
        operands = [t for t in (dr, dx, h, y, w_pre, w_post, gate) if t is not None and t.numel()]
        for i, t in enumerate(sums):
            if any(_rows_meet(_rows_at(t), _rows_at(o)) for o in operands + sums[:i]):
                raise ValueError("a gradient buffer overlaps another operand")
    if rows == 0:
        if not accumulate:
            for t in sums:
                t.zero_()
        return BlockNormGrads(dh, dy, dgate, dw_pre, dw_post)
    ws, nws = None, 0
    if sums:
        nws = L.pf8_block_norm_bwd_workspace(rows, cols)
        ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    _call(L.pf8_block_norm_bwd, dev, rows, cols, pdr, ldr, pdx, ldx, *args, p_dh, cols, p_dy, cols,
          p_gate, ld_dg, p_pre, p_post, int(accumulate), 0 if ws is None else ws.data_ptr(), nws)
    return BlockNormGrads(dh, dy, dgate, dw_pre, dw_post)


def _as_rows(t: Optional[Tensor], cols: int) -> Optional[Tensor]:
    if t is None:
        return None
    t = t.reshape(-1, cols)
    if t.shape[0] > 1 and (t.stride(0) < cols or (t.stride(1) != 1 and cols != 1)) or t.shape[0] == 1 and not t.is_contiguous():
        t = t.contiguous()
    return t


class BlockNormFunction(torch.autograd.Function):
    """Autograd function of the block norm; saves its inputs only (the backward makes the rest again)."""

    @staticmethod
    def forward(ctx, h, y, w_pre, w_post, gate, residual_scale, branch_scale, eps, unit_offset, main_grads):
        ctx.set_materialize_grads(False)
        cols = h.shape[-1]
        full = gate is not None and gate.dim() > 1
        g2 = _as_rows(gate, cols) if full else gate
        h2, y2 = _as_rows(h, cols), _as_rows(y, cols)
        ctx.save_for_backward(h2, y2, w_pre, w_post, g2)
        ctx.scalars = (residual_scale, branch_scale, eps, unit_offset)
        ctx.main_grads, ctx.shape, ctx.full = main_grads, h.shape, full
        ctx.leaves = [t is not None and t.requires_grad and t.is_leaf for t in (h, y, w_pre, w_post, gate)]
        r, x = block_norm(h2, y2, w_pre, w_post, g2, *ctx.scalars)
        r = None if y is None else r.reshape(h.shape)
        x = None if x is None else x.reshape(h.shape)
        return r, x

    @staticmethod
    @once_differentiable
    def backward(ctx, dr, dx):
        h, y, w_pre, w_post, gate = ctx.saved_tensors
        need = ctx.needs_input_grad[:5]
        main = dict(zip((2, 3, 4), ctx.main_grads)) if ctx.main_grads is not None else {}
        if torch.cuda.is_current_stream_capturing():
            # autograd's accumulator of a leaf belongs to the stream of the first graph that used the
            # leaf; from inside a capture it may wait on that stream, which breaks the capture
            if any(leaf and n and main.get(i) is None for i, (leaf, n) in enumerate(zip(ctx.leaves, need))):
                raise RuntimeError("a captured backward cannot hand gradients to leaf tensors: capture "
                                   "block_norm_backward, or give the weights a main_grad")
        none = (None,) * 10
        if dr is None and dx is None:
            return none
        cols = ctx.shape[-1]

        def rows_of(t):
            return None if t is None else _as_rows(t.to(torch.bfloat16), cols)

        outs = [None, None, None]
        present = (dx is not None, w_post is not None, gate is not None and not ctx.full)
        accumulate = any(main.get(i) is not None and need[i] for i in (2, 3, 4))
        if accumulate:
            outs = [None if not p else main[i] if main.get(i) is not None and need[i]
                    else torch.zeros(cols, dtype=torch.float32, device=h.device)
                    for i, p in zip((2, 3, 4), present)]
        g = block_norm_backward(rows_of(dr), rows_of(dx), h, y, w_pre, w_post, gate, *ctx.scalars, *outs,
                                accumulate=accumulate)

        def column(i, grad, like):
            if not need[i] or grad is None or main.get(i) is not None:
                return None
            return grad.to(like.dtype)

        dgate = None
        if gate is not None and need[4]:
            dgate = g.dgate.reshape(ctx.shape) if ctx.full else column(4, g.dgate, gate)
        return (g.dh.reshape(ctx.shape) if need[0] else None,
                g.dy.reshape(ctx.shape) if y is not None and need[1] else None,
                column(2, g.dw_pre, w_pre), column(3, g.dw_post, w_post), dgate, *none[5:])


def fp8_block_norm(h: Tensor, y: Optional[Tensor] = None, w_pre: Optional[Tensor] = None,
                   w_post: Optional[Tensor] = None, gate: Optional[Tensor] = None, residual_scale: float = 1.0,
                   branch_scale: float = 1.0, eps: float = 1e-6, unit_offset: bool = False, main_grads=None
                   ) -> Tuple[Tensor, Optional[Tensor]]:
    """The block norm under autograd, for h and y [..., cols]; returns (r, x) as ``block_norm`` does.

    A gate is [cols] or of h's shape. Weights' gradients come in the weights' type, or, where
    ``main_grads`` = (of w_pre, of w_post, of a [cols] gate) holds a float32 buffer, are added to it in
    FP32 while autograd receives none. A backward pass that is being captured into a graph hands no
    gradient to leaf tensors: it raises, unless they go to ``main_grads``.
    """
    if not isinstance(h, Tensor) or h.dim() < 1 or (y is not None and y.shape != h.shape):
        raise ValueError("h and y must be tensors of one shape")
    if gate is not None and gate.dim() != 1 and gate.shape != h.shape:
        raise ValueError(f"gate must be [cols] or of h's shape {tuple(h.shape)}, got {tuple(gate.shape)}")
    if main_grads is not None:
        for m, w in zip(main_grads, (w_pre, w_post, gate)):
            if m is not None and (w is None or w.dim() != 1 or m.dtype != torch.float32 or m.shape != w.shape):
                raise ValueError("a main_grad must be a float32 tensor of its weight's shape")
    r, x = BlockNormFunction.apply(h, y, w_pre, w_post, gate, float(residual_scale), float(branch_scale), float(eps),
                                   bool(unit_offset), None if main_grads is None else tuple(main_grads))
    return (h if r is None else r), x


class BlockNorm(torch.nn.Module):
    """Post-norm, gate, residual sum and pre-norm between two blocks: ``r, x = norm(h, y)``.

    ``pre`` / ``post`` choose which of the two norms there are; ``gate`` adds a learned [cols] gate
    (started at ``gate_init``), and a gate per token can be passed to ``forward`` instead. Without y (before
    a model's first block) x is h's pre-norm and the rest stands aside. Weights are
    kept in ``dtype`` (BF16 as the rest of the model, or FP32). With ``fp32_main_grad`` every weight
    carries a float32 ``main_grad`` that each backward pass adds to, and its ``grad`` stays None.
    """

    def __init__(self, cols: int, pre: bool = True, post: bool = True, gate: bool = False, gate_init: float = 1.0,
                 residual_scale: float = 1.0, branch_scale: float = 1.0, eps: float = 1e-6, unit_offset: bool = False,
                 dtype: torch.dtype = torch.bfloat16, device=None, fp32_main_grad: bool = False):
        super().__init__()
        if not (pre or post or gate):
            raise ValueError("a BlockNorm has at least one of pre, post and gate")
        fill = 0.0 if unit_offset else 1.0
        self.cols, self.residual_scale, self.branch_scale = cols, residual_scale, branch_scale
        self.eps, self.unit_offset = eps, unit_offset

        def weight(there, value):
            if not there:
                return None
            w = torch.nn.Parameter(torch.full((cols,), value, dtype=dtype, device=device))
            if fp32_main_grad:
                w.main_grad = torch.zeros(cols, dtype=torch.float32, device=w.device)
            return w

        self.w_pre = weight(pre, fill)
        self.w_post = weight(post, fill)
        self.gate = weight(gate, gate_init)

    def _operands(self, y, gate):
        if gate is not None and self.gate is not None:
            raise ValueError("this BlockNorm has a learned gate: none can be passed")
        if gate is not None and y is None:
            raise ValueError("without a branch y there is no gate")
        return self.w_pre, self.w_post, self.gate if gate is None else gate

    def forward(self, h: Tensor, y: Optional[Tensor] = None, gate: Optional[Tensor] = None
                ) -> Tuple[Tensor, Optional[Tensor]]:
        w_pre, w_post, g = self._operands(y, gate)
        main = tuple(getattr(w, "main_grad", None) for w in (w_pre, w_post, g if gate is None else None))
        if y is None:
            return fp8_block_norm(h, None, w_pre, eps=self.eps, unit_offset=self.unit_offset,
                                  main_grads=(main[0], None, None))
        return fp8_block_norm(h, y, w_pre, w_post, g, self.residual_scale, self.branch_scale, self.eps,
                              self.unit_offset, main)

    @torch.no_grad()
    def quantised(self, h: Tensor, y: Optional[Tensor] = None, gate: Optional[Tensor] = None
                  ) -> Tuple[Tensor, Tensor, Tensor]:
        """(r, codes, scales) of 2-D h and y, for ``fprop`` (no gradients; see ``block_norm_quant``)."""
        w_pre, w_post, g = self._operands(y, gate)
        if y is None:
            return block_norm_quant(h, None, w_pre, eps=self.eps, unit_offset=self.unit_offset)
        return block_norm_quant(h, y, w_pre, w_post, g, self.residual_scale, self.branch_scale, self.eps,
                                self.unit_offset)
