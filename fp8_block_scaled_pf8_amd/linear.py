"""FP8 linear layer for PyTorch autograd: every matmul and every quantisation runs in libpf8.

Y = X . W^T with X [..., K] bf16 and W [N, K] bf16 (a torch.nn.Linear weight without bias).

forward:  X -> row-mode codes (groups along K) and col-mode codes (groups along the tokens) in one
          read (pf8_quant_act_dual); W -> 128x128-tile codes and the transposed codes; Y = fprop.
backward: dY -> row-mode codes (along N) and col-mode codes (along the tokens) in one read;
          dX = dgrad(dY codes, W^T codes); dW = wgrad(dY^T codes, X^T codes).
Only codes and scales are saved for the backward pass (1 byte per element plus 1/32 of that).

FP32 weight gradients: given ``main_grad`` (an FP32 [N, K] buffer), the backward pass adds dW to
it in FP32 inside the GEMM's epilogue (pf8_block_gemm_f32 with accumulate = 1), the way gradients
are summed over the micro-batches of an optimizer step, and autograd receives no gradient for W.

Weight codes: W changes only at an optimizer step, so ``Fp8Linear`` quantises it once per weight
version (codes, transposed codes and tile scales) and reuses them for every micro-batch until W is
modified. An in-place update of the parameter (as optimizers do) bumps its version counter. An
update through ``weight.data`` bypasses that counter; call ``invalidate_weight_codes()`` after one.

Bias, activation and residual: ``fp8_linear_act`` and an ``Fp8Linear`` made with them run the product's
epilogue (``epilogue.fprop_act``): d = act(X . W^T + bias) + residual, or gated act(g) * u + residual from the
two halves of W's rows. For an activation the backward pass keeps z = X . W^T + bias in BF16; its gradient dz
(``epilogue.act_backward_quant``, with the bias's in FP32) is made as codes and takes dY's place above. ``Fp8Linear.infer`` runs any number of
tokens without gradients.

Tokens (the product of the leading dimensions), N and K must be multiples of 128. Zero tokens give
an empty result and no weight-gradient contribution, without a launch.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from torch.autograd.function import once_differentiable

from . import epilogue, ops

GROUP = 128


def _check_shapes(m: int, n: int, k: int) -> None:
    if m % GROUP or n % GROUP or k % GROUP:
        raise ValueError(f"fp8_linear needs tokens, out_features and in_features to be multiples of 128 "
                         f"(got tokens={m}, out={n}, in={k})")


class Fp8LinearFunction(torch.autograd.Function):
    """Autograd function of the FP8 linear layer (see the module docstring)."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, w: torch.Tensor, main_grad: Optional[torch.Tensor] = None,
                w_codes: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None):
        lead = x.shape[:-1]
        k = x.shape[-1]
        x2 = x.reshape(-1, k)
        if x2.stride(1) != 1 or x2.stride(0) % 8:
            x2 = x2.contiguous()
        n = w.shape[0]
        _check_shapes(x2.shape[0], n, k)
        ctx.lead, ctx.k, ctx.main_grad = lead, k, main_grad
        if x2.shape[0] == 0:
            # no tokens: an empty result, and no gradient contribution in the backward pass (the
            # library rejects empty dimensions, so nothing is launched)
            ctx.empty = True
            return x.new_empty((*lead, n))
        ctx.empty = False
        qx, sx, qxt, sxt = ops.quant_act_dual(x2)
        qw, qwt, sw = w_codes if w_codes is not None else ops.quant_w_128x128(w.contiguous(), transposed=True)
        # results handed to the caller are plain contiguous tensors (the library's own workspaces
        # use padded row pitches instead)
        y = ops.fprop(qx, sx, qw, sw, out=torch.empty((x2.shape[0], n), dtype=torch.bfloat16, device=x.device))
        ctx.save_for_backward(qxt, sxt, qwt, sw)
        return y.reshape(*lead, n)

    @staticmethod
    def backward(ctx, dy: torch.Tensor):
        if ctx.empty:
            dx = dy.new_empty((*ctx.lead, ctx.k), dtype=torch.bfloat16) if ctx.needs_input_grad[0] else None
            return dx, None, None, None
        qxt, sxt, qwt, sw = ctx.saved_tensors
        n = qwt.shape[1]
        dy2 = dy.reshape(-1, n)
        if dy2.dtype != torch.bfloat16:
            dy2 = dy2.to(torch.bfloat16)
        if dy2.stride(1) != 1 or dy2.stride(0) % 8:
            dy2 = dy2.contiguous()
        qdy, sdy, qdyt, sdyt = ops.quant_act_dual(dy2)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = ops.dgrad(qdy, sdy, qwt, sw, out=torch.empty((dy2.shape[0], ctx.k), dtype=torch.bfloat16,
                                                              device=dy2.device)).reshape(*ctx.lead, ctx.k)
        if ctx.main_grad is not None:
            ops.wgrad_f32(qdyt, sdyt, qxt, sxt, out=ctx.main_grad, accumulate=True)
        elif ctx.needs_input_grad[1]:
            dw = ops.wgrad(qdyt, sdyt, qxt, sxt, out=torch.empty((n, ctx.k), dtype=torch.bfloat16, device=dy2.device))
        return dx, dw, None, None


def _rows(t: torch.Tensor, cols: int) -> torch.Tensor:
    """[..., cols] as rows that the quantisers and the epilogue take, copied only where it has to be."""
    t = t.reshape(-1, cols)
    if t.stride(1) != 1 or t.stride(0) % 8 or t.stride(0) < cols or t.data_ptr() % 16:
        t = t.contiguous()
        if t.data_ptr() % 16:
            t = t.clone()
    return t


def _act_forward(x, w, bias, residual, activation, gated, w_codes, keep):
    """(d, what the backward pass needs beside the arguments: None where it is not kept)."""
    lead, k, n = x.shape[:-1], x.shape[-1], w.shape[0]
    cols = n // 2 if gated else n
    x2 = _rows(x, k)
    _check_shapes(x2.shape[0], n, k)
    if x2.shape[0] == 0:
        return x.new_empty((*lead, cols)), None
    if keep:
        qx, sx, qxt, sxt = ops.quant_act_dual(x2)
    else:
        qx, sx = ops.quant_act_1x128(x2)
    qw, qwt, sw = w_codes if w_codes is not None else ops.quant_w_128x128(w.contiguous(), transposed=keep)
    d = torch.empty((x2.shape[0], cols), dtype=torch.bfloat16, device=x.device)
    got = epilogue.fprop_act(qx, sx, qw, sw, bias, activation, gated, None if residual is None else _rows(residual, cols),
                             save_z=keep and activation is not None, out=d)
    saved = (qxt, sxt, qwt, sw, got[1] if activation is not None else None) if keep else None
    return d.reshape(*lead, cols), saved


class Fp8LinearActFunction(torch.autograd.Function):
    """Autograd function of the FP8 linear layer with its epilogue (see the module docstring)."""

    @staticmethod
    def forward(ctx, x, w, bias, residual, activation, gated, main_grad, bias_main_grad, w_codes):
        ctx.lead, ctx.k, ctx.n, ctx.activation, ctx.gated = x.shape[:-1], x.shape[-1], w.shape[0], activation, gated
        ctx.main_grad, ctx.bias_main_grad, ctx.bias = main_grad, bias_main_grad, None if bias is None else bias.dtype
        ctx.leaves = [t is not None and t.requires_grad and t.is_leaf for t in (x, w, bias, residual)]
        ctx.empty = x.numel() == 0
        # (a gradient of the residual alone is the result's)
        d, saved = _act_forward(x, w, bias, residual, activation, gated, w_codes, any(ctx.needs_input_grad[:3]))
        if saved is not None:
            ctx.save_for_backward(*saved)
        return d

    @staticmethod
    @once_differentiable
    def backward(ctx, dd):
        need = ctx.needs_input_grad[:4]
        if torch.cuda.is_current_stream_capturing():
            # autograd's accumulator of a leaf belongs to the stream of the first graph that used the
            # leaf; from inside a capture it may wait on that stream, which breaks the capture
            if any(leaf and nd and m is None
                   for leaf, nd, m in zip(ctx.leaves, need, (None, ctx.main_grad, ctx.bias_main_grad, None))):
                raise RuntimeError("a captured backward cannot hand gradients to leaf tensors: give the weight and the "
                                   "bias a main_grad, and capture no leaf inputs")
        none = (None,) * 5
        dres = dd if need[3] else None
        if ctx.empty:
            dx = dd.new_empty((*ctx.lead, ctx.k), dtype=torch.bfloat16) if need[0] else None
            dw = dd.new_zeros((ctx.n, ctx.k), dtype=torch.bfloat16) if need[1] and ctx.main_grad is None else None
            db = dd.new_zeros((ctx.n,), dtype=ctx.bias) if need[2] and ctx.bias_main_grad is None else None
            return (dx, dw, db, dres, *none)
        if not any(need[:3]):
            return (None, None, None, dres, *none)
        qxt, sxt, qwt, sw, z = ctx.saved_tensors
        n = ctx.n
        dz = _rows(dd.to(torch.bfloat16), n // 2 if ctx.gated else n)
        add = need[2] and ctx.bias_main_grad is not None
        bias = dict(bias_grad=need[2], dbias_out=ctx.bias_main_grad if add else None, accumulate=add)
        if dz.shape[1] % GROUP:  # a gate over an odd number of 64 columns: a scale's columns are of both halves
            dz, dbias = epilogue.act_backward(dz, z, ctx.activation, ctx.gated, **bias)
            qdz, sdz, qdzt, sdzt = ops.quant_act_dual(dz)
        else:
            qdz, sdz, qdzt, sdzt, dbias = epilogue.act_backward_quant(dz, z, ctx.activation, ctx.gated, **bias)
        dbias = None if add or dbias is None else dbias.to(ctx.bias)
        dx = dw = None
        if need[0]:
            dx = ops.dgrad(qdz, sdz, qwt, sw, out=torch.empty((dz.shape[0], ctx.k), dtype=torch.bfloat16,
                                                              device=dz.device)).reshape(*ctx.lead, ctx.k)
        if need[1] and ctx.main_grad is not None:
            ops.wgrad_f32(qdzt, sdzt, qxt, sxt, out=ctx.main_grad, accumulate=True)
        elif need[1]:
            dw = ops.wgrad(qdzt, sdzt, qxt, sxt, out=torch.empty((n, ctx.k), dtype=torch.bfloat16, device=dz.device))
        return (dx, dw, dbias, dres, *none)


def _check_layer(x, w, bias, residual, activation, gated, main_grad, bias_main_grad) -> None:
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("fp8_linear_act takes bfloat16 X and W")
    epilogue._activation(activation, gated)
    n = w.shape[0]
    if bias is not None and (bias.shape != (n,) or bias.dtype not in (torch.bfloat16, torch.float32)):
        raise ValueError(f"bias must be a bfloat16 or float32 tensor of the shape ({n},)")
    if residual is not None and (residual.dtype != torch.bfloat16 or
                                 tuple(residual.shape) != (*x.shape[:-1], n // 2 if gated else n)):
        raise ValueError("residual must be a bfloat16 tensor of the result's shape")
    if main_grad is not None and (main_grad.dtype != torch.float32 or tuple(main_grad.shape) != tuple(w.shape)):
        raise ValueError("main_grad must be a float32 tensor of W's shape")
    if bias_main_grad is not None and (bias is None or bias_main_grad.dtype != torch.float32 or
                                       bias_main_grad.shape != bias.shape):
        raise ValueError("bias_main_grad must be a float32 tensor of bias's shape")


def _check_codes(w: torch.Tensor, w_codes) -> None:
    n, k = w.shape
    qw, qwt, sw = w_codes
    if (tuple(qw.shape) != (n, k) or tuple(qwt.shape) != (k, n) or tuple(sw.shape) != (n // GROUP, k // GROUP)
            or qw.dtype != torch.uint8 or qwt.dtype != torch.uint8 or sw.dtype != torch.float32):
        raise ValueError("w_codes must be (codes [N,K] uint8, transposed codes [K,N] uint8, scales [N/128,K/128] float32)")


def fp8_linear_act(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   activation: Optional[str] = None, gated: bool = False, residual: Optional[torch.Tensor] = None,
                   main_grad: Optional[torch.Tensor] = None, bias_main_grad: Optional[torch.Tensor] = None,
                   w_codes: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None) -> torch.Tensor:
    """``fp8_linear`` with bias, activation and residual in the product's epilogue (see ``fprop_act``).

    Differentiable in X, W, bias and residual. The bias's gradient comes in its own type, or is added to
    ``bias_main_grad`` (float32) while autograd receives none; ``main_grad`` and ``w_codes`` are as ``fp8_linear`` takes
    them. A backward pass that is being captured into a graph hands no gradient to leaf tensors: it raises, unless
    they go to main gradients.
    """
    _check_layer(x, w, bias, residual, activation, gated, main_grad, bias_main_grad)
    if w_codes is not None:
        _check_codes(w, w_codes)
    if not (torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, w, bias, residual))):
        # (a function's own needs_input_grad is true of a parameter under no_grad, too)
        return _act_forward(x, w, bias, residual, activation, bool(gated), w_codes, False)[0]
    return Fp8LinearActFunction.apply(x, w, bias, residual, activation, bool(gated), main_grad, bias_main_grad, w_codes)


def fp8_linear(x: torch.Tensor, w: torch.Tensor, main_grad: Optional[torch.Tensor] = None,
               w_codes: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None) -> torch.Tensor:
    """Y = X . W^T through libpf8's block-scaled FP8 path, differentiable in X and W.

    Without ``main_grad`` W's gradient is returned to autograd in BF16. With it (FP32, W's shape,
    16-byte row pitch) the backward pass adds dW to ``main_grad`` in FP32 instead. ``w_codes``
    are W's codes, transposed codes and tile scales from ``ops.quant_w_128x128(w, transposed=True)``
    for the current W; without them W is quantised here.
    """
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("fp8_linear takes bfloat16 X and W")
    if main_grad is not None and (main_grad.dtype != torch.float32 or tuple(main_grad.shape) != tuple(w.shape)):
        raise ValueError("main_grad must be a float32 tensor of W's shape")
    if w_codes is not None:
        _check_codes(w, w_codes)
    return Fp8LinearFunction.apply(x, w, main_grad, w_codes)


class Fp8Linear(torch.nn.Module):
    """Linear layer whose three GEMMs run in block-scaled FP8 (weights kept in BF16), without a bias by default.

    With ``fp32_main_grad`` the weight carries an FP32 ``main_grad`` buffer that every backward
    pass accumulates into (zero it once per optimizer step); ``weight.grad`` then stays None.
    The weight's codes are made once per weight version and shared by the micro-batches (see the
    module docstring). ``bias`` (of ``bias_dtype``, from zeros), ``activation`` and a residual passed to ``forward`` go
    into the product's epilogue; ``gated`` takes out_features as gate and factor, and the result has half of them.
    """

    def __init__(self, in_features: int, out_features: int, device=None, fp32_main_grad: bool = False,
                 weight: Optional[torch.Tensor] = None, bias: bool = False, activation: Optional[str] = None,
                 gated: bool = False, bias_dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        epilogue._activation(activation, gated)
        if weight is None:
            weight = torch.empty((out_features, in_features), dtype=torch.bfloat16, device=device)
            torch.nn.init.normal_(weight, std=0.02)
        self.weight = torch.nn.Parameter(weight)
        self.activation, self.gated = activation, bool(gated)
        rows = self.weight.shape[0]
        self.bias = torch.nn.Parameter(torch.zeros(rows, dtype=bias_dtype, device=self.weight.device)) if bias else None
        if fp32_main_grad:
            self.weight.main_grad = torch.zeros(self.weight.shape, dtype=torch.float32, device=self.weight.device)
            if bias:
                self.bias.main_grad = torch.zeros(rows, dtype=torch.float32, device=self.weight.device)
        self._codes = None
        self._codes_key = None
        self._codes_ready = None  # event recorded on the stream that made the codes
        self._codes_users = set()  # streams the codes were handed to
        self._codes_held = []  # codes that graphs were captured with

    def weight_codes(self) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """W's codes, transposed codes and tile scales, made once per version of the weight.

        They are made on the current stream. A later call from another stream makes that stream
        wait for them, and marks them as used there, so that the allocator keeps their memory
        until that stream's work is done even after new codes replace them. Codes that are made while
        the stream is being captured belong to that graph and are not kept. A graph that is captured with
        kept codes reads those at every replay, whatever becomes of the weight: they stay in memory as
        long as the layer, and the graph is to be captured again after an update."""
        w = self.weight
        key = (w.data_ptr(), w._version, tuple(w.shape), w.device)
        cur = torch.cuda.current_stream(w.device)
        capturing = torch.cuda.is_current_stream_capturing()
        if self._codes is None or self._codes_key != key:
            # (codes made in inference mode could not be saved for a later training pass)
            with torch.inference_mode(False), torch.no_grad():
                codes = ops.quant_w_128x128(w.detach().contiguous(), transposed=True)
            if capturing:
                return codes  # made by the graph's replays, in its memory: not there for an eager pass
            self._codes = codes
            self._codes_key = key
            self._codes_ready = torch.cuda.Event()
            self._codes_ready.record(cur)
            self._codes_users = {cur.cuda_stream}
        elif cur.cuda_stream not in self._codes_users:
            cur.wait_event(self._codes_ready)
            for t in self._codes:
                t.record_stream(cur)
            self._codes_users.add(cur.cuda_stream)
        if capturing and not any(c is self._codes for c in self._codes_held):
            self._codes_held.append(self._codes)
        return self._codes

    def invalidate_weight_codes(self) -> None:
        """Forget the cached weight codes (after a change to W that its version counter misses)."""
        self._codes = None
        self._codes_key = None
        self._codes_ready = None
        self._codes_users = set()

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        main_grad = getattr(self.weight, "main_grad", None)
        if self.bias is None and self.activation is None and residual is None:
            return fp8_linear(x, self.weight, main_grad, self.weight_codes())
        return fp8_linear_act(x, self.weight, self.bias, self.activation, self.gated, residual, main_grad,
                              getattr(self.bias, "main_grad", None), self.weight_codes())

    @torch.no_grad()
    def infer(self, x, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The layer without gradients, for any number of tokens: x is BF16 [..., in_features], or the (codes, scales) of
        ``quant_act_1x128`` or ``BlockNorm.quantised`` for a 2-D result."""
        n, k = self.weight.shape
        cols = n // 2 if self.gated else n
        qw, _, sw = self.weight_codes()
        if isinstance(x, tuple):
            (qx, sx), lead = x, None
            if residual is not None and tuple(residual.shape) != (qx.shape[0], cols):
                raise ValueError("residual must have the result's shape")
        else:
            _check_layer(x, self.weight, None, residual, self.activation, self.gated, None, None)
            lead = x.shape[:-1]
            x2 = _rows(x, k)
            if x2.shape[0] == 0:
                return x.new_empty((*lead, cols))
            qx, sx = ops.quant_act_1x128(x2)
        d = epilogue.fprop_act(qx, sx, qw, sw, self.bias, self.activation, self.gated,
                               None if residual is None else _rows(residual, cols))
        return d if lead is None else d.reshape(*lead, cols)
