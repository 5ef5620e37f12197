"""What stands around the FP8 product in a layer: bias, activation, residual, and their backward pass.

    z = X W^T + bias
    d = act(z) + residual                 or, gated, with z = [g | u]:  d = act(g) * u + residual

Activations: "relu", "relu2" (its square), "silu", "gelu" (by erf), "gelu_tanh"; None for none. include/pf8_layer.h
has the details.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib as L
from .norm import _call, _may_write, _rows, _rows_at, _rows_meet, _vector

Tensor = torch.Tensor

ACTIVATIONS = {None: L.PF8_ACT_NONE, "relu": L.PF8_ACT_RELU, "relu2": L.PF8_ACT_RELU2, "silu": L.PF8_ACT_SILU,
               "gelu": L.PF8_ACT_GELU, "gelu_tanh": L.PF8_ACT_GELU_TANH}


class ActGrads(NamedTuple):
    """Gradients of an activation: bf16 dz; float32 dbias, the column sums of dz before its rounding."""
    dz: Tensor
    dbias: Optional[Tensor]


def _activation(activation: Optional[str], gated: bool) -> int:
    code = ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
    if gated and not code:
        raise ValueError("a gated product needs an activation for its gate")
    return code


def act_backward(dd: Tensor, z: Optional[Tensor], activation: Optional[str], gated: bool = False,
                 bias_grad: bool = False, dz_out: Optional[Tensor] = None, dbias_out: Optional[Tensor] = None,
                 accumulate: bool = False) -> ActGrads:
    """Gradient dz of the value before an activation, and of the bias in it, from bf16 dd [rows, cols].

    z is that value as the forward rounded it: bf16 [rows, cols], or [rows, 2 cols] with its gate first. dz has
    z's shape. Without an activation z is None and dz is dd itself. ``bias_grad``: dbias, float32 column sums formed
    in a fixed order; given dbias_out they are written there, or with ``accumulate`` added. dz_out may be z, or
    without a gate dd. No rows: empty results, a dbias of zeros.
    """
    if not isinstance(dd, Tensor) or dd.dim() != 2:
        raise ValueError("dd must be a 2-D tensor")
    if not dd.is_cuda:
        raise ValueError("dd must be on a HIP device")
    code = _activation(activation, gated)
    (rows, cols), dev = dd.shape, dd.device
    if cols < 1:
        raise ValueError("dd must have at least one column")
    pd, ldd = _rows(dd, "dd", dd.shape, dev)
    width = 2 * cols if gated else cols
    pz = ldz = po = ldo = 0
    if not code:
        if z is not None or dz_out is not None:
            raise ValueError("without an activation there is no z and no dz_out: dz is dd")
        if not bias_grad:
            raise ValueError("nothing to do: neither an activation nor bias_grad")
        dz = dd
    else:
        if z is None:
            raise ValueError("an activation's gradient needs z")
        shape = torch.Size((rows, width))
        pz, ldz = _rows(z, "z", shape, dev)
        if dz_out is None:
            dz = torch.empty(shape, dtype=torch.bfloat16, device=dev)
            po, ldo = dz.data_ptr(), width
        else:
            dz = dz_out
            po, ldo = _rows(dz_out, "dz_out", shape, dev)
    dbias, pb, ws, nws = None, 0, None, 0
    if bias_grad:
        dbias = dbias_out
        if dbias is None:
            if accumulate:
                raise ValueError("accumulate needs dbias_out")
            dbias = torch.empty(width, dtype=torch.float32, device=dev)
            pb = dbias.data_ptr()
        else:
            pb = _vector(dbias_out, "dbias_out", width, torch.float32, dev)
    elif dbias_out is not None or accumulate:
        raise ValueError("dbias_out and accumulate need bias_grad")
    if rows == 0:
        if bias_grad and not accumulate:
            dbias.zero_()
        return ActGrads(dz, dbias)
    if dz_out is not None:
        _may_write(dz_out, "dz_out", [(z, True), (dd, not gated), (dbias, False)])
    if dbias_out is not None and any(_rows_meet(_rows_at(dbias), _rows_at(t)) for t in (dd, z) if t is not None):
        raise ValueError("dbias_out overlaps another operand")
    if bias_grad:
        nws = L.pf8_act_bwd_workspace(rows, cols, int(gated))
        ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    _call(L.pf8_act_bwd, dev, rows, cols, pd, ldd, pz, ldz, code, int(gated), po, ldo, pb, int(accumulate),
          0 if ws is None else ws.data_ptr(), nws)
    return ActGrads(dz, dbias)
