"""What stands around the FP8 product in a layer: bias, activation, residual, and their backward pass.

    z = X W^T + bias
    d = act(z) + residual                 or, gated, with z = [g | u]:  d = act(g) * u + residual

Activations: "relu", "relu2" (its square), "silu", "gelu" (by erf), "gelu_tanh"; None for none. include/pf8_layer.h
has the details.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import _lib as L
from .norm import _call, _may_write, _rows, _rows_at, _rows_meet, _vector
from .ops import GROUP, code_buffer, out_pitch

Tensor = torch.Tensor

ACTIVATIONS = {None: L.PF8_ACT_NONE, "relu": L.PF8_ACT_RELU, "relu2": L.PF8_ACT_RELU2, "silu": L.PF8_ACT_SILU,
               "gelu": L.PF8_ACT_GELU, "gelu_tanh": L.PF8_ACT_GELU_TANH}


class ActGrads(NamedTuple):
    """Gradients of an activation: bf16 dz; float32 dbias, the column sums of dz before its rounding."""
    dz: Tensor
    dbias: Optional[Tensor]


class ActQuantGrads(NamedTuple):
    """An activation's gradient as ``quant_act_dual`` has it: codes and scales along the rows, and transposed; dbias."""
    q: Tensor
    s: Tensor
    qt: Tensor
    st: Tensor
    dbias: Optional[Tensor]


def _activation(activation: Optional[str], gated: bool) -> int:
    code = ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
    if gated and not code:
        raise ValueError("a gated product needs an activation for its gate")
    return code


def _aligned_rows(t: Tensor, name: str, shape, device) -> Tuple[int, int]:
    """(address, pitch) of a bf16 matrix that the product's epilogue reads or writes 16 bytes at a time."""
    p, ld = _rows(t, name, shape, device)
    if shape[0] <= 1:  # no second row: a pitch of any size
        ld = -(-shape[1] // 8) * 8
    if p % 16 or ld % 8:
        raise ValueError(f"{name} must be 16-byte aligned with a row pitch of a multiple of 8")
    return p, ld


def _codes(t: Tensor, name: str) -> Tuple[int, int, int, int]:
    """(rows, columns, address, pitch) of a tensor of codes after its checks."""
    shape = t.shape if isinstance(t, Tensor) else ()
    if len(shape) != 2 or t.dtype is not torch.uint8:
        raise TypeError(f"{name} must be a 2-D uint8 tensor of codes")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a HIP device")
    rows, cols = shape
    ld, one = t.stride()
    if one != 1 or rows > 1 and ld < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return rows, cols, t.data_ptr(), cols if rows == 1 else ld


def _scales(t: Tensor, name: str, rows: int, cols: int, device) -> Tuple[int, int]:
    shape = t.shape if isinstance(t, Tensor) else ()
    if len(shape) != 2 or t.dtype is not torch.float32:
        raise TypeError(f"{name} must be a 2-D float32 tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if shape[0] < rows or shape[1] < cols:
        raise ValueError(f"{name} must cover [{rows}, {cols}], got {tuple(shape)}")
    ld, one = t.stride()
    if one != 1 and cols > 1 or rows > 1 and ld < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), max(ld, cols)


def _new_result(rows: int, cols: int, device) -> Tuple[Tensor, int, int]:
    """A bf16 result in rows that are multiples of 16 bytes apart (in one call: a slice of a wider tensor takes as long
    as the tensor)."""
    pitch = out_pitch(cols, 2) if rows > 1 else -(-cols // 8) * 8
    t = torch.empty_strided((rows, cols), (pitch, 1), dtype=torch.bfloat16, device=device)
    return t, t.data_ptr(), pitch


def fprop_act(qx: Tensor, sx: Tensor, qw: Tensor, sw: Tensor, bias: Optional[Tensor] = None,
              activation: Optional[str] = None, gated: bool = False, residual: Optional[Tensor] = None,
              save_z: bool = False, out: Optional[Tensor] = None, z_out: Optional[Tensor] = None
              ) -> Union[Tensor, Tuple[Tensor, Tensor]]:
    """d = act(X W^T + bias) + residual from X's row-mode codes and W's tile codes, as ``fprop`` takes them.

    ``gated``: the first half of W's rows makes the gate g, the second u, and d = act(g) * u + residual has half
    the columns; W's rows are then a multiple of 128. bias is bf16 or float32 [rows of W], residual bf16 of d's
    shape. d is bf16, and so is z = X W^T + bias, which ``act_backward`` takes: returned as (d, z) with ``save_z`` or
    z_out. out may be residual itself. No tokens: empty results.
    """
    m, k, pa, lda = _codes(qx, "qx")
    n, kw, pb, ldb = _codes(qw, "qw")
    dev = qx.device
    if kw != k:
        raise ValueError(f"reduction dims differ: qx {(m, k)}, qw {(n, kw)}")
    if qw.device != dev:
        raise ValueError(f"qw must be on {dev}, got {qw.device}")
    if k < GROUP or k % GROUP:
        raise ValueError(f"the reduction dimension must be a multiple of {GROUP}, got {k}")
    if n < 1:
        raise ValueError("qw must have at least one row")
    code = _activation(activation, gated)
    if gated and n % GROUP:
        raise ValueError(f"a gated product needs a multiple of {GROUP} weight rows, got {n}")
    pas, ld_as = _scales(sx, "sx", k // GROUP, m, dev)
    pbs, ld_bs = _scales(sw, "sw", -(-n // GROUP), k // GROUP, dev)
    cols = n // 2 if gated else n
    pbias, btype = 0, L.PF8_BF16
    if bias is not None:
        if bias.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"bias must be bfloat16 or float32, got {bias.dtype}")
        pbias = _vector(bias, "bias", n, bias.dtype, dev)
        btype = L.PF8_F32 if bias.dtype == torch.float32 else L.PF8_BF16
    shape = (m, cols)
    pr = ldr = pz = ldz = 0
    if residual is not None:
        pr, ldr = _aligned_rows(residual, "residual", shape, dev)
    if out is None:
        out, pd, ldd = _new_result(m, cols, dev)
    else:
        pd, ldd = _aligned_rows(out, "out", shape, dev)
        if m:
            _may_write(out, "out", [(residual, True), (qx, False), (qw, False), (sx, False), (sw, False), (bias, False),
                                    (z_out, False)])
    z = z_out
    if z is not None:
        pz, ldz = _aligned_rows(z, "z_out", torch.Size((m, n)), dev)
        if m:
            _may_write(z, "z_out", [(t, False) for t in (residual, qx, qw, sx, sw, bias)])
    elif save_z:
        z, pz, ldz = _new_result(m, n, dev)
    if m:
        _call(L.pf8_fprop_act, dev, m, n, k, pa, lda, pas, ld_as, pb, ldb, pbs, ld_bs, pbias, btype, code, int(gated), pr,
              ldr, pz, ldz, pd, ldd)
    return out if z is None else (out, z)


def _dbias(bias_grad, dbias_out, accumulate, width, dev) -> Tuple[Optional[Tensor], int]:
    """A bias's gradient, new or as given, and its address."""
    if not bias_grad:
        if dbias_out is not None or accumulate:
            raise ValueError("dbias_out and accumulate need bias_grad")
        return None, 0
    if dbias_out is not None:
        return dbias_out, _vector(dbias_out, "dbias_out", width, torch.float32, dev)
    if accumulate:
        raise ValueError("accumulate needs dbias_out")
    dbias = torch.empty(width, dtype=torch.float32, device=dev)
    return dbias, dbias.data_ptr()


def _alone(dbias_out: Optional[Tensor], dd: Tensor, z: Optional[Tensor]) -> None:
    if dbias_out is not None and any(_rows_meet(_rows_at(dbias_out), _rows_at(t)) for t in (dd, z) if t is not None):
        raise ValueError("dbias_out overlaps another operand")


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
            dz = torch.empty_like(z, memory_format=torch.contiguous_format)
            po, ldo = dz.data_ptr(), width
        else:
            dz = dz_out
            po, ldo = _rows(dz_out, "dz_out", shape, dev)
    dbias, pb = _dbias(bias_grad, dbias_out, accumulate, width, dev)
    if rows == 0:
        if bias_grad and not accumulate:
            dbias.zero_()
        return ActGrads(dz, dbias)
    if dz_out is not None:
        _may_write(dz_out, "dz_out", [(z, True), (dd, not gated), (dbias, False)])
    _alone(dbias_out, dd, z)
    ws, nws = None, 0
    if bias_grad:
        nws = L.pf8_act_bwd_workspace(rows, cols, int(gated))
        ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    _call(L.pf8_act_bwd, dev, rows, cols, pd, ldd, pz, ldz, code, int(gated), po, ldo, pb, int(accumulate),
          0 if ws is None else ws.data_ptr(), nws)
    return ActGrads(dz, dbias)


def act_backward_quant(dd: Tensor, z: Optional[Tensor], activation: Optional[str], gated: bool = False,
                       bias_grad: bool = False, dbias_out: Optional[Tensor] = None, accumulate: bool = False
                       ) -> ActQuantGrads:
    """``act_backward`` with dz as the codes of both groupings, what ``dgrad`` and ``wgrad`` take.

    Bit for bit ``quant_act_dual(act_backward(...).dz)``, without dz in memory; rows and columns of dd are multiples of
    128. Without an activation the codes are those of dd, and z is None. dbias comes as from ``act_backward``, its sums
    formed in another fixed order.
    """
    if not isinstance(dd, Tensor) or dd.dim() != 2:
        raise ValueError("dd must be a 2-D tensor")
    if not dd.is_cuda:
        raise ValueError("dd must be on a HIP device")
    code = _activation(activation, gated)
    (rows, cols), dev = dd.shape, dd.device
    if rows % GROUP or cols % GROUP or not rows or not cols:
        raise ValueError(f"act_backward_quant needs multiples of {GROUP} rows and columns, got {tuple(dd.shape)}")
    if (z is None) != (code == 0):
        raise ValueError("z comes with an activation")
    width = 2 * cols if gated else cols
    pd, ldd = _aligned_rows(dd, "dd", dd.shape, dev)
    pz, ldz = (0, 0) if z is None else _aligned_rows(z, "z", torch.Size((rows, width)), dev)
    dbias, pb = _dbias(bias_grad, dbias_out, accumulate, width, dev)
    _alone(dbias_out, dd, z)
    q, qt = code_buffer(rows, width, dev), code_buffer(width, rows, dev)
    s = torch.empty((width // GROUP, rows), dtype=torch.float32, device=dev)
    st = torch.empty((rows // GROUP, width), dtype=torch.float32, device=dev)
    ws, nws = None, 0
    if bias_grad:
        nws = L.pf8_act_bwd_quant_workspace(rows, cols, int(gated))
        ws = torch.empty(nws, dtype=torch.uint8, device=dev)
    _call(L.pf8_act_bwd_quant, dev, rows, cols, pd, ldd, pz, ldz, code, int(gated), q.data_ptr(), q.stride(0), s.data_ptr(),
          rows, qt.data_ptr(), qt.stride(0), st.data_ptr(), width, pb, int(accumulate), 0 if ws is None else ws.data_ptr(), nws)
    return ActQuantGrads(q, s, qt, st, dbias)
