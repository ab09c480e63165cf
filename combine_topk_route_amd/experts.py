"""Binding of the experts' products and of the gradients: argument marshalling
only, as in ``binding``.

The rows are dispatch's: expert ``e`` owns rows ``expert_offsets[e]`` to
``expert_offsets[e + 1]`` of ``x``, and rows behind the last expert are left
as they were in every output.  A training step runs

    send, buf = moe_dispatch(idx, x, E)
    h, gate_up = moe_expert_gated(buf, send.expert_offsets, w_gate_up, save_gate_up=True)
    y, _ = moe_expert_matmul(h, send.expert_offsets, w_down)
    out = moe_combine(y, send.pair_row, w)

and back

    dy, dw_route = moe_combine_backward(dout, y, send.pair_row, w)
    down = moe_expert_matmul_backward(dy, h, send.expert_offsets, w_down)
    gated = moe_expert_gated_backward(down.dx, gate_up, buf, send.expert_offsets, w_gate_up)
    dx = moe_combine(gated.dx, send.pair_row, torch.ones_like(w))   # dispatch's gradient
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .binding import MoeError, _dev, _empty, _stream

_BF16 = torch.bfloat16


class GatedGrads(NamedTuple):
    dx: Optional[torch.Tensor]        # bf16 [rows, H]
    dw: Optional[torch.Tensor]        # bf16 or fp32 [E, 2*I, H]
    dgate_up: torch.Tensor            # bf16 [rows, 2*I]


class MatmulGrads(NamedTuple):
    dx: Optional[torch.Tensor]        # bf16 [rows, K]
    dw: Optional[torch.Tensor]        # bf16 or fp32 [E, N, K]
    dbias: Optional[torch.Tensor]     # fp32 [E, N]
    dpre: Optional[torch.Tensor]      # bf16 [rows, N]; None without an activation


def _act(act: str) -> int:
    try:
        return _lib.ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {sorted(_lib.ACTS)}, got {act!r}") from None


# The current device without the checks of torch.cuda.current_device, which
# cost as much as the rest of a small call's marshalling.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name: str, device: int, *args) -> None:
    """The library's entry point `name`, with `device` the current one: a
    launch goes to the current device, so tensors elsewhere need the switch."""
    fn = getattr(_lib.load(), name)
    if device == _current_device():
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status != _lib.MOE_OK:
        raise MoeError(name, status)


def _given(t: Optional[torch.Tensor], name: str, shape, dtype, device: int) -> Optional[int]:
    """Pointer of an optional tensor after the checks every tensor gets."""
    if t is None:
        return None
    p = _dev(t, name, dtype, len(shape), device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return p


def _out(t: Optional[torch.Tensor], name: str, shape, dtype, like: torch.Tensor, stream):
    """(tensor, pointer) of an output, allocated on the launch stream if not given."""
    if t is None:
        t = like.new_empty(shape, dtype=dtype) if stream is None else _empty(shape, dtype, like,
                                                                            stream)
        return t, t.data_ptr()
    return t, _given(t, name, shape, dtype, like.get_device())


def _offsets(expert_offsets: torch.Tensor, E: int, device: int) -> int:
    return _given(expert_offsets, "expert_offsets", (E + 1,), torch.int32, device)


def _dw_dtype(dw: Optional[torch.Tensor], dw_dtype) -> torch.dtype:
    dtype = dw.dtype if dw is not None else dw_dtype
    if dtype not in (_BF16, torch.float32):
        raise TypeError(f"dw must be torch.bfloat16 or torch.float32, got {dtype}")
    return dtype


def moe_expert_gated(x: torch.Tensor, expert_offsets: torch.Tensor, w_gate_up: torch.Tensor,
                     act: str = "silu", *, h: Optional[torch.Tensor] = None,
                     gate_up: Optional[torch.Tensor] = None, save_gate_up: bool = False,
                     stream=None):
    """act(x W_gate^T) * (x W_up^T) of every expert's rows: returns (h bf16
    [rows, I], gate_up bf16 [rows, 2*I] or None).  ``w_gate_up`` is bf16
    [E, 2*I, H], the gate rows first.  ``save_gate_up`` keeps both factors for
    the backward pass."""
    xp = _dev(x, "x", _BF16, 2)
    d = x.get_device()
    wp = _dev(w_gate_up, "w_gate_up", _BF16, 3, d)
    rows, H = x.shape
    E, I2 = w_gate_up.shape[:2]
    if w_gate_up.shape[2] != H or I2 % 2:
        raise ValueError(f"w_gate_up must be [E, 2*I, {H}], got {list(w_gate_up.shape)}")
    op = _offsets(expert_offsets, E, d)
    a = _act(act)
    h, hp = _out(h, "h", (rows, I2 // 2), _BF16, x, stream)
    gp = None
    if save_gate_up or gate_up is not None:
        gate_up, gp = _out(gate_up, "gate_up", (rows, I2), _BF16, x, stream)
    _call("moe_expert_gated", d, xp, op, wp, rows, E, H, I2 // 2, a, hp, gp, _stream(stream, x))
    return h, gate_up


def moe_expert_gated_backward(dh: torch.Tensor, gate_up: torch.Tensor, x: torch.Tensor,
                              expert_offsets: torch.Tensor, w_gate_up: torch.Tensor,
                              act: str = "silu", *, dgate_up: Optional[torch.Tensor] = None,
                              dx: Optional[torch.Tensor] = None,
                              dw: Optional[torch.Tensor] = None, need_dx: bool = True,
                              need_dw: bool = True, dw_dtype: torch.dtype = _BF16,
                              stream=None) -> GatedGrads:
    """Gradients of moe_expert_gated from dh [rows, I] and the factors it kept.
    ``dw`` is bf16 unless ``dw_dtype`` (or a given ``dw``) is fp32."""
    xp = _dev(x, "x", _BF16, 2)
    d = x.get_device()
    wp = _dev(w_gate_up, "w_gate_up", _BF16, 3, d)
    rows, H = x.shape
    E, I2 = w_gate_up.shape[:2]
    if w_gate_up.shape[2] != H or I2 % 2:
        raise ValueError(f"w_gate_up must be [E, 2*I, {H}], got {list(w_gate_up.shape)}")
    op = _offsets(expert_offsets, E, d)
    hp = _given(dh, "dh", (rows, I2 // 2), _BF16, d)
    gp = _given(gate_up, "gate_up", (rows, I2), _BF16, d)
    a = _act(act)
    dgate_up, dgp = _out(dgate_up, "dgate_up", (rows, I2), _BF16, x, stream)
    dxp = dwp = None
    wt = _dw_dtype(dw, dw_dtype)
    if need_dx or dx is not None:
        dx, dxp = _out(dx, "dx", (rows, H), _BF16, x, stream)
    if need_dw or dw is not None:
        dw, dwp = _out(dw, "dw", (E, I2, H), wt, x, stream)
    _call("moe_expert_gated_backward", d, hp, gp, xp, op, wp, rows, E, H, I2 // 2, a, dgp, dxp,
          dwp, int(wt is torch.float32), _stream(stream, x))
    return GatedGrads(dx, dw, dgate_up)


def moe_expert_matmul(x: torch.Tensor, expert_offsets: torch.Tensor, w: torch.Tensor, *,
                      bias: Optional[torch.Tensor] = None, act: str = "none",
                      residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                      pre: Optional[torch.Tensor] = None, save_pre: bool = False, stream=None):
    """act(x W^T + bias) + residual of every expert's rows: returns (y bf16
    [rows, N], pre bf16 [rows, N] or None).  ``w`` is bf16 [E, N, K], ``bias``
    bf16 [E, N]; ``save_pre`` keeps the activation's argument for the backward
    pass."""
    xp = _dev(x, "x", _BF16, 2)
    d = x.get_device()
    wp = _dev(w, "w", _BF16, 3, d)
    rows, K = x.shape
    E, N = w.shape[:2]
    if w.shape[2] != K:
        raise ValueError(f"w must be [E, N, {K}], got {list(w.shape)}")
    op = _offsets(expert_offsets, E, d)
    bp = _given(bias, "bias", (E, N), _BF16, d)
    rp = _given(residual, "residual", (rows, N), _BF16, d)
    a = _act(act)
    y, yp = _out(y, "y", (rows, N), _BF16, x, stream)
    pp = None
    if save_pre or pre is not None:
        pre, pp = _out(pre, "pre", (rows, N), _BF16, x, stream)
    _call("moe_expert_matmul", d, xp, op, wp, bp, rp, rows, E, K, N, a, yp, pp, _stream(stream, x))
    return y, pre


def moe_expert_matmul_backward(dy: torch.Tensor, x: torch.Tensor, expert_offsets: torch.Tensor,
                               w: torch.Tensor, *, act: str = "none",
                               pre: Optional[torch.Tensor] = None,
                               dpre: Optional[torch.Tensor] = None,
                               dx: Optional[torch.Tensor] = None,
                               dw: Optional[torch.Tensor] = None,
                               dbias: Optional[torch.Tensor] = None, need_dx: bool = True,
                               need_dw: bool = True, need_dbias: bool = False,
                               dw_dtype: torch.dtype = _BF16, stream=None) -> MatmulGrads:
    """Gradients of moe_expert_matmul from dy [rows, N] (the residual's is dy
    itself).  With an activation ``pre`` is the forward call's.  ``dw`` is bf16
    unless ``dw_dtype`` (or a given ``dw``) is fp32; ``dbias`` is fp32 [E, N]."""
    xp = _dev(x, "x", _BF16, 2)
    d = x.get_device()
    wp = _dev(w, "w", _BF16, 3, d)
    rows, K = x.shape
    E, N = w.shape[:2]
    if w.shape[2] != K:
        raise ValueError(f"w must be [E, N, {K}], got {list(w.shape)}")
    op = _offsets(expert_offsets, E, d)
    yp = _given(dy, "dy", (rows, N), _BF16, d)
    a = _act(act)
    pp = dpp = None
    if act != "none":
        if pre is None:
            raise ValueError("pre (the forward call's) is needed with an activation")
        pp = _given(pre, "pre", (rows, N), _BF16, d)
        dpre, dpp = _out(dpre, "dpre", (rows, N), _BF16, x, stream)
    elif dpre is not None:
        raise ValueError("dpre is written with an activation only (without one it is dy)")
    dxp = dwp = dbp = None
    wt = _dw_dtype(dw, dw_dtype)
    if need_dx or dx is not None:
        dx, dxp = _out(dx, "dx", (rows, K), _BF16, x, stream)
    if need_dw or dw is not None:
        dw, dwp = _out(dw, "dw", (E, N, K), wt, x, stream)
    if need_dbias or dbias is not None:
        dbias, dbp = _out(dbias, "dbias", (E, N), torch.float32, x, stream)
    _call("moe_expert_matmul_backward", d, yp, pp, xp, op, wp, rows, E, K, N, a, dpp, dxp, dwp,
          int(wt is torch.float32), dbp, _stream(stream, x))
    return MatmulGrads(dx, dw, dbias, dpre)


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, pair_row: torch.Tensor,
                         topk_w: torch.Tensor, *, dy: Optional[torch.Tensor] = None,
                         dtopk_w: Optional[torch.Tensor] = None, capacity: Optional[int] = None,
                         stream=None):
    """Gradients of moe_combine: returns (dy bf16 [capacity, H], dtopk_w fp32
    [T, k]).  Rows of dy that no pair maps to are left as they were."""
    yp = _dev(y, "y", _BF16, 2)
    d = y.get_device()
    if pair_row.dim() != 2:
        raise ValueError("pair_row must be [T, k]")
    T, k = pair_row.shape
    H = y.shape[1]
    op = _given(dout, "dout", (T, H), _BF16, d)
    pp = _dev(pair_row, "pair_row", torch.int32, 2, d)
    wp = _given(topk_w, "topk_w", (T, k), torch.float32, d)
    if capacity is None:
        capacity = y.shape[0]
    if capacity > y.shape[0]:
        raise ValueError("capacity exceeds y's rows")
    dy, dyp = _out(dy, "dy", (y.shape[0], H), _BF16, y, stream)
    dtopk_w, dwp = _out(dtopk_w, "dtopk_w", (T, k), torch.float32, y, stream)
    _call("moe_combine_backward", d, op, yp, pp, wp, T, H, k, capacity, dyp, dwp, _stream(stream, y))
    return dy, dtopk_w
