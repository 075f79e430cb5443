"""Python binding of the projection with the low-rank adapters of many requests
beside it (``include/moe_adapter.h``).

Argument marshalling only, as in the module ``ffn``, whose conventions hold
here too: tensors are checked, outputs and a workspace are allocated when the
caller gives none, and the backward pass is a call of its own.

    adapter_linear(x, w, a, b, ids)                    -> moe_adapter_linear
    adapter_linear_backward(dy, x, w, a, b, ids, s)    -> moe_adapter_linear_backward
"""
from __future__ import annotations

import ctypes
import struct
from typing import Dict, Optional

import torch

from .block import _m, _plain, _SizedEntry
from .ffn import (_MATRIX, _NONE, Matrix, _c_i32, _c_i64, _c_vp, _fail, _first, _number, _out)


class AdapterLinearArgs(ctypes.Structure):
    _fields_ = [("dtype", _c_i32), ("rank", _c_i32), ("tokens", _c_i64), ("in_", _c_i32),
                ("out", _c_i32), ("adapters", _c_i32), ("reserved", _c_i32)] + \
        [(n, Matrix) for n in ("x", "w", "a", "b", "bias", "residual", "y")] + \
        [(n, _c_vp) for n in ("ids", "scale", "s")] + \
        [(n, Matrix) for n in ("dy", "dx", "da", "db")]


_ENTRY = (ctypes.c_int, [_c_vp, _c_vp, ctypes.c_size_t, _c_vp])
EXPORTS = {
    "moe_adapter_linear_workspace_bytes": (_c_i64, [_c_vp, _c_i32]),
    "moe_adapter_linear": _ENTRY,
    "moe_adapter_linear_backward": _ENTRY,
}

_PACK = struct.Struct("@iiqiiii" + 7 * _MATRIX + "PPP" + 4 * _MATRIX).pack
_ADAPTER = _SizedEntry("moe_adapter_linear", "moe_adapter_linear_workspace_bytes")
_ADAPTER_BACKWARD = _SizedEntry("moe_adapter_linear_backward", "moe_adapter_linear_workspace_bytes",
                                1)


def _adapters(x, w, a, b, ids, scale):
    """What both calls pass on, checked: (dtype, device, tokens, in, out, rank, adapters),
    the sizes, the matrices x, w, a and b, ids and scale."""
    d = _first(x, "x")
    for t, name, ndim in ((w, "w", 2), (a, "a", 3), (b, "b", 3)):
        if not isinstance(t, torch.Tensor) or t.dim() != ndim:
            _fail(f"{name} must be a tensor of {ndim} dimensions")
    if ids is None:
        _fail("ids are needed")
    dt, dev = x.dtype, x.device
    tokens, n_in = x.shape
    n_out = w.shape[0]
    n, rank, _ = a.shape
    head = (d, _number(rank, "rank"), tokens, _number(n_in, "in"), _number(n_out, "out"),
            _number(n, "adapters"), 0)
    mats = (*_m(x, "x", (tokens, n_in), dt, dev, x), *_m(w, "w", (n_out, n_in), dt, dev, x),
            *_m(a, "a", (n, rank, n_in), dt, dev, x), *_m(b, "b", (n, n_out, rank), dt, dev, x))
    tail = (_plain(ids, "ids", torch.int32, (tokens,), dev),
            _plain(scale, "scale", torch.float32, (n,), dev))
    return (dt, dev, tokens, n_in, n_out, rank, n), head, mats, tail


def adapter_linear(x: torch.Tensor, w: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                   ids: torch.Tensor, *, scale: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                   save: bool = False, out: Optional[Dict[str, torch.Tensor]] = None,
                   ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_adapter_linear: y [T, O] = x W^T + bias + s B[id]^T + residual with
    s [T, R] = scale[id] x A[id]^T, from x [T, I], w [O, I], a [n, R, I], b [n, O, R],
    ids [T] (int32; a number outside 0 .. n-1: the token has no adapter) and scale [n]
    (fp32). With `save` also s (fp32), which adapter_linear_backward reads."""
    (dt, dev, tokens, _, n_out, rank, _), head, mats, tail = _adapters(x, w, a, b, ids, scale)
    if out is None:
        out = {"y": x.new_empty((tokens, n_out))}
    if save and out.get("s") is None:
        out["s"] = torch.empty((tokens, rank), dtype=torch.float32, device=dev)
    s = out.get("s") if save else None
    shape = (tokens, n_out)
    args = _PACK(*head, *mats, *_m(bias, "bias", (n_out,), dt, dev, x),
                 *_m(residual, "residual", shape, dt, dev, x),
                 *_m(_out(out, "y"), "y", shape, dt, dev, x), *tail,
                 _plain(s, "s", torch.float32, (tokens, rank), dev), *_NONE * 4)
    _ADAPTER(args, dev, ws)
    return out


def adapter_linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, a: torch.Tensor,
                            b: torch.Tensor, ids: torch.Tensor, s: torch.Tensor, *,
                            scale: Optional[torch.Tensor] = None,
                            out: Optional[Dict[str, torch.Tensor]] = None,
                            ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_adapter_linear_backward: dx [T, I], da [n, R, I] and db [n, O, R] (zeros for
    an adapter without tokens) from dy [T, O] and the forward pass's s [T, R]. An
    `out` dict without one of them leaves it out; s may be None without db. The
    residual's gradient is dy, and w has none here."""
    (dt, dev, tokens, n_in, n_out, rank, n), head, mats, tail = _adapters(x, w, a, b, ids, scale)
    if dy is None:
        _fail("dy is needed")
    if out is None:
        out = {"dx": x.new_empty((tokens, n_in)),
               "da": x.new_empty((n, rank, n_in)),
               "db": x.new_empty((n, n_out, rank))}
    args = _PACK(*head, *mats, *_NONE * 3, *tail,
                 _plain(s, "s", torch.float32, (tokens, rank), dev),
                 *_m(dy, "dy", (tokens, n_out), dt, dev, x),
                 *_m(out.get("dx"), "dx", (tokens, n_in), dt, dev, x),
                 *_m(out.get("da"), "da", (n, rank, n_in), dt, dev, x),
                 *_m(out.get("db"), "db", (n, n_out, rank), dt, dev, x))
    _ADAPTER_BACKWARD(args, dev, ws)
    return out
