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

from .block import _plain
from .ffn import (_MATRIX, _NONE, Matrix, _c_i32, _c_i64, _c_vp, _Entry, _fail, _first, _mat,
                  _number, _out)


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
_ADAPTER = _Entry("moe_adapter_linear", "moe_adapter_linear_workspace_bytes")
_ADAPTER_BACKWARD = _Entry("moe_adapter_linear_backward", "moe_adapter_linear_workspace_bytes", 1)


def _adapters(x, w, a, b, ids, scale):
    """Checked sizes of an adapter call: (dtype, tokens, in, out, rank, adapters)."""
    d = _first(x, "x")
    for t, name, ndim in ((w, "w", 2), (a, "a", 3), (b, "b", 3)):
        if not isinstance(t, torch.Tensor) or t.dim() != ndim:
            _fail(f"{name} must be a tensor of {ndim} dimensions")
    if ids is None:
        _fail("ids are needed")
    n, rank, _ = a.shape
    return (d, x.shape[0], _number(x.shape[1], "in"), _number(w.shape[0], "out"),
            _number(rank, "rank"), _number(n, "adapters"))


def adapter_linear(x: torch.Tensor, w: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                   ids: torch.Tensor, *, scale: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                   save: bool = False, out: Optional[Dict[str, torch.Tensor]] = None,
                   ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_adapter_linear: y [T, O] = x W^T + bias + s B[id]^T + residual with
    s [T, R] = scale[id] x A[id]^T, from x [T, I], w [O, I], a [n, R, I], b [n, O, R],
    ids [T] (int32; a number outside 0 .. n-1: the token has no adapter) and scale [n]
    (fp32). With `save` also s (fp32), which adapter_linear_backward reads."""
    d, tokens, n_in, n_out, rank, n = _adapters(x, w, a, b, ids, scale)
    if out is None:
        out = {"y": torch.empty((tokens, n_out), dtype=x.dtype, device=x.device)}
    if save and out.get("s") is None:
        out["s"] = torch.empty((tokens, rank), dtype=torch.float32, device=x.device)
    s = out.get("s") if save else None
    args = _PACK(
        d, rank, tokens, n_in, n_out, n, 0, *_mat(x, "x", (tokens, n_in), x),
        *_mat(w, "w", (n_out, n_in), x), *_mat(a, "a", (n, rank, n_in), x),
        *_mat(b, "b", (n, n_out, rank), x), *_mat(bias, "bias", (n_out,), x),
        *_mat(residual, "residual", (tokens, n_out), x),
        *_mat(_out(out, "y"), "y", (tokens, n_out), x),
        _plain(ids, "ids", torch.int32, (tokens,), x.device),
        _plain(scale, "scale", torch.float32, (n,), x.device),
        _plain(s, "s", torch.float32, (tokens, rank), x.device), *_NONE * 4)
    _ADAPTER(args, x.device, ws)
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
    d, tokens, n_in, n_out, rank, n = _adapters(x, w, a, b, ids, scale)
    if dy is None:
        _fail("dy is needed")
    if out is None:
        out = {"dx": torch.empty((tokens, n_in), dtype=x.dtype, device=x.device),
               "da": torch.empty((n, rank, n_in), dtype=x.dtype, device=x.device),
               "db": torch.empty((n, n_out, rank), dtype=x.dtype, device=x.device)}
    args = _PACK(
        d, rank, tokens, n_in, n_out, n, 0, *_mat(x, "x", (tokens, n_in), x),
        *_mat(w, "w", (n_out, n_in), x), *_mat(a, "a", (n, rank, n_in), x),
        *_mat(b, "b", (n, n_out, rank), x), *_NONE * 3,
        _plain(ids, "ids", torch.int32, (tokens,), x.device),
        _plain(scale, "scale", torch.float32, (n,), x.device),
        _plain(s, "s", torch.float32, (tokens, rank), x.device),
        *_mat(dy, "dy", (tokens, n_out), x), *_mat(out.get("dx"), "dx", (tokens, n_in), x),
        *_mat(out.get("da"), "da", (n, rank, n_in), x),
        *_mat(out.get("db"), "db", (n, n_out, rank), x))
    _ADAPTER_BACKWARD(args, x.device, ws)
    return out
