"""Python binding of the operators around the feed-forward block
(``include/moe_block.h``): the norm in front of the router and the experts, and
dropout.

Argument marshalling only, as in the module ``ffn``, whose conventions hold
here too: tensors are checked, outputs and a workspace are allocated when the
caller gives none, the backward passes are calls of their own.

    rms_norm(x, weight, residual=, p=, rng=, quant=)   -> moe_rms_norm
    rms_norm_backward(dy, h, weight, rstd, dh=)        -> moe_rms_norm_backward
    dropout(x, p, rng, residual=)                      -> moe_dropout
    dropout_backward(dout, p, rng)                     -> moe_dropout
    mxfp8_values(act_q, act_scale)                     -> moe_mxfp8_values

``rng`` is an int64 tensor [seed, offset] on the device, read when the kernels
run: a program adds to the offset between its steps (``rng[1] += 1``, in a
captured graph too), and a backward pass has to run with the numbers of its
forward pass. ``site`` tells the dropouts of one step apart. ``p`` is taken as
the nearest multiple of 2^-16.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Dict, Optional

import torch

from . import ffn as _ffn
from .ffn import (_MATRIX, _NONE, DTYPES, Matrix, _c_i32, _c_i64, _c_vp, _Entry, _fail, _first,
                  _mat, _number, _out)

_c_u32 = ctypes.c_uint32


class DropoutSpec(ctypes.Structure):
    _fields_ = [("state", _c_vp), ("level", _c_u32), ("site", _c_i32)]


class RmsNormArgs(ctypes.Structure):
    _fields_ = [("dtype", _c_i32), ("width", _c_i32), ("tokens", _c_i64),
                ("eps", ctypes.c_float), ("reserved", _c_i32), ("drop", DropoutSpec)] + \
        [(n, Matrix) for n in ("x", "residual", "h", "y")] + \
        [(n, _c_vp) for n in ("weight", "rstd", "q", "q_scale")] + \
        [(n, Matrix) for n in ("dy", "dh", "dx", "dresidual")] + [("dweight", _c_vp)]


class DropoutArgs(ctypes.Structure):
    _fields_ = [("dtype", _c_i32), ("width", _c_i32), ("tokens", _c_i64),
                ("drop", DropoutSpec)] + [(n, Matrix) for n in ("x", "residual", "out")]


EXPORTS = {
    "moe_rms_norm": (ctypes.c_int, [_c_vp, _c_vp]),
    "moe_rms_norm_backward_workspace_bytes": (_c_i64, [_c_vp, _c_i32]),
    "moe_rms_norm_backward": (ctypes.c_int, [_c_vp, _c_vp, ctypes.c_size_t, _c_vp]),
    "moe_dropout": (ctypes.c_int, [_c_vp, _c_vp]),
    "moe_mxfp8_values": (ctypes.c_int, [_c_vp, _c_vp, _c_i64, _c_i32, _c_vp, _c_vp]),
}

_DROP = "PIi"
_PACK_NORM = struct.Struct("@iiqfi" + _DROP + 4 * _MATRIX + "PPPP" + 4 * _MATRIX + "P").pack
_PACK_DROPOUT = struct.Struct("@iiq" + _DROP + 3 * _MATRIX).pack



class _SizedEntry(_Entry):
    """An entry whose calls nearly always need a workspace: its size is asked for
    first, which saves a call that would only say so."""

    def __call__(self, args: bytes, dev: torch.device, ws: Optional[torch.Tensor] = None) -> None:
        if ws is None:
            need = getattr(_ffn._pkg.lib(), self.size)(args, self.backward)
            if need > 0:
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
        super().__call__(args, dev, ws)


_NORM = _Entry("moe_rms_norm")
_NORM_BACKWARD = _SizedEntry("moe_rms_norm_backward", "moe_rms_norm_backward_workspace_bytes", 1)
_DROPOUT = _Entry("moe_dropout")


class _Values(_Entry):
    """moe_mxfp8_values, whose arguments are no structure."""

    def __call__(self, args: tuple, dev: torch.device, ws: Optional[torch.Tensor] = None) -> None:
        if self.fn is None:
            fn = getattr(_ffn._pkg.lib(), self.name)
            self.fn = lambda a, stream: fn(*a, stream)
        super().__call__(args, dev, ws)


_VALUES = _Values("moe_mxfp8_values")


def _m(t: Optional[torch.Tensor], name: str, shape: tuple, dtype, dev, like) -> tuple:
    """_mat, in less host time where the tensor is as it should be and contiguous."""
    if t is None:
        return _NONE
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and \
            t.is_contiguous() and t.device == dev:
        cols = shape[-1]
        return (t.data_ptr(), cols, cols * shape[-2] if len(shape) == 3 else 0)
    return _mat(t, name, shape, like)


def _plain(t: Optional[torch.Tensor], name: str, dtype, shape: tuple, dev) -> int:
    """The pointer of a contiguous tensor of a fixed type, checked; 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev or \
            not t.is_contiguous():
        _fail(f"{name} must be a contiguous {dtype} tensor on {dev}")
    if t.shape != shape:
        _fail(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    return t.data_ptr()


def _drop(p, rng, site, dev) -> tuple:
    """(state, level, site) of a dropout."""
    if not isinstance(p, (int, float)) or not 0.0 <= p <= 1.0:
        _fail(f"p must be between 0 and 1, not {p!r}")
    level = int(round(p * 65536))
    site = _number(site, "site")
    if rng is None and level:
        _fail("rng is needed where something is dropped")
    return _plain(rng, "rng", torch.int64, (2,), dev), level, site


def rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6, p: float = 0.0, rng: Optional[torch.Tensor] = None, site: int = 0,
             quant: Optional[str] = None,
             out: Optional[Dict[str, torch.Tensor]] = None) -> Dict[str, torch.Tensor]:
    """moe_rms_norm: y [T, W] = h rstd weight with h = residual + x, x dropped out
    with probability p, and rstd [T] (fp32) = 1 / sqrt(mean(h^2) + eps). Returns y,
    rstd and, with a residual or dropout, h [T, W] (without them it is x).
    quant="mxfp8" returns act_q (uint8 E4M3 codes [T, W]) and act_scale (uint8
    E8M0 codes [T, W/32]) in the place of y, as route_quant_local does. An `out`
    dict gives the outputs' memory: y and rstd are left out where it has none, h
    may be the residual itself, and with quant a y in it is written too."""
    d = _first(x, "x")
    shape = tokens, width = x.shape
    dt, dev = x.dtype, x.device
    if quant not in (None, "mxfp8"):
        _fail(f"quant must be None or 'mxfp8', not {quant!r}")
    drop = _drop(p, rng, site, dev)
    if not isinstance(eps, (int, float)) or not 0.0 <= eps <= 3.4e38:
        _fail(f"eps must be a number of 0 or more, not {eps!r}")
    if out is None:
        out = {"rstd": torch.empty(tokens, dtype=torch.float32, device=dev)}
        if quant is None:
            out["y"] = torch.empty_like(x)
        if residual is not None or drop[1]:
            out["h"] = torch.empty_like(x)
    q = scale = 0
    if quant:
        if width % 32:
            _fail("quant needs a width that is a multiple of 32")
        for name, cols in (("act_q", width), ("act_scale", width // 32)):
            if out.get(name) is None:
                out[name] = torch.empty((tokens, cols), dtype=torch.uint8, device=dev)
        q = _plain(out["act_q"], "act_q", torch.uint8, shape, dev)
        scale = _plain(out["act_scale"], "act_scale", torch.uint8, (tokens, width // 32), dev)
    elif out.get("y") is None:
        _fail("out must have y")
    h = _out(out, "h") if residual is not None or drop[1] else out.get("h")
    a = _PACK_NORM(d, _number(width, "width"), tokens, eps, 0, *drop,
                   *_m(x, "x", shape, dt, dev, x), *_m(residual, "residual", shape, dt, dev, x),
                   *_m(h, "h", shape, dt, dev, x), *_m(out.get("y"), "y", shape, dt, dev, x),
                   _weight(weight, width, x),
                   _plain(out.get("rstd"), "rstd", torch.float32, (tokens,), dev), q, scale,
                   *_NONE * 4, 0)
    _NORM(a, dev)
    return out


def _weight(weight, width: int, like: torch.Tensor) -> int:
    if weight is None:
        _fail("weight is needed")
    return _m(weight, "weight", (width,), like.dtype, like.device, like)[0]


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                      *, dh: Optional[torch.Tensor] = None, p: float = 0.0,
                      rng: Optional[torch.Tensor] = None, site: int = 0,
                      out: Optional[Dict[str, torch.Tensor]] = None,
                      ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_rms_norm_backward: from dy [T, W], the forward pass's h and rstd, and dh
    [T, W], the gradient that reaches h from behind (None: 0): dx [T, W], the gradient
    of x and, without dropout, of the residual too; dweight [W]; with dropout
    also dresidual [T, W]. An `out` dict without one of them leaves it out."""
    d = _first(h, "h")
    shape = tokens, width = h.shape
    dt, dev = h.dtype, h.device
    drop = _drop(p, rng, site, dev)
    if out is None:
        out = {"dx": torch.empty_like(h),
               "dweight": h.new_empty(width)}
        if drop[1]:
            out["dresidual"] = torch.empty_like(h)
    if dy is None or rstd is None:
        _fail("dy and rstd are needed")
    a = _PACK_NORM(d, _number(width, "width"), tokens, 0.0, 0, *drop, *_NONE * 2,
                   *_m(h, "h", shape, dt, dev, h), *_NONE, _weight(weight, width, h),
                   _plain(rstd, "rstd", torch.float32, (tokens,), dev), 0, 0,
                   *_m(dy, "dy", shape, dt, dev, h), *_m(dh, "dh", shape, dt, dev, h),
                   *_m(out.get("dx"), "dx", shape, dt, dev, h),
                   *_m(out.get("dresidual"), "dresidual", shape, dt, dev, h),
                   _m(out.get("dweight"), "dweight", (width,), dt, dev, h)[0])
    _NORM_BACKWARD(a, dev, ws)
    return out


def dropout(x: torch.Tensor, p: float, rng: Optional[torch.Tensor], *, site: int = 0,
            residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_dropout: out [T, W] = residual + x, x dropped out with probability p and
    scaled by 1 / (1 - p). `out` may be x or the residual."""
    d = _first(x, "x")
    shape = tokens, width = x.shape
    dt, dev = x.dtype, x.device
    drop = _drop(p, rng, site, dev)
    if out is None:
        out = torch.empty_like(x)
    a = _PACK_DROPOUT(d, _number(width, "width"), tokens, *drop, *_m(x, "x", shape, dt, dev, x),
                      *_m(residual, "residual", shape, dt, dev, x),
                      *_m(out, "out", shape, dt, dev, x))
    _DROPOUT(a, dev)
    return out


def dropout_backward(dout: torch.Tensor, p: float, rng: Optional[torch.Tensor], *, site: int = 0,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of dropout's x from dout [T, W], with the rng and site of the
    forward pass. The residual's gradient is dout."""
    return dropout(dout, p, rng, site=site, out=out)


def mxfp8_values(act_q: torch.Tensor, act_scale: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_mxfp8_values: what act_q [T, W] and act_scale [T, W/32] of rms_norm or
    route_quant_local stand for, [T, W] in bfloat16 or float16."""
    if not isinstance(act_q, torch.Tensor) or not act_q.is_cuda or act_q.dim() != 2:
        _fail("act_q must be a GPU tensor of 2 dimensions")
    if dtype not in DTYPES:
        _fail(f"dtype must be bfloat16 or float16, not {dtype}")
    tokens, width = act_q.shape
    if width % 32:
        _fail("act_q must have a width that is a multiple of 32")
    dev = act_q.device
    if act_scale is None:
        _fail("act_scale is needed")
    if out is None:
        out = torch.empty((tokens, width), dtype=dtype, device=dev)
    _VALUES((_plain(act_q, "act_q", torch.uint8, (tokens, width), dev),
             _plain(act_scale, "act_scale", torch.uint8, (tokens, width // 32), dev),
             tokens * width, DTYPES[dtype], _plain(out, "out", dtype, (tokens, width), dev)), dev)
    return out
