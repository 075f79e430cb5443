"""Python binding of the feed-forward operators (``include/moe_ffn.h``): the
gated block, the linear product with its epilogue and the combination of the
experts' rows, dense or over a routing call's grouped layout, forward and
backward.

Argument marshalling only, as in the package's own module: tensors are
checked, outputs and a workspace are allocated when the caller gives none, and
the HIP kernels behind the C ABI do every step. The backward passes are calls
of their own: outputs carry no autograd graph, also where inputs require
gradients, and nothing is kept between calls.

    gated_ffn(x, w_gate, w_up)                 -> moe_gated_ffn
    gated_ffn_backward(dh, pre, x, w_gate, w_up) -> moe_gated_ffn_backward
    linear(x, w)                               -> moe_linear
    linear_backward(dy, x, w)                  -> moe_linear_backward
    expert_gated_ffn(x, w_gate, w_up, lay, tile_m=, top_k=)   and so on:
        the same over the experts' rows of a layout
    combine(y, lay, num_experts=)              -> moe_combine
    combine_backward(dout, y, lay, num_experts=) -> moe_combine_backward

``lay`` is what ``route_local_grouped`` returns (or a dict with the same
names from ``route_local`` and ``grouped_layout``). Its m_indices and
row_entry may be cut to the rows that the caller's buffers have. ``ws``, a
contiguous tensor on the operands' device, is a workspace of the caller's own;
without it a call that needs one takes one for itself.
"""
from __future__ import annotations

import ctypes
import operator
import struct
from typing import Dict, Optional

import torch

_c_i32, _c_i64, _c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class Matrix(ctypes.Structure):
    _fields_ = [("p", _c_vp), ("ld", _c_i64), ("stride", _c_i64)]


class ExpertRows(ctypes.Structure):
    _fields_ = [("counts", _c_vp), ("padded_offsets", _c_vp), ("m_indices", _c_vp),
                ("row_entry", _c_vp), ("rows", _c_i64), ("num_experts", _c_i32),
                ("tile_m", _c_i32), ("top_k", _c_i32)]


class GatedFfnArgs(ctypes.Structure):
    _fields_ = [("dtype", _c_i32), ("activation", _c_i32), ("tokens", _c_i64),
                ("hidden", _c_i32), ("inter", _c_i32), ("rows", ExpertRows)] + \
        [(n, Matrix) for n in ("x", "w_gate", "w_up", "h", "pre", "dh", "dx", "dw_gate", "dw_up")]


class LinearArgs(ctypes.Structure):
    _fields_ = [("dtype", _c_i32), ("activation", _c_i32), ("tokens", _c_i64),
                ("in_", _c_i32), ("out", _c_i32), ("rows", ExpertRows)] + \
        [(n, Matrix) for n in ("x", "w", "bias", "residual", "y", "pre", "dy", "dx", "dw",
                               "dbias")]


class CombineArgs(ctypes.Structure):
    _fields_ = [("dtype", _c_i32), ("width", _c_i32), ("tokens", _c_i64), ("rows", _c_i64),
                ("top_k", _c_i32), ("num_experts", _c_i32), ("num_ids", _c_i32)] + \
        [(n, _c_vp) for n in ("packed", "inv_perm", "offsets", "padded_offsets", "m_indices",
                              "row_entry", "weights")] + \
        [(n, Matrix) for n in ("y", "residual", "out", "dout", "dy")] + [("dweights", _c_vp)]


EXPORTS = {
    "moe_gated_ffn_workspace_bytes": (_c_i64, [_c_vp, _c_i32]),
    "moe_gated_ffn": (ctypes.c_int, [_c_vp, _c_vp, ctypes.c_size_t, _c_vp]),
    "moe_gated_ffn_backward": (ctypes.c_int, [_c_vp, _c_vp, ctypes.c_size_t, _c_vp]),
    "moe_linear_workspace_bytes": (_c_i64, [_c_vp, _c_i32]),
    "moe_linear": (ctypes.c_int, [_c_vp, _c_vp, ctypes.c_size_t, _c_vp]),
    "moe_linear_backward": (ctypes.c_int, [_c_vp, _c_vp, ctypes.c_size_t, _c_vp]),
    "moe_combine": (ctypes.c_int, [_c_vp, _c_vp]),
    "moe_combine_backward": (ctypes.c_int, [_c_vp, _c_vp]),
}

DTYPES = {torch.bfloat16: 0, torch.float16: 1}
ACTIVATIONS = {"none": 0, None: 0, "silu": 1, "gelu": 2}

_pkg = None  # the package module, set by it on import


def _fail(msg: str):
    raise _pkg.MoeRouteError(msg)


# The structures above as bytes (native sizes and alignment): packing them is
# several times faster than filling ctypes fields, which small calls notice.
_MATRIX = "Pqq"
_PACK_GATED = struct.Struct("@iiqii" + "PPPPqiii0q" + 9 * _MATRIX).pack
_PACK_LINEAR = struct.Struct("@iiqii" + "PPPPqiii0q" + 10 * _MATRIX).pack
_PACK_COMBINE = struct.Struct("@iiqqiii0q" + 7 * "P" + 5 * _MATRIX + "P").pack
_NONE = (0, 0, 0)
_ERR_WORKSPACE = -5
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class _Entry:
    """A C entry on the current stream of a device. One that needs a workspace
    says so and gets one of this call alone, which a captured call keeps in its
    graph's memory."""

    def __init__(self, name: str, size: Optional[str] = None, backward: int = 0):
        self.name, self.size, self.backward, self.fn = name, size, backward, None

    def __call__(self, args: bytes, dev: torch.device, ws: Optional[torch.Tensor] = None) -> None:
        if self.fn is None:
            self.fn = getattr(_pkg.lib(), self.name)
        if dev.index != _current_device():
            with torch.cuda.device(dev):
                return self(args, dev, ws)
        stream = _pkg._stream_handle(dev)
        if self.size is None:
            st = self.fn(args, stream)
        elif ws is not None:
            if not isinstance(ws, torch.Tensor) or ws.device != dev or not ws.is_contiguous():
                _fail(f"ws must be a contiguous tensor on {dev}")
            st = self.fn(args, ws.data_ptr(), ws.numel() * ws.element_size(), stream)
        else:
            st = self.fn(args, None, 0, stream)
            if st == _ERR_WORKSPACE:
                need = getattr(_pkg.lib(), self.size)(args, self.backward)
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
                st = self.fn(args, ws.data_ptr(), need, stream)
        if st:
            _pkg._check(st, self.name)


_GATED = _Entry("moe_gated_ffn", "moe_gated_ffn_workspace_bytes")
_GATED_BACKWARD = _Entry("moe_gated_ffn_backward", "moe_gated_ffn_workspace_bytes", 1)
_LINEAR = _Entry("moe_linear", "moe_linear_workspace_bytes")
_LINEAR_BACKWARD = _Entry("moe_linear_backward", "moe_linear_workspace_bytes", 1)
_COMBINE = _Entry("moe_combine")
_COMBINE_BACKWARD = _Entry("moe_combine_backward")


def _mat(t: Optional[torch.Tensor], name: str, shape: tuple, like: torch.Tensor) -> tuple:
    """(pointer, ld, stride) of a matrix or a stack of them, checked."""
    if t is None:
        return _NONE
    if not isinstance(t, torch.Tensor) or t.dtype != like.dtype or t.device != like.device:
        _fail(f"{name} must be a {like.dtype} tensor on {like.device}")
    if t.shape != shape:
        _fail(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    st = t.stride()
    p = t.data_ptr()
    if p == 0 or 0 in shape:
        return (0, shape[-1], 0)
    if st[-1] != 1 and shape[-1] > 1:
        _fail(f"{name} must have contiguous columns")
    n = len(st)
    if n == 1:
        return (p, shape[0], 0)
    ld = st[-2] if shape[-2] > 1 else max(st[-2], shape[-1])
    if n == 2:
        return (p, ld, 0)
    return (p, ld, st[0] if shape[0] > 1 else ld * shape[1])


def _vec(t: Optional[torch.Tensor], name: str, shape: tuple, like: torch.Tensor) -> tuple:
    """(pointer, ld, stride) of a vector, or of one vector for each expert."""
    if t is None or len(shape) == 1:
        return _mat(t, name, shape, like)
    p, ld, _ = _mat(t, name, shape, like)
    return (p, shape[1], ld)


def _first(x, name: str, ndim: int = 2) -> int:
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        _fail(f"{name} must be a GPU tensor")
    d = DTYPES.get(x.dtype)
    if d is None:
        _fail(f"{name} must be bfloat16 or float16, not {x.dtype}")
    if x.dim() != ndim:
        _fail(f"{name} must have {ndim} dimensions")
    return d


def _activation(name) -> int:
    a = ACTIVATIONS.get(name)
    if a is None:
        _fail(f"activation must be one of 'none', 'silu', 'gelu', not {name!r}")
    return a


def _index(t, name: str, dev, least: int = 0) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != dev or \
            not t.is_contiguous():
        _fail(f"{name} must be a contiguous int32 tensor on {dev}")
    if t.numel() < least:
        _fail(f"{name} must have at least {least} elements")
    return t.data_ptr()


def _number(v, name: str) -> int:
    try:
        v = operator.index(v)
    except TypeError:
        _fail(f"{name} must be a whole number, not {v!r}")
    if not -1 << 31 <= v < 1 << 31:
        _fail(f"{name} must fit 32 bits")
    return v


def _of(lay, name: str):
    """A tensor of the layout."""
    t = lay.get(name)
    if t is None:
        _fail(f"the layout has no {name}")
    return t


def _out(out, name: str):
    """An output that a caller's dict may not leave out."""
    t = out.get(name)
    if t is None:
        _fail(f"out must have {name}")
    return t


def _lead(w, name: str, lay) -> torch.Size:
    """() or (experts,), the leading dimensions of a weight."""
    ndim = 2 if lay is None else 3
    if not isinstance(w, torch.Tensor) or w.dim() != ndim:
        _fail(f"{name} must be a tensor of {ndim} dimensions")
    return w.shape[:-2]


def _zeros(out: Dict[str, torch.Tensor], *names: str) -> Dict[str, torch.Tensor]:
    """The outputs of a call over no experts, checked like any other's."""
    for n in names:
        if out.get(n) is not None:
            out[n].zero_()
    return out


_DENSE = (0, 0, 0, 0, 0, 0, 0, 0)


def _rows(lay, n_experts: int, tile_m: int, top_k: int, dev, gather: bool) -> tuple:
    m = _of(lay, "m_indices")
    p = _index(m, "m_indices", dev)
    rows = m.numel()
    entry = lay.get("row_entry") if gather else None
    e = 0 if entry is None else _index(entry, "row_entry", dev)
    if entry is not None and entry.numel() != rows:
        _fail("row_entry must have as many elements as m_indices")
    return (_index(_of(lay, "counts"), "counts", dev, n_experts),
            _index(_of(lay, "padded_offsets"), "padded_offsets", dev, n_experts + 1),
            p, e, rows, n_experts, _number(tile_m, "tile_m"), _number(top_k, "top_k"))


def _gated(x, w_gate, w_up, activation, save_pre, out, ws, lay, tile_m, top_k):
    d = _first(x, "x")
    act = _activation(activation)
    tokens, hidden = x.shape
    lead = _lead(w_gate, "w_gate", lay)
    inter = w_gate.shape[-2]
    rows, desc = tokens, _DENSE
    if lay is not None:
        desc = _rows(lay, lead[0], tile_m, top_k, x.device, True)
        rows = desc[4]
    wshape = (*lead, inter, hidden)
    if out is None:
        out = {"h": torch.empty((rows, inter), dtype=x.dtype, device=x.device)}
    if save_pre and out.get("pre") is None:
        out["pre"] = torch.empty((rows, 2 * inter), dtype=x.dtype, device=x.device)
    pre = out.get("pre") if save_pre else None
    a = _PACK_GATED(d, act, tokens, hidden, inter, *desc, *_mat(x, "x", (tokens, hidden), x),
                    *_mat(w_gate, "w_gate", wshape, x), *_mat(w_up, "w_up", wshape, x),
                    *_mat(_out(out, "h"), "h", (rows, inter), x),
                    *_mat(pre, "pre", (rows, 2 * inter), x), *_NONE * 4)
    if lay is not None and lead[0] == 0:  # no experts here: every row is zero
        return _zeros(out, "h", "pre" if save_pre else "h")
    _GATED(a, x.device, ws)
    return out


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, *,
              activation: str = "silu", save_pre: bool = False,
              out: Optional[Dict[str, torch.Tensor]] = None,
              ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_gated_ffn, dense: h [T, F] = act(x Wg^T) * (x Wu^T) from x [T, H] and
    w_gate, w_up [F, H]; with save_pre also pre [T, 2F], the two projections,
    which gated_ffn_backward reads."""
    return _gated(x, w_gate, w_up, activation, save_pre, out, ws, None, 0, 0)


def expert_gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                     lay: Dict[str, torch.Tensor], *, tile_m: int, top_k: int,
                     activation: str = "silu", save_pre: bool = False,
                     out: Optional[Dict[str, torch.Tensor]] = None,
                     ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_gated_ffn over experts: h [rows, F] for the rows of a grouped
    layout, from token rows x [T, H] (gathered through row_entry; without it
    x has one row per row) and w_gate, w_up [E, F, H] of the ids 0 .. E-1. Rows
    without an entry of these experts are zero."""
    return _gated(x, w_gate, w_up, activation, save_pre, out, ws, lay, tile_m, top_k)


def _gated_backward(dh, pre, x, w_gate, w_up, activation, out, ws, lay, tile_m, top_k):
    d = _first(x, "x")
    act = _activation(activation)
    tokens, hidden = x.shape
    lead = _lead(w_gate, "w_gate", lay)
    inter = w_gate.shape[-2]
    rows, desc = tokens, _DENSE
    if lay is not None:
        desc = _rows(lay, lead[0], tile_m, top_k, x.device, True)
        rows = desc[4]
    wshape = (*lead, inter, hidden)
    if out is None:
        out = {"dx": torch.empty((rows, hidden), dtype=x.dtype, device=x.device),
               "dw_gate": torch.empty(wshape, dtype=x.dtype, device=x.device),
               "dw_up": torch.empty(wshape, dtype=x.dtype, device=x.device)}
    a = _PACK_GATED(d, act, tokens, hidden, inter, *desc, *_mat(x, "x", (tokens, hidden), x),
                    *_mat(w_gate, "w_gate", wshape, x), *_mat(w_up, "w_up", wshape, x), *_NONE,
                    *_mat(pre, "pre", (rows, 2 * inter), x), *_mat(dh, "dh", (rows, inter), x),
                    *_mat(out.get("dx"), "dx", (rows, hidden), x),
                    *_mat(out.get("dw_gate"), "dw_gate", wshape, x),
                    *_mat(out.get("dw_up"), "dw_up", wshape, x))
    if lay is not None and lead[0] == 0:
        return _zeros(out, "dx")
    _GATED_BACKWARD(a, x.device, ws)
    return out


def gated_ffn_backward(dh: torch.Tensor, pre: torch.Tensor, x: torch.Tensor,
                       w_gate: torch.Tensor, w_up: torch.Tensor, *, activation: str = "silu",
                       out: Optional[Dict[str, torch.Tensor]] = None,
                       ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_gated_ffn_backward, dense: dx [T, H], dw_gate and dw_up [F, H] from dh
    [T, F] and the forward pass's pre [T, 2F]. An `out` dict without dx, or
    without the two weight gradients, leaves them out."""
    return _gated_backward(dh, pre, x, w_gate, w_up, activation, out, ws, None, 0, 0)


def expert_gated_ffn_backward(dh: torch.Tensor, pre: torch.Tensor, x: torch.Tensor,
                              w_gate: torch.Tensor, w_up: torch.Tensor,
                              lay: Dict[str, torch.Tensor], *, tile_m: int, top_k: int,
                              activation: str = "silu",
                              out: Optional[Dict[str, torch.Tensor]] = None,
                              ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_gated_ffn_backward over experts: dx [rows, H] (one row per row;
    ``combine(dx, lay, num_experts=E, weighted=False)`` sums them into tokens),
    dw_gate and dw_up [E, F, H], zeros for an expert without rows."""
    return _gated_backward(dh, pre, x, w_gate, w_up, activation, out, ws, lay, tile_m, top_k)


def _linear(x, w, bias, activation, residual, save_pre, out, ws, lay, tile_m):
    d = _first(x, "x")
    act = _activation(activation)
    rows, n_in = x.shape
    lead = _lead(w, "w", lay)
    n_out = w.shape[-2]
    desc = _DENSE
    if lay is not None:
        desc = _rows(lay, lead[0], tile_m, 0, x.device, False)
        if desc[4] != rows:
            _fail("x must have as many rows as m_indices")
    if out is None:
        out = {"y": torch.empty((rows, n_out), dtype=x.dtype, device=x.device)}
    if save_pre and out.get("pre") is None:
        out["pre"] = torch.empty((rows, n_out), dtype=x.dtype, device=x.device)
    pre = out.get("pre") if save_pre else None
    a = _PACK_LINEAR(d, act, rows, n_in, n_out, *desc, *_mat(x, "x", (rows, n_in), x),
                     *_mat(w, "w", (*lead, n_out, n_in), x),
                     *_vec(bias, "bias", (*lead, n_out), x),
                     *_mat(residual, "residual", (rows, n_out), x),
                     *_mat(_out(out, "y"), "y", (rows, n_out), x),
                     *_mat(pre, "pre", (rows, n_out), x), *_NONE * 4)
    if lay is not None and lead[0] == 0:
        return _zeros(out, "y", "pre" if save_pre else "y")
    _LINEAR(a, x.device, ws)
    return out


def linear(x: torch.Tensor, w: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
           activation: Optional[str] = None, residual: Optional[torch.Tensor] = None,
           save_pre: bool = False, out: Optional[Dict[str, torch.Tensor]] = None,
           ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_linear, dense: y [T, O] = act(x W^T + bias) + residual from x [T, I]
    and w [O, I]; with save_pre also pre [T, O] = x W^T + bias, which
    linear_backward reads when there is an activation."""
    return _linear(x, w, bias, activation, residual, save_pre, out, ws, None, 0)


def expert_linear(x: torch.Tensor, w: torch.Tensor, lay: Dict[str, torch.Tensor], *, tile_m: int,
                  bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                  residual: Optional[torch.Tensor] = None, save_pre: bool = False,
                  out: Optional[Dict[str, torch.Tensor]] = None,
                  ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_linear over experts: y [rows, O] from x [rows, I], w [E, O, I] and
    bias [E, O]. Rows without an entry of these experts are zero."""
    return _linear(x, w, bias, activation, residual, save_pre, out, ws, lay, tile_m)


def _linear_backward(dy, x, w, pre, activation, bias_grad, out, ws, lay, tile_m):
    d = _first(x, "x")
    act = _activation(activation)
    rows, n_in = x.shape
    lead = _lead(w, "w", lay)
    n_out = w.shape[-2]
    if act and pre is None:
        _fail("pre is needed where there is an activation")
    desc = _DENSE
    if lay is not None:
        desc = _rows(lay, lead[0], tile_m, 0, x.device, False)
        if desc[4] != rows:
            _fail("x must have as many rows as m_indices")
    wshape = (*lead, n_out, n_in)
    if out is None:
        out = {"dx": torch.empty((rows, n_in), dtype=x.dtype, device=x.device),
               "dw": torch.empty(wshape, dtype=x.dtype, device=x.device)}
        if bias_grad:
            out["dbias"] = torch.empty((*lead, n_out), dtype=x.dtype, device=x.device)
    a = _PACK_LINEAR(d, act, rows, n_in, n_out, *desc, *_mat(x, "x", (rows, n_in), x),
                     *_mat(w, "w", wshape, x), *_NONE * 3,
                     *(_mat(pre, "pre", (rows, n_out), x) if act else _NONE),
                     *_mat(dy, "dy", (rows, n_out), x),
                     *_mat(out.get("dx"), "dx", (rows, n_in), x),
                     *_mat(out.get("dw"), "dw", wshape, x),
                     *_vec(out.get("dbias"), "dbias", (*lead, n_out), x))
    if lay is not None and lead[0] == 0:
        return _zeros(out, "dx")
    _LINEAR_BACKWARD(a, x.device, ws)
    return out


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, *,
                    pre: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                    bias_grad: bool = False, out: Optional[Dict[str, torch.Tensor]] = None,
                    ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_linear_backward, dense: dx [T, I], dw [O, I] and (bias_grad) dbias [O]
    from dy [T, O]; pre [T, O] where there is an activation. An `out` dict
    without one of them leaves it out. The residual's gradient is dy."""
    return _linear_backward(dy, x, w, pre, activation, bias_grad, out, ws, None, 0)


def expert_linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                           lay: Dict[str, torch.Tensor], *, tile_m: int,
                           pre: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                           bias_grad: bool = False,
                           out: Optional[Dict[str, torch.Tensor]] = None,
                           ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_linear_backward over experts: dx [rows, I], dw [E, O, I] and
    (bias_grad) dbias [E, O], zeros for an expert without rows."""
    return _linear_backward(dy, x, w, pre, activation, bias_grad, out, ws, lay, tile_m)


def _tokens(lay) -> torch.Size:
    """(tokens, entries a token) of the layout."""
    packed = _of(lay, "packed")
    if not isinstance(packed, torch.Tensor) or packed.dim() != 2:
        _fail("packed must be a tensor of 2 dimensions")
    return packed.shape


def _combine_args(y_rows, width, d, lay, num_experts, weighted, like, backward, mats, dweights):
    dev = like.device
    tokens, top_k = _tokens(lay)
    packed = lay["packed"]
    w = _of(lay, "topk_weights") if weighted else None
    if w is not None and (not isinstance(w, torch.Tensor) or w.dtype != torch.float32 or
                          w.shape != packed.shape or w.device != dev or not w.is_contiguous()):
        _fail(f"topk_weights must be a contiguous float32 tensor like packed on {dev}")
    n = tokens * top_k
    offsets = _of(lay, "offsets")
    o = _index(offsets, "offsets", dev, 1)
    num_ids = offsets.numel() - 1
    num_experts = _number(num_experts, "num_experts")
    if not 0 <= num_experts <= num_ids:
        _fail(f"num_experts must be between 0 and the {num_ids} ids of the layout")
    rows = (0, 0)
    if backward:
        rows = [_index(_of(lay, k), k, dev, y_rows) for k in ("m_indices", "row_entry")]
    return _PACK_COMBINE(d, width, tokens, y_rows, top_k, num_experts, num_ids,
                         _index(packed, "packed", dev),
                         _index(_of(lay, "inv_perm"), "inv_perm", dev, n), o,
                         _index(_of(lay, "padded_offsets"), "padded_offsets", dev, num_ids + 1),
                         *rows, 0 if w is None else w.data_ptr(), *mats, dweights)


def combine(y: torch.Tensor, lay: Dict[str, torch.Tensor], *, num_experts: int,
            weighted: bool = True, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_combine: out [T, W] = residual + the sum over k of topk_weights[t, k]
    (1 without `weighted`) times the row of y [rows, W] of entry (t, k), for
    the entries of the experts 0 .. num_experts-1."""
    d = _first(y, "y")
    rows, width = y.shape
    tokens, _ = _tokens(lay)
    if out is None:
        out = torch.empty((tokens, width), dtype=y.dtype, device=y.device)
    a = _combine_args(rows, width, d, lay, num_experts, weighted, y, False,
                      (*_mat(y, "y", (rows, width), y),
                       *_mat(residual, "residual", (tokens, width), y),
                       *_mat(out, "out", (tokens, width), y), *_NONE * 2), 0)
    _COMBINE(a, y.device)
    return out


def combine_backward(dout: torch.Tensor, y: Optional[torch.Tensor],
                     lay: Dict[str, torch.Tensor], *, num_experts: int, weighted: bool = True,
                     out: Optional[Dict[str, torch.Tensor]] = None) -> Dict[str, torch.Tensor]:
    """moe_combine_backward: dy [rows, W] and dweights [T, K] (fp32) from dout
    [T, W] and the forward pass's y. Without `weighted`, or with an `out` dict
    without dweights, only dy is computed and y is not read (it may be None:
    the rows are then those of m_indices). The residual's gradient is dout."""
    d = _first(dout, "dout")
    tokens, width = dout.shape
    entries = _tokens(lay)
    if y is None:
        _index(_of(lay, "m_indices"), "m_indices", dout.device)
    elif not isinstance(y, torch.Tensor) or y.dim() != 2:
        _fail("y must be a tensor of 2 dimensions")
    rows = lay["m_indices"].numel() if y is None else y.shape[0]
    if out is None:
        out = {"dy": torch.empty((rows, width), dtype=dout.dtype, device=dout.device)}
        if weighted:
            out["dweights"] = torch.empty(entries, dtype=torch.float32,
                                          device=dout.device)
    dw = out.get("dweights")
    if dw is not None:
        if y is None:
            _fail("y is needed for dweights")
        if dw.dtype != torch.float32 or dw.shape != entries or \
                not dw.is_contiguous() or dw.device != dout.device:
            _fail("dweights must be a contiguous float32 tensor like packed")
    if entries[0] != tokens:
        _fail("dout must have one row for each token of the layout")
    a = _combine_args(rows, width, d, lay, num_experts, weighted, dout, True,
                      (*_mat(y, "y", (rows, width), dout), *_NONE * 2,
                       *_mat(dout, "dout", (tokens, width), dout),
                       *_mat(_out(out, "dy"), "dy", (rows, width), dout)),
                      0 if dw is None else dw.data_ptr())
    _COMBINE_BACKWARD(a, dout.device)
    return out
