"""Host-side checks of the feed-forward operators, with no GPU: what the C
entries refuse before anything is launched, the workspace sizes, and that the
binding's structures match the header's."""
import ctypes
import os
import re

import pytest
import torch

import moe_expert_routing_amd as M
from moe_expert_routing_amd import ffn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUP, WS = 0, -1, -2, -4, -5
P = 0x10000  # never dereferenced: every call below is refused, or has no rows


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("library not built")
    return M.lib()


def test_header_and_binding_agree(L):
    text = open(os.path.join(ROOT, "include", "moe_ffn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(moe_\w+)\s*\(", text))
    assert names == set(ffn.EXPORTS)
    for n in names:
        assert hasattr(L, n)


def test_packed_arguments_have_the_structures_layout():
    """The binding packs bytes; every field has to land where the structure has it."""
    def numbers(n):
        return list(range(1, n + 1))

    def flat(v):
        if isinstance(v, ctypes.Structure):
            return [x for name, _ in v._fields_ for x in flat(getattr(v, name))]
        return [v or 0]
    for pack, cls, n in ((ffn._PACK_GATED, ffn.GatedFfnArgs, 13 + 27),
                         (ffn._PACK_LINEAR, ffn.LinearArgs, 13 + 30),
                         (ffn._PACK_COMBINE, ffn.CombineArgs, 7 + 7 + 15 + 1)):
        raw = pack(*numbers(n))
        assert len(raw) == ctypes.sizeof(cls)
        assert flat(cls.from_buffer_copy(raw)) == numbers(n)


def rows(**kw):
    d = dict(counts=P, padded_offsets=P, m_indices=P, row_entry=P, rows=64, num_experts=4,
             tile_m=16, top_k=2)
    d.update(kw)
    return ffn.ExpertRows(**d)


def mat(p=P, ld=64, stride=0):
    return ffn.Matrix(p, ld, stride)


def gated(experts=False, **kw):
    d = dict(dtype=0, activation=1, tokens=8, hidden=64, inter=64, x=mat(),
             w_gate=mat(stride=64 * 64), w_up=mat(stride=64 * 64), h=mat(), pre=mat(ld=128),
             dh=mat(), dx=mat(), dw_gate=mat(stride=64 * 64), dw_up=mat(stride=64 * 64))
    if experts:
        d["rows"] = rows()
    d.update(kw)
    return ffn.GatedFfnArgs(**d)


BAD_GATED = [
    (dict(dtype=2), UNSUP), (dict(activation=3), UNSUP), (dict(activation=-1), UNSUP),
    (dict(tokens=-1), SHAPE), (dict(hidden=0), SHAPE), (dict(inter=-3), SHAPE),
    (dict(hidden=(1 << 20) + 1), UNSUP), (dict(tokens=1 << 31), UNSUP),
    (dict(x=mat(None)), NULL), (dict(w_up=mat(None)), NULL), (dict(x=mat(P + 1)), SHAPE),
    (dict(x=mat(ld=63)), SHAPE), (dict(x=mat(ld=(1 << 22) + 1)), UNSUP), (dict(x=mat(ld=-64)), SHAPE),
    (dict(rows=rows(num_experts=-1)), SHAPE), (dict(rows=rows(num_experts=5000)), UNSUP),
    (dict(rows=rows(tile_m=0)), SHAPE), (dict(rows=rows(tile_m=24)), UNSUP),
    (dict(rows=rows(tile_m=8192)), SHAPE), (dict(rows=rows(m_indices=None)), NULL),
    (dict(rows=rows(rows=-1)), SHAPE), (dict(rows=rows(top_k=0)), SHAPE),
    (dict(rows=rows(), w_gate=mat(stride=64)), SHAPE),
    (dict(rows=rows(row_entry=None)), SHAPE),  # 64 rows, but x has 8
]


@pytest.mark.parametrize("kw,want", BAD_GATED)
def test_gated_refuses(L, kw, want):
    a = gated(**kw)
    assert L.moe_gated_ffn(ctypes.byref(a), P, 1 << 40, None) == want
    assert L.moe_gated_ffn_backward(ctypes.byref(a), P, 1 << 40, None) == want
    assert L.moe_gated_ffn_workspace_bytes(ctypes.byref(a), 0) == -1


def test_gated_refuses_more(L):
    def fwd(**kw):
        return L.moe_gated_ffn(ctypes.byref(gated(**kw)), None, 0, None)

    def bwd(ws=P, n=1 << 40, **kw):
        return L.moe_gated_ffn_backward(ctypes.byref(gated(**kw)), ws, n, None)
    assert L.moe_gated_ffn(None, None, 0, None) == NULL
    assert fwd(h=mat(None)) == NULL
    assert fwd(h=mat(ld=8)) == SHAPE
    assert fwd(pre=mat(ld=64)) == SHAPE  # two projections wide
    assert bwd(pre=mat(None)) == NULL
    assert bwd(dh=mat(None)) == NULL
    assert bwd(dw_up=mat(None)) == NULL  # the two weight gradients go together
    assert bwd(rows=rows(counts=None)) == NULL
    assert bwd(rows=rows(padded_offsets=None)) == NULL
    assert bwd(None, 0) == WS and bwd(P, 16) == WS and bwd(P + 8) == WS
    # misaligned operands need their copies' workspace
    assert fwd(x=mat(P + 2)) == WS
    assert fwd(hidden=63, x=mat(ld=63), w_gate=mat(ld=63), w_up=mat(ld=63)) == WS


def test_gated_workspace(L):
    size = L.moe_gated_ffn_workspace_bytes
    assert size(ctypes.byref(gated()), 0) == 0
    assert size(ctypes.byref(gated()), 1) == 8 * 128 * 2  # dz
    assert size(ctypes.byref(gated(x=mat(P + 2))), 0) == 8 * 64 * 2
    odd = gated(hidden=63, x=mat(ld=63), w_gate=mat(ld=63), w_up=mat(ld=63))
    assert size(ctypes.byref(odd), 0) == 8 * 64 * 2 + 2 * 64 * 64 * 2


def linear(**kw):
    d = dict(dtype=1, activation=2, tokens=8, in_=64, out=64, x=mat(), w=mat(stride=64 * 64),
             bias=mat(), residual=mat(), y=mat(), pre=mat(), dy=mat(), dx=mat(),
             dw=mat(stride=64 * 64), dbias=mat())
    d.update(kw)
    return ffn.LinearArgs(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=-1), UNSUP), (dict(tokens=-2), SHAPE), (dict(in_=0), SHAPE), (dict(out=0), SHAPE),
    (dict(x=mat(None)), NULL), (dict(w=mat(None)), NULL), (dict(x=mat(ld=32)), SHAPE),
    (dict(pre=mat(ld=3)), SHAPE), (dict(rows=rows(m_indices=None)), NULL),
    (dict(rows=rows(), w=mat(stride=1)), SHAPE),
])
def test_linear_refuses(L, kw, want):
    a = linear(**kw)
    assert L.moe_linear(ctypes.byref(a), P, 1 << 40, None) == want
    assert L.moe_linear_backward(ctypes.byref(a), P, 1 << 40, None) == want
    assert L.moe_linear_workspace_bytes(ctypes.byref(a), 1) == -1


def test_linear_refuses_more(L):
    def fwd(**kw):
        return L.moe_linear(ctypes.byref(linear(**kw)), P, 1 << 40, None)

    def bwd(ws=P, n=1 << 40, **kw):
        return L.moe_linear_backward(ctypes.byref(linear(**kw)), ws, n, None)
    assert fwd(y=mat(None)) == NULL
    assert fwd(residual=mat(ld=8)) == SHAPE
    assert fwd(rows=rows(), bias=mat(stride=8)) == SHAPE
    assert bwd(dy=mat(None)) == NULL
    assert bwd(pre=mat(None)) == NULL
    assert bwd(None, 0) == WS
    size = L.moe_linear_workspace_bytes
    assert size(ctypes.byref(linear()), 0) == 0
    # the bias gradient's partial sums and dz
    assert size(ctypes.byref(linear()), 1) == 64 * 4 + 8 * 64 * 2
    assert size(ctypes.byref(linear(activation=0, dbias=mat(None))), 1) == 0


def combine(**kw):
    d = dict(dtype=0, width=64, tokens=8, rows=64, top_k=2, num_experts=4, num_ids=8, packed=P,
             inv_perm=P, offsets=P, padded_offsets=P, m_indices=P, row_entry=P, weights=P, y=mat(),
             residual=mat(), out=mat(), dout=mat(), dy=mat(), dweights=P)
    d.update(kw)
    return ffn.CombineArgs(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=9), UNSUP), (dict(width=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(rows=-1), SHAPE),
    (dict(top_k=0), SHAPE), (dict(top_k=65), UNSUP), (dict(num_experts=9), SHAPE),
    (dict(packed=None), NULL), (dict(offsets=None), NULL), (dict(y=mat(None)), NULL),
    (dict(y=mat(ld=32)), SHAPE), (dict(tokens=1 << 30, top_k=4), UNSUP),
])
def test_combine_refuses(L, kw, want):
    a = combine(**kw)
    assert L.moe_combine(ctypes.byref(a), None) == want
    assert L.moe_combine_backward(ctypes.byref(a), None) == want


def test_combine_refuses_more(L):
    def fwd(**kw):
        return L.moe_combine(ctypes.byref(combine(**kw)), None)

    def bwd(**kw):
        return L.moe_combine_backward(ctypes.byref(combine(**kw)), None)
    assert fwd(out=mat(None)) == NULL and fwd(residual=mat(ld=8)) == SHAPE
    assert bwd(dout=mat(None)) == NULL and bwd(dy=mat(None)) == NULL
    assert bwd(m_indices=None) == NULL and bwd(row_entry=None) == NULL
    assert fwd(tokens=0, rows=0, out=mat(None), y=mat(None)) == OK  # nothing to do


def test_binding_refuses_host_tensors(L):
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16)
    with pytest.raises(M.MoeRouteError, match="GPU tensor"):
        M.gated_ffn(x, w, w)
    with pytest.raises(M.MoeRouteError, match="GPU tensor"):
        M.linear(x, w)
    with pytest.raises(M.MoeRouteError, match="GPU tensor"):
        M.combine(x, {}, num_experts=1)
