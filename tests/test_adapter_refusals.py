"""Host-side checks of the product with adapters, with no GPU: what the C entries
refuse before anything is launched, the workspace, and that the binding matches
the header."""
import ctypes
import os
import re

import pytest

import moe_expert_routing_amd as M
from moe_expert_routing_amd import adapters
from moe_expert_routing_amd.ffn import Matrix

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUP, WS = 0, -1, -2, -4, -5
P = 0x10000  # never dereferenced: every call below is refused, or has no tokens and no gradients


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("library not built")
    return M.lib()


def test_header_and_binding_agree(L):
    text = open(os.path.join(ROOT, "include", "moe_adapter.h")).read()
    names = set(re.findall(r"\b(moe_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(adapters.EXPORTS)
    for n in names:
        assert hasattr(L, n)


def flat(v):
    if isinstance(v, ctypes.Structure):
        return [x for name, _ in v._fields_ for x in flat(getattr(v, name))]
    return [v or 0]


def test_packed_arguments_have_the_structures_layout():
    n = 7 + 21 + 3 + 12
    raw = adapters._PACK(*range(1, n + 1))
    assert len(raw) == ctypes.sizeof(adapters.AdapterLinearArgs)
    assert flat(adapters.AdapterLinearArgs.from_buffer_copy(raw)) == list(range(1, n + 1))


def mat(p=P, ld=64, stride=0):
    return Matrix(p, ld, stride)


def call(**kw):
    d = dict(dtype=0, rank=16, tokens=8, in_=64, out=64, adapters=3, x=mat(), w=mat(), a=mat(stride=64 * 16),
             b=mat(ld=16, stride=64 * 16), bias=mat(), residual=mat(), y=mat(), ids=P, scale=P, s=P, dy=mat(), dx=mat(),
             da=mat(stride=64 * 16), db=mat(ld=16, stride=64 * 16))
    d.update(kw)
    return adapters.AdapterLinearArgs(**d)


BAD_BOTH = [
    (dict(dtype=2), UNSUP), (dict(tokens=-1), SHAPE), (dict(in_=0), SHAPE), (dict(out=-5), SHAPE), (dict(rank=0), SHAPE), (dict(adapters=0), SHAPE),
    (dict(reserved=3), SHAPE), (dict(rank=129), UNSUP), (dict(adapters=4097), UNSUP), (dict(in_=(1 << 20) + 1), UNSUP),
    (dict(out=(1 << 20) + 1), UNSUP), (dict(tokens=(1 << 30) + 1), UNSUP), (dict(x=mat(None)), NULL), (dict(w=mat(None)), NULL),
    (dict(a=mat(None)), NULL), (dict(b=mat(None)), NULL), (dict(ids=None), NULL), (dict(ids=P + 1), SHAPE), (dict(scale=P + 2), SHAPE),
    (dict(s=P + 2), SHAPE), (dict(a=mat(stride=64 * 15)), SHAPE), (dict(b=mat(ld=15, stride=64 * 16)), SHAPE),
    (dict(b=mat(ld=16, stride=64 * 16 - 1)), SHAPE), (dict(x=mat(P + 1)), SHAPE), (dict(w=mat(ld=63)), SHAPE),
    (dict(x=mat(ld=(1 << 22) + 1)), UNSUP)]


@pytest.mark.parametrize("kw,want", BAD_BOTH + [(dict(y=mat(None)), NULL), (dict(residual=mat(ld=1)), SHAPE), (dict(bias=mat(P + 1)), SHAPE)])
def test_forward_refuses(L, kw, want):
    a = call(**kw)
    assert L.moe_adapter_linear(ctypes.byref(a), P, 1 << 50, None) == want
    assert L.moe_adapter_linear_workspace_bytes(ctypes.byref(a), 0) == -1


@pytest.mark.parametrize("kw,want", BAD_BOTH + [(dict(dy=mat(None)), NULL), (dict(s=None), NULL), (dict(dx=mat(ld=1)), SHAPE),
                                               (dict(da=mat(stride=5)), SHAPE), (dict(db=mat(ld=16, stride=5)), SHAPE)])
def test_backward_refuses(L, kw, want):
    a = call(**kw)
    assert L.moe_adapter_linear_backward(ctypes.byref(a), P, 1 << 50, None) == want
    assert L.moe_adapter_linear_workspace_bytes(ctypes.byref(a), 1) == -1


def test_workspace(L):
    a = call(s=None)
    need = L.moe_adapter_linear_workspace_bytes(ctypes.byref(a), 0)
    assert need >= 8 * 16 * 4
    # many tokens need memory for s alone, which may be the caller's
    assert L.moe_adapter_linear_workspace_bytes(ctypes.byref(call(tokens=100, s=None)), 0) >= 100 * 16 * 4
    assert L.moe_adapter_linear_workspace_bytes(ctypes.byref(call(tokens=100)), 0) == 0
    for ws, n in ((None, need), (P, need - 1), (P + 8, need)):
        assert L.moe_adapter_linear(ctypes.byref(a), ws, n, None) == WS
    back = L.moe_adapter_linear_workspace_bytes(ctypes.byref(call()), 1)
    assert back > 8 * 16 * 4
    assert L.moe_adapter_linear_backward(ctypes.byref(call()), P, back - 1, None) == WS


def test_calls_without_arguments_or_work(L):
    for f in (L.moe_adapter_linear, L.moe_adapter_linear_backward):
        assert f(None, None, 0, None) == NULL
    none = Matrix(None, 0, 0)
    empty = call(tokens=0, x=none, y=none, residual=none, ids=None, s=None, dy=none, dx=none, da=none, db=none)
    assert L.moe_adapter_linear(ctypes.byref(empty), None, 0, None) == OK
    assert L.moe_adapter_linear_backward(ctypes.byref(empty), None, 0, None) == OK
    nothing = call(dx=none, da=none, db=none)
    assert L.moe_adapter_linear_backward(ctypes.byref(nothing), None, 0, None) == OK
