"""Host-side checks of the norm and dropout, with no GPU: what the C entries
refuse before anything is launched, and that the binding matches the header."""
import ctypes
import os
import re

import pytest

import moe_expert_routing_amd as M
from moe_expert_routing_amd import block
from moe_expert_routing_amd.ffn import Matrix

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUP, WS = 0, -1, -2, -4, -5
P = 0x10000  # never dereferenced: every call below is refused, or has no tokens


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("library not built")
    return M.lib()


def test_header_and_binding_agree(L):
    text = open(os.path.join(ROOT, "include", "moe_block.h")).read()
    names = set(re.findall(r"\b(moe_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == set(block.EXPORTS)
    for n in names:
        assert hasattr(L, n)


def flat(v):
    if isinstance(v, ctypes.Structure):
        return [x for name, _ in v._fields_ for x in flat(getattr(v, name))]
    return [v or 0]


def test_packed_arguments_have_the_structures_layout():
    for pack, cls, n in ((block._PACK_NORM, block.RmsNormArgs, 8 + 12 + 4 + 12 + 1),
                         (block._PACK_DROPOUT, block.DropoutArgs, 6 + 9)):
        raw = pack(*range(1, n + 1))
        assert len(raw) == ctypes.sizeof(cls)
        assert flat(cls.from_buffer_copy(raw)) == list(range(1, n + 1))


def mat(p=P, ld=64, stride=0):
    return Matrix(p, ld, stride)


def drop(state=P, level=6554, site=0):
    return block.DropoutSpec(state, level, site)


def norm(**kw):
    d = dict(dtype=0, width=64, tokens=8, eps=1e-6, drop=drop(), x=mat(), residual=mat(), h=mat(), y=mat(), weight=P, rstd=P,
             q=P, q_scale=P, dy=mat(), dh=mat(), dx=mat(), dresidual=mat(), dweight=P)
    d.update(kw)
    return block.RmsNormArgs(**d)


BAD_BOTH = [
    (dict(dtype=2), UNSUP), (dict(dtype=-1), UNSUP), (dict(width=0), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(reserved=1), SHAPE), (dict(width=32769), UNSUP), (dict(tokens=(1 << 30) + 1), UNSUP), (dict(weight=None), NULL),
    (dict(weight=P + 1), SHAPE), (dict(rstd=P + 2), SHAPE), (dict(drop=drop(None)), NULL), (dict(drop=drop(P + 4)), SHAPE),
    (dict(drop=drop(level=65537)), SHAPE), (dict(drop=drop(site=-1)), SHAPE), (dict(drop=drop(site=32768)), UNSUP),
    (dict(h=mat(None)), NULL), (dict(h=mat(ld=63)), SHAPE), (dict(h=mat(P + 1)), SHAPE), (dict(h=mat(ld=(1 << 22) + 1)), UNSUP)]
BAD_FORWARD = BAD_BOTH + [
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(x=mat(None)), NULL),
    (dict(y=mat(None), q=None, q_scale=None), NULL), (dict(q=None), NULL), (dict(q_scale=None), NULL), (dict(width=48), SHAPE),
    (dict(residual=mat(ld=63)), SHAPE), (dict(residual=mat(None), h=mat(None)), NULL), (dict(drop=drop(level=0), h=mat(None)), NULL)]
BAD_BACKWARD = BAD_BOTH + [
    (dict(dy=mat(None)), NULL), (dict(rstd=None), NULL), (dict(dweight=P + 1), SHAPE), (dict(dx=mat(ld=10)), SHAPE),
    (dict(dh=mat(P + 1)), SHAPE), (dict(dresidual=mat(ld=-1)), SHAPE)]


@pytest.mark.parametrize("kw,want", BAD_FORWARD)
def test_norm_refuses(L, kw, want):
    assert L.moe_rms_norm(ctypes.byref(norm(**kw)), None) == want


@pytest.mark.parametrize("kw,want", BAD_BACKWARD)
def test_norm_backward_refuses(L, kw, want):
    a = norm(**kw)
    assert L.moe_rms_norm_backward(ctypes.byref(a), P, 1 << 40, None) == want
    assert L.moe_rms_norm_backward_workspace_bytes(ctypes.byref(a), 1) == -1


def test_norm_calls_without_arguments_or_tokens(L):
    assert L.moe_rms_norm(None, None) == NULL
    assert L.moe_rms_norm_backward(None, None, 0, None) == NULL
    assert L.moe_rms_norm_backward_workspace_bytes(None, 1) == -1
    none = Matrix(None, 0, 0)
    empty = norm(tokens=0, x=none, residual=none, h=none, y=none, q=None, q_scale=None, rstd=None, dy=none, dh=none, dx=none,
                 dresidual=none, dweight=None)
    assert L.moe_rms_norm(ctypes.byref(empty), None) == OK
    assert L.moe_rms_norm_backward(ctypes.byref(empty), None, 0, None) == OK


def test_norm_workspace(L):
    a = norm()
    need = L.moe_rms_norm_backward_workspace_bytes(ctypes.byref(a), 1)
    assert need >= 64 * 4
    for ws, n in ((None, need), (P, need - 1), (P + 8, need)):
        assert L.moe_rms_norm_backward(ctypes.byref(a), ws, n, None) == WS
    assert L.moe_rms_norm_backward_workspace_bytes(ctypes.byref(norm(dweight=None)), 1) == 0
    assert L.moe_rms_norm_backward_workspace_bytes(ctypes.byref(a), 0) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=7), UNSUP), (dict(width=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(width=(1 << 20) + 1), UNSUP), (dict(tokens=1 << 31), UNSUP),
    (dict(drop=drop(None)), NULL), (dict(drop=drop(level=70000)), SHAPE), (dict(x=mat(None)), NULL), (dict(out=mat(None)), NULL),
    (dict(residual=mat(ld=3)), SHAPE), (dict(out=mat(P + 1)), SHAPE)])
def test_dropout_refuses(L, kw, want):
    d = dict(dtype=0, width=64, tokens=8, drop=drop(), x=mat(), residual=mat(), out=mat())
    d.update(kw)
    assert L.moe_dropout(ctypes.byref(block.DropoutArgs(**d)), None) == want


def test_dropout_without_arguments_or_tokens(L):
    assert L.moe_dropout(None, None) == NULL
    none = Matrix(None, 0, 0)
    a = block.DropoutArgs(dtype=1, width=5, tokens=0, drop=drop(), x=none, residual=none, out=none)
    assert L.moe_dropout(ctypes.byref(a), None) == OK


@pytest.mark.parametrize("args,want", [
    ((P, P, 64, 3, P), UNSUP), ((P, P, -32, 0, P), SHAPE), ((P, P, 33, 0, P), SHAPE), ((None, P, 32, 0, P), NULL),
    ((P, None, 32, 0, P), NULL), ((P, P, 32, 0, None), NULL), ((P, P, 32, 0, P + 1), SHAPE), ((P, P, 1 << 55, 0, P), UNSUP),
    ((None, None, 0, 0, None), OK)])
def test_mxfp8_values_refuses(L, args, want):
    assert L.moe_mxfp8_values(*args, None) == want
