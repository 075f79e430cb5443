"""The binding of the feed-forward operators on its own, with no GPU: what it
hands to the library, seen through an entry that records its calls."""
import pytest
import torch

import moe_expert_routing_amd as M
from moe_expert_routing_amd import ffn

DEV = torch.device("cuda", 0)


@pytest.fixture
def entry(monkeypatch):
    """An entry with a workspace, whose calls are recorded instead of made."""
    monkeypatch.setattr(ffn, "_current_device", lambda: 0)
    monkeypatch.setattr(M, "_stream_handle", lambda dev: 0)
    e = ffn._Entry("moe_linear", "moe_linear_workspace_bytes")
    e.calls = []
    e.fn = lambda *a: e.calls.append(a) or 0
    return e


@pytest.mark.parametrize("ws", [
    torch.empty(1 << 12, dtype=torch.uint8),                    # host memory
    torch.empty(1 << 12, dtype=torch.uint8, device="meta"),     # no memory at all
    bytearray(1 << 12),
], ids=["host", "meta", "bytes"])
def test_workspace_has_to_be_on_the_device(entry, ws):
    with pytest.raises(M.MoeRouteError, match="ws must be"):
        entry(b"", DEV, ws)
    assert not entry.calls


class GpuTensor(torch.Tensor):
    """Host memory that passes for the GPU's."""
    device = DEV


def test_workspace_has_to_be_contiguous(entry):
    """The bytes behind a strided or expanded tensor are not its elements'."""
    t = torch.empty(1 << 12, dtype=torch.uint8)
    for bad in (t[::2].as_subclass(GpuTensor), t[:1].expand(1 << 20).as_subclass(GpuTensor)):
        with pytest.raises(M.MoeRouteError, match="ws must be"):
            entry(b"", DEV, bad)
    assert not entry.calls


def test_workspace_is_counted_in_bytes(entry):
    for t in (torch.empty(1 << 12, dtype=torch.uint8), torch.empty(1 << 10, dtype=torch.float32)):
        entry(b"args", DEV, t.as_subclass(GpuTensor))
        assert entry.calls.pop() == (b"args", t.data_ptr(), 1 << 12, 0)


class AnyGpuTensor(GpuTensor):
    is_cuda = True

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        return torch._C._disabled_torch_function_impl(func, types, args, kwargs or {})


def gpu(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt).as_subclass(AnyGpuTensor)


def layout(n, rows=32, tokens=4, k=2):
    i = torch.int32
    return dict(counts=gpu(n, dt=i), padded_offsets=gpu(n + 1, dt=i), m_indices=gpu(rows, dt=i),
                row_entry=gpu(rows, dt=i), packed=gpu(tokens, k, dt=i), offsets=gpu(n + 1, dt=i),
                inv_perm=gpu(tokens, k, dt=i), topk_weights=gpu(tokens, k, dt=torch.float32))


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, recorded instead of made."""
    made = []
    monkeypatch.setattr(ffn, "_current_device", lambda: 0)
    monkeypatch.setattr(M, "_stream_handle", lambda dev: 0)
    for e in (ffn._GATED, ffn._GATED_BACKWARD, ffn._LINEAR, ffn._LINEAR_BACKWARD, ffn._COMBINE,
              ffn._COMBINE_BACKWARD):
        monkeypatch.setattr(e, "fn", lambda *a: made.append(a) or 0)
    return made


H, F, R = 16, 8, 32


def some_calls(n=3):
    """(what, call of everything but what is wrong in it) of each operator."""
    lay, kw = layout(n), dict(tile_m=16, top_k=2)
    x, w, xr, h, y = gpu(4, H), gpu(n, F, H), gpu(R, H), gpu(R, F), gpu(R, H)
    return dict(
        gated=lambda lay=lay, w=w, out={"h": h}, **k: M.expert_gated_ffn(
            x, w, w, lay, out=out, **{**kw, **k}),
        gated_backward=lambda lay=lay, w=w, out={"dx": xr}, **k: M.expert_gated_ffn_backward(
            h, gpu(R, 2 * F), x, w, w, lay, out=out, **{**kw, **k}),
        linear=lambda lay=lay, w=w, out={"y": h}, **k: M.expert_linear(
            xr, w, lay, out=out, **{"tile_m": 16, **k}),
        linear_backward=lambda lay=lay, w=w, out={"dx": xr}, **k: M.expert_linear_backward(
            h, xr, w, lay, out=out, **{"tile_m": 16, **k}),
        combine=lambda lay=lay, out=gpu(4, H), **k: M.combine(
            y, lay, out=out, **{"num_experts": n, **k}),
        combine_backward=lambda lay=lay, out={"dy": y}, **k: M.combine_backward(
            gpu(4, H), y, lay, out=out, **{"num_experts": n, **k}))


def test_the_calls_below_are_right_but_for_one_thing(calls):
    for call in some_calls().values():
        call()
    assert len(calls) == 6


@pytest.mark.parametrize("op,kw", [
    ("gated", dict(out={})), ("linear", dict(out={})), ("combine_backward", dict(out={})),
    ("gated", dict(out={"h": None})), ("combine_backward", dict(out={"dy": None})),
    ("gated", dict(w=None)), ("gated_backward", dict(w=[])), ("linear", dict(w=None)),
    ("linear_backward", dict(w=3)),
    ("gated", dict(tile_m=None)), ("gated_backward", dict(top_k=2.0)), ("linear", dict(tile_m="16")),
    ("linear_backward", dict(tile_m=1 << 31)), ("gated", dict(tile_m=-1 << 40)),
    ("combine", dict(num_experts=None)), ("combine_backward", dict(num_experts=1.5)),
])
def test_refusals_are_the_packages_own(calls, op, kw):
    with pytest.raises(M.MoeRouteError):
        some_calls()[op](**kw)
    assert not calls


@pytest.mark.parametrize("op,need", [
    ("gated", ("counts", "padded_offsets", "m_indices")),
    ("gated_backward", ("counts", "padded_offsets", "m_indices")),
    ("linear", ("padded_offsets", "m_indices")), ("linear_backward", ("counts", "m_indices")),
    ("combine", ("packed", "inv_perm", "offsets", "padded_offsets", "topk_weights")),
    ("combine_backward", ("packed", "m_indices", "row_entry")),
])
def test_what_a_layout_lacks_is_named(calls, op, need):
    for k in need:
        for lay in ({a: b for a, b in layout(3).items() if a != k}, {**layout(3), k: None}):
            with pytest.raises(M.MoeRouteError, match=k):
                some_calls()[op](lay=lay)
    assert not calls


def test_no_experts_here(calls):
    """Without experts the rows are zeroed, after the same checks as ever."""
    ops = some_calls(0)
    h, x = gpu(R, F), gpu(R, H)
    for t in (h, x):
        t.fill_(1)
    ops["gated"](out={"h": h})
    ops["gated_backward"](out={"dx": x})
    assert not bool(h.any()) and not bool(x.any())
    for t in (h, x):
        t.fill_(1)
    ops["linear"](out={"y": h})
    ops["linear_backward"](out={"dx": x})
    assert not bool(h.any()) and not bool(x.any())
    for op, key, good in (("gated", "h", F), ("gated_backward", "dx", H), ("linear", "y", F),
                          ("linear_backward", "dx", H)):
        for bad in (gpu(R, good + 1), gpu(R - 1, good), gpu(R, good, dt=torch.float32)):
            bad.fill_(1)
            with pytest.raises(M.MoeRouteError):
                ops[op](out={key: bad})
            assert bool(bad.all())
    assert not calls
