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
