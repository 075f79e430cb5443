"""The workspace of the adapters' backward pass: transposed copies of A and B for no more
adapters than there are tokens, sums that do not grow with the adapters, and the results
where adapters outnumber tokens."""
import ctypes
import os

import pytest
import torch

import moe_expert_routing_amd as M
from moe_expert_routing_amd import adapters
from moe_expert_routing_amd.ffn import Matrix

BF, FP = torch.bfloat16, torch.float16
P = 0x10000  # never dereferenced


@pytest.mark.parametrize("T,I,O,R,n", [(128, 7168, 7168, 64, 512), (40, 7168, 7168, 16, 1024), (8192, 7168, 7168, 64, 4096), (1, 4096, 4096, 128, 4096),
                                       (3000, 2048, 4096, 32, 3001), (100000, 1024, 1024, 128, 4096)])
def test_size(T, I, O, R, n):
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("library not built")
    a = adapters.AdapterLinearArgs(dtype=0, rank=R, tokens=T, in_=I, out=O, adapters=n, x=Matrix(P, I, 0), w=Matrix(P, I, 0),
                                   a=Matrix(P, I, R * I), b=Matrix(P, R, O * R), ids=P, scale=P, s=P, dy=Matrix(P, O, 0), dx=Matrix(P, I, 0),
                                   da=Matrix(P, I, R * I), db=Matrix(P, R, O * R))
    need = M.lib().moe_adapter_linear_workspace_bytes(ctypes.byref(a), 1)
    copies = 2 * min(n, T) * R * (I + O)
    # two sums a chunk, of 4 tokens and more for each of the rank: 2 T / (4 R) R (I + O) fp32; at most some 512
    # blocks' chunks of 256 columns
    sums = min(2 * T * (I + O), 2 * (512 * 256 // (I + O) + 2) * R * (I + O) * 4)
    assert 0 < need <= copies + sums + 4 * (T * (R + 8) + n) + (1 << 16)


def ids_of(kind, T, n, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "spread":
        ids = torch.randint(0, n, (T,), generator=g)
    elif kind == "few":  # the same few again and again, some without, some out of range
        ids = torch.randint(0, n, (6,), generator=g)[torch.randint(0, 6, (T,), generator=g)]
        ids[1::7], ids[3::11] = -1, n
    elif kind == "one":
        ids = torch.full((T,), n - 1)
    else:  # a request after the other
        ids = torch.randint(0, n, (5,), generator=g)[torch.arange(T) * 5 // T]
    return ids.int().cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["spread", "few", "one", "requests"])
@pytest.mark.parametrize("T,I,O,R,n", [(1, 64, 72, 8, 2), (40, 96, 264, 4, 1000), (300, 200, 72, 7, 301), (1500, 130, 64, 16, 1600), (700, 512, 520, 40, 701)])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_more_adapters_than_tokens(T, I, O, R, n, kind, dt):
    """The outputs over all adapters are those over the live ones alone, which take the
    places of the adapters, and zeros for the others."""
    from block_util import normal
    x, w, dy = normal(1, T, I, dt=dt), normal(2, O, I, dt=dt, scale=I ** -0.5), normal(3, T, O, dt=dt)
    ids = ids_of(kind, T, n, T)
    live, at = torch.unique(ids.long().clamp(-1, n), return_inverse=True)
    real = (live >= 0) & (live < n)
    at = torch.where(real[at], (real.cumsum(0) - 1)[at], -1).int()
    live = live[real]
    assert 0 < len(live) <= T
    a, b = normal(4, n, R, I, dt=dt, scale=I ** -0.5), normal(5, n, O, R, dt=dt, scale=R ** -0.5)
    s = normal(6, T, R, dt=torch.float32)
    for scale in (None, 0.5 + torch.rand(n, device="cuda")):
        all_ = M.adapter_linear_backward(dy, x, w, a, b, ids, s, scale=scale,
                                         out={"dx": torch.empty_like(x), "da": torch.full_like(a, 9.0), "db": torch.full_like(b, 9.0)})
        few = M.adapter_linear_backward(dy, x, w, a[live].contiguous(), b[live].contiguous(), at, s, scale=None if scale is None else scale[live].contiguous())
        for k in ("da", "db"):
            assert torch.equal(all_[k][live], few[k]), k
            all_[k][live] = 0
            assert bool((all_[k] == 0).all()), k
        assert torch.equal(all_["dx"], few["dx"])
        alone = M.adapter_linear_backward(dy, x, w, a, b, ids, None, scale=scale, out={"dx": torch.empty_like(x)})
        assert torch.equal(alone["dx"], few["dx"])
