"""GPU tests of the feed-forward operators at sizes past what 32 bits, a grid
or an even spread of the rows would allow."""
import pytest
import torch

from ffn_util import normal
from test_gpu_ffn import check_expert_gated

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("T,H", [
    (2_130_000, 1001),  # x and its padded copy below 4 GB
    (2_131_000, 1001),  # x below, the copy above
    (2_146_000, 1001),  # both above
    (300_032, 7168),    # no copy, x above
])
def test_gathered_tiles_beyond_32_bits(T, H):
    """Rows at x's end, enough of them for the tiled kernels in both directions."""
    n, tile = 2, 128
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    far = T - 1 - torch.randperm(500, generator=torch.Generator().manual_seed(1))[:200]
    x[far.cuda()] = normal(1, 200, H, dt=BF)
    i32 = dict(dtype=torch.int32, device="cuda")
    m, entry = torch.full((256,), -1, **i32), torch.full((256,), -1, **i32)
    m[:104], m[128:224] = 0, 1
    entry[:104], entry[128:224] = far[:104].int().cuda(), far[104:].int().cuda()
    lay = dict(m_indices=m, row_entry=entry, counts=torch.tensor([104, 96], **i32),
               padded_offsets=torch.tensor([0, 128, 256], **i32))
    check_expert_gated(lay, n, 1, x, 64, tile, BF)
