"""GPU tests of the feed-forward operators at sizes past what 32 bits, a grid
or an even spread of the rows would allow."""
import pytest
import torch

import moe_expert_routing_amd as M
from ffn_util import (F32, TINY, assert_close, gated_grads, gated_oracle, groups, hand_layout,
                      normal)
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


@pytest.mark.parametrize("T", [12, 400])  # weight gradients of few rows, and on the matrix cores
def test_layout_of_tokens_that_x_does_not_have(T):
    """x of no rows with a layout of entries: nothing to gather, so h and the weight
    gradients are zeros; dx is made of the rows alone and is whole."""
    n, H, F, tile = 3, 72, 40, 16
    ids = torch.randint(0, n, (T, 1), generator=torch.Generator().manual_seed(T))
    lay = hand_layout(ids, n, tile)
    rows = lay["m_indices"].numel()
    x, dt = normal(1, 0, H, dt=BF), BF
    wg, wu = normal(2, n, F, H, dt=dt), normal(3, n, F, H, dt=dt)
    pre, dh = normal(4, rows, 2 * F, dt=dt), normal(5, rows, F, dt=dt)
    kw = dict(tile_m=tile, top_k=1)
    r = M.expert_gated_ffn(x, wg, wu, lay, save_pre=True, **kw)
    assert not bool(r["h"].any()) and not bool(r["pre"].any())
    b = M.expert_gated_ffn_backward(dh, pre, x, wg, wu, lay, **kw)
    assert not bool(b["dw_gate"].any()) and not bool(b["dw_up"].any())
    some = normal(6, T, H, dt=dt)
    for e, at, tok in groups(lay, n, rows, 1):
        ref, bd = gated_grads(dh[at], pre[at], some[tok], wg[e], wu[e], "silu", dt)["dx"]
        assert_close(b["dx"][at], ref, bd, f"dx of {e}")


def test_combine_of_more_rows_than_one_grid_takes():
    """2^24 tokens and more, one block each: a launch's 2^32 work items hold 2^24 - 1
    of them. Each entry has weight 1, so the rows come back as they are."""
    T, W, n = (1 << 24) + 77, 8, 3
    ids = torch.randint(0, n, (T, 1), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    lay = hand_layout(ids, n, 16)
    real = lay["row_entry"] >= 0
    entry = lay["row_entry"][real].long()
    y = normal(1, real.numel(), W, dt=BF)
    want = torch.empty((T, W), dtype=BF, device="cuda")
    want[entry] = y[real]
    assert torch.equal(M.combine(y, lay, num_experts=n), want)
    dout = normal(2, T, W, dt=BF)
    r = M.combine_backward(dout, y, lay, num_experts=n)
    assert torch.equal(r["dy"][real], dout[entry]) and not bool(r["dy"][~real].any())
    d, v = dout[entry].double(), y[real].double()
    S = (d * v).abs().sum(1)
    assert_close(r["dweights"][entry, 0], (d * v).sum(1), (W + 8) * F32 * S + TINY[torch.float32], "dw")
    # and entries without a row, past the rows' blocks: their gradient is 0
    half = {**lay, "m_indices": lay["m_indices"][:64], "row_entry": lay["row_entry"][:64]}
    r = M.combine_backward(dout, y[:64], half, num_experts=n)
    kept = torch.zeros(T, dtype=torch.bool, device="cuda")
    kept[half["row_entry"][half["row_entry"] >= 0].long()] = True
    assert not bool(r["dweights"][~kept].any()) and bool(r["dweights"][kept].all())


def test_product_of_more_tiles_than_one_grid_takes():
    """4096 experts of 64 rows, 32832 wide: 2^23 blocks of 512 threads and some."""
    n, each, H, F = 4096, 64, 8, 32832
    T = n * each
    ids = (torch.arange(T, device="cuda") // each)[:, None]
    lay = hand_layout(ids, n, 16)
    x = normal(1, T, H, dt=BF)
    g = torch.Generator("cuda").manual_seed(2)
    w = torch.randn((n, F, H), device="cuda", dtype=BF, generator=g)
    r = M.expert_gated_ffn(x, w, w, lay, tile_m=16, top_k=1)
    for e in (0, 1, 2047, 4094, 4095):
        at = slice(e * each, (e + 1) * each)
        h, bh, _, _ = gated_oracle(x[at], w[e], w[e], "silu", BF)
        assert_close(r["h"][at], h, bh, f"h of {e}")


@pytest.mark.parametrize("n,tile,live,each", [(64, 256, 2, 700), (32, 4096, 1, 900), (64, 64, 10, 40),
                                              (48, 128, 9, 3), (64, 16, 1, 500)])
def test_few_of_the_experts_have_rows(n, tile, live, each):
    """Tight layouts in which most experts have no rows."""
    ids = (torch.arange(live * each) % live * (n // live))[:, None]
    lay = hand_layout(ids, n, tile)
    check_expert_gated(lay, n, 1, normal(1, live * each, 136, dt=BF), 72, tile, BF)


def test_weight_gradients_of_few_rows_have_the_range_of_fp32():
    """fp16, dh u act'(g) up to 1e6 on 8 rows: dW takes it unrounded."""
    T, H, F = 8, 40, 24
    x = normal(1, T, H, dt=FP, scale=1e-3)
    dh, pre = normal(2, T, F, dt=FP, scale=300.0), normal(3, T, 2 * F, dt=FP, scale=300.0)
    wg = normal(4, F, H, dt=FP)
    out = {"dw_gate": torch.empty_like(wg), "dw_up": torch.empty_like(wg)}
    r = M.gated_ffn_backward(dh, pre, x, wg, wg, out=out)
    grads = gated_grads(dh, pre, x, wg, wg, "silu", FP)
    for k in out:
        ref, b = grads[k]
        assert bool(torch.isfinite(r[k]).all()) and float((dh.double() * pre[:, F:].double()).abs().max()) > 65504
        assert_close(r[k], ref, b, k)
