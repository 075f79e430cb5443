"""GPU tests of the feed-forward operators against the 64-bit oracle: sizes
around the tiles' edges, both types and every activation, strided and
misaligned operands, the expert form over real routing calls (experts without
rows, other ranks' rows, buffers cut short), padding that holds NaN, streams
and graphs."""
import pytest
import torch

import moe_expert_routing_amd as M
from ffn_util import (ACT_ULP, F32, TINY, act, assert_close, gated_grads, gated_oracle, groups,
                      half_step, hand_layout, linear_grads, linear_oracle, local_layout, normal,
                      slope)

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

BF, FP = torch.bfloat16, torch.float16


def check_gated(x, wg, wu, name, r):
    h, bh, pre, bp = gated_oracle(x, wg, wu, name, x.dtype)
    assert_close(r["h"], h, bh, "h")
    if "pre" in r:
        assert_close(r["pre"], pre, bp, "pre")


@pytest.mark.parametrize("T,H,F", [
    (1, 64, 64), (1, 7168, 256), (2, 8, 8), (5, 136, 72), (15, 64, 32), (16, 512, 128),
    (17, 200, 40), (33, 320, 264), (64, 1024, 64), (65, 1000, 100), (128, 128, 128),
    (200, 72, 520), (257, 640, 130), (1000, 256, 1000),
])
@pytest.mark.parametrize("dt,name", [(BF, "silu"), (FP, "gelu")])
def test_gated(T, H, F, dt, name):
    x = normal(1, T, H, dt=dt)
    wg, wu = normal(2, F, H, dt=dt, scale=H ** -0.5), normal(3, F, H, dt=dt, scale=H ** -0.5)
    check_gated(x, wg, wu, name, M.gated_ffn(x, wg, wu, activation=name, save_pre=True))
    r = M.gated_ffn(x, wg, wu, activation=name)
    assert set(r) == {"h"}
    check_gated(x, wg, wu, name, r)


def test_gated_fills_the_chip():
    x, wg, wu = normal(1, 4000, 512, dt=BF), normal(2, 2040, 512, dt=BF), normal(3, 2040, 512, dt=BF)
    check_gated(x, wg, wu, "silu", M.gated_ffn(x, wg, wu, save_pre=True))


@pytest.mark.parametrize("T,H,F", [(3, 65, 33), (20, 1, 1), (70, 127, 63), (130, 1001, 515), (9, 7, 1500)])
@pytest.mark.parametrize("dt", [BF, FP])
def test_gated_odd_widths(T, H, F, dt):
    x = normal(1, T, H, dt=dt)
    wg, wu = normal(2, F, H, dt=dt), normal(3, F, H, dt=dt)
    check_gated(x, wg, wu, "silu", M.gated_ffn(x, wg, wu, save_pre=True))
    pre, dh = normal(4, T, 2 * F, dt=dt), normal(5, T, F, dt=dt)
    r = M.gated_ffn_backward(dh, pre, x, wg, wu)
    for k, (ref, b) in gated_grads(dh, pre, x, wg, wu, "silu", dt).items():
        assert_close(r[k], ref, b, k)


def test_gated_strided_and_misaligned():
    """One fused weight, rows of wider buffers, starts off the 16-byte grid."""
    T, H, F = 70, 256, 96
    for shift in (0, 1, 4, 8):
        base = normal(1, T, H + 24, dt=BF)
        x = base[:, shift:shift + H]
        fused = normal(2, 2 * F, H + 8, dt=BF, scale=H ** -0.5)
        wg, wu = fused[:F, :H], fused[F:, :H]
        out = {"h": torch.full((T, F + 7), 7.0, dtype=BF, device="cuda")[:, :F],
               "pre": torch.full((T, 2 * F + 5), 7.0, dtype=BF, device="cuda")[:, 1:2 * F + 1]}
        r = M.gated_ffn(x, wg, wu, save_pre=True, out=out)
        check_gated(x, wg, wu, "silu", r)
        assert bool((out["h"]._base[:, F:] == 7).all()) and bool((out["pre"]._base[:, 0] == 7).all())
    # gate and up of different alignment and stride
    wu2 = normal(5, F, H + 3, dt=BF, scale=H ** -0.5)[:, 3:]
    check_gated(x, wg, wu2, "silu", M.gated_ffn(x, wg, wu2, save_pre=True))


@pytest.mark.parametrize("T,H,F", [(1, 64, 64), (7, 256, 136), (64, 128, 264), (130, 520, 128),
                                   (300, 1000, 200), (1021, 264, 520)])
@pytest.mark.parametrize("dt,name", [(BF, "gelu"), (FP, "silu"), (BF, "none")])
def test_gated_backward(T, H, F, dt, name):
    x = normal(1, T, H, dt=dt)
    wg, wu = normal(2, F, H, dt=dt, scale=H ** -0.5), normal(3, F, H, dt=dt, scale=H ** -0.5)
    pre, dh = normal(4, T, 2 * F, dt=dt), normal(5, T, F, dt=dt)
    r = M.gated_ffn_backward(dh, pre, x, wg, wu, activation=name)
    for k, (ref, b) in gated_grads(dh, pre, x, wg, wu, name, dt).items():
        assert_close(r[k], ref, b, k)
    only = M.gated_ffn_backward(dh, pre, x, wg, wu, activation=name,
                                out={"dx": torch.empty_like(x)})
    assert torch.equal(only["dx"], r["dx"]) and set(only) == {"dx"}


def test_gated_backward_fills_the_chip():
    T, H, F, dt = 2000, 4096, 2048, BF
    x = normal(1, T, H, dt=dt)
    wg, wu = normal(2, F, H, dt=dt, scale=H ** -0.5), normal(3, F, H, dt=dt, scale=H ** -0.5)
    pre, dh = normal(4, T, 2 * F, dt=dt), normal(5, T, F, dt=dt)
    r = M.gated_ffn_backward(dh, pre, x, wg, wu)
    for k, (ref, b) in gated_grads(dh, pre, x, wg, wu, "silu", dt).items():
        assert_close(r[k], ref, b, k)


def test_extreme_pre_activations():
    """Large and infinite gates: finite results where the formula has them."""
    dt, F, H = BF, 64, 64
    g = torch.tensor([0.0, -0.0, 1e-30, 88.0, -88.0, 100.0, -100.0, 3e4, -3e4, 20.0, -20.0, 5.0],
                     device="cuda").to(dt)
    T = g.numel()
    pre = normal(1, T, 2 * F, dt=dt)
    pre[:, 0] = g
    dh, x = normal(2, T, F, dt=dt), normal(3, T, H, dt=dt)
    wg, wu = normal(4, F, H, dt=dt), normal(5, F, H, dt=dt)
    for name in ("silu", "gelu"):
        r = M.gated_ffn_backward(dh, pre, x, wg, wu, activation=name)
        for k, (ref, b) in gated_grads(dh, pre, x, wg, wu, name, dt).items():
            assert_close(r[k], ref, b, k)


def test_nan_stays_in_its_row():
    x = normal(1, 40, 128, dt=BF)
    x[7, 3] = float("nan")
    x[9, 5] = float("inf")
    wg, wu = normal(2, 64, 128, dt=BF), normal(3, 64, 128, dt=BF)
    clean = x.clone()
    clean[7], clean[9] = 0, 0
    r, c = M.gated_ffn(x, wg, wu)["h"], M.gated_ffn(clean, wg, wu)["h"]
    assert bool(torch.isnan(r[7]).all()) and not bool(torch.isfinite(r[9]).all())
    keep = [i for i in range(40) if i not in (7, 9)]
    assert torch.equal(r[keep], c[keep])


# ------------------------------------------------------------------- linear

@pytest.mark.parametrize("T,I,O", [(1, 64, 64), (3, 2048, 7168), (16, 8, 8), (31, 264, 200),
                                   (64, 1024, 130), (129, 72, 257), (500, 1000, 640), (77, 63, 31)])
@pytest.mark.parametrize("dt,name,bias,res", [(BF, "none", False, False), (BF, "gelu", True, True),
                                              (FP, "silu", True, False), (FP, "none", False, True)])
def test_linear(T, I, O, dt, name, bias, res):
    x, w = normal(1, T, I, dt=dt), normal(2, O, I, dt=dt, scale=I ** -0.5)
    b = normal(3, O, dt=dt) if bias else None
    rs = normal(4, T, O, dt=dt) if res else None
    r = M.linear(x, w, bias=b, activation=name, residual=rs, save_pre=True)
    y, by, z, bz = linear_oracle(x, w, b, name, rs, dt)
    assert_close(r["y"], y, by, "y")
    assert_close(r["pre"], z, bz, "pre")
    assert torch.equal(M.linear(x, w, bias=b, activation=name, residual=rs)["y"], r["y"])


def test_linear_residual_in_place():
    """The output may be the residual's own memory."""
    x, w, rs = normal(1, 300, 256, dt=BF), normal(2, 520, 256, dt=BF), normal(3, 300, 520, dt=BF)
    want = M.linear(x, w, residual=rs)["y"]
    got = M.linear(x, w, residual=rs, out={"y": rs})["y"]
    assert got is rs and torch.equal(got, want)


def test_linear_fills_the_chip():
    x, w = normal(1, 4100, 320, dt=FP), normal(2, 4104, 320, dt=FP, scale=320 ** -0.5)
    b, rs = normal(3, 4104, dt=FP), normal(4, 4100, 4104, dt=FP)
    y, by, _, _ = linear_oracle(x, w, b, "gelu", rs, FP)
    assert_close(M.linear(x, w, bias=b, activation="gelu", residual=rs)["y"], y, by, "y")


@pytest.mark.parametrize("T,I,O", [(1, 64, 64), (9, 136, 72), (65, 256, 520), (700, 200, 1000),
                                   (130, 61, 35)])
@pytest.mark.parametrize("dt,name", [(BF, "none"), (BF, "silu"), (FP, "gelu")])
def test_linear_backward(T, I, O, dt, name):
    x, w = normal(1, T, I, dt=dt), normal(2, O, I, dt=dt, scale=I ** -0.5)
    dy, pre = normal(3, T, O, dt=dt), normal(4, T, O, dt=dt)
    r = M.linear_backward(dy, x, w, pre=pre, activation=name, bias_grad=True)
    for k, (ref, b) in linear_grads(dy, pre, x, w, name, dt).items():
        assert_close(r[k], ref, b, k)
    only = M.linear_backward(dy, x, w, pre=pre, activation=name,
                             out={"dbias": torch.empty(O, dtype=dt, device="cuda")})
    assert torch.equal(only["dbias"], r["dbias"])


def test_no_tokens():
    x, w = normal(1, 0, 64, dt=BF), normal(2, 32, 64, dt=BF)
    assert M.gated_ffn(x, w, w, save_pre=True)["pre"].shape == (0, 64)
    assert M.linear(x, w)["y"].shape == (0, 32)
    r = M.linear_backward(normal(3, 0, 32, dt=BF), x, w, bias_grad=True)
    assert not bool(r["dw"].any()) and not bool(r["dbias"].any())
    r = M.gated_ffn_backward(normal(3, 0, 32, dt=BF), normal(3, 0, 64, dt=BF), x, w, w)
    assert not bool(r["dw_gate"].any()) and not bool(r["dw_up"].any())


# ------------------------------------------------------------------ experts

CASES = [  # T, H, F, tile, experts, top_k, offset, count, rows kept (None: all)
    (1, 64, 40, 16, 128, 8, 0, 0, None),
    (16, 256, 64, 16, 128, 8, 32, 16, None),
    (40, 136, 72, 32, 128, 4, 64, 48, None),
    (200, 128, 136, 64, 128, 8, 0, 16, None),
    (300, 200, 64, 128, 128, 2, 16, 32, None),
    (300, 65, 33, 48, 128, 4, 16, 24, None),
    (900, 64, 128, 256, 128, 8, 96, 32, None),
    (130, 64, 64, 80, 128, 8, 0, 16, 200),
    (0, 64, 64, 16, 128, 8, 0, 16, None),
]


@pytest.mark.parametrize("case", CASES, ids=[f"T{c[0]}_tile{c[3]}" for c in CASES])
@pytest.mark.parametrize("dt,name", [(BF, "silu"), (FP, "gelu")])
def test_experts(case, dt, name):
    T, H, F, tile, e, k, off, cnt, cut = case
    lay, n = local_layout(T, tile, e=e, top_k=k, off=off, cnt=cnt, seed=T)
    if cut is not None:
        lay["m_indices"], lay["row_entry"] = lay["m_indices"][:cut], lay["row_entry"][:cut]
    rows = lay["m_indices"].numel()
    gr = groups(lay, n, rows, k)
    x = normal(1, T, H, dt=dt)
    wg, wu = normal(2, n, F, H, dt=dt, scale=H ** -0.5), normal(3, n, F, H, dt=dt, scale=H ** -0.5)
    kw = dict(tile_m=tile, top_k=k, activation=name)
    r = M.expert_gated_ffn(x, wg, wu, lay, save_pre=True, **kw)
    rest = torch.ones(rows, dtype=torch.bool)
    for e_, at, tok in gr:
        rest[at] = False
        h, bh, pre, bp = gated_oracle(x[tok], wg[e_], wu[e_], name, dt)
        assert_close(r["h"][at], h, bh, f"h of {e_}")
        assert_close(r["pre"][at], pre, bp, f"pre of {e_}")
    assert not bool(r["h"][rest].any()) and not bool(r["pre"][rest].any())

    # backward: what rows without an entry hold does not matter
    pre, dh = normal(4, rows, 2 * F, dt=dt), normal(5, rows, F, dt=dt)
    pre[rest], dh[rest] = float("nan"), float("nan")
    b = M.expert_gated_ffn_backward(dh, pre, x, wg, wu, lay, **kw)
    for e_, at, tok in gr:
        for key, (ref, bd) in gated_grads(dh[at], pre[at], x[tok], wg[e_], wu[e_], name, dt).items():
            assert_close(b[key][at] if key == "dx" else b[key][e_], ref, bd, f"{key} of {e_}")
    assert not bool(b["dx"][rest].any())

    # the down projection on the rows
    xr, w = normal(6, rows, F, dt=dt), normal(7, n, H, F, dt=dt, scale=F ** -0.5)
    xr[rest] = float("nan")
    bias, res = normal(8, n, H, dt=dt), normal(9, rows, H, dt=dt)
    y = M.expert_linear(xr, w, lay, tile_m=tile, bias=bias, activation=name, residual=res,
                        save_pre=True)
    dy = normal(10, rows, H, dt=dt)
    dy[rest] = float("nan")
    lb = M.expert_linear_backward(dy, xr, w, lay, tile_m=tile, pre=y["pre"], activation=name,
                                  bias_grad=True)
    plain = M.expert_linear_backward(dy, xr, w, lay, tile_m=tile, bias_grad=True)
    for e_, at, _ in gr:
        ref, bd, z, bz = linear_oracle(xr[at], w[e_], bias[e_], name, res[at], dt)
        assert_close(y["y"][at], ref, bd, f"y of {e_}")
        assert_close(y["pre"][at], z, bz, f"z of {e_}")
        for got, nm, pr in ((lb, name, y["pre"][at]), (plain, "none", None)):
            for key, (ref, bd) in linear_grads(dy[at], pr, xr[at], w[e_], nm, dt).items():
                assert_close(got[key][at] if key == "dx" else got[key][e_], ref, bd,
                             f"{key} of {e_}")
    for t in (y["y"], y["pre"], lb["dx"], plain["dx"]):
        assert not bool(t[rest].any())


@pytest.mark.parametrize("case", CASES, ids=[f"T{c[0]}_tile{c[3]}" for c in CASES])
@pytest.mark.parametrize("dt,W", [(BF, 64), (FP, 1000), (BF, 61), (BF, 7168)])
def test_combine(case, dt, W):
    T, _, _, tile, e, k, off, cnt, cut = case
    lay, n = local_layout(T, tile, e=e, top_k=k, off=off, cnt=cnt, seed=T)
    rows = lay["m_indices"].numel() if cut is None else cut
    gr = groups(lay, n, rows, k)
    y, res, dout = normal(1, rows, W, dt=dt), normal(2, T, W, dt=dt), normal(3, T, W, dt=dt)
    rest = torch.ones(rows, dtype=torch.bool)
    for _, at, _ in gr:
        rest[at] = False
    y[rest] = float("nan")
    u = half_step(dt)
    w = lay["topk_weights"].double()
    for weighted in (True, False):
        for residual in (None, res):
            ref = residual.double() if residual is not None else torch.zeros(T, W, device="cuda").double()
            S = ref.abs()
            for _, at, tok in gr:
                entry = lay["row_entry"][at.cuda()].long()
                f = w.reshape(-1)[entry][:, None] if weighted else 1.0
                ref[tok] += f * y[at].double()
                S[tok] += f * y[at].double().abs()
            got = M.combine(y, lay, num_experts=n, weighted=weighted, residual=residual)
            assert_close(got, ref, u * ref.abs() * 1.01 + (k + 2) * F32 * S + TINY[dt], "out")
        b = M.combine_backward(dout, y if weighted else None,
                               lay if weighted else {**lay, "m_indices": lay["m_indices"][:rows]},
                               num_experts=n, weighted=weighted)
        dy = torch.zeros(rows, W, device="cuda").double()
        dw, Sw = torch.zeros_like(w).reshape(-1), torch.zeros_like(w).reshape(-1)
        for _, at, tok in gr:
            entry = lay["row_entry"][at.cuda()].long()
            d = dout[tok].double()
            dy[at] = (w.reshape(-1)[entry][:, None] if weighted else 1.0) * d
            dw[entry] = (d * y[at].double()).sum(1)
            Sw[entry] = (d * y[at].double()).abs().sum(1)
        assert_close(b["dy"], dy, (u * 1.01 + F32) * dy.abs() + TINY[dt], "dy")
        if weighted:
            assert_close(b["dweights"].reshape(-1), dw, (W + 8) * F32 * Sw + TINY[torch.float32], "dw")
        else:
            assert set(b) == {"dy"}


def test_experts_without_gather():
    """Without row_entry x has a row per row, as a dispatched batch has."""
    lay, n = local_layout(100, 32, top_k=4, off=0, cnt=32)
    rows = lay["m_indices"].numel()
    tok = (lay["row_entry"].long() // 4).clamp(min=0)
    x = normal(1, 100, 128, dt=BF)
    wg, wu = normal(2, n, 64, 128, dt=BF), normal(3, n, 64, 128, dt=BF)
    a = M.expert_gated_ffn(x, wg, wu, lay, tile_m=32, top_k=4)["h"]
    cut = {k: v for k, v in lay.items() if k != "row_entry"}
    b = M.expert_gated_ffn(x[tok].contiguous(), wg, wu, cut, tile_m=32, top_k=4)["h"]
    assert a.shape == (rows, 64) and torch.equal(a, b)


def test_results_are_the_same_every_call():
    T = 3000
    x, wg, wu = normal(1, T, 512, dt=BF), normal(2, 320, 512, dt=BF), normal(3, 320, 512, dt=BF)
    pre, dh = normal(4, T, 640, dt=BF), normal(5, T, 320, dt=BF)
    first = M.gated_ffn_backward(dh, pre, x, wg, wu)
    for _ in range(3):
        again = M.gated_ffn_backward(dh, pre, x, wg, wu)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_side_stream_and_graph():
    """A training step on a side stream, and captured: every replay gives the
    eager result on new inputs, with eager work between the replays."""
    lay, n = local_layout(200, 64, top_k=8, off=0, cnt=16)
    T, H, F = 200, 256, 136
    x = normal(1, T, H, dt=BF)
    wg, wu = normal(2, n, F, H, dt=BF, scale=H ** -0.5), normal(3, n, F, H, dt=BF, scale=H ** -0.5)
    wd = normal(4, n, H, F, dt=BF, scale=F ** -0.5)
    dout = normal(5, T, H, dt=BF)
    kw = dict(tile_m=64, top_k=8)

    def step():
        f = M.expert_gated_ffn(x, wg, wu, lay, save_pre=True, **kw)
        y = M.expert_linear(f["h"], wd, lay, tile_m=64)["y"]
        out = M.combine(y, lay, num_experts=n, residual=x)
        c = M.combine_backward(dout, y, lay, num_experts=n)
        d = M.expert_linear_backward(c["dy"], f["h"], wd, lay, tile_m=64)
        b = M.expert_gated_ffn_backward(d["dx"], f["pre"], x, wg, wu, lay, **kw)
        dx = M.combine(b["dx"], lay, num_experts=n, weighted=False, residual=dout)
        return [out, c["dweights"], d["dw"], b["dw_gate"], b["dw_up"], dx]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        x.copy_(normal(20 + i, T, H, dt=BF))
        dout.copy_(normal(30 + i, T, H, dt=BF))
        for t in held:
            t.fill_(9)
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


def test_gradients_against_differences():
    """The block's loss <dout, out> moved along random directions of x and of
    every weight, by the 64-bit oracle: the operators' gradients predict it."""
    T, H, F, k = 24, 64, 40, 4
    lay, n = local_layout(T, 16, top_k=k, off=0, cnt=16)
    gr = groups(lay, n, lay["m_indices"].numel(), k)
    dt = FP
    x = normal(1, T, H, dt=dt)
    p = {"x": x, "wg": normal(2, n, F, H, dt=dt, scale=H ** -0.5),
         "wu": normal(3, n, F, H, dt=dt, scale=H ** -0.5),
         "wd": normal(4, n, H, F, dt=dt, scale=F ** -0.5), "w": lay["topk_weights"]}
    dout = normal(5, T, H, dt=dt)
    kw = dict(tile_m=16, top_k=k)
    f = M.expert_gated_ffn(x, p["wg"], p["wu"], lay, save_pre=True, **kw)
    y = M.expert_linear(f["h"], p["wd"], lay, tile_m=16)["y"]
    c = M.combine_backward(dout, y, lay, num_experts=n)
    d = M.expert_linear_backward(c["dy"], f["h"], p["wd"], lay, tile_m=16)
    b = M.expert_gated_ffn_backward(d["dx"], f["pre"], x, p["wg"], p["wu"], lay, **kw)
    grad = {"x": M.combine(b["dx"], lay, num_experts=n, weighted=False), "wg": b["dw_gate"],
            "wu": b["dw_up"], "wd": d["dw"], "w": c["dweights"]}

    def loss(q):
        out = torch.zeros(T, H, device="cuda", dtype=torch.float64)
        for e, at, tok in gr:
            entry = lay["row_entry"][at.cuda()].long()
            xe = q["x"][tok]
            h = act(xe @ q["wg"][e].T, "silu") * (xe @ q["wu"][e].T)
            out[tok] += q["w"].reshape(-1)[entry][:, None] * (h @ q["wd"][e].T)
        return float((out * dout.double()).sum())

    full = {key: v.double() for key, v in p.items()}
    for key in p:
        dirn = normal(40, *p[key].shape, dt=torch.float32).double()
        eps = 1e-4
        num = (loss({**full, key: full[key] + eps * dirn}) -
               loss({**full, key: full[key] - eps * dirn})) / (2 * eps)
        ana = float((grad[key].double() * dirn).sum())
        # every factor of the chain was rounded to fp16 at most 6 times; errors
        # of the summed products add up like their absolute sizes at worst,
        # like random signs in the mean: 6 half steps of the gradient's norm
        scale = float(grad[key].double().norm()) * float(dirn.norm()) / dirn.numel() ** 0.5
        assert abs(num - ana) <= 6 * half_step(dt) * scale * 10 + 1e-6 * abs(num), (key, num, ana)


def check_expert_gated(lay, n, k, x, F, tile, dt, name="silu", backward=True):
    H, rows = x.shape[1], lay["m_indices"].numel()
    wg, wu = normal(2, n, F, H, dt=dt, scale=H ** -0.5), normal(3, n, F, H, dt=dt, scale=H ** -0.5)
    kw = dict(tile_m=tile, top_k=k, activation=name)
    r = M.expert_gated_ffn(x, wg, wu, lay, save_pre=True, **kw)
    pre, dh = normal(4, rows, 2 * F, dt=dt), normal(5, rows, F, dt=dt)
    b = M.expert_gated_ffn_backward(dh, pre, x, wg, wu, lay, **kw) if backward else None
    for e, at, tok in groups(lay, n, rows, k):
        at, tok = at.cuda(), tok.cuda()
        h, bh, ref, bp = gated_oracle(x[tok], wg[e], wu[e], name, dt)
        assert_close(r["h"][at], h, bh, f"h of {e}")
        assert_close(r["pre"][at], ref, bp, f"pre of {e}")
        if b is not None:
            for key, (ref, bd) in gated_grads(dh[at], pre[at], x[tok], wg[e], wu[e], name, dt).items():
                assert_close(b[key][at] if key == "dx" else b[key][e], ref, bd, f"{key} of {e}")


@pytest.mark.parametrize("k", [1, 3, 6])
def test_entries_per_token_need_not_be_a_power_of_two(k):
    T, n = 90, 7
    g = torch.Generator().manual_seed(k)
    ids = torch.stack([torch.randperm(n, generator=g)[:k] for _ in range(T)])
    lay = hand_layout(ids, n, 32)
    check_expert_gated(lay, n, k, normal(1, T, 136, dt=BF), 72, 32, BF)


def test_many_rows_an_expert():
    """Experts with thousands of rows, one with a single row and one with none."""
    T, n = 5200, 4
    ids = torch.randint(0, 2, (T, 1), generator=torch.Generator().manual_seed(1))
    ids[77] = 3
    lay = hand_layout(ids, n, 256, rows=9216)
    check_expert_gated(lay, n, 1, normal(1, T, 264, dt=FP), 136, 256, FP, "gelu")


def test_one_expert_gets_everything():
    lay = hand_layout(torch.full((300, 1), 5), 8, 64)
    check_expert_gated(lay, 8, 1, normal(1, 300, 128, dt=BF), 256, 64, BF)


def test_gathered_rows_beyond_32_bits():
    """x of more than 4 GB: rows at its end are the ones that are gathered."""
    T, H, F, n = 300_032, 7168, 64, 2
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    far = T - 1 - torch.arange(40) * 3
    x[far.cuda()] = normal(1, 40, H, dt=BF)
    i32 = dict(dtype=torch.int32, device="cuda")
    m = torch.full((64,), -1, **i32)
    entry = torch.full((64,), -1, **i32)
    m[:25], m[32:47] = 0, 1
    entry[:25], entry[32:47] = far[:25].int().cuda(), far[25:].int().cuda()
    lay = dict(m_indices=m, row_entry=entry, counts=torch.tensor([25, 15], **i32),
               padded_offsets=torch.tensor([0, 32, 64], **i32))
    check_expert_gated(lay, n, 1, x, F, 32, BF)


def test_outputs_beyond_32_bits():
    """Outputs of more than 4 GB, by the last rows."""
    T, I, O = 300_032, 8, 8192
    x, w = normal(1, T, I, dt=BF), normal(2, O, I, dt=BF)
    res = torch.zeros((1, O), dtype=BF, device="cuda").expand(T, O)
    with pytest.raises(M.MoeRouteError):
        M.linear(x, w, residual=res)  # rows that overlap
    y = M.linear(x, w)["y"]
    ref, b, _, _ = linear_oracle(x[-300:], w, None, "none", None, BF)
    assert_close(y[-300:], ref, b, "y")
    lay = hand_layout(torch.zeros((T, 1), dtype=torch.long), 1, 16)
    out = M.combine(y, lay, num_experts=1)
    assert torch.equal(out[-300:], y[-300:])
    dy = M.combine_backward(out, y, lay, num_experts=1)
    assert torch.equal(dy["dy"][-300:], y[-300:])
    d = y[-300:].double()
    assert_close(dy["dweights"][-300:, 0], (d * d).sum(1), (O + 8) * F32 * (d * d).sum(1), "dw")


@pytest.mark.parametrize("T,I,O", [(40, 4480, 384), (64, 7168, 256), (100, 512, 4096), (1000, 2560, 384),
                                   (3000, 1024, 1024), (2100, 2048, 4096)])
def test_linear_tiles(T, I, O):
    """Shapes that lie on each side of the tile choice, forward and backward."""
    x, w = normal(1, T, I, dt=BF), normal(2, O, I, dt=BF, scale=I ** -0.5)
    dy, pre = normal(3, T, O, dt=BF), normal(4, T, O, dt=BF)
    y, by, z, bz = linear_oracle(x, w, None, "silu", None, BF)
    r = M.linear(x, w, activation="silu", save_pre=True)
    assert_close(r["y"], y, by, "y")
    assert_close(r["pre"], z, bz, "pre")
    r = M.linear_backward(dy, x, w, pre=pre, activation="silu", bias_grad=True)
    for k, (ref, b) in linear_grads(dy, pre, x, w, "silu", BF).items():
        assert_close(r[k], ref, b, k)


def test_two_streams_at_once():
    """Calls on two streams with nothing between them give what each gives alone."""
    xs = [normal(i, 700, 512, dt=BF) for i in range(2)]
    ws = [normal(5 + i, 1024, 512, dt=BF) for i in range(2)]
    dys = [normal(9 + i, 700, 1024, dt=BF) for i in range(2)]
    pre = normal(20, 700, 1024, dt=BF)
    want = [M.linear_backward(dys[i], xs[i], ws[i], pre=pre, activation="gelu", bias_grad=True)
            for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(M.linear_backward(dys[i], xs[i], ws[i], pre=pre, activation="gelu",
                                                bias_grad=True))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(r[k], want[i][k]) for k in want[i])


def test_refusals_on_the_gpu():
    x, w = normal(1, 8, 64, dt=BF), normal(2, 32, 64, dt=BF)
    bad = [
        lambda: M.gated_ffn(x, w, w.to(FP)),                       # another type
        lambda: M.gated_ffn(x.float(), w.float(), w.float()),      # no such type
        lambda: M.gated_ffn(x, w, w[:, :32]),                      # another shape
        lambda: M.gated_ffn(x.t(), w, w),                          # columns not contiguous
        lambda: M.gated_ffn(x, w, w, activation="tanh"),
        lambda: M.gated_ffn(x, w, w, out={"h": x}),                # output of another shape
        lambda: M.linear(x, w.unsqueeze(0)),
        lambda: M.linear(x, w, bias=x[0]),
        lambda: M.linear_backward(normal(3, 8, 32, dt=BF), x, w, activation="silu"),  # no pre
        lambda: M.linear(x, w, residual=normal(4, 9, 32, dt=BF)),
        lambda: M.linear(x, w.cpu()),
    ]
    lay, n = local_layout(20, 16, top_k=4, off=0, cnt=16)
    rows = lay["m_indices"].numel()
    we = normal(5, n, 32, 64, dt=BF)
    xt = normal(6, 20, 64, dt=BF)
    bad += [
        lambda: M.expert_gated_ffn(xt, we, we, lay, tile_m=24, top_k=4),   # no multiple of 16
        lambda: M.expert_gated_ffn(xt, we, we, lay, tile_m=16, top_k=0),
        lambda: M.expert_gated_ffn(xt, we[0], we[0], lay, tile_m=16, top_k=4),
        lambda: M.expert_linear(xt, we, lay, tile_m=16),                   # rows, not tokens
        lambda: M.expert_gated_ffn(xt, we, we, {**lay, "m_indices": lay["m_indices"].long()},
                                   tile_m=16, top_k=4),
        lambda: M.combine(normal(7, rows, 64, dt=BF), lay, num_experts=1000),
        lambda: M.combine(normal(7, rows, 64, dt=BF), lay, num_experts=n, residual=xt[:, :32]),
        lambda: M.combine_backward(xt[:10], None, lay, num_experts=n, weighted=False),
        lambda: M.combine_backward(xt, None, lay, num_experts=n),          # dweights need y
    ]
    for f in bad:
        with pytest.raises(M.MoeRouteError):
            f()


@pytest.mark.parametrize("tokens", [16, 500])
def test_moe_block_example(tokens):
    """The example's block, forward and backward, against plain torch. The chain
    rounds to bf16 at most 6 times on the way to any output, each by at most
    half a step; in the 2-norm independent roundings add up to less than their
    plain sum."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import moe_block as E
    block = E.MoeBlock(256, 128, offset=112, count=112)
    x, dout = normal(1, tokens, 256, dt=BF), normal(2, tokens, 256, dt=BF)
    out, saved = block.forward(x, train=True)
    grads = block.backward(dout, saved)
    want, ref = E.plain(block, x, dout, saved)
    assert E.off(out, want) <= 6 * half_step(BF)
    for k in ref:
        assert E.off(grads[k], ref[k]) <= 6 * half_step(BF), k
    plain, _ = block.forward(x)
    assert torch.equal(plain, out)


@pytest.mark.parametrize("T,n,k,tile,extra", [(60, 8, 4, 16, 0), (130, 8, 4, 16, 100), (400, 8, 3, 16, 0),
                                              (400, 8, 3, 48, 200), (3000, 2, 1, 16, 70), (3000, 3, 1, 80, 0),
                                              (900, 20, 4, 64, 33)])
def test_tiles_that_follow_the_experts(T, n, k, tile, extra):
    """More rows an expert than the layout's alignment: tiles that do not divide
    it, with rows past the experts' to be cleared."""
    g = torch.Generator().manual_seed(T)
    ids = torch.stack([torch.randperm(n, generator=g)[:k] for _ in range(T)])
    ids = torch.where(ids == 1, 0, ids) if k == 1 else ids  # an expert without rows
    full = hand_layout(ids, n, tile)
    lay = hand_layout(ids, n, tile, rows=full["m_indices"].numel() + extra)
    check_expert_gated(lay, n, k, normal(1, T, 200, dt=BF), 136, tile, BF)
    rows = lay["m_indices"].numel()
    w, b = normal(6, n, 264, 136, dt=BF, scale=136 ** -0.5), normal(7, n, 264, dt=BF)
    x, res = normal(8, rows, 136, dt=BF), normal(9, rows, 264, dt=BF)
    r = M.expert_linear(x, w, lay, tile_m=tile, bias=b, activation="gelu", residual=res,
                        save_pre=True, out={"y": torch.full((rows, 264), 9.0, dtype=BF, device="cuda")})
    rest = torch.ones(rows, dtype=torch.bool)
    for e, at, _ in groups(lay, n, rows, k):
        rest[at] = False
        ref, bd, z, bz = linear_oracle(x[at], w[e], b[e], "gelu", res[at], BF)
        assert_close(r["y"][at], ref, bd, f"y of {e}")
        assert_close(r["pre"][at], z, bz, f"z of {e}")
    assert not bool(r["y"][rest].any()) and not bool(r["pre"][rest].any())


@pytest.mark.parametrize("T,H,F", [(1, 2112, 322), (3, 513, 33), (8, 1088, 448), (5, 7, 1500)])
@pytest.mark.parametrize("dt,name", [(BF, "silu"), (FP, "gelu"), (FP, "none")])
def test_weight_gradients_of_few_rows_are_rounded_once(T, H, F, dt, name):
    """Up to 8 rows: fp32 up to the result, so half a step of it, the fp32 sum
    and the activation's own error are all there is."""
    x, dh, pre = normal(1, T, H, dt=dt), normal(2, T, F, dt=dt), normal(3, T, 2 * F, dt=dt)
    wg, wu = normal(4, F, H, dt=dt), normal(5, F, H, dt=dt)
    d, g, u, xd = dh.double(), pre[:, :F].double(), pre[:, F:].double(), x.double()
    out = {"dw_gate": torch.empty_like(wg), "dw_up": torch.empty_like(wu)}
    r = M.gated_ffn_backward(dh, pre, x, wg, wu, activation=name, out=out)
    y = M.linear_backward(dh, x, wg, pre=pre[:, :F], activation=name, out={"dw": torch.empty_like(wg)})
    for got, f, size in ((r["dw_gate"], slope(g, name) * u, (1 + g.abs()) * u.abs()),
                         (r["dw_up"], act(g, name), g.abs()), (y["dw"], slope(g, name), 1 + g.abs())):
        dz = d * f
        S = (dz.abs() * (T + 8) + 2 * ACT_ULP * d.abs() * size).T @ xd.abs()
        ref = dz.T @ xd
        assert_close(got, ref, half_step(dt) * 1.01 * ref.abs() + F32 * S * 1.01 + TINY[dt], name)
