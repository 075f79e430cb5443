"""GPU tests of the norm, dropout and the 8-bit outputs against 64 bits."""
import numpy as np
import pytest
import torch

import moe_expert_routing_amd as M
from block_util import check_mx, drop, e4m3_values, norm_grads, norm_h, norm_y, normal, numbers
from ffn_util import F32, TINY, assert_close, half_step

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
RNG = (0x9E3779B97F4A7C15 - 2 ** 64, 0x1_2345_6789)


def rng_tensor(rng=RNG):
    return torch.tensor(rng, dtype=torch.int64, device="cuda")


# (tokens, width): every row shape's least, largest and odd widths, one row to many
SIZES = [(1, 1), (3, 7), (1, 128), (257, 64), (1000, 128), (5, 129), (33, 512), (130, 513),
         (7, 1000), (2, 2048), (19, 2049), (64, 4096), (3, 4097), (700, 7168), (2, 8192),
         (5, 8193), (3, 16384), (2, 20001), (2, 32768)]


@pytest.mark.parametrize("T,W", SIZES)
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_norm_forward(T, W, dt):
    for k, (res, p) in enumerate([(False, 0.0), (True, 0.0), (True, 0.1), (False, 0.5)]):
        x, w = normal(k, T, W, dt=dt), normal(k + 10, W, dt=dt)
        r = normal(k + 20, T, W, dt=dt, scale=3.0) if res else None
        out = M.rms_norm(x, w, residual=r, eps=1e-5, p=p, rng=rng_tensor() if p else None, site=k)
        h = x
        if res or p:
            h = out["h"]
            assert_close(h, *norm_h(x, r, p, RNG, k, dt), "h")
        else:
            assert "h" not in out
        y, by, rstd, br = norm_y(h, w, 1e-5, dt)
        assert_close(out["rstd"], rstd, br, "rstd")
        assert_close(out["y"], y, by, "y")


@pytest.mark.parametrize("T,W", SIZES)
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_norm_backward(T, W, dt):
    for k, (with_dh, p) in enumerate([(True, 0.0), (False, 0.0), (True, 0.25)]):
        h, dy, w = normal(k, T, W, dt=dt, scale=2.0), normal(k + 1, T, W, dt=dt), normal(k + 2, W, dt=dt)
        dh = normal(k + 3, T, W, dt=dt) if with_dh else None
        rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
        out = M.rms_norm_backward(dy, h, w, rstd, dh=dh, p=p, rng=rng_tensor() if p else None, site=k)
        ref = norm_grads(dy, h, w, rstd, dh, dt)
        assert_close(out["dweight"], *ref["dweight"], "dweight")
        v, b = ref["dtotal"]
        if p:
            assert_close(out["dresidual"], v, b, "dresidual")
            assert_close(out["dx"], drop(v, p, RNG, k), drop(b + 3 * F32 * v.abs(), p, RNG, k) + TINY[dt], "dx")
        else:
            assert "dresidual" not in out
            assert_close(out["dx"], v, b, "dx")


def test_norm_gradients_are_the_differences():
    """The formulas of the gradients against central differences of the forward
    formula in 64 bits: sum(y gy + h gh) in x, residual and weight, with dropout."""
    T, W, eps, p, site = 3, 40, 1e-5, 0.3, 2
    g = torch.Generator().manual_seed(1)
    x, r, gy, gh = (torch.randn(T, W, generator=g, dtype=torch.float64) for _ in range(4))
    w = torch.randn(W, generator=g, dtype=torch.float64)

    def loss(x, r, w):
        h = r + drop(x, p, RNG, site)
        return ((h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * w) * gy + h * gh).sum()
    h = r + drop(x, p, RNG, site)
    rstd = 1 / torch.sqrt(h.square().mean(1) + eps)
    ref = norm_grads(gy, h, w, rstd, gh, BF)
    d = 1e-5
    for t, grad in ((x, drop(ref["dtotal"][0], p, RNG, site)), (r, ref["dtotal"][0]), (w, ref["dweight"][0])):
        flat, want = t.reshape(-1), grad.reshape(-1)
        for i in range(0, flat.numel(), 7):
            was = float(flat[i])
            flat[i] = was + d
            up = loss(x, r, w)
            flat[i] = was - d
            down = loss(x, r, w)
            flat[i] = was
            assert abs((up - down) / (2 * d) - want[i]) < 1e-6


@pytest.mark.parametrize("T,W", [(1, 32), (9, 96), (257, 128), (3, 2048), (5, 4128), (64, 7168), (2, 12288), (1, 32768)])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_norm_mxfp8(T, W, dt):
    x, w, r = normal(1, T, W, dt=dt), normal(2, W, dt=dt), normal(3, T, W, dt=dt)
    x[:, :32] *= 2.0 ** -20
    r[:, :32] *= 2.0 ** -20
    w[-32:] = 0
    out = M.rms_norm(x, w, residual=r, quant="mxfp8")
    assert "y" not in out
    y, by, _, _ = norm_y(out["h"], w, 1e-6, dt)
    err = by - half_step(dt) * 1.01 * y.abs()
    check_mx(out["act_q"], out["act_scale"], y, err)
    v = M.mxfp8_values(out["act_q"], out["act_scale"], dt)
    want = e4m3_values(out["act_q"]).reshape(T, -1, 32) * \
        torch.exp2(out["act_scale"].cpu().double() - 127)[:, :, None]
    assert torch.equal(v.cpu(), want.reshape(T, W).to(dt))
    # beside y, and into the caller's memory: the same codes
    mine = {"y": torch.empty_like(x), "h": torch.empty_like(x)}
    both = M.rms_norm(x, w, residual=r, quant="mxfp8", out=mine)
    assert both is mine and "rstd" not in both
    assert torch.equal(both["act_q"], out["act_q"]) and torch.equal(both["act_scale"], out["act_scale"])
    assert_close(both["y"], y, by, "y")


def test_norm_mxfp8_is_the_routing_calls_form():
    """A norm that changes nothing (a mean square of 1, a weight of 1) writes the codes
    and scales that route_quant_local writes for the same activations."""
    T, H = 32, 2048
    g = torch.Generator(device="cuda").manual_seed(0)
    # pairs a, b with a^2 + b^2 = 2 and any signs: their sums are exact in fp32
    a = torch.where(torch.rand(T, H // 2, device="cuda", generator=g) < 0.5, 1.0, 0.2)
    b = torch.where(a == 1, 1.0, 1.4)  # 0.04 + 1.96
    sign = torch.where(torch.rand(T, H, device="cuda", generator=g) < 0.5, 1.0, -1.0)
    x = (torch.stack([a, b], 2).view(T, H) * sign).to(BF)
    one = torch.ones(H, dtype=BF, device="cuda")
    eps = float(1 - x[0].double().square().mean())  # what the rounding of 0.2 and 1.4 takes away
    out = M.rms_norm(x, one, eps=max(eps, 0.0), quant="mxfp8")
    logits = torch.randn(T, 896, device="cuda", generator=g)
    q = M.route_quant_local(logits, torch.zeros(896, device="cuda"), x, 0, 112)
    check_mx(q["act_q"], q["act_scale"], x.double().cpu(), torch.zeros(T, H, dtype=torch.float64))
    assert torch.equal(q["act_q"], out["act_q"]) and torch.equal(q["act_scale"], out["act_scale"])
    v = M.mxfp8_values(q["act_q"], q["act_scale"])
    assert float((v - x).abs().max()) <= 2.0 ** -4 * 1.4


def test_mxfp8_values_of_all_codes():
    q = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).repeat(256, 1).contiguous()
    scale = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8)[:, None].repeat(1, 8).contiguous()
    for dt in (BF, FP):
        v = M.mxfp8_values(q, scale, dt).cpu()
        exact = e4m3_values(q) * torch.exp2(scale[:, :1].cpu().double() - 127)
        exact[255] = float("nan")
        want = exact.float().to(dt)  # fp32 holds every one of them, or overflows in both
        assert torch.equal(torch.isnan(v), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(v[fine], want[fine])


def test_norm_special_values():
    """Rows of zeros give zeros and finite gradients (eps > 0); NaN and infinities stay
    in their rows, and dropped ones have no effect."""
    W = 512
    x, w = normal(1, 4, W, dt=BF), torch.ones(W, dtype=BF, device="cuda")
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 6] = float("inf")
    out = M.rms_norm(x, w, quant="mxfp8", out={"y": torch.empty_like(x), "rstd": torch.empty(4, device="cuda")})
    assert bool((out["y"][0] == 0).all()) and bool((out["act_q"][0] & 0x7F == 0).all())
    assert bool((out["act_scale"][0] == 0).all())
    assert bool(torch.isnan(out["y"][1]).all()) and bool((out["act_q"][1] & 0x7F == 0x7F).all())
    assert bool(torch.isnan(out["y"][2, 6])) and bool((out["y"][2, :6] == 0).all())
    assert bool(torch.isfinite(out["y"][3]).all())
    dy = normal(2, 4, W, dt=BF)
    g = M.rms_norm_backward(dy[:1], x[:1], w, out["rstd"][:1])
    assert bool(torch.isfinite(g["dx"]).all())
    # dropped everywhere: h is the residual whatever x holds
    r = normal(3, 4, W, dt=BF)
    h = M.rms_norm(x, w, residual=r, p=1.0, rng=rng_tensor())["h"]
    assert torch.equal(h, r)
    kept = torch.from_numpy(numbers(*RNG, 0, 4, W) >= 32768)
    x[~kept.cuda()] = float("nan")
    v = M.dropout(x, 0.5, rng_tensor())
    assert bool((v[~kept.cuda()] == 0).all())


@pytest.mark.parametrize("W", [5, 130, 1001, 2056, 7168, 20000])
def test_norm_of_squares_outside_fp32(W):
    """bf16 rows whose squares overflow or vanish, between ordinary ones."""
    T = 37
    x = normal(1, T, W, dt=BF)
    size = torch.tensor([1.0, 2.0 ** 70, 2.0 ** 118, 2.0 ** -70, 2.0 ** -110, 2.0 ** 62, 2.0 ** -50], device="cuda")[torch.arange(T, device="cuda") % 7]
    x = (x.float() * size[:, None]).to(BF)
    weight = normal(2, W, dt=BF)
    for eps in (0.0, 1e-6, 1e-35):
        out = M.rms_norm(x, weight, eps=eps)
        y, bound, rstd, rbound = norm_y(x, weight, eps, BF)
        assert bool(((out["rstd"].double().cpu() - rstd).abs() <= rbound).all()), eps
        assert bool(((out["y"].double().cpu() - y).abs() <= bound).all()), eps


def test_norm_large_values_in_fp16():
    """The squares of fp16's largest values pass its range; fp32 sums hold them."""
    x = torch.full((2, 7168), 60000.0, dtype=FP, device="cuda")
    w = torch.ones(7168, dtype=FP, device="cuda")
    assert bool((M.rms_norm(x, w)["y"] == 1).all())


@pytest.mark.parametrize("T,W", [(1, 1), (3, 5), (17, 8), (300, 100), (33, 2047), (1, 40000), (5000, 64), (70000, 9)])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.9, 1.0])
def test_dropout(T, W, dt, p):
    x, r = normal(1, T, W, dt=dt), normal(2, T, W, dt=dt)
    for res in (None, r):
        want = drop(x.double().cpu(), p, RNG, 77)
        size = want.abs()
        if res is not None:
            want = want + res.double().cpu()
            size = size + res.double().cpu().abs()
        bound = half_step(dt) * want.abs() * 1.01 + 3 * F32 * size + TINY[dt]
        got = M.dropout(x, p, rng_tensor(), site=77, residual=res)
        assert_close(got, want, bound, "out")
    assert torch.equal(M.dropout_backward(x, p, rng_tensor(), site=77),
                       M.dropout(x, p, rng_tensor(), site=77))


def test_dropout_numbers_are_the_generators():
    """Known answers of Philox4x32-10 (the authors' published test vectors) in the
    oracle: a counter of zeros with a key of zeros, and all ones."""
    z = numbers(0, 0, 0, 1, 8)[0]
    assert [int(v) for v in z.view(np.uint32)] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def test_dropout_share_and_independence():
    """The share of kept elements, and of pairs kept by two sites, seeds, offsets or
    rows, is within 6 standard deviations."""
    T, W, p = 512, 4096, 0.25
    one = torch.ones(T, W, dtype=BF, device="cuda")

    def kept(rng=RNG, site=0):
        return M.dropout(one, p, rng_tensor(rng), site=site) != 0
    a = kept()
    n = T * W

    def near(share, q, n):
        return abs(float(share) - q) < 6 * (q * (1 - q) / n) ** 0.5
    assert near(a.float().mean(), 1 - p, n)
    q = (1 - p) ** 2
    for b in (kept(site=1), kept((RNG[0] + 1, RNG[1])), kept((RNG[0], RNG[1] + 1)), kept((RNG[0], RNG[1] + (1 << 32))), a.roll(1, 0), a.roll(1, 1), a.roll(8, 1)):
        assert near((a & b).float().mean(), q, n)


def test_strides_and_alignment():
    """Rows further apart than they are long, and pointers at any element."""
    T, W = 37, 515
    for dt in (BF, FP):
        def odd(seed):
            base = normal(seed, T, W + 14, dt=dt)
            return base[:, 3:3 + W]
        x, r, dy, dh = odd(1), odd(2), odd(3), odd(4)
        w = normal(5, W + 1, dt=dt)[1:]
        guard = torch.full((T, W + 6), 7.0, dtype=dt, device="cuda")
        out = {"y": guard[:, 1:1 + W], "h": torch.empty(T, W + 3, dtype=dt, device="cuda")[:, :W],
               "rstd": torch.empty(T, device="cuda")}
        M.rms_norm(x, w, residual=r, out=out)
        flat = M.rms_norm(x.contiguous(), w.clone(), residual=r.contiguous())
        for k in ("y", "h", "rstd"):
            assert torch.equal(out[k], flat[k])
        assert bool((guard[:, 0] == 7).all()) and bool((guard[:, 1 + W:] == 7).all())
        guard.fill_(7)
        g = M.rms_norm_backward(dy, out["h"], w, out["rstd"], dh=dh,
                                out={"dx": guard[:, 1:1 + W], "dweight": torch.empty(W + 1, dtype=dt, device="cuda")[1:]})
        f = M.rms_norm_backward(dy.contiguous(), flat["h"], w.clone(), flat["rstd"], dh=dh.contiguous())
        assert torch.equal(g["dx"], f["dx"]) and torch.equal(g["dweight"], f["dweight"])
        assert bool((guard[:, 0] == 7).all()) and bool((guard[:, 1 + W:] == 7).all())
        assert torch.equal(M.dropout(x, 0.3, rng_tensor(), residual=r),
                           M.dropout(x.contiguous(), 0.3, rng_tensor(), residual=r.contiguous()))


def test_in_place():
    T, W = 50, 1003
    x, r, w = normal(1, T, W, dt=BF), normal(2, T, W, dt=BF), normal(3, W, dt=BF)
    want = M.rms_norm(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    out = M.rms_norm(x2, w, residual=r2, out={"h": r2, "y": x2})
    assert torch.equal(out["h"], want["h"]) and torch.equal(out["y"], want["y"])
    d = M.dropout(x, 0.2, rng_tensor(), residual=r)
    x2, r2 = x.clone(), r.clone()
    assert torch.equal(M.dropout(x2, 0.2, rng_tensor(), residual=r2, out=r2), d)
    dy, dh = normal(4, T, W, dt=BF), normal(5, T, W, dt=BF)
    g = M.rms_norm_backward(dy, want["h"], w, want["rstd"], dh=dh)
    M.rms_norm_backward(dy, want["h"], w, want["rstd"], dh=dh, out={"dx": dh})
    assert torch.equal(dh, g["dx"])


def test_parts_of_the_outputs_and_no_tokens():
    T, W = 12, 96
    h, dy, w = normal(1, T, W, dt=BF), normal(2, T, W, dt=BF), normal(3, W, dt=BF)
    rstd = M.rms_norm(h, w)["rstd"]
    full = M.rms_norm_backward(dy, h, w, rstd)
    for k in ("dx", "dweight"):
        one = M.rms_norm_backward(dy, h, w, rstd, out={k: torch.empty_like(full[k])})
        assert list(one) == [k] and torch.equal(one[k], full[k])
    none = h[:0]
    out = M.rms_norm(none, w, residual=none, quant="mxfp8")
    assert out["h"].shape == (0, W) and out["act_q"].shape == (0, W)
    g = M.rms_norm_backward(none, none, w, rstd[:0])
    assert g["dx"].shape == (0, W) and bool((g["dweight"] == 0).all())
    assert M.dropout(none, 0.5, rng_tensor()).shape == (0, W)
    assert M.mxfp8_values(out["act_q"], out["act_scale"]).shape == (0, W)


def test_same_bits_every_time_and_on_another_stream():
    T, W = 3000, 1024
    h, dy, w, dh = (normal(k, *s, dt=BF) for k, s in enumerate([(T, W), (T, W), (W,), (T, W)]))
    rstd = M.rms_norm(h, w)["rstd"]
    first = M.rms_norm_backward(dy, h, w, rstd, dh=dh, p=0.1, rng=rng_tensor())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = M.rms_norm_backward(dy, h, w, rstd, dh=dh, p=0.1, rng=rng_tensor())
    again = M.rms_norm_backward(dy, h, w, rstd, dh=dh, p=0.1, rng=rng_tensor())
    torch.cuda.synchronize()
    for k in first:
        assert torch.equal(first[k], other[k]) and torch.equal(first[k], again[k])


def test_captured_step_draws_new_numbers():
    """Forward and backward captured with the offset's step: each replay drops by
    new numbers, forward and backward alike, as the eager calls with them do."""
    T, W, p = 64, 768, 0.3
    x, r, w, dy = normal(1, T, W, dt=BF), normal(2, T, W, dt=BF), normal(3, W, dt=BF), normal(4, T, W, dt=BF)
    rng = rng_tensor((5, 0))

    def step():
        f = M.rms_norm(x, w, residual=r, p=p, rng=rng, site=1)
        d = M.dropout(f["y"], p, rng, site=2)
        b = M.rms_norm_backward(dy, f["h"], w, f["rstd"], dh=d, p=p, rng=rng, site=1)
        rng[1] += 1
        return f, d, b
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, d, b = step()
    seen = []
    for k in range(4):
        rng.copy_(torch.tensor((5, 10 + k)))
        graph.replay()
        got = [t.clone() for t in (*f.values(), d, *b.values())]
        rng.copy_(torch.tensor((5, 10 + k)))
        ef, ed, eb = step()
        for a, e in zip(got, (*ef.values(), ed, *eb.values())):
            assert torch.equal(a, e)
        torch.cuda.synchronize()
        seen.append(got[1])
    assert not torch.equal(seen[0], seen[1])


def test_rows_beyond_32_bits_of_bytes():
    """More than 4 GB a matrix: the last rows."""
    T, W = 300_001, 7168
    x = torch.zeros(T, W, dtype=BF, device="cuda")
    x[-3:] = normal(1, 3, W, dt=BF)
    w = normal(2, W, dt=BF)
    out = M.rms_norm(x, w, quant="mxfp8", out={"y": torch.empty_like(x), "rstd": torch.empty(T, device="cuda")})
    y, by, rstd, br = norm_y(x[-3:], w, 1e-6, BF)
    assert_close(out["y"][-3:], y, by, "y")
    check_mx(out["act_q"][-3:], out["act_scale"][-3:], y, by)
    del out
    d = M.dropout(x, 0.5, rng_tensor(), out=x)
    keep = torch.from_numpy(numbers(*RNG, 0, T, 8)[-3:] >= 32768)
    assert bool((d[-3:, :8].cpu()[~keep] == 0).all()) and bool((d[-3:, :8].cpu()[keep] != 0).all())
