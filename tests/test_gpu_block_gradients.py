"""GPU tests of what the library's backward passes write: against differences of the
forward formulas in 64 bits, and on rows whose squares leave fp32's range.

A central difference with step d of a smooth function is off by its third derivative
times d^2 / 6 and by 64-bit rounding over d: below 1e-6 here. The gradients' own bounds
are those of the tests against the formulas.
"""
import pytest
import torch

import moe_expert_routing_amd as M
from block_util import drop, norm_grads, normal
from ffn_util import F32, TINY, assert_close, half_step

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
DEV = "cuda"
RNG = (12345, 678)


def differences(loss, tensors, d=1e-4):
    """The gradient of loss() in each tensor (float64 on the CPU, changed in place)."""
    out = []
    for t in tensors:
        g = torch.zeros_like(t)
        flat, to = t.view(-1), g.view(-1)
        for i in range(flat.numel()):
            was = float(flat[i])
            flat[i] = was + d
            up = float(loss())
            flat[i] = was - d
            to[i] = (up - float(loss())) / (2 * d)
            flat[i] = was
        out.append(g)
    return out


@pytest.mark.parametrize("p", [0.0, 0.5])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_norm(dt, p):
    T, W, eps, site = 3, 40, 1e-2, 7
    g = torch.Generator().manual_seed(4)
    # quarters, whose sums and doubles both types hold: h is not rounded
    x, r = (torch.randint(-8, 9, (T, W), generator=g).double() / 4 for _ in range(2))
    w, gy, gh = (torch.randn(*s, generator=g).to(dt).double() for s in ((W,), (T, W), (T, W)))

    def loss():
        h = r + drop(x, p, RNG, site)
        return ((h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * w) * gy + h * gh).sum()
    dx, dr, dw = differences(loss, (x, r, w))
    rng = torch.tensor(RNG, dtype=torch.int64, device=DEV)
    put = lambda t: t.to(dt).to(DEV)  # noqa: E731
    kw = dict(p=p, rng=rng, site=site) if p else {}
    f = M.rms_norm(put(x), put(w), residual=put(r), eps=eps, **kw)
    h = r + drop(x, p, RNG, site)
    assert torch.equal(f["h"].double().cpu(), h)
    b = M.rms_norm_backward(put(gy), f["h"], put(w), f["rstd"], dh=put(gh), **kw)
    bound = norm_grads(gy, h, w, f["rstd"], gh, dt)
    # rstd is the forward pass's, (W + 16) F32 off at most, and its error times what it multiplies
    more = 1e-6 + (W + 16) * F32 * (dr.abs() + gh.abs()).max()
    assert_close(b["dresidual" if p else "dx"], dr, bound["dtotal"][1] + more, "dresidual")
    assert_close(b["dx"], dx, 2 * bound["dtotal"][1] + 2 * more, "dx")
    assert_close(b["dweight"], dw, bound["dweight"][1] + 1e-6 + (W + 16) * F32 * dw.abs().max(), "dweight")


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_dropout(dt):
    """out is linear in x: a step of 1 in x changes it by what the backward pass says."""
    T, W = 9, 77
    g = torch.Generator(device=DEV).manual_seed(4)
    x, one = (torch.randint(lo, 9, (T, W), device=DEV, generator=g).to(dt) for lo in (-8, 8))
    one = one / 8
    rng = torch.tensor(RNG, dtype=torch.int64, device=DEV)
    step = M.dropout(x + one, 0.5, rng, site=3) - M.dropout(x, 0.5, rng, site=3)
    assert torch.equal(step, M.dropout_backward(one, 0.5, rng, site=3)) and bool((step == 2).any()) and bool((step == 0).any())


@pytest.mark.parametrize("T", [7, 61])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_adapters(dt, T):
    I, O, R, n = 12, 10, 5, 3
    g = torch.Generator().manual_seed(T)
    x, w, a, b, gy = (torch.randn(*s, generator=g).to(dt).double() for s in ((T, I), (O, I), (n, R, I), (n, O, R), (T, O)))
    ids = torch.randint(-1, n + 1, (T,), generator=g)
    has = ((ids >= 0) & (ids < n)).double()
    at = ids.clamp(0, n - 1)
    c = torch.tensor([0.5, 2.0, -1.25])

    def loss():
        s = c.double()[at][:, None] * (x[:, None] @ a[at].transpose(1, 2))[:, 0] * has[:, None]
        return ((x @ w.T + (b[at] @ s[:, :, None])[:, :, 0]) * gy).sum()
    dx, da, db = differences(loss, (x, a, b))
    put = lambda t: t.to(dt).to(DEV)  # noqa: E731
    on = ids.int().to(DEV)
    f = M.adapter_linear(put(x), put(w), put(a), put(b), on, scale=c.to(DEV), save=True)
    got = M.adapter_linear_backward(put(gy), put(x), put(w), put(a), put(b), on, f["s"], scale=c.to(DEV))
    # every gradient is a sum of products of at most (I + O + R + T) terms, whose sizes' sum is at most S;
    # s and u are fp32 sums themselves
    S = {"dx": 2 * gy.abs().sum(1).max() * (w.abs().max() + (a.abs().sum(1).max() * b.abs().max())),
         "da": 2 * (gy.abs().sum(1) * x.abs().amax(1)).sum() * b.abs().max(),
         "db": 2 * (gy.abs().amax(1) * x.abs().sum(1)).sum() * a.abs().max()}
    for k, want in (("dx", dx), ("da", da), ("db", db)):
        assert_close(got[k], want, half_step(dt) * want.abs() * 1.01 + (I + O + R + T + 16) * F32 * S[k] + 1e-6 + TINY[dt], k)


@pytest.mark.parametrize("W", [5, 130, 1001, 2056, 7168, 20000])
def test_norm_backward_of_squares_outside_fp32(W):
    """bf16 rows whose squares overflow or vanish, between ordinary ones, with the rstd
    that the forward pass writes."""
    T = 37
    size = torch.tensor([1.0, 2.0 ** 70, 2.0 ** 118, 2.0 ** -70, 2.0 ** -110, 2.0 ** 62, 2.0 ** -50], device=DEV)[torch.arange(T, device=DEV) % 7]
    h = (normal(1, T, W, dt=torch.float32) * size[:, None]).to(BF)
    weight, dy, dh = normal(2, W, dt=BF), normal(3, T, W, dt=BF), normal(4, T, W, dt=BF)
    for eps in (0.0, 1e-6, 1e-35):
        rstd = M.rms_norm(h, weight, eps=eps)["rstd"]
        for more in (None, dh):
            out = M.rms_norm_backward(dy, h, weight, rstd, dh=more)
            want = norm_grads(dy, h, weight, rstd, more, BF)
            assert bool(torch.isfinite(want["dtotal"][0]).all())
            assert_close(out["dx"], *want["dtotal"], "dx")
            assert_close(out["dweight"], *want["dweight"], "dweight")
