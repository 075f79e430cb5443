"""Oracle of the feed-forward operators in 64 bits (plain loops over experts,
on the tensors' own device), grouped layouts for tests, and the error bounds.

Bounds. A product's inputs are exact, its sum is fp32, its result is rounded
once to the output's type. With u = eps / 2 of that type, S the same sum over
absolute values and n the number of terms:
    |err| <= u |ref| + n 2^-24 S                         (a product)
    + u S where one factor was rounded before it         (backward products)
Activations are evaluated in fp32 with an error below ACT_ULP 2^-24 of their
largest intermediate. Subnormal results round to half the smallest subnormal.
"""
import math

import torch

import moe_expert_routing_amd as M

ACT_ULP = 32.0
F32 = 2.0 ** -24
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2))


def act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * phi(z)
    return z.clone()


def slope(z, name):
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def half_step(dt):
    return torch.finfo(dt).eps / 2


def groups(lay, n_exp, rows, top_k):
    """[(expert, rows, tokens)] of the experts here, rows past the buffers cut."""
    m = lay["m_indices"][:rows].cpu()
    entry = lay["row_entry"][:rows].cpu().long()
    out = []
    for e in range(n_exp):
        at = torch.nonzero(m == e).reshape(-1)
        out.append((e, at, entry[at] // top_k))
    return out


def assert_close(got, ref, bound, what):
    """|got - ref| <= bound elementwise; NaN and infinities have to agree."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    g = got.double().cpu()
    r, b = ref.double().cpu(), bound.double().cpu()
    fine = torch.isfinite(r)
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{what}: NaN in other places"
    assert torch.equal(g[~fine & ~torch.isnan(r)], r[~fine & ~torch.isnan(r)]), f"{what}: infinities"
    over = ((g - r).abs() - b)[fine]
    if over.numel():
        worst = int(over.argmax())
        assert float(over[worst]) <= 0, (
            f"{what}: off by {float((g - r).abs()[fine][worst]):.4g}, bound "
            f"{float(b[fine][worst]):.4g} at value {float(r[fine][worst]):.6g}")


def product_bound(ref, S, n, dt, rounded=False):
    u = half_step(dt)
    return u * ref.abs() * 1.01 + (n + 8) * F32 * S + (u * S * 1.01 if rounded else 0) + TINY[dt]


def local_layout(T, tile, *, e=128, top_k=8, off=0, cnt=0, seed=0, scale=1.0):
    """A routing call and its layout, by the framework: (lay, experts)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    logits = torch.randn(T, e, device="cuda", generator=g) * scale
    bias = 0.01 * torch.randn(e, device="cuda", generator=g)
    lay = M.route_local_grouped(logits, bias, off, cnt, tile_m=tile, top_k=top_k)
    return lay, (cnt if cnt and lay["num_experts_out"] != e else e)


def hand_layout(ids, n_ids, tile, rows=None):
    """The grouped layout of ids [T, K] (int64, 0 .. n_ids-1, one entry each), with
    uniform weights; rows beyond the entries are padding."""
    dev = "cuda"
    T, k = ids.shape
    flat = ids.reshape(-1).to(dev)
    perm = torch.argsort(flat, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=dev)
    counts = torch.bincount(flat, minlength=n_ids)
    zero = torch.zeros(1, dtype=torch.long, device=dev)
    offsets = torch.cat([zero, counts.cumsum(0)])
    padded = torch.cat([zero, ((counts + tile - 1) // tile * tile).cumsum(0)])
    rows = int(padded[-1]) if rows is None else rows
    row = inv - offsets[flat] + padded[flat]
    m = torch.full((rows,), -1, dtype=torch.int32, device=dev)
    entry = torch.full((rows,), -1, dtype=torch.int32, device=dev)
    here = row < rows
    m[row[here]] = flat[here].int()
    entry[row[here]] = torch.nonzero(here).reshape(-1).int()
    i = torch.int32
    return dict(counts=counts.to(i), offsets=offsets.to(i), padded_offsets=padded.to(i),
                m_indices=m, row_entry=entry, inv_perm=inv.to(i),
                packed=(flat.view(T, k) << 16).to(i),
                topk_weights=torch.full((T, k), 1.0 / k, device=dev))


def normal(seed, *shape, dt, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)


def gated_oracle(x, wg, wu, name, dt):
    """(h, pre) and their bounds for one expert's rows, 64-bit."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    n = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    Sg, Su = x.abs() @ wg.abs().T, x.abs() @ wu.abs().T
    h = act(g, name) * u
    eg, eu = (n + 8) * F32 * Sg, (n + 8) * F32 * Su
    # |act'| <= 1.13; the activation's own error is relative to its argument
    bh = half_step(dt) * h.abs() * 1.01 + 1.2 * eg * (u.abs() + eu) + \
        act(g, name).abs() * eu + ACT_ULP * F32 * g.abs() * u.abs() + TINY[dt]
    pre = torch.cat([g, u], 1)
    bp = half_step(dt) * pre.abs() * 1.01 + torch.cat([eg, eu], 1) + TINY[dt]
    return h, bh, pre, bp


def gated_grads(dh, pre, x, wg, wu, name, dt):
    """{name: (value, bound)} of one expert's gradients."""
    dh, pre, x, wg, wu = (t.double() for t in (dh, pre, x, wg, wu))
    F = wg.shape[0]
    g, u = pre[:, :F], pre[:, F:]
    dg, du = dh * u * slope(g, name), dh * act(g, name)
    # size of what dg and du are rounded relative to: their own, and the
    # activation's error relative to its terms
    ag = dg.abs() + 2 * ACT_ULP * F32 / half_step(dt) * (dh * u).abs() * (1 + g.abs()) + \
        TINY[dt] / half_step(dt)
    au = du.abs() + 2 * ACT_ULP * F32 / half_step(dt) * (dh * g).abs() + TINY[dt] / half_step(dt)
    out = {}
    ref = dg @ wg + du @ wu
    S = ag @ wg.abs() + au @ wu.abs()
    out["dx"] = (ref, product_bound(ref, S, 2 * F, dt, True))
    for k, d, a in (("dw_gate", dg, ag), ("dw_up", du, au)):
        ref, S = d.T @ x, a.T @ x.abs()
        out[k] = (ref, product_bound(ref, S, x.shape[0], dt, True))
    return out


def linear_oracle(x, w, bias, name, residual, dt):
    x, w = x.double(), w.double()
    n = x.shape[1] + 2
    z, S = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, S = z + bias.double(), S + bias.double().abs()
    ez = (n + 8) * F32 * S
    y = act(z, name)
    ey = ez if name == "none" else 1.2 * ez + ACT_ULP * F32 * z.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + F32 * (residual.double().abs() + act(z, name).abs())
    u = half_step(dt)
    return y, u * y.abs() * 1.01 + ey * 1.01 + TINY[dt], z, u * z.abs() * 1.01 + ez + TINY[dt]


def linear_grads(dy, pre, x, w, name, dt):
    dy, x, w = dy.double(), x.double(), w.double()
    s = torch.ones_like(dy) if name == "none" else slope(pre.double(), name)
    dz = dy * s
    u = half_step(dt)
    err = 0 if name == "none" else \
        2 * ACT_ULP * F32 * dy.abs() * (1 + pre.double().abs())
    a = dz.abs() + err / u + (0 if name == "none" else TINY[dt] / u)
    out = {}
    for k, ref, S, n in (("dx", dz @ w, a @ w.abs(), w.shape[0]),
                         ("dw", dz.T @ x, a.T @ x.abs(), x.shape[0])):
        out[k] = (ref, product_bound(ref, S, n, dt, name != "none"))
    ref = dz.sum(0)
    S = dz.abs().sum(0) + (err.sum(0) / F32 if name != "none" else 0) / (x.shape[0] + 8)
    out["dbias"] = (ref, product_bound(ref, S, x.shape[0], dt))
    return out
