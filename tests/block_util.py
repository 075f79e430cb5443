"""Oracle of the norm, dropout and the 8-bit outputs in 64 bits, by numpy and
torch on the CPU, and the error bounds.

Bounds, with u = eps / 2 of the output's type and F32 = 2^-24:
  h        u |h| of the exact sum + F32 of the terms (the fp32 sum, and the
           product with 2^16 / (2^16 - level), whose factor is rounded too)
  rstd     the sum of W squares in fp32: (W + 8) F32 relative at most, half of it
           after the root; 4 F32 for the root, the division and eps' addition
  y        of the stored h: u |y| + (rstd's relative error + 4 F32) |y|
  dtotal   terms a = dh, b = rstd g, c = n mean(g n): u |ref| + F32 (8 |a| + 8 |b|)
           + F32 (W + 16) |n| rstd mean|g n|
  dweight  u |ref| + (T + 8) F32 sum |dy n|
"""
import numpy as np
import torch

from ffn_util import F32, TINY, half_step


def numbers(seed, offset, site, T, W):
    """The 16-bit numbers of a [T, W] matrix, Philox4x32-10."""
    seed, offset = int(seed) % 2 ** 64, int(offset) % 2 ** 64
    chunks, u = -(-W // 8), np.uint64
    low = u(0xFFFFFFFF)
    x = [np.broadcast_to(np.arange(chunks, dtype=u) + u(site << 17), (T, chunks)),
         np.broadcast_to(np.arange(T, dtype=u)[:, None], (T, chunks)),
         np.full((T, chunks), offset & 0xFFFFFFFF, u), np.full((T, chunks), offset >> 32, u)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p0, p1 = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(p1 >> u(32)) ^ x[1] ^ u(k0), p1 & low, (p0 >> u(32)) ^ x[3] ^ u(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    out = np.empty((T, chunks, 8), np.uint16)
    for i in range(8):
        out[:, :, i] = (x[i // 2] >> u(16 * (i % 2))).astype(np.uint16)
    return out.reshape(T, chunks * 8)[:, :W]


def drop(v, p, rng, site):
    """drop(v) of a float64 CPU matrix; rng: (seed, offset)."""
    level = int(round(p * 65536))
    if not level:
        return v
    keep = torch.from_numpy((numbers(*rng, site, *v.shape) >= level))
    times = 65536.0 / (65536 - level) if level < 65536 else 0.0
    return torch.where(keep, v * times, torch.zeros_like(v))


def norm_h(x, residual, p, rng, site, dt):
    """(h, bound) before the rounding to dt, float64 on the CPU."""
    v = drop(x.double().cpu(), p, rng, site)
    h = v if residual is None else v + residual.double().cpu()
    size = v.abs() + (0 if residual is None else residual.double().cpu().abs())
    return h, half_step(dt) * h.abs() * 1.01 + 3 * F32 * size + TINY[dt]


def norm_y(h, weight, eps, dt):
    """(y unrounded, bound of its rounded form, rstd, bound) from the stored h."""
    h, w = h.double().cpu(), weight.double().cpu()
    W = h.shape[1]
    mean = h.square().mean(1)
    rstd = 1 / torch.sqrt(mean + eps)
    e = (W + 8) / 2 * F32 + 4 * F32
    y = h * rstd[:, None] * w
    return y, (half_step(dt) * 1.01 + e + 4 * F32) * y.abs() + TINY[dt], rstd, e * rstd


def norm_grads(dy, h, weight, rstd, dh, dt):
    """{name: (value, bound)}: dtotal and dweight."""
    dy, h, w, r = (t.double().cpu() for t in (dy, h, weight, rstd))
    r = r[:, None]
    T, W = h.shape
    n, g = h * r, dy * w
    a = torch.zeros_like(dy) if dh is None else dh.double().cpu()
    b, m = r * g, (g * n).mean(1, keepdim=True)
    ref = a + b - r * n * m
    e = F32 * (8 * a.abs() + 8 * b.abs() + (W + 16) * r * n.abs() * (g * n).abs().mean(1, keepdim=True))
    s = (dy * n).sum(0)
    return {"dtotal": (ref, half_step(dt) * ref.abs() * 1.01 + e + TINY[dt]),
            "dweight": (s, half_step(dt) * s.abs() * 1.01 + (T + 8) * F32 * (dy * n).abs().sum(0) + TINY[dt])}


def e4m3_values(codes):
    """Real values of E4M3 codes (uint8 tensor), float64; NaN for 0x7F and 0xFF."""
    c = codes.to(torch.int64).cpu()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m * 2.0 ** -9)
    v = torch.where((c & 0x7F) == 0x7F, torch.full_like(v, float("nan")), v)
    return torch.where(c >= 128, -v, v)


def check_mx(q, scale, y, err):
    """q and scale against y (float64 [T, W], each known within err): the scale's
    exponent is that of the largest of 32 values, either one next to a power of two
    within err, and each element is within half a step of the value."""
    T, W = y.shape
    y, err = y.reshape(T, W // 32, 32), err.reshape(T, W // 32, 32)
    top, at = y.abs().max(2)
    shared = scale.to(torch.int64).cpu() - 127
    slack = err.amax(2)

    def exponent(v):
        return torch.where(v > 0, torch.floor(torch.log2(v.clamp(min=2.0 ** -1000))) - 8,
                           torch.full_like(v, -127.0)).clamp(min=-127).to(torch.int64)
    low, high = exponent((top - slack).clamp(min=0)), exponent(top + slack)
    assert bool(((shared >= low) & (shared <= high)).all()), "a scale is of another power of two"
    one = torch.exp2(shared.double())[:, :, None]
    v = (y / one)
    got = e4m3_values(q).reshape(T, W // 32, 32)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    over = (v.abs() - 448).clamp(min=0)  # saturated
    off = (got - v).abs() - over - step / 2 - err / one
    # next to a binade's upper end the rounded value's step is the larger one's half
    assert float(off.max()) <= 1e-12, f"an element is off by {float(off.max()):.3g} too much"


def normal(seed, *shape, dt, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)
