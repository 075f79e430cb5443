"""What is measured of the operators around the feed-forward block: the root-mean-square norm with the residual's
addition (outputs in 16 bits, or in 8 bits with a scale for each 32 values), dropout from a counter-based generator,
and the projection with the low-rank adapters of many requests beside it, forward and backward.

A case says its operator and direction:
  norm      h = residual + drop(x) (without a residual h is x itself), rounded to the type;
            y = h rstd weight with rstd = 1 / sqrt(mean(h^2) + eps); `mx` True: y as E4M3 values with a power of two for
            each 32 of them; backward: from dy, h, weight, rstd and dh, the gradient that reaches h from behind,
            the gradients of h (and of x, where it is dropped out) and of the weight
  dropout   out = residual + drop(x); backward: drop(dout)
  adapters  y = x W^T + bias + scale[a] (x A[a]^T) B[a]^T with a = ids[t], no adapter where that is negative; `save` True:
            also s = scale[a] x A[a]^T, which the backward pass reads; backward: dx, dA and dB (W is not trained)
drop(x) keeps element (t, c) where its 16-bit number is at least round(p 2^16), times 2^16 / (2^16 - round(p 2^16)). The
numbers are Philox4x32-10's (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011): 8 of them to a counter
(c / 8 + 2^17 site, t, offset), key seed, low halves first.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
SITE = 5


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the norm before the router for a decode batch: latency alone
        dict(name="norm_decode", op="norm", dir="forward", tokens=8, width=7168, dtype="bf16", residual=True, p=0.0, mx=False),
        # the same for a long prefill, with the activations that the experts take in 8 bits: memory traffic alone
        dict(name="norm_prefill_mx", op="norm", dir="forward", tokens=16384, width=7168, dtype="bf16", residual=True, p=0.0, mx=True),
        # a norm over short rows, as of the heads of a prefill's queries
        dict(name="norm_short_rows", op="norm", dir="forward", tokens=131071, width=128, dtype="fp16", residual=False, p=0.0, mx=False),
        # training: the block's own gradient and the residual stream's meet
        dict(name="norm_backward", op="norm", dir="backward", tokens=8192, width=7168, dtype="bf16", residual=True, p=0.0, mx=False),
        # training with dropout before the residual, at a width that is no multiple of any vector
        dict(name="norm_backward_odd", op="norm", dir="backward", tokens=1021, width=1001, dtype="fp16", residual=True, p=0.1, mx=False),
        # a block's output dropped out and added to the residual stream
        dict(name="dropout_prefill", op="dropout", dir="forward", tokens=8192, width=7168, dtype="bf16", residual=True, p=0.1),
        # its backward pass on a small odd batch: latency alone
        dict(name="dropout_backward_odd", op="dropout", dir="backward", tokens=333, width=2047, dtype="fp16", residual=False, p=0.25),
        # decode of 16 requests with adapters of their own: the shared weights streamed once, and each live adapter
        dict(name="adapters_decode", op="adapters", dir="forward", tokens=16, hidden=7168, out=2048, rank=16, adapters=64, requests=16, dtype="bf16", bias=False, save=False),
        # a larger decode batch on a wide output
        dict(name="adapters_decode_batch", op="adapters", dir="forward", tokens=128, hidden=2048, out=7168, rank=32, adapters=112, requests=128, dtype="fp16", bias=True, save=False),
        # prompts of 16 requests together: one large product, the adapters beside it
        dict(name="adapters_prefill", op="adapters", dir="forward", tokens=8192, hidden=7168, out=2048, rank=16, adapters=64, requests=16, dtype="bf16", bias=False, save=False),
        # training 8 adapters at once
        dict(name="adapters_backward", op="adapters", dir="backward", tokens=8192, hidden=2048, out=4096, rank=64, adapters=8, requests=24, dtype="bf16", bias=False, save=True),
        # training at sizes that are no multiple of any tile
        dict(name="adapters_backward_odd", op="adapters", dir="backward", tokens=1021, hidden=1000, out=1412, rank=12, adapters=3, requests=7, dtype="fp16", bias=False, save=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    # model widths: mostly multiples of 64, some of 8, a few odd
    v, kind = _log(rng, lo, hi), rng.random()
    return max(64, v // 64 * 64) if kind < 0.7 else max(8, v // 8 * 8) if kind < 0.9 else v


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm", "dropout", "adapters", "adapters", "adapters"])
        back = rng.random() < 0.4
        c = dict(op=op, dir="backward" if back else "forward", dtype=rng.choice(["bf16", "fp16"]))
        if op == "norm":
            short = rng.random() < 0.25
            c |= dict(tokens=_log(rng, 64, 262144) if short else _log(rng, 1, 32768), width=rng.choice([64, 96, 128, 192, 256]) if short else _width(rng, 256, 16384))
            c |= dict(residual=back or rng.random() < 0.6, p=0.0, mx=not back and c["width"] % 32 == 0 and rng.random() < 0.4)
            if c["residual"] and rng.random() < 0.3:
                c["p"] = rng.choice([0.05, 0.1, 0.5])
        elif op == "dropout":
            c |= dict(tokens=_log(rng, 1, 32768), width=_width(rng, 256, 16384), residual=not back and rng.random() < 0.6, p=rng.choice([0.05, 0.1, 0.25, 0.5]))
        else:
            decode = not back and rng.random() < 0.5
            t = _log(rng, 1, 256) if decode else _log(rng, 128, 8192)
            c |= dict(tokens=t, hidden=_width(rng, 256, 7168), out=_width(rng, 256, 7168), rank=rng.choice([4, 8, 8, 16, 16, 16, 32, 32, 64, 12, 7, 40]),
                      adapters=_log(rng, 1, 16) if back else _log(rng, 1, 128), requests=t if decode else min(t, _log(rng, 1, 64)), bias=not back and rng.random() < 0.3, save=back or rng.random() < 0.3)
        w = work(c)
        if w["bytes"] < 9.3e8 and w["flops"] < 2.4e11:
            return c


# ---------------------------------------------------------------------------------------------------- what a pass cannot do without

def _live(c):
    """Adapters that some token has, in expectation."""
    n = c["adapters"]
    return n * (1 - (1 - 7 / 8 / n) ** c["requests"])


def work(c):
    t = c["tokens"]
    if c["op"] == "norm":
        w = c["width"]
        if c["dir"] == "forward":
            return {"bytes": 2 * t * w * (4 if c["residual"] else 2) + 2 * w + 4 * t, "flops": 5 * t * w}
        return {"bytes": 2 * t * w * (5 if c["p"] else 4) + 4 * w + 4 * t, "flops": 11 * t * w}
    if c["op"] == "dropout":
        return {"bytes": 2 * t * c["width"] * (3 if c["residual"] else 2), "flops": 2 * t * c["width"]}
    i, o, r, live = c["hidden"], c["out"], c["rank"], _live(c)
    share = 7 / 8  # of the tokens have an adapter
    if c["dir"] == "forward":
        return {"bytes": 2 * (t * i + o * i + live * r * (i + o) + t * o) + (4 * t * r if c["save"] else 0), "flops": 2 * t * i * o + 2 * share * t * r * (i + o)}
    return {"bytes": 2 * (2 * t * i + t * o + o * i + live * r * (i + o) + c["adapters"] * r * (i + o)) + 4 * t * r, "flops": 2 * t * i * o + 4 * share * t * r * (i + o)}


# ---------------------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[c["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device=DEV, dtype=dt, generator=g).mul_(scale)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, device=DEV, generator=g)

    s, t = dict(case=dict(c)), c["tokens"]
    if c["op"] in ("norm", "dropout"):
        w = c["width"]
        s["rng"] = torch.cat([whole(0, 1 << 62, 1), whole(0, 1 << 40, 1)])  # seed, offset
        s["residual"] = None
        if c["op"] == "dropout":
            s["x"] = normal(t, w)
            s["residual"] = normal(t, w, scale=4.0) if c["residual"] else None
            return s
        s["weight"] = (1 + 0.2 * torch.randn(w, device=DEV, generator=g)).to(dt)
        if c["dir"] == "forward":
            s["x"] = normal(t, w)
            # a residual stream has a few columns that are much larger than the others
            big = 1 + 20 * (whole(0, 256, w) == 0).to(dt)
            s["residual"] = normal(t, w, scale=4.0).mul_(big) if c["residual"] else None
            return s
        s["h"], s["dy"], s["dh"] = normal(t, w, scale=4.0), normal(t, w), normal(t, w)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        return s
    i, o, r, n, q = c["hidden"], c["out"], c["rank"], c["adapters"], c["requests"]
    # tokens of a request lie together; one request in eight has no adapter
    of = torch.where(whole(0, 8, q) == 0, torch.full((q,), -1, device=DEV), whole(0, n, q))
    if q == t:
        s["ids"] = of.int()
    else:
        cuts = torch.sort(whole(0, t, q - 1)).values
        s["ids"] = of[torch.searchsorted(cuts, torch.arange(t, device=DEV), right=True)].int()
    s["x"], s["w"] = normal(t, i), normal(o, i, scale=i ** -0.5)
    s["a"], s["b"] = normal(n, r, i, scale=i ** -0.5), normal(n, o, r, scale=0.3 * r ** -0.5)
    s["scale"] = 0.5 + 1.5 * torch.rand(n, device=DEV, generator=g)
    s["bias"] = normal(o, scale=0.1) if c["bias"] else None
    if c["dir"] == "backward":
        s["dy"] = normal(t, o)
        at = s["ids"].long()
        full = (s["x"].float() @ s["a"].float().view(n * r, i).T).view(t, n, r)
        s["s"] = torch.where(at[:, None] >= 0, full[torch.arange(t, device=DEV), at.clamp(min=0)] * s["scale"][at.clamp(min=0)][:, None], 0.0)
    return s


# ---------------------------------------------------------------------------------------------------- the framework's operators

def _own(s):
    import moe_expert_routing_amd as M
    c = s["case"]
    forward = c["dir"] == "forward"
    if c["op"] == "dropout":
        if forward:
            return {"out": M.dropout(s["x"], c["p"], s["rng"], site=SITE, residual=s["residual"])}
        return {"dx": M.dropout_backward(s["x"], c["p"], s["rng"], site=SITE)}
    if c["op"] == "norm":
        drop = dict(p=c["p"], rng=s["rng"], site=SITE) if c["p"] else {}
        if forward:
            r = M.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant="mxfp8" if c["mx"] else None, **drop)
            out = {"y": M.mxfp8_values(r["act_q"], r["act_scale"], s["x"].dtype) if c["mx"] else r["y"], "rstd": r["rstd"]}
            return out | {"h": r["h"]} if c["residual"] else out
        r = M.rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dh=s["dh"], **drop)
        out = {"dx": r["dx"], "dweight": r["dweight"]}
        return out | {"dresidual": r["dresidual"]} if c["p"] else out
    if forward:
        r = M.adapter_linear(s["x"], s["w"], s["a"], s["b"], s["ids"], scale=s["scale"], bias=s["bias"], save=c["save"])
        return {"y": r["y"], "s": r["s"]} if c["save"] else {"y": r["y"]}
    r = M.adapter_linear_backward(s["dy"], s["x"], s["w"], s["a"], s["b"], s["ids"], s["s"], scale=s["scale"])
    return {"dx": r["dx"], "da": r["da"], "db": r["db"]}


# ---------------------------------------------------------------------------------------------------- the plain forms, in 32 bits

def _round(k0, k1, x):
    # whole numbers below 2^32 in 64 bits: a product's low 64 bits are right, and so are both halves of them
    low = 0xFFFFFFFF
    p0, p1 = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
    return (p1 >> 32 & low) ^ x[1] ^ k0, p1 & low, (p0 >> 32 & low) ^ x[3] ^ k1, p0 & low


def _kept(s):
    """Which elements dropout keeps, and what they are multiplied with."""
    c, low = s["case"], 0xFFFFFFFF
    t, chunks = c["tokens"], (c["width"] + 7) // 8
    seed, offset = s["rng"][0], s["rng"][1]
    x = ((torch.arange(chunks, device=DEV) + (SITE << 17)).expand(t, chunks), torch.arange(t, device=DEV)[:, None].expand(t, chunks),
         (offset & low).expand(t, chunks), (offset >> 32 & low).expand(t, chunks))
    k = [((seed & low) + j * 0x9E3779B9 & low, (seed >> 32 & low) + j * 0xBB67AE85 & low) for j in range(10)]
    x = _round(*k[4], _round(*k[3], _round(*k[2], _round(*k[1], _round(*k[0], x)))))
    x = _round(*k[9], _round(*k[8], _round(*k[7], _round(*k[6], _round(*k[5], x)))))
    words = torch.stack(x, 2)
    u = torch.stack([words & 0xFFFF, words >> 16], 3).view(t, chunks * 8)[:, : c["width"]]
    level = round(c["p"] * 65536)
    return u >= level, 65536 / (65536 - level)


def _drop(s, v):
    if not s["case"]["p"]:
        return v
    kept, times = _kept(s)
    return torch.where(kept, v * times, 0.0)


def _e4m3(y, dt):
    """y as E4M3 values with a power of two for each 32 of them."""
    b = y.view(y.shape[0], -1, 32)
    top = torch.frexp(b.abs().amax(2, keepdim=True))
    shared = torch.where(top.mantissa > 0, top.exponent - 1 - 8, -127).clamp(min=-127)
    v = torch.ldexp(b, -shared).clamp(-448, 448)
    quantum = torch.frexp(v).exponent.clamp(min=-5) - 4  # of its binade; below 2^-6 the step stays
    return torch.ldexp(torch.round(torch.ldexp(v, -quantum)), quantum + shared).view(y.shape).to(dt)


def _norm(s):
    c, dt, w = s["case"], DT[s["case"]["dtype"]], s["weight"].float()
    if c["dir"] == "forward":
        h = (_drop(s, s["x"].float()) + s["residual"].float()).to(dt) if c["residual"] else s["x"]
        f = h.float()
        rstd = torch.rsqrt(f.square().mean(1) + EPS)
        y = f * rstd[:, None] * w
        out = {"y": _e4m3(y, dt) if c["mx"] else y.to(dt), "rstd": rstd}
        return out | {"h": h} if c["residual"] else out
    f, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    n = f * rstd
    g = dy * w
    d = rstd * (g - n * (g * n).mean(1, keepdim=True)) + s["dh"].float()
    out = {"dx": _drop(s, d).to(dt), "dweight": (dy * n).sum(0).to(dt)}
    return out | {"dresidual": d.to(dt)} if c["p"] else out


def _dropout(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    v = _drop(s, s["x"].float())
    if c["dir"] == "backward":
        return {"dx": v.to(dt)}
    return {"out": (v + s["residual"].float() if c["residual"] else v).to(dt)}


def _adapters(s):
    c, dt = s["case"], DT[s["case"]["dtype"]]
    i, o, r, n, t = c["hidden"], c["out"], c["rank"], c["adapters"], c["tokens"]
    x, w = s["x"].float(), s["w"].float()
    a, b = s["a"].float().view(n * r, i), s["b"].float().transpose(0, 1).reshape(o, n * r)
    # every token against every adapter, and those that are not its own left out
    times = (s["ids"][:, None] == torch.arange(n, device=DEV)) * s["scale"]
    mine = times[:, :, None].expand(t, n, r).reshape(t, n * r)
    if c["dir"] == "forward":
        every = (x @ a.T) * mine
        y = x @ w.T + every @ b.T
        if c["bias"]:
            y = y + s["bias"].float()
        return {"y": y.to(dt), "s": every.view(t, n, r).sum(1)} if c["save"] else {"y": y.to(dt)}
    dy = s["dy"].float()
    u = (dy @ b) * mine
    every = s["s"].repeat(1, n) * (mine != 0)
    return {"dx": (dy @ w + u @ a).to(dt), "da": (u.T @ x).view(n, r, i).to(dt), "db": (dy.T @ every).view(o, n, r).transpose(0, 1).to(dt).contiguous()}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "dropout": _dropout, "adapters": _adapters}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------- the definition, in 64 bits

def _numbers(seed, offset, t, w):
    """The generator's 16-bit numbers of a matrix, by numpy."""
    chunks, u = -(-w // 8), np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    ctr = [np.broadcast_to(np.arange(chunks, dtype=u) + u(SITE * 2 ** 17), (t, chunks)), np.broadcast_to(np.arange(t, dtype=u)[:, None], (t, chunks)),
           np.full((t, chunks), offset % 2 ** 32, u), np.full((t, chunks), offset >> 32, u)]
    key = [seed % 2 ** 32, seed >> 32]
    for _ in range(10):
        first, second = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = [(second >> half) ^ ctr[1] ^ u(key[0]), second & low, (first >> half) ^ ctr[3] ^ u(key[1]), first & low]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    words = np.stack([v.astype(np.uint32) for v in ctr], 2)
    return np.ascontiguousarray(words).view(np.uint16).reshape(t, chunks * 8)[:, :w]  # little-endian: low halves first


def exact(case, seed):
    s, c, d = prepare(case, seed), case, torch.float64
    t = c["tokens"]

    def dropped(v):
        if not c["p"]:
            return v
        numbers = _numbers(int(s["rng"][0]), int(s["rng"][1]), t, c["width"])
        level = int(round(c["p"] * 65536))
        keep = torch.from_numpy(numbers >= level).to(DEV)
        v = v * (65536.0 / (65536 - level))
        v[~keep] = 0
        return v

    if c["op"] == "dropout":
        v = dropped(s["x"].to(d))
        if c["dir"] == "backward":
            return {"dx": v}
        return {"out": v if s["residual"] is None else s["residual"].to(d) + v}
    if c["op"] == "norm":
        w = s["weight"].to(d)
        if c["dir"] == "forward":
            # the norm is of the h that is stored
            total = s["x"].to(d) if s["residual"] is None else s["residual"].to(d) + dropped(s["x"].to(d))
            h = total.to(DT[c["dtype"]]).to(d)
            rstd = 1 / torch.sqrt((h * h).sum(1) / c["width"] + EPS)
            y = h * (rstd[:, None] * w)
            if c["mx"]:
                v = y.reshape(-1, 32)
                most = v.abs().max(1, keepdim=True).values
                one = torch.exp2(torch.where(most > 0, torch.floor(torch.log2(most)) - 8, -127.0).clamp(min=-127.0))
                v = v / one
                step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
                y = ((torch.round(v / step) * step).clamp(-448.0, 448.0) * one).reshape(y.shape)
            out = {"y": y, "rstd": rstd}
            return out | {"h": total} if c["residual"] else out
        h, dy, rstd = s["h"].to(d), s["dy"].to(d), s["rstd"].to(d)[:, None]
        g = dy * w
        along = (g * h).sum(1, keepdim=True) / c["width"]
        total = s["dh"].to(d) + g * rstd - h * (rstd ** 3 * along)
        out = {"dx": dropped(total.clone()), "dweight": (dy * (h * rstd)).sum(0)}
        return out | {"dresidual": total} if c["p"] else out
    ids, scale = s["ids"].long(), s["scale"].to(d)
    x, w, r = s["x"].to(d), s["w"].to(d), c["rank"]
    if c["dir"] == "forward":
        y = x @ w.T
        inner = torch.zeros(t, r, dtype=d, device=DEV)
        for e in range(c["adapters"]):
            at = torch.nonzero(ids == e).reshape(-1)
            if at.numel():
                inner[at] = scale[e] * (x[at] @ s["a"][e].to(d).T)
                y[at] += inner[at] @ s["b"][e].to(d).T
        if s["bias"] is not None:
            y += s["bias"].to(d)
        return {"y": y, "s": inner} if c["save"] else {"y": y}
    dy = s["dy"].to(d)
    dx = dy @ w
    da, db = torch.zeros(*s["a"].shape, dtype=d, device=DEV), torch.zeros(*s["b"].shape, dtype=d, device=DEV)
    for e in range(c["adapters"]):
        at = torch.nonzero(ids == e).reshape(-1)
        if at.numel():
            u = scale[e] * (dy[at] @ s["b"][e].to(d))
            dx[at] += u @ s["a"][e].to(d)
            da[e], db[e] = u.T @ x[at], dy[at].T @ s["s"][at].to(d)
    return {"dx": dx, "da": da, "db": db}
