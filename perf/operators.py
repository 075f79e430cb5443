"""What is measured of the feed-forward operators: the gated feed-forward block, the linear product with its
epilogue and the combination of the experts' rows, each dense or over routed experts, forward and backward.

A case says its operator and direction:
  gated    h = act(x Wg^T) * (x Wu^T); `pre` True: also the pre-activations [x Wg^T, x Wu^T] that the backward pass reads;
           backward: from dh, pre, x, Wg, Wu the gradients dx, dWg, dWu
  linear   y = act(x W^T + bias) + residual; backward: dx, dW and, with a bias, dbias
  combine  out[t] = residual[t] + sum_k w[t, k] y[row(t, k)]; backward: dy and dw
`experts` 0 is the dense form. Above 0 it is the number of experts whose weights are here, out of `routed` experts
that every token chooses `top_k` of; the rows are in expert order, each expert's padded to `tile`. The program's
buffers have a fixed number of rows, more than the experts here usually need: rows without an entry of theirs are zero.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    e = dict(experts=112, routed=896, top_k=16)
    d = dict(experts=0, routed=0, top_k=0, tile=0)
    return [
        # a shared expert's up projections for one decoded token: the smallest call, two weight matrices streamed once
        dict(name="gated_decode_one", op="gated", dir="forward", tokens=1, hidden=7168, inter=2048, dtype="bf16", act="silu", pre=False, **d),
        # 16 decoded tokens on one of eight expert-parallel ranks: about 28 of its 112 experts get a row or two
        dict(name="gated_decode_experts", op="gated", dir="forward", tokens=16, hidden=7168, inter=1024, dtype="bf16", act="silu", pre=False, tile=16, **e),
        # a shared expert over a prefill chunk in training: the pre-activations are kept for the backward pass
        dict(name="gated_prefill_train", op="gated", dir="forward", tokens=4096, hidden=7168, inter=2048, dtype="bf16", act="silu", pre=True, **d),
        # one rank's experts over a prefill chunk: about 150 rows an expert, unevenly
        dict(name="gated_prefill_experts", op="gated", dir="forward", tokens=8192, hidden=2048, inter=1024, dtype="bf16", act="silu", pre=False, tile=128, **e),
        # a dense block's backward pass at sizes that are no multiple of any tile
        dict(name="gated_backward_odd", op="gated", dir="backward", tokens=1021, hidden=1000, inter=1412, dtype="fp16", act="gelu", pre=True, **d),
        # the backward pass of one rank's experts
        dict(name="gated_backward_experts", op="gated", dir="backward", tokens=8192, hidden=2048, inter=1024, dtype="bf16", act="silu", pre=True, tile=128, **e),
        # the down projection of one rank's experts in decode
        dict(name="linear_decode_experts", op="linear", dir="forward", tokens=16, hidden=1024, out=7168, dtype="bf16", act="none", bias=False, residual=False, tile=16, **e),
        # a prefill's projection with everything in its epilogue
        dict(name="linear_prefill", op="linear", dir="forward", tokens=8192, hidden=2048, out=7168, dtype="fp16", act="gelu", bias=True, residual=True, **d),
        # the backward pass of a projection with bias and activation
        dict(name="linear_backward", op="linear", dir="backward", tokens=4096, hidden=2048, out=4096, dtype="bf16", act="silu", bias=True, residual=False, **d),
        # the experts' rows of a decode batch summed into its tokens: latency alone
        dict(name="combine_decode", op="combine", dir="forward", tokens=8, hidden=7168, dtype="bf16", residual=True, tile=16, **e),
        # the same for a long prefill: memory traffic alone
        dict(name="combine_prefill", op="combine", dir="forward", tokens=32768, hidden=7168, dtype="bf16", residual=True, tile=128, **e),
        # its backward pass: the gradients of the rows and of the routing weights
        dict(name="combine_backward", op="combine", dir="backward", tokens=8192, hidden=7168, dtype="bf16", residual=True, tile=128, **e),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    # model widths: mostly multiples of 64, some of 8, a few odd
    v, kind = _log(rng, lo, hi), rng.random()
    return max(64, v // 64 * 64) if kind < 0.7 else max(8, v // 8 * 8) if kind < 0.9 else v


def draw(rng):
    while True:
        op = rng.choice(["gated", "gated", "linear", "linear", "combine"])
        back = rng.random() < 0.4
        c = dict(op=op, dir="backward" if back else "forward", tokens=_log(rng, 1, 8192), dtype=rng.choice(["bf16", "fp16"]))
        if op == "combine" or rng.random() < 0.5:
            n = rng.choice([8, 16, 32, 64, 112])
            c |= dict(experts=n, routed=n * rng.choice([1, 2, 8]), top_k=rng.choice([2, 4, 8, 16]), tile=16 if c["tokens"] <= 256 else rng.choice([64, 128, 256]))
            c["top_k"] = min(c["top_k"], n)
        else:
            c |= dict(experts=0, routed=0, top_k=0, tile=0)
        c["hidden"] = _width(rng, 256, 7168)
        if op == "gated":
            c |= dict(inter=_width(rng, 256, 4096), act=rng.choice(["silu", "gelu"]), pre=back or rng.random() < 0.5)
        elif op == "linear":
            c |= dict(out=_width(rng, 256, 7168), act=rng.choice(["none", "silu", "gelu"]), bias=rng.random() < 0.5, residual=not back and rng.random() < 0.5)
        else:
            c |= dict(residual=rng.random() < 0.5)
        w = work(c)
        if w["bytes"] < 1.5e9 and w["flops"] < 2e11 and _rows(c) * c["hidden"] < 4e8:
            return c


# ---------------------------------------------------------------------------------------------------- what a pass cannot do without

def _rows(c):
    """Expected rows: the tokens, or the entries that go to the experts here."""
    return c["tokens"] * c["top_k"] * c["experts"] / c["routed"] if c["experts"] else c["tokens"]


def _capacity(c):
    """Rows of the program's buffers: the expected entries with room for uneven routing, and every expert's padding."""
    r = _rows(c)
    return math.ceil(min(c["tokens"] * c["top_k"], 1.3 * r + 8 * math.sqrt(r)) / c["tile"]) * c["tile"] + c["experts"] * (c["tile"] - 1)


def work(c):
    t, r, h = c["tokens"], _rows(c), c["hidden"]
    # experts with at least one row, in expectation
    live = c["experts"] * (1 - (1 - c["top_k"] / c["routed"]) ** t) if c["experts"] else 1
    n_exp = max(1, c["experts"])
    xin = min(t, r) if c["experts"] and c["op"] == "gated" else r  # gathered rows are read once a token
    if c["op"] == "gated":
        f = c["inter"]
        if c["dir"] == "forward":
            return {"bytes": 2 * (xin * h + live * 2 * f * h + r * f + (2 * r * f if c["pre"] else 0)), "flops": 4 * r * f * h}
        return {"bytes": 2 * (r * f + 2 * r * f + xin * h + live * 2 * f * h + r * h + n_exp * 2 * f * h), "flops": 8 * r * f * h}
    if c["op"] == "linear":
        o = c["out"]
        if c["dir"] == "forward":
            return {"bytes": 2 * (r * h + live * o * h + r * o * (2 if c["residual"] else 1)), "flops": 2 * r * o * h}
        return {"bytes": 2 * (r * o * (1 if c["act"] == "none" else 2) + 2 * r * h + live * o * h + n_exp * o * h), "flops": 4 * r * o * h}
    if c["dir"] == "forward":
        return {"bytes": 2 * h * (r + t + (t if c["residual"] else 0)), "flops": 2 * r * h}
    return {"bytes": 2 * h * (2 * r + min(t, r)), "flops": 3 * r * h}


# ---------------------------------------------------------------------------------------------------- inputs

def _routing(c, g):
    """A routing call's outputs for one rank (its experts are ids 0 .. experts-1), and the grouped layout of them."""
    t, k, n, total, tile = c["tokens"], c["top_k"], c["experts"], c["routed"], c["tile"]
    score = torch.randn(t, total, device=DEV, generator=g) + 0.3 * torch.randn(total, device=DEV, generator=g)
    s, ids = torch.topk(score, k, dim=1)
    s = 1 / (1 + torch.exp(-s))
    n_out = n if n == total else (n + k + 3) // 4 * 4
    slot = torch.arange(k, device=DEV)
    local = ids if n == total else torch.where(ids < n, ids, n + slot)
    flat = local.reshape(-1)
    perm = torch.argsort(flat, stable=True)
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(t * k, device=DEV)
    counts = torch.bincount(flat, minlength=n_out)
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    offsets = torch.cat([zero, torch.cumsum(counts, 0)])
    padded = torch.cat([zero, torch.cumsum((counts + tile - 1) // tile * tile, 0)])
    rows = _capacity(c)
    row = inv - offsets[flat] + padded[flat]
    here = row < rows
    m_indices = torch.full((rows,), -1, dtype=torch.long, device=DEV)
    row_entry = torch.full((rows,), -1, dtype=torch.long, device=DEV)
    m_indices[row[here]] = flat[here]
    row_entry[row[here]] = torch.nonzero(here).reshape(-1)
    weights = s / s.sum(1, keepdim=True)
    bits = weights.to(torch.bfloat16).view(torch.int16).long() & 0xFFFF
    i = torch.int32
    return dict(topk_weights=weights, packed=((local << 16) | bits).to(i), counts=counts.to(i), offsets=offsets.to(i), inv_perm=inv.to(i),
                padded_offsets=padded.to(i), m_indices=m_indices.to(i), row_entry=row_entry.to(i))


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[c["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device=DEV, dtype=dt, generator=g).mul_(scale)

    s = dict(case=dict(c))
    lead = (c["experts"],) if c["experts"] else ()
    t, h = c["tokens"], c["hidden"]
    rows = t
    if c["experts"]:
        s["lay"] = _routing(c, g)
        rows = s["lay"]["m_indices"].shape[0]
    # rows of padding hold zeros, as the operators leave them
    m = s["lay"]["m_indices"] if c["experts"] else None
    real = ((m >= 0) & (m < c["experts"])).to(dt).unsqueeze(1) if c["experts"] else 1
    if c["op"] == "gated":
        f = c["inter"]
        s["x"] = normal(t, h)
        s["w_gate"], s["w_up"] = normal(*lead, f, h, scale=h ** -0.5), normal(*lead, f, h, scale=h ** -0.5)
        if c["dir"] == "backward":
            s["pre"], s["dh"] = normal(rows, 2 * f) * real, normal(rows, f) * real
    elif c["op"] == "linear":
        o = c["out"]
        s["x"] = normal(rows, h) * real
        s["w"] = normal(*lead, o, h, scale=h ** -0.5)
        s["bias"] = normal(*lead, o, scale=0.1) if c["bias"] else None
        s["residual"] = normal(rows, o) if c["residual"] else None
        if c["dir"] == "backward":
            s["dy"] = normal(rows, o) * real
            s["pre"] = normal(rows, o) * real if c["act"] != "none" else None
    else:
        s["y"] = normal(rows, h) * real
        s["residual"] = normal(t, h) if c["residual"] else None
        if c["dir"] == "backward":
            s["dout"] = normal(t, h)
    return s


# ---------------------------------------------------------------------------------------------------- the framework's operators

def _own(s):
    import moe_expert_routing_amd as M
    c = s["case"]
    if c["op"] == "combine":
        if c["dir"] == "forward":
            return {"out": M.combine(s["y"], s["lay"], num_experts=c["experts"], residual=s["residual"])}
        r = M.combine_backward(s["dout"], s["y"], s["lay"], num_experts=c["experts"])
        return {"dy": r["dy"], "dweights": r["dweights"]}
    where = dict(lay=s["lay"], tile_m=c["tile"], top_k=c["top_k"]) if c["experts"] else {}
    if c["op"] == "gated":
        if c["dir"] == "forward":
            r = (M.expert_gated_ffn if where else M.gated_ffn)(s["x"], s["w_gate"], s["w_up"], activation=c["act"], save_pre=c["pre"], **where)
            return {"h": r["h"], "pre": r["pre"]} if c["pre"] else {"h": r["h"]}
        r = (M.expert_gated_ffn_backward if where else M.gated_ffn_backward)(s["dh"], s["pre"], s["x"], s["w_gate"], s["w_up"], activation=c["act"], **where)
        return {"dx": r["dx"], "dw_gate": r["dw_gate"], "dw_up": r["dw_up"]}
    where.pop("top_k", None)
    if c["dir"] == "forward":
        r = (M.expert_linear if where else M.linear)(s["x"], s["w"], bias=s["bias"], activation=c["act"], residual=s["residual"], **where)
        return {"y": r["y"]}
    r = (M.expert_linear_backward if where else M.linear_backward)(s["dy"], s["x"], s["w"], pre=s["pre"], activation=c["act"], bias_grad=c["bias"], **where)
    return {"dx": r["dx"], "dw": r["dw"], "dbias": r["dbias"]} if c["bias"] else {"dx": r["dx"], "dw": r["dw"]}


# ---------------------------------------------------------------------------------------------------- the plain forms, in 32 bits

def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _slope(z, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


class _Groups:
    """Rows to and from one padded matrix an expert, [experts, most rows of one, width]; the dense form is one group."""

    def __init__(self, s):
        c = s["case"]
        self.n = c["experts"]
        if self.n:
            lay = s["lay"]
            self.rows = lay["m_indices"].shape[0]
            self.at = torch.nonzero((lay["m_indices"] >= 0) & (lay["m_indices"] < self.n)).reshape(-1)
            self.e = lay["m_indices"][self.at].long()
            self.j = self.at - lay["padded_offsets"][self.e].long()
            self.cap = max(1, int(lay["counts"][: self.n].max()))
            self.token = lay["row_entry"][self.at].long() // c["top_k"]

    def split(self, v, by_token=False):
        if not self.n:
            return v.float().unsqueeze(0)
        out = torch.zeros(self.n, self.cap, v.shape[1], device=v.device)
        out[self.e, self.j] = v[self.token if by_token else self.at].float()
        return out

    def join(self, v, dt):
        if not self.n:
            return v[0].to(dt)
        out = torch.zeros(self.rows, v.shape[2], dtype=dt, device=v.device)
        out[self.at] = v[self.e, self.j].to(dt)
        return out

    def weight(self, w):
        return w.float() if self.n else w.float().unsqueeze(0)

    def weight_grad(self, dw, dt):
        return dw.to(dt) if self.n else dw[0].to(dt)


def _gated(s):
    c, q, dt = s["case"], _Groups(s), s["x"].dtype
    x = q.split(s["x"], by_token=True)
    wg, wu = q.weight(s["w_gate"]), q.weight(s["w_up"])
    if c["dir"] == "forward":
        g, u = torch.bmm(x, wg.transpose(1, 2)), torch.bmm(x, wu.transpose(1, 2))
        out = {"h": q.join(_act(g, c["act"]) * u, dt)}
        if c["pre"]:
            out["pre"] = q.join(torch.cat([g, u], 2), dt)
        return out
    f = c["inter"]
    dh, pre = q.split(s["dh"]), q.split(s["pre"])
    g, u = pre[..., :f], pre[..., f:]
    dg, du = dh * u * _slope(g, c["act"]), dh * _act(g, c["act"])
    return {"dx": q.join(torch.bmm(dg, wg) + torch.bmm(du, wu), dt),
            "dw_gate": q.weight_grad(torch.bmm(dg.transpose(1, 2), x), dt), "dw_up": q.weight_grad(torch.bmm(du.transpose(1, 2), x), dt)}


def _linear(s):
    c, q, dt = s["case"], _Groups(s), s["x"].dtype
    x, w = q.split(s["x"]), q.weight(s["w"])
    if c["dir"] == "forward":
        z = torch.bmm(x, w.transpose(1, 2))
        if c["bias"]:
            z = z + q.weight(s["bias"]).unsqueeze(-2 if q.n else 0)
        y = _act(z, c["act"])
        if c["residual"]:
            y = y + q.split(s["residual"])
        return {"y": q.join(y, dt)}
    dz = q.split(s["dy"])
    if c["act"] != "none":
        dz = dz * _slope(q.split(s["pre"]), c["act"])
    out = {"dx": q.join(torch.bmm(dz, w), dt), "dw": q.weight_grad(torch.bmm(dz.transpose(1, 2), x), dt)}
    if c["bias"]:
        out["dbias"] = q.weight_grad(dz.sum(1), dt)
    return out


def _combine(s):
    c, lay, dt = s["case"], s["lay"], s["y"].dtype
    t, k = lay["packed"].shape
    e = (lay["packed"] >> 16).long()
    row = lay["inv_perm"].long().view(t, k) - lay["offsets"][e].long() + lay["padded_offsets"][e].long()
    here = (e < c["experts"]) & (row < s["y"].shape[0])
    if c["dir"] == "forward":
        out = s["residual"].float() if c["residual"] else torch.zeros(t, c["hidden"], device=DEV)
        tok, slot = torch.nonzero(here, as_tuple=True)
        return {"out": out.index_add(0, tok, s["y"][row[tok, slot]].float() * lay["topk_weights"][tok, slot].unsqueeze(1)).to(dt)}
    tok, slot = torch.nonzero(here, as_tuple=True)
    r, w = row[tok, slot], lay["topk_weights"]
    d = s["dout"][tok].float()
    dy = torch.zeros_like(s["y"])
    dy[r] = (d * w[tok, slot].unsqueeze(1)).to(dt)
    dw = torch.zeros_like(w)
    dw[tok, slot] = (d * s["y"][r].float()).sum(1)
    return {"dy": dy, "dweights": dw}


def run(state):
    if own:
        return _own(state)
    return {"gated": _gated, "linear": _linear, "combine": _combine}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s, c, d = prepare(case, seed), case, torch.float64
    # [(weights' index, the rows' range or places, the tokens of these rows)], an expert at a time
    if c["experts"]:
        lay = s["lay"]
        starts, counts = lay["padded_offsets"].tolist(), lay["counts"].tolist()
        rows = lay["m_indices"].shape[0]
        groups = [(e, slice(starts[e], min(rows, starts[e] + counts[e]))) for e in range(c["experts"]) if counts[e] and starts[e] < rows]
        token = lay["row_entry"].long() // c["top_k"]
    else:
        groups, rows = [(Ellipsis, slice(0, c["tokens"]))], c["tokens"]

    def sigma(z):
        return torch.sigmoid(z)

    def phi(z):
        return 0.5 * torch.special.erfc(-z / math.sqrt(2))

    value = {"silu": lambda z: z * sigma(z), "gelu": lambda z: z * phi(z), "none": lambda z: z}
    slope = {"silu": lambda z: sigma(z) + z * sigma(z) * sigma(-z),
             "gelu": lambda z: phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), "none": torch.ones_like}

    def empty(*shape):
        return torch.zeros(*shape, dtype=d, device=DEV)

    if c["op"] == "combine":
        y, w, k = s["y"].to(d), s["lay"]["topk_weights"].to(d), c["top_k"]
        if c["dir"] == "forward":
            out = s["residual"].to(d) if c["residual"] else empty(c["tokens"], c["hidden"])
        else:
            dy, dw = torch.zeros_like(y), torch.zeros_like(w)
        for _, at in groups:  # a token has an expert at most once
            entry = s["lay"]["row_entry"][at].long()
            tok, slot = entry // k, entry % k
            if c["dir"] == "forward":
                out[tok] += w[tok, slot][:, None] * y[at]
            else:
                do = s["dout"][tok].to(d)
                dy[at] = w[tok, slot][:, None] * do
                dw[tok, slot] = torch.linalg.vecdot(do, y[at])
        return {"out": out} if c["dir"] == "forward" else {"dy": dy, "dweights": dw}

    value, slope = value[c["act"]], slope[c["act"]]
    if c["op"] == "gated":
        f = c["inter"]
        if c["dir"] == "forward":
            out = {"h": empty(rows, f)} | ({"pre": empty(rows, 2 * f)} if c["pre"] else {})
        else:
            out = {"dx": empty(rows, c["hidden"]), "dw_gate": empty(*s["w_gate"].shape), "dw_up": empty(*s["w_up"].shape)}
        for e, at in groups:
            x = s["x"][token[at] if c["experts"] else at].to(d)
            wg, wu = s["w_gate"][e].to(d), s["w_up"][e].to(d)
            if c["dir"] == "forward":
                g, u = x @ wg.T, x @ wu.T
                out["h"][at] = value(g) * u
                if c["pre"]:
                    out["pre"][at, :f], out["pre"][at, f:] = g, u
                continue
            g, u, dh = s["pre"][at, :f].to(d), s["pre"][at, f:].to(d), s["dh"][at].to(d)
            dg, du = dh * u * slope(g), dh * value(g)
            out["dx"][at] = dg @ wg + du @ wu
            out["dw_gate"][e], out["dw_up"][e] = dg.T @ x, du.T @ x
        return out
    if c["dir"] == "forward":
        out = {"y": empty(rows, c["out"])}
    else:
        out = {"dx": empty(rows, c["hidden"]), "dw": empty(*s["w"].shape)} | ({"dbias": empty(*s["bias"].shape)} if c["bias"] else {})
    for e, at in groups:
        x, w = s["x"][at].to(d), s["w"][e].to(d)
        if c["dir"] == "forward":
            z = x @ w.T
            z = z + s["bias"][e].to(d) if c["bias"] else z
            out["y"][at] = value(z) + s["residual"][at].to(d) if c["residual"] else value(z)
            continue
        dz = s["dy"][at].to(d) * slope(s["pre"][at].to(d)) if c["act"] != "none" else s["dy"][at].to(d)
        out["dx"][at], out["dw"][e] = dz @ w, dz.T @ x
        if c["bias"]:
            out["dbias"][e] = dz.sum(0)
    return out
