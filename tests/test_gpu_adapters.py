"""GPU tests of the product with low-rank adapters against 64 bits.

Bounds, with u = eps / 2 of the output's type, F32 = 2^-24 and H the relative error of
an fp32 number in two halves of the type, (eps / 2)^2:
  s        (in + 8) F32 sum|c x a| + 2 F32 |s|
  y        u |y| + (in + rank + 8) F32 (sum|x w| + |s| |B|^T + |bias| + |residual|)
           + (error of s + H |s|) |B|^T
  dx       the same with u = c dy B in the place of s
  da, db   u |ref| + (tokens + 8) F32 S + (error of u + H |u|)^T |x|, and H |s| for db
In fp16 the halves are taken at a power of two of their own, which leaves 2^-38 of the
largest value beside a small one.
"""
import pytest
import torch

import moe_expert_routing_amd as M
from block_util import normal
from ffn_util import F32, TINY, assert_close, half_step

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
DEV = "cuda"


def split_error(v, dt):
    return half_step(dt) ** 2 * 1.01 * v.abs() + 2.0 ** -36 * v.abs().amax()


def inner(x, a, ids, scale):
    """(s, bound) with a [n, R, K]: c x a^T of each token's own adapter."""
    T, K = x.shape
    n, R = a.shape[:2]
    s = torch.zeros(T, R, dtype=torch.float64, device=DEV)
    S = torch.zeros_like(s)
    x = x.double()
    for e in range(n):
        at = torch.nonzero(ids == e).reshape(-1)
        if at.numel():
            c = 1.0 if scale is None else float(scale[e])
            s[at] = c * (x[at] @ a[e].double().T)
            S[at] = abs(c) * (x[at].abs() @ a[e].double().abs().T)
    return s, (K + 8) * F32 * S + 2 * F32 * s.abs() + 1e-42


def outer(s, es, b, ids, dt):
    """(s b^T, the sum of its terms' sizes, the error that s brings) with b [n, N, R]."""
    T, N = s.shape[0], b.shape[1]
    d = torch.zeros(T, N, dtype=torch.float64, device=DEV)
    S, E = torch.zeros_like(d), torch.zeros_like(d)
    for e in range(b.shape[0]):
        at = torch.nonzero(ids == e).reshape(-1)
        if at.numel():
            w = b[e].double()
            d[at] = s[at] @ w.T
            S[at] = s[at].abs() @ w.abs().T
            E[at] = (es[at] + split_error(s[at], dt)) @ w.abs().T
    return d, S, E


def check_forward(x, w, a, b, ids, scale, bias, res, out):
    dt, (T, K), R = x.dtype, x.shape, a.shape[1]
    s, es = inner(x, a, ids, scale)
    if "s" in out:
        assert_close(out["s"], s, es, "s")
    d, S, E = outer(s, es, b, ids, dt)
    y = x.double() @ w.double().T + d
    S = S + x.double().abs() @ w.double().abs().T
    for t in (bias, res):
        if t is not None:
            y, S = y + t.double(), S + t.double().abs()
    assert_close(out["y"], y, half_step(dt) * y.abs() * 1.01 + (K + R + 8) * F32 * S + E + TINY[dt], "y")


def check_backward(dy, x, w, a, b, ids, scale, s, out):
    dt, T, R = x.dtype, x.shape[0], a.shape[1]
    N = dy.shape[1]
    u, eu = inner(dy, b.transpose(1, 2), ids, scale)
    if "dx" in out:
        d, S, E = outer(u, eu, a.transpose(1, 2), ids, dt)
        ref = dy.double() @ w.double() + d
        S = S + dy.double().abs() @ w.double().abs()
        assert_close(out["dx"], ref, half_step(dt) * ref.abs() * 1.01 + (N + R + 8) * F32 * S + E + TINY[dt], "dx")
    for e in range(a.shape[0]):
        at = torch.nonzero(ids == e).reshape(-1)
        for name, left, err, right in (("da", u[at], eu[at], x[at].double()), ("db", s[at].double(), 0 * eu[at], dy[at].double())):
            if name not in out:
                continue
            ref, S = left.T @ right, left.abs().T @ right.abs()
            E = (err + split_error(left, dt) if at.numel() else err).T @ right.abs()
            bound = half_step(dt) * ref.abs() * 1.01 + (len(at) + 8) * F32 * S + E + TINY[dt]
            if name == "db":
                ref, bound = ref.T, bound.T
            assert_close(out[name][e], ref, bound, f"{name} of adapter {e}")


def make_ids(kind, T, n, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        ids = torch.full((T,), n - 1)
    elif kind == "none":
        ids = torch.full((T,), -1)
    elif kind == "each":  # a decode batch
        ids = torch.arange(T) % n
    elif kind == "random":  # some without, some out of range
        ids = torch.randint(-2, n + 2, (T,), generator=g)
    else:  # requests of any length
        cuts = torch.sort(torch.randint(0, T + 1, (max(1, T // 40),), generator=g)).values
        of = torch.randint(-1, n, (len(cuts) + 1,), generator=g)
        ids = of[torch.searchsorted(cuts, torch.arange(T), right=True)]
    return ids.int().to(DEV)


def problem(T, I, O, R, n, kind, dt, seed=0):
    x, w = normal(seed, T, I, dt=dt), normal(seed + 1, O, I, dt=dt, scale=I ** -0.5)
    a, b = normal(seed + 2, n, R, I, dt=dt, scale=I ** -0.5), normal(seed + 3, n, O, R, dt=dt, scale=R ** -0.5)
    scale = 0.5 + torch.rand(n, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))
    return x, w, a, b, make_ids(kind, T, n, seed), scale


# tokens of one block of the gradients that fill its list of tokens more than once,
# few rows of one, two and four 16s and of several groups of 64, the tiles of 32 to 256 rows, split ranges of k, widths of no tile
CASES = [(20000, 7168, 64, 8, 1, "one"), (100, 4096, 512, 16, 70, "each"), (200, 2100, 72, 12, 5, "random"), (128, 4096, 264, 8, 128, "each"), (150, 512, 1000, 16, 9, "each"), (40, 2048, 300, 24, 9, "requests"), (64, 96, 7168, 128, 64, "each"), (32, 1000, 33, 16, 2, "random"), (65, 4096, 128, 16, 65, "each"),
         (1, 64, 64, 16, 1, "one"), (1, 7168, 2048, 16, 4, "one"), (3, 1000, 17, 7, 5, "each"), (16, 512, 7168, 16, 16, "each"),
         (16, 129, 515, 1, 3, "random"), (17, 320, 200, 8, 17, "each"), (33, 1024, 96, 12, 40, "each"), (64, 7168, 1024, 16, 64, "each"),
         (100, 2000, 1001, 40, 6, "requests"), (257, 640, 768, 128, 3, "random"), (300, 96, 64, 17, 9, "requests"), (1000, 1000, 1412, 64, 5, "requests"),
         (1500, 256, 512, 32, 20, "each"), (4500, 512, 2304, 16, 7, "requests"), (4111, 777, 300, 100, 3, "random"), (5000, 64, 264, 33, 2, "none"),
         (6000, 320, 520, 64, 4, "requests"), (4200, 130, 260, 24, 5, "each")]


@pytest.mark.parametrize("T,I,O,R,n,kind", CASES)
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_forward(T, I, O, R, n, kind, dt):
    x, w, a, b, ids, scale = problem(T, I, O, R, n, kind, dt)
    out = M.adapter_linear(x, w, a, b, ids, scale=scale, save=True)
    check_forward(x, w, a, b, ids, scale, None, None, out)
    bias, res = normal(9, O, dt=dt), normal(10, T, O, dt=dt)
    out = M.adapter_linear(x, w, a, b, ids, bias=bias, residual=res)
    assert "s" not in out
    check_forward(x, w, a, b, ids, None, bias, res, out)


@pytest.mark.parametrize("T,I,O,R,n,kind", CASES)
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_backward(T, I, O, R, n, kind, dt):
    x, w, a, b, ids, scale = problem(T, I, O, R, n, kind, dt)
    dy = normal(11, T, O, dt=dt)
    s = inner(x, a, ids, scale)[0].float()
    out = M.adapter_linear_backward(dy, x, w, a, b, ids, s, scale=scale)
    check_backward(dy, x, w, a, b, ids, scale, s, out)
    for k in ("dx", "da", "db"):  # each alone gives the same bits
        one = M.adapter_linear_backward(dy, x, w, a, b, ids, s if k == "db" else None, scale=scale, out={k: torch.full_like(out[k], 5.0)})
        assert list(one) == [k]
        if k == "dx":
            assert torch.equal(one[k], out[k])
        else:
            check_backward(dy, x, w, a, b, ids, scale, s, one)


def test_gradients_are_the_differences():
    """The formulas of the gradients against central differences in 64 bits."""
    T, I, O, R, n = 5, 6, 4, 3, 2
    g = torch.Generator().manual_seed(3)
    x, w, a, b, gy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((T, I), (O, I), (n, R, I), (n, O, R), (T, O)))
    ids, c = torch.tensor([0, 1, -1, 1, 0]), [0.5, 2.0]

    def loss(x, a, b):
        y = x @ w.T
        for t in range(T):
            if ids[t] >= 0:
                y = y.index_add(0, torch.tensor([t]), (c[ids[t]] * (x[t] @ a[ids[t]].T) @ b[ids[t]].T)[None])
        return (y * gy).sum()
    dx, da, db = gy @ w, torch.zeros_like(a), torch.zeros_like(b)
    for t in range(T):
        e = int(ids[t])
        if e >= 0:
            u, s = c[e] * (gy[t] @ b[e]), c[e] * (x[t] @ a[e].T)
            dx[t] += u @ a[e]
            da[e] += torch.outer(u, x[t])
            db[e] += torch.outer(gy[t], s)
    h = 1e-5
    for t, want in ((x, dx), (a, da), (b, db)):
        flat = t.view(-1)
        for i in range(flat.numel()):
            was = float(flat[i])
            flat[i] = was + h
            up = loss(x, a, b)
            flat[i] = was - h
            down = loss(x, a, b)
            flat[i] = was
            assert abs((up - down) / (2 * h) - want.reshape(-1)[i]) < 1e-7


@pytest.mark.parametrize("T", [9, 200, 4500])
def test_infinities_and_nan_stay_in_their_requests(T):
    """One adapter full of NaN, another of infinities, and a NaN in a token's x and dy:
    the other requests' outputs and the other adapters' gradients are the same."""
    I, O, R, n = 256, 320, 16, 5
    for dt in (BF, FP):
        x, w, a, b, ids, scale = problem(T, I, O, R, n, "each", dt)
        dy, s = normal(11, T, O, dt=dt), normal(12, T, R, dt=torch.float32)
        clean = M.adapter_linear(x, w, a, b, ids, scale=scale)["y"]
        grads = M.adapter_linear_backward(dy, x, w, a, b, ids, s, scale=scale)
        a2, b2, x2, dy2, s2 = (t.clone() for t in (a, b, x, dy, s))
        a2[1], b2[1], a2[2], b2[2] = float("nan"), float("nan"), float("inf"), float("inf")
        x2[3, 5] = dy2[3, 7] = s2[3, 1] = float("nan")  # of adapter 3
        y = M.adapter_linear(x2, w, a2, b2, ids, scale=scale)["y"]
        fine = (ids == 0) | (ids == 4)
        assert torch.equal(y[fine], clean[fine])
        assert bool(torch.isnan(y[ids == 1]).all()) and bool(torch.isnan(y[3]).all())
        later = torch.nonzero(ids == 3).reshape(-1)[1:]
        assert torch.equal(y[later], clean[later])
        g = M.adapter_linear_backward(dy2, x2, w, a2, b2, ids, s2, scale=scale)
        assert torch.equal(g["dx"][fine], grads["dx"][fine])
        for e in (0, 4):
            assert torch.equal(g["da"][e], grads["da"][e]) and torch.equal(g["db"][e], grads["db"][e])


@pytest.mark.parametrize("T", [4, 300])
def test_inner_values_past_fp16(T):
    """s and u above fp16's range, with small factors behind them, and tiny ones."""
    I, O, R, n = 512, 256, 16, 2
    for size in (2.0 ** 9, 2.0 ** -9):
        x, w, a, b, ids, scale = problem(T, I, O, R, n, "each", FP)
        x, a = x * min(size, 16.0), a * size
        scale = scale * (64.0 if size > 1 else 2.0 ** -10)
        b = b * (2.0 ** -13 if size > 1 else 2.0 ** 8)
        out = M.adapter_linear(x, w, a, b, ids, scale=scale, save=True)
        if size > 1:
            assert float(out["s"].abs().max()) > 65504
        check_forward(x, w, a, b, ids, scale, None, None, out)
        dy = normal(4, T, O, dt=FP, scale=16.0 if size > 1 else 2.0 ** -6)
        b3 = normal(5, n, O, R, dt=FP, scale=64.0 if size > 1 else 2.0 ** -6)
        a3 = normal(6, n, R, I, dt=FP, scale=2.0 ** -13 if size > 1 else 1.0)
        x3 = normal(7, T, I, dt=FP, scale=2.0 ** -13 if size > 1 else 1.0)
        s3 = normal(8, T, R, dt=torch.float32, scale=2.0 ** 18 if size > 1 else 2.0 ** -20)
        dy3 = dy * 2.0 ** -12 if size > 1 else dy
        check_backward(dy, x3, w, a3, b3, ids, scale, s3, M.adapter_linear_backward(dy, x3, w, a3, b3, ids, s3, scale=scale, out={
            "dx": torch.empty_like(x3), "da": torch.empty_like(a3)}))
        check_backward(dy3, x3, w, a3, b3, ids, scale, s3, M.adapter_linear_backward(dy3, x3, w, a3, b3, ids, s3, scale=scale, out={
            "db": torch.empty_like(b3)}))


@pytest.mark.parametrize("T", [5, 150, 4300])
def test_strides_and_alignment(T):
    """Rows and adapters further apart than they are long, at any element, and nothing
    written beside the outputs."""
    I, O, R, n = 203, 301, 13, 4

    def inside(*shape, seed, dt):
        base = normal(seed, *shape[:-2], shape[-2] + 1, shape[-1] + 9, dt=dt)
        return base[..., :shape[-2], 3:3 + shape[-1]]
    for dt in (BF, FP):
        x, w, res, dy = (inside(*s, seed=k, dt=dt) for k, s in enumerate(((T, I), (O, I), (T, O), (T, O))))
        a, b = inside(n, R, I, seed=5, dt=dt) * 0.1, inside(n, O, R, seed=6, dt=dt)
        a = torch.cat([a, a], 1)[:, :R]  # adapters 2 R rows apart
        ids = make_ids("random", T, n, 1)
        guard = torch.full((T, O + 6), 7.0, dtype=dt, device=DEV)
        out = M.adapter_linear(x, w, a, b, ids, residual=res, save=True, out={"y": guard[:, 1:1 + O]})
        flat = M.adapter_linear(x.contiguous(), w.contiguous(), a.contiguous(), b.contiguous(), ids, residual=res.contiguous(), save=True)
        assert torch.equal(out["y"], flat["y"]) and torch.equal(out["s"], flat["s"])
        assert bool((guard[:, 0] == 7).all()) and bool((guard[:, 1 + O:] == 7).all())
        full = {"dx": torch.full((T, I + 4), 7.0, dtype=dt, device=DEV), "da": torch.full((n, R + 2, I + 4), 7.0, dtype=dt, device=DEV),
                "db": torch.full((n, O + 2, R + 4), 7.0, dtype=dt, device=DEV)}
        view = {"dx": full["dx"][:, 1:1 + I], "da": full["da"][:, :R, 1:1 + I], "db": full["db"][:, :O, 1:1 + R]}
        M.adapter_linear_backward(dy, x, w, a, b, ids, out["s"], out=view)
        g = M.adapter_linear_backward(dy.contiguous(), x.contiguous(), w.contiguous(), a.contiguous(), b.contiguous(), ids, out["s"])
        for k in g:
            assert torch.equal(view[k], g[k]), k
            outside = full[k].clone()
            {"dx": outside, "da": outside[:, :R], "db": outside[:, :O]}[k][..., 1:1 + g[k].shape[-1]] = 7
            assert bool((outside == 7).all()), k


def test_no_tokens():
    x, w, a, b, ids, scale = problem(0, 64, 32, 8, 3, "one", BF)
    out = M.adapter_linear(x, w, a, b, ids, scale=scale, save=True)
    assert out["y"].shape == (0, 32) and out["s"].shape == (0, 8)
    g = M.adapter_linear_backward(torch.empty(0, 32, dtype=BF, device=DEV), x, w, a, b, ids, out["s"], scale=scale,
                                  out={"dx": torch.empty_like(x), "da": torch.full_like(a, 3.0), "db": torch.full_like(b, 3.0)})
    assert bool((g["da"] == 0).all()) and bool((g["db"] == 0).all())


def test_without_adapters_it_is_the_linear_product():
    """Tokens without an adapter get moe_linear's y and dx, to the bit where both run on
    its tiles."""
    for T, I, O in ((300, 256, 1024), (4500, 512, 2304)):
        x, w, a, b, ids, _ = problem(T, I, O, 8, 2, "none", BF)
        bias, dy = normal(3, O, dt=BF), normal(4, T, O, dt=BF)
        assert torch.equal(M.adapter_linear(x, w, a, b, ids, bias=bias)["y"], M.linear(x, w, bias=bias)["y"])
        dx = M.adapter_linear_backward(dy, x, w, a, b, ids, None, out={"dx": torch.empty_like(x)})["dx"]
        assert torch.equal(dx, M.linear_backward(dy, x, w)["dx"])


@pytest.mark.parametrize("T,K,R,n,kind", [(1025, 520, 16, 30, "each"), (1400, 7168, 8, 40, "requests"), (2100, 200, 48, 9, "random"), (4096, 264, 32, 3, "requests"),
                                          (1030, 96, 64, 1, "random"), (1100, 203, 13, 25, "each")])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_rows_between_a_thousand_and_four(T, K, R, n, kind, dt):
    """16 rows a block of s, whose adapters several blocks share."""
    x, w, a, b, ids, scale = problem(T, K, 72, R, n, kind, dt)
    check_forward(x, w, a, b, ids, scale, None, None, M.adapter_linear(x, w, a, b, ids, scale=scale, save=True))
    x, w, a, b, ids, scale = problem(T, 72, K, R, n, kind, dt)
    dy, s = normal(11, T, K, dt=dt), normal(12, T, R, dt=torch.float32)
    check_backward(dy, x, w, a, b, ids, scale, s, M.adapter_linear_backward(dy, x, w, a, b, ids, s, scale=scale))


@pytest.mark.parametrize("T,I,O,R,n,kind", [(65, 4101, 130, 16, 5, "random"), (500, 5002, 200, 12, 40, "each"), (130, 4097, 64, 7, 9, "requests"),
                                            (512, 7168, 512, 16, 16, "requests"), (48, 8000, 100, 8, 48, "each"), (33, 2048, 4100, 32, 20, "each")])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_ranges_of_a_long_way(T, I, O, R, n, kind, dt):
    """Small tiles whose ranges of k meet in the workspace, with the term on one of them."""
    x, w, a, b, ids, scale = problem(T, I, O, R, n, kind, dt)
    bias, res = normal(9, O, dt=dt), normal(10, T, O, dt=dt)
    check_forward(x, w, a, b, ids, scale, bias, res, M.adapter_linear(x, w, a, b, ids, scale=scale, bias=bias, residual=res, save=True))


def test_many_adapters():
    """More adapters than tokens, and the largest number of them."""
    T, I, O, R, n = 40, 64, 48, 4, 4096
    x, w, a, b, _, scale = problem(T, I, O, R, n, "one", FP)
    ids = torch.randint(0, n, (T,), device=DEV, dtype=torch.int32)
    out = M.adapter_linear(x, w, a, b, ids, scale=scale, save=True)
    live = torch.unique(ids.long())
    at = torch.searchsorted(live, ids.long()).int()
    check_forward(x, w, a[live], b[live], at, scale[live], None, None, out)
    dy = normal(3, T, O, dt=FP)
    g = M.adapter_linear_backward(dy, x, w, a, b, ids, out["s"], scale=scale)
    check_backward(dy, x, w, a[live], b[live], at, scale[live], out["s"], {"dx": g["dx"], "da": g["da"][live], "db": g["db"][live]})
    g["da"][live] = 0
    g["db"][live] = 0
    assert bool((g["da"] == 0).all()) and bool((g["db"] == 0).all())


def test_same_bits_on_two_streams_and_in_a_graph():
    T, I, O, R, n = 700, 512, 768, 16, 6
    x, w, a, b, ids, scale = problem(T, I, O, R, n, "requests", BF)
    dy = normal(3, T, O, dt=BF)

    def step():
        f = M.adapter_linear(x, w, a, b, ids, scale=scale, save=True)
        return [*f.values(), *M.adapter_linear_backward(dy, x, w, a, b, ids, f["s"], scale=scale).values()]
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append([step() for _ in range(3)][-1])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        ids.copy_(make_ids("requests", T, n, 20 + k))
        x.copy_(normal(30 + k, T, I, dt=BF))
        for t in out:
            t.zero_()
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, eager))


def test_rows_beyond_32_bits_of_bytes():
    """An x of more than 4 GB: the last rows, forward and backward."""
    T, I, O, R, n = 300_100, 7168, 64, 8, 2
    x = torch.zeros(T, I, dtype=BF, device=DEV)
    x[-40:] = normal(1, 40, I, dt=BF)
    _, w, a, b, _, scale = problem(1, I, O, R, n, "one", BF)
    ids = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    ids[-40:] = make_ids("each", 40, n, 0)
    out = M.adapter_linear(x, w, a, b, ids, scale=scale, save=True)
    assert bool((out["y"][:-40] == 0).all()) and bool((out["s"][:-40] == 0).all())
    check_forward(x[-40:], w, a, b, ids[-40:], scale, None, None, {k: v[-40:] for k, v in out.items()})
    dy = torch.zeros(T, O, dtype=BF, device=DEV)
    dy[-40:] = normal(2, 40, O, dt=BF)
    g = M.adapter_linear_backward(dy, x, w, a, b, ids, out["s"], scale=scale)
    check_backward(dy[-40:], x[-40:], w, a, b, ids[-40:], scale, out["s"][-40:], {"dx": g["dx"][-40:], "da": g["da"], "db": g["db"]})
