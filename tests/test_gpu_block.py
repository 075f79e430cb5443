"""The operators as they are used together: one residual block in training,

    h, y = norm(x + drop(attention's output)),   f = silu(y Wg^T) * (y Wu^T)
    z = f Wd^T + adapters,   out = h + drop(z)

forward and backward, eager and captured, against the same block in 64 bits."""
import pytest
import torch

import moe_expert_routing_amd as M
from block_util import normal, numbers

pytestmark = pytest.mark.gpu
DEV = "cuda"
SEED = 77


class Block:
    def __init__(self, T, H, F, R, n, dt):
        self.T, self.H, self.dt, self.p = T, H, dt, 0.1
        self.x, self.o, self.dout = normal(1, T, H, dt=dt, scale=2.0), normal(2, T, H, dt=dt), normal(3, T, H, dt=dt)
        self.w = (1 + 0.1 * normal(4, H, dt=torch.float32)).to(dt)
        self.wg, self.wu = normal(5, F, H, dt=dt, scale=H ** -0.5), normal(6, F, H, dt=dt, scale=H ** -0.5)
        self.wd = normal(7, H, F, dt=dt, scale=F ** -0.5)
        self.a, self.b = normal(8, n, R, F, dt=dt, scale=F ** -0.5), normal(9, n, H, R, dt=dt, scale=R ** -0.5)
        self.scale = torch.linspace(0.5, 2.0, n, device=DEV)
        cuts = torch.linspace(0, n + 1, T + 1)[:T].long() - 1  # the first request has no adapter
        self.ids = cuts.int().to(DEV)
        self.rng = torch.tensor((SEED, 5), dtype=torch.int64, device=DEV)

    def step(self):
        drop = dict(p=self.p, rng=self.rng)
        n = M.rms_norm(self.o, self.w, residual=self.x, site=1, **drop)
        g = M.gated_ffn(n["y"], self.wg, self.wu, save_pre=True)
        z = M.adapter_linear(g["h"], self.wd, self.a, self.b, self.ids, scale=self.scale, save=True)
        out = M.dropout(z["y"], self.p, self.rng, site=2, residual=n["h"])
        dz = M.dropout_backward(self.dout, self.p, self.rng, site=2)
        ad = M.adapter_linear_backward(dz, g["h"], self.wd, self.a, self.b, self.ids, z["s"], scale=self.scale)
        dg = M.gated_ffn_backward(ad["dx"], g["pre"], n["y"], self.wg, self.wu)
        dn = M.rms_norm_backward(dg["dx"], n["h"], self.w, n["rstd"], dh=self.dout, site=1, **drop)
        return {"out": out, "da": ad["da"], "db": ad["db"], "dwg": dg["dw_gate"], "dwu": dg["dw_up"],
                "dw": dn["dweight"], "dx": dn["dresidual"], "do": dn["dx"]}

    def exact(self, offset):
        """The block and its gradients by autograd in 64 bits on the CPU."""
        leaf = {k: getattr(self, k).detach().double().cpu().requires_grad_() for k in ("x", "o", "w", "wg", "wu", "a", "b")}
        keep = [torch.from_numpy(numbers(SEED, offset, site, self.T, self.H) >= 6554) * (65536 / (65536 - 6554)) for site in (1, 2)]
        h = leaf["x"] + keep[0] * leaf["o"]
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * leaf["w"]
        f = torch.nn.functional.silu(y @ leaf["wg"].T) * (y @ leaf["wu"].T)
        z = f @ self.wd.double().cpu().T
        ids = self.ids.cpu()
        for e in range(self.a.shape[0]):
            at = torch.nonzero(ids == e).reshape(-1)
            z = z.index_add(0, at, float(self.scale[e]) * (f[at] @ leaf["a"][e].T) @ leaf["b"][e].T)
        out = h + keep[1] * z
        out.backward(self.dout.double().cpu())
        g = {k: v.grad for k, v in leaf.items()}
        return {"out": out.detach(), "da": g["a"], "db": g["b"], "dwg": g["wg"], "dwu": g["wu"], "dw": g["w"], "dx": g["x"], "do": g["o"]}


def off(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


# Each value on the way is rounded once, by at most u = eps / 2 of itself: out passes h,
# y, f, z and its own rounding; a gradient also dz, the gradient of f, the one inside the
# gated block's backward pass, dy and its own. In the 2-norm these add up to no more than
# their number times u, for a block whose parts do not amplify: 16 u leaves room for
# the products (and f) that meet two rounded factors.
@pytest.mark.parametrize("T,H,F,R,n", [(37, 256, 96, 8, 3), (300, 512, 704, 16, 4), (1030, 264, 520, 12, 2)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_block(T, H, F, R, n, dt):
    b = Block(T, H, F, R, n, dt)
    want, got = b.exact(5), b.step()
    for k in want:
        assert off(got[k], want[k]) < 16 * torch.finfo(dt).eps / 2, k


def test_block_captured():
    """A captured training step, its dropout's offset counted up inside the graph."""
    b = Block(200, 256, 320, 16, 3, torch.bfloat16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b.step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.step()
        b.rng[1] += 1
    b.rng.copy_(torch.tensor((SEED, 9)))
    last = None
    for k in range(3):
        for t in got.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = {name: t.clone() for name, t in got.items()}
        now = b.rng.clone()
        assert now.tolist() == [SEED, 10 + k]
        b.rng[1] -= 1
        eager = b.step()
        b.rng.copy_(now)
        for name in replayed:
            assert torch.equal(replayed[name], eager[name]), name
        assert last is None or not torch.equal(last, replayed["out"])
        last = replayed["out"]
    want = b.exact(11)
    assert off(last, want["out"]) < 16 * torch.finfo(torch.bfloat16).eps / 2


def test_norm_into_the_router_and_back():
    """The norm's y through the routing and one rank's experts, whose rows combine onto
    the norm's h, as a serving program has them; its 8-bit form for the same tokens."""
    T, H, F, n = 48, 512, 128, 28
    x, res, w = normal(1, T, H, dt=torch.bfloat16), normal(2, T, H, dt=torch.bfloat16), normal(3, H, dt=torch.bfloat16)
    y = {"y": torch.empty_like(x), "h": torch.empty_like(x)}
    q = M.rms_norm(x, w, residual=res, quant="mxfp8", out=y)
    back = M.mxfp8_values(q["act_q"], q["act_scale"])
    # E4M3 is off by 2^-4 of a value, or half its smallest step, 2^-10, of the block's scale,
    # whose largest value is at least 2^8; y itself by 2^-8. The scale puts that value below
    # 512, and E4M3 ends at 448: one between them is off by what it is above 448 (by up to
    # 64 / 512 = 2^-3 of it) in place of a rounding.
    v = q["y"].float().abs()
    one = torch.exp2(q["act_scale"].float() - 127).repeat_interleave(32, 1)
    most = v.view(T, H // 32, 32).amax(2).repeat_interleave(32, 1)
    above = (v * (1 + 2.0 ** -7) - 448 * one).clamp(min=0)
    bound = (2.0 ** -4 + 2.0 ** -7) * v + 2.0 ** -17 * most + above
    assert bool(((back.float() - q["y"].float()).abs() <= bound).all())
    g = torch.Generator(device=DEV).manual_seed(0)
    router = (torch.randn(896, H, device=DEV, generator=g) * H ** -0.5).bfloat16()
    lay = M.router_gemm_route(q["y"], router, torch.zeros(896, device=DEV), 0, n, top_k=8)
    lay.update(M.grouped_layout(lay["counts"], lay["perm"], 16))
    wg, wu, wd = (normal(k, n, *s, dt=torch.bfloat16, scale=0.05) for k, s in ((5, (F, H)), (6, (F, H)), (7, (H, F))))
    f = M.expert_gated_ffn(q["y"], wg, wu, lay, tile_m=16, top_k=8)
    rows = M.expert_linear(f["h"], wd, lay, tile_m=16)["y"]
    out = M.combine(rows, lay, num_experts=n, residual=q["h"])
    want = q["h"].double().cpu()
    yd = q["y"].double().cpu()
    ids, weight = (lay["packed"] >> 16).cpu(), lay["topk_weights"].double().cpu()
    for t in range(T):
        for k in range(8):
            e = int(ids[t, k])
            if e < n:
                hh = torch.nn.functional.silu(wg[e].double().cpu() @ yd[t]) * (wu[e].double().cpu() @ yd[t])
                want[t] += weight[t, k] * (wd[e].double().cpu() @ hh)
    assert off(out, want) < 4 * torch.finfo(torch.bfloat16).eps / 2
