"""One mixture-of-experts block on one MI355X, from the router's logits to the
gradients of every weight:

    out = x + down_s(act(x Wg_s^T) * (x Wu_s^T)) + sum over the token's experts of
          w_e down_e(act(x Wg_e^T) * (x Wu_e^T))

with a shared expert (the dense operators) and one expert-parallel rank's routed
experts (the expert operators on the layout that the routing writes).

    python examples/moe_block.py [--tokens 4096] [--hidden 2048] [--inter 1024]

prints the time of a forward pass, of a training step and of a decode step, and
how far the outputs and gradients are from the same block in plain torch.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_routing_amd as M  # noqa: E402

EXPERTS, TOP_K = 896, 16


class MoeBlock:
    """Weights of the block; `offset`, `count`: the experts of this rank. `hidden`
    is a multiple of 64 and `dtype` bf16, as the router product has it."""

    def __init__(self, hidden, inter, offset=0, count=112, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, device="cuda", generator=g) * shape[-1] ** -0.5).to(dtype)
        self.offset, self.count = offset, count
        self.router = weight(EXPERTS, hidden)
        self.bias = 0.01 * torch.randn(EXPERTS, device="cuda", generator=g)
        self.w_gate, self.w_up = weight(count, inter, hidden), weight(count, inter, hidden)
        self.w_down = weight(count, hidden, inter)
        self.s_gate, self.s_up = weight(inter, hidden), weight(inter, hidden)
        self.s_down = weight(hidden, inter)

    def route(self, x, tile_m):
        """The rank's layout, cut to the rows that its buffers have: every entry
        of a small batch, and twice the mean share of a large one."""
        lay = M.router_gemm_route(x, self.router, self.bias, self.offset, self.count, top_k=TOP_K)
        lay.update(M.grouped_layout(lay["counts"], lay["perm"], tile_m))
        entries = x.shape[0] * TOP_K
        share = entries if x.shape[0] <= 256 else 2 * entries * self.count // EXPERTS
        rows = min(lay["m_indices"].numel(), share + self.count * (tile_m - 1))
        lay["m_indices"], lay["row_entry"] = lay["m_indices"][:rows], lay["row_entry"][:rows]
        return lay

    def forward(self, x, train=False):
        tile_m = 16 if x.shape[0] <= 256 else 128
        lay = self.route(x, tile_m)
        s = M.gated_ffn(x, self.s_gate, self.s_up, save_pre=train)
        shared = M.linear(s["h"], self.s_down, residual=x)["y"]
        f = M.expert_gated_ffn(x, self.w_gate, self.w_up, lay, tile_m=tile_m, top_k=TOP_K,
                               save_pre=train)
        y = M.expert_linear(f["h"], self.w_down, lay, tile_m=tile_m)["y"]
        out = M.combine(y, lay, num_experts=self.count, residual=shared)
        return out, (x, tile_m, lay, s, f, y)

    def backward(self, dout, saved):
        x, tile_m, lay, s, f, y = saved
        n = self.count
        c = M.combine_backward(dout, y, lay, num_experts=n)
        d = M.expert_linear_backward(c["dy"], f["h"], self.w_down, lay, tile_m=tile_m)
        e = M.expert_gated_ffn_backward(d["dx"], f["pre"], x, self.w_gate, self.w_up, lay,
                                        tile_m=tile_m, top_k=TOP_K)
        sd = M.linear_backward(dout, s["h"], self.s_down)
        sg = M.gated_ffn_backward(sd["dx"], s["pre"], x, self.s_gate, self.s_up)
        dx = M.combine(e["dx"], lay, num_experts=n, weighted=False, residual=sg["dx"])
        return {"x": dx.add_(dout), "weights": c["dweights"], "w_gate": e["dw_gate"],
                "w_up": e["dw_up"], "w_down": d["dw"], "s_gate": sg["dw_gate"],
                "s_up": sg["dw_up"], "s_down": sd["dw"]}


def plain(block, x, dout, saved):
    """The block and its gradients in 32 bits by torch, an expert at a time, with
    the routing that the block used: (out, gradients)."""
    lay, n = saved[2], block.count
    leaves = {k: getattr(block, k).float().requires_grad_() for k in
              ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")}
    leaves["x"] = x.float().requires_grad_()
    leaves["weights"] = lay["topk_weights"].clone().requires_grad_()
    p, xf = leaves, leaves["x"]

    def ffn(v, gate, up, down):
        return (torch.nn.functional.silu(v @ gate.t()) * (v @ up.t())) @ down.t()
    out = xf + ffn(xf, p["s_gate"], p["s_up"], p["s_down"])
    m, entry = lay["m_indices"], lay["row_entry"].long()
    for e in range(n):
        en = entry[m == e]
        if en.numel():
            tok = en // TOP_K
            w = p["weights"].reshape(-1)[en].unsqueeze(1)
            out = out.index_add(0, tok, w * ffn(xf[tok], p["w_gate"][e], p["w_up"][e], p["w_down"][e]))
    out.backward(dout.float())
    return out.detach(), {k: v.grad for k, v in leaves.items()}


def off(a, b):
    return float((a.float() - b).norm() / b.norm().clamp(min=1e-30))


def timed(f, n=20):
    for _ in range(3):
        f()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(n):
        f()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / n * 1e6


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1024)
    a = ap.parse_args()
    block = MoeBlock(a.hidden, a.inter)
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    dout = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    out, saved = block.forward(x, train=True)
    grads = block.backward(dout, saved)
    want, ref = plain(block, x, dout, saved)
    print("out off by %.2g; gradients: %s" % (off(out, want), ", ".join(
        "%s %.2g" % (k, off(grads[k], ref[k])) for k in ref)))

    def step():
        o, s = block.forward(x, train=True)
        block.backward(dout, s)
    print("forward %.0f us, training step %.0f us (%d tokens)" % (
        timed(lambda: block.forward(x)), timed(step), a.tokens))
    print("decode of 16 tokens %.0f us" % timed(lambda: block.forward(x[:16])))


if __name__ == "__main__":
    main()
