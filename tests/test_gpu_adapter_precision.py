"""GPU tests that s and u of the adapters keep the bits of fp32 on their way through the
matrix cores, for few tokens and many: outputs in which nearly everything cancels.

An fp32 number v is the sum of three parts of the type: hi = v rounded, mid = v - hi
rounded, lo = the rest, which both types hold exactly here. Where every other operation
is exact too, an output that v - hi - mid has to give is lo itself. In the gradients
two tokens cancel to 2^-14 of their terms S: beside the output's own rounding there is
one of each u (F32 |u x|) and no more than 6 of sums that are at most S.
"""
import pytest
import torch

import moe_expert_routing_amd as M
from ffn_util import F32, TINY, assert_close, half_step

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
DEV = "cuda"
N = 3
# few tokens, and the tiles of 32 to 256 rows
SIZES = [(5, 136, 96), (150, 136, 96), (700, 200, 640), (4500, 264, 2304)]
RANKS = [4, 16, 20, 64, 128]


def scales(seed):
    """N numbers of 24 bits in [1, 1.5), odd in their last bit."""
    g = torch.Generator().manual_seed(seed)
    k = torch.randint(0, 1 << 22, (N,), generator=g) | 1
    return (1 + k.double() * 2.0 ** -23).float().to(DEV)


def parts(v, dt):
    hi = v.to(dt).double()
    mid = (v - hi).to(dt).double()
    lo = v - hi - mid
    assert torch.equal(lo.to(dt).double(), lo)
    return hi, mid, lo


def token_ids(T):
    ids = torch.arange(T, device=DEV) * 7 // 5 % (N + 1)  # N: none
    return ids.int()


@pytest.mark.parametrize("R", RANKS)
@pytest.mark.parametrize("T,I,O", SIZES)
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_y_of_what_s_leaves(T, I, O, R, dt):
    ids, c = token_ids(T), scales(R)
    at, has = ids.long().clamp(max=N - 1), ids < N
    a, b, x, w = (torch.zeros(*s, dtype=dt, device=DEV) for s in ((N, R, I), (N, O, R), (T, I), (O, I)))
    power = 2.0 ** (4 + torch.arange(R, device=DEV) % 5).double()
    a[:, :, 0] = power.to(dt)
    col = torch.arange(O, device=DEV)
    b[:, col, col % R] = 1
    x[:, 0] = 1
    x[torch.arange(T, device=DEV), 1 + at] = has.to(dt)
    hi, mid, lo = parts(c.double()[:, None] * power[col % R], dt)
    w[:, 1:1 + N] = -mid.T.to(dt)
    res = torch.where(has[:, None], -hi[at], 0.0).to(dt)
    want = torch.where(has[:, None], lo[at], 0.0)
    assert bool((want != 0).any())
    out = M.adapter_linear(x, w, a, b, ids, scale=c, residual=res, save=True)
    assert torch.equal(out["s"].double(), torch.where(has[:, None], c.double()[at][:, None] * power, 0.0))
    assert torch.equal(out["y"].double(), want)


@pytest.mark.parametrize("R", RANKS)
@pytest.mark.parametrize("T,O,I", SIZES)
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_dx_of_what_u_leaves(T, I, O, R, dt):
    ids, c = token_ids(T), scales(R + 1)
    at, has = ids.long().clamp(max=N - 1), ids < N
    a, b, dy, w = (torch.zeros(*s, dtype=dt, device=DEV) for s in ((N, R, I), (N, O, R), (T, O), (O, I)))
    power = 2.0 ** (4 + torch.arange(R, device=DEV) % 5).double()
    b[:, 0] = power.to(dt)
    col, row = torch.arange(I, device=DEV), torch.arange(T, device=DEV)
    a[:, col % R, col] = 1
    hi, mid, lo = parts(c.double()[:, None] * power[col % R], dt)
    w[1:1 + N], w[1 + N:1 + 2 * N] = -hi.to(dt), -mid.to(dt)
    dy[:, 0] = 1
    dy[row, 1 + at] = has.to(dt)
    dy[row, 1 + N + at] = has.to(dt)
    want = torch.where(has[:, None], lo[at], 0.0)
    dx = M.adapter_linear_backward(dy, torch.zeros(T, I, dtype=dt, device=DEV), w, a, b, ids, None, scale=c,
                                   out={"dx": torch.empty(T, I, dtype=dt, device=DEV)})["dx"]
    assert torch.equal(dx.double(), want)


@pytest.mark.parametrize("R", RANKS)
@pytest.mark.parametrize("T,I,O", [(6, 72, 96), (600, 200, 264), (5000, 264, 520)])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_gradients_of_two_tokens_that_cancel(T, I, O, R, dt):
    g = torch.Generator(device=DEV).manual_seed(R)
    c, p, q = scales(R + 2), 1 - 2.0 ** -7, 1 + 2.0 ** -7  # p q = 1 - 2^-14
    ids = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    pair = torch.stack([torch.arange(N), T - 1 - torch.arange(N)]).to(DEV)  # adapter e's two tokens
    ids[pair] = torch.arange(N, device=DEV).int()
    a = torch.zeros(N, R, I, dtype=dt, device=DEV)
    b = torch.zeros(N, O, R, dtype=dt, device=DEV)
    b[:, 0] = (1 + torch.rand(N, R, device=DEV, generator=g)).to(dt)
    x, dy = torch.zeros(T, I, dtype=dt, device=DEV), torch.zeros(T, O, dtype=dt, device=DEV)
    v = 2.0 ** torch.randint(-3, 4, (N, I), device=DEV, generator=g).double()
    x[pair[0]], x[pair[1]] = v.to(dt), (-v * q).to(dt)
    dy[pair[0], 0], dy[pair[1], 0] = 1, p
    w = torch.zeros(O, I, dtype=dt, device=DEV)
    da = M.adapter_linear_backward(dy, x, w, a, b, ids, None, scale=c, out={"da": torch.empty_like(a)})["da"]
    base = c.double()[:, None] * b[:, 0].double()  # u of the first token
    ref, S = base[:, :, None] * v[:, None] * 2.0 ** -14, 2 * base[:, :, None] * v[:, None]
    assert_close(da, ref, half_step(dt) * ref.abs() * 1.01 + 7 * F32 * S + TINY[dt], "da")
    s = torch.zeros(T, R, device=DEV)
    s[pair[0]] = 1 + torch.rand(N, R, device=DEV, generator=g)
    s[pair[1]] = s[pair[0]] * p
    v = 2.0 ** torch.randint(-3, 4, (N, O), device=DEV, generator=g).double()
    dy[pair[0]], dy[pair[1]] = v.to(dt), (-v * q).to(dt)
    db = M.adapter_linear_backward(dy, x, w, a, b, ids, s, scale=c, out={"db": torch.empty_like(b)})["db"]
    s = s.double()
    ref = v[:, :, None] * (s[pair[0]] - s[pair[1]] * q)[:, None]
    S = v[:, :, None] * (s[pair[0]] + s[pair[1]] * q)[:, None]
    assert_close(db, ref, half_step(dt) * ref.abs() * 1.01 + 6 * F32 * S + TINY[dt], "db")
