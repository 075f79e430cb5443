"""The binding of the norm, dropout and the adapters on its own, with no GPU: what
it refuses, and what it hands to the library, seen through recorded calls."""
import pytest
import torch

import moe_expert_routing_amd as M
from moe_expert_routing_amd import adapters, block, ffn

DEV = torch.device("cuda", 0)


class AnyGpuTensor(torch.Tensor):
    """Host memory that passes for the GPU's."""
    device = DEV
    is_cuda = True

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        return torch._C._disabled_torch_function_impl(func, types, args, kwargs or {})


def gpu(*shape, dt=torch.bfloat16):
    return torch.zeros(shape, dtype=dt).as_subclass(AnyGpuTensor)


ENTRIES = (block._NORM, block._NORM_BACKWARD, block._DROPOUT, block._VALUES, adapters._ADAPTER,
           adapters._ADAPTER_BACKWARD)


class Library:
    """Sizes of workspaces: none."""

    def __getattr__(self, name):
        return lambda *a: 0


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, recorded instead of made."""
    made = []
    monkeypatch.setattr(ffn, "_current_device", lambda: 0)
    monkeypatch.setattr(M, "_stream_handle", lambda dev: 0)
    monkeypatch.setattr(M, "lib", Library)
    for e in ENTRIES:
        monkeypatch.setattr(e, "fn", lambda *a, name=e.name: made.append((name, a)) or 0)
    return made


T, W, I, O, R, N = 6, 64, 32, 24, 8, 3
F32, U8, I32, I64 = torch.float32, torch.uint8, torch.int32, torch.int64


def some_calls():
    """A call of each operator, of everything but what is wrong in it."""
    m, v = gpu(T, W), gpu(W)
    ad = dict(x=gpu(T, I), w=gpu(O, I), a=gpu(N, R, I), b=gpu(N, O, R), ids=gpu(T, dt=I32))
    return dict(
        norm=lambda **k: M.rms_norm(**{**dict(x=m, weight=v, out={"y": gpu(T, W)}), **k}),
        norm_backward=lambda **k: M.rms_norm_backward(**{**dict(dy=m, h=m, weight=v, rstd=gpu(T, dt=F32), out={"dx": gpu(T, W)}), **k}),
        dropout=lambda **k: M.dropout(**{**dict(x=m, p=0.5, rng=gpu(2, dt=I64), out=gpu(T, W)), **k}),
        values=lambda **k: M.mxfp8_values(**{**dict(act_q=gpu(T, W, dt=U8), act_scale=gpu(T, W // 32, dt=U8), out=gpu(T, W)), **k}),
        adapters=lambda **k: M.adapter_linear(**{**ad, "out": {"y": gpu(T, O)}, **k}),
        adapters_backward=lambda **k: M.adapter_linear_backward(**{**ad, "dy": gpu(T, O), "s": gpu(T, R, dt=F32), "out": {"dx": gpu(T, I)}, **k}))


def test_the_calls_below_are_right_but_for_one_thing(calls):
    for call in some_calls().values():
        call()
    assert [c[0] for c in calls] == [e.name for e in ENTRIES]


@pytest.mark.parametrize("op,kw", [
    ("norm", dict(x=None)), ("norm", dict(x=gpu(T, W, dt=F32))), ("norm", dict(x=gpu(W))), ("norm", dict(x=torch.zeros(T, W).bfloat16())),
    ("norm", dict(weight=None)), ("norm", dict(weight=gpu(W + 1))), ("norm", dict(weight=3)), ("norm", dict(weight=gpu(W, dt=torch.float16))),
    ("norm", dict(residual=gpu(T, W))), ("norm", dict(residual=gpu(T + 1, W))), ("norm", dict(residual=5)), ("norm", dict(out={})),
    ("norm", dict(out={"y": gpu(T, W), "rstd": gpu(T)})), ("norm", dict(out={"y": gpu(W, T).t()})),
    ("norm", dict(p=0.5)), ("norm", dict(p=-0.1)), ("norm", dict(p=1.5)), ("norm", dict(p=float("nan"))), ("norm", dict(p="0.1")),
    ("norm", dict(rng=gpu(2, dt=I32))), ("norm", dict(rng=gpu(3, dt=I64))), ("norm", dict(site=1.5)), ("norm", dict(site=1 << 40)),
    ("norm", dict(eps=-1.0)), ("norm", dict(eps=float("nan"))), ("norm", dict(eps=None)), ("norm", dict(quant="fp8")),
    ("norm", dict(quant="mxfp8", x=gpu(T, 48), weight=gpu(48), out={})), ("norm", dict(quant="mxfp8", out={"act_q": gpu(T, W), "act_scale": gpu(T, 2, dt=U8)})),
    ("norm", dict(quant="mxfp8", out={"act_q": gpu(T, W, dt=U8), "act_scale": gpu(T, 3, dt=U8)})),
    ("norm_backward", dict(dy=None)), ("norm_backward", dict(rstd=None)), ("norm_backward", dict(rstd=gpu(T))), ("norm_backward", dict(dy=gpu(T, W + 8))),
    ("norm_backward", dict(dh=gpu(T))), ("norm_backward", dict(weight=None)), ("norm_backward", dict(out={"dweight": gpu(W, dt=F32)})), ("norm_backward", dict(p=0.5)),
    ("dropout", dict(rng=None)), ("dropout", dict(p=2)), ("dropout", dict(x=gpu(T, W, dt=F32))), ("dropout", dict(residual=gpu(W))), ("dropout", dict(out=gpu(T, W - 1))),
    ("values", dict(act_q=gpu(T, W))), ("values", dict(act_q=None)), ("values", dict(act_scale=None)), ("values", dict(act_scale=gpu(T, 1, dt=U8))),
    ("values", dict(dtype=F32)), ("values", dict(act_q=gpu(T, 40, dt=U8))), ("values", dict(out=gpu(T, W, dt=torch.float16))),
    ("adapters", dict(ids=None)), ("adapters", dict(ids=gpu(T, dt=I64))), ("adapters", dict(ids=gpu(T + 1, dt=I32))), ("adapters", dict(w=None)),
    ("adapters", dict(a=gpu(R, I))), ("adapters", dict(a=gpu(N, R, I + 1))), ("adapters", dict(b=gpu(N, R, O))), ("adapters", dict(b=gpu(N + 1, O, R))),
    ("adapters", dict(scale=gpu(N))), ("adapters", dict(scale=2.0)), ("adapters", dict(bias=gpu(O + 1))), ("adapters", dict(residual=gpu(T, I))), ("adapters", dict(out={})),
    ("adapters", dict(save=True, out={"y": gpu(T, O), "s": gpu(T, R)})), ("adapters", dict(x=gpu(T, I, dt=torch.float16))),
    ("adapters_backward", dict(dy=None)), ("adapters_backward", dict(dy=gpu(T, I))), ("adapters_backward", dict(s=gpu(R, T, dt=F32).t())),
    ("adapters_backward", dict(out={"da": gpu(N, R, O)})), ("adapters_backward", dict(out={"db": gpu(N, O, R, dt=F32)}))])
def test_refusals_are_the_packages_own(calls, op, kw):
    with pytest.raises(M.MoeRouteError):
        some_calls()[op](**kw)
    assert not calls


def test_level_is_the_nearest_multiple(calls):
    for p, level in ((0.0, 0), (1e-7, 0), (0.1, 6554), (0.5, 32768), (1.0, 65536), (1, 65536)):
        some_calls()["dropout"](p=p)
        a = block.DropoutArgs.from_buffer_copy(calls.pop()[1][0])
        assert a.drop.level == level


@pytest.mark.parametrize("op", ["norm", "norm_backward", "dropout", "values", "adapters", "adapters_backward"])
def test_calls_run_on_their_tensors_device(calls, monkeypatch, op):
    """With another device current the call is made inside its own."""
    now = [1]

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            now.append(self.dev.index)

        def __exit__(self, *a):
            now.pop()
    monkeypatch.setattr(ffn, "_current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    seen = []
    monkeypatch.setattr(M, "_stream_handle", lambda dev: seen.append(now[-1]) or 7)
    some_calls()[op]()
    assert len(calls) == 1 and seen == [0] and now == [1] and calls[0][1][-1] == 7
