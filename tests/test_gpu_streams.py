"""Arguments that are freed as soon as a call on another stream returns: their
memory is not given out again before the call's work has ended."""
import pytest
import torch

from lossless_bf16_tensor_sign_amd import zc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, E, k, H = 4096, 512, 4, 1024


def inputs():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, E, generator=g, device=DEV)
    h = torch.randn(T, H, generator=g, device=DEV)
    e, w = zc.route(x, k)
    s, _ = zc.expert_slots(e, E)
    y = zc.dispatch(h, s)
    return dict(x=x, bias=0.1 * torch.randn(E, generator=g, device=DEV), valid=x[:, 0] < 1.0, h=h, e=e, w=w, s=s, y=y,
                base=h * 0.5, gw=torch.randn(T, k, generator=g, device=DEV), one=torch.full((1,), 0.5, device=DEV))


CALLS = {
    "route": (("x", "bias", "valid"), lambda a, st: zc.route(a["x"], k, bias=a["bias"], valid=a["valid"], stream=st)),
    "route_grad": (("x", "e", "gw"), lambda a, st: zc.route_grad(a["x"], a["e"], a["gw"], stream=st)),
    "expert_slots": (("e",), lambda a, st: zc.expert_slots(a["e"], E, stream=st)),
    "dispatch": (("h", "s"), lambda a, st: zc.dispatch(a["h"], a["s"], stream=st)),
    "combine": (("y", "s", "w", "base"),
                lambda a, st: zc.combine(a["y"], a["s"], weights=a["w"], base=a["base"], stream=st)),
    "combine_grad": (("h", "y", "s", "w"), lambda a, st: zc.combine_grad(a["h"], a["y"], a["s"], a["w"], stream=st)),
    "grad_norm": (("x", "h"), lambda a, st: zc.grad_norm((t for t in (a["x"], a["h"])), max_norm=1.0, stream=st)),
}


def outputs(r):
    return r if isinstance(r, tuple) else (r,)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_arguments_may_be_freed_at_once(name):
    needs, call = CALLS[name]
    a = inputs()
    want = outputs(call(a, None))
    side = torch.cuda.Stream()
    m = torch.zeros(8192, 8192, dtype=torch.bfloat16, device=DEV)
    m2 = torch.zeros_like(m)
    temps = {n: a[n].clone() for n in needs}
    torch.cuda.synchronize()
    with torch.cuda.stream(side):                        # some 50 ms of work before the call's
        for _ in range(50):
            torch.mm(m, m, out=m2)
    got = outputs(call(temps, side))
    at = {t.data_ptr() for t in temps.values()}
    temps.clear()
    fresh = [torch.full_like(a[n], 0 if a[n].dtype is torch.bool else 3) for n in needs for _ in range(6)]
    assert not at & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_factor_of_a_step_may_be_freed_at_once():
    def tensors():
        g = torch.Generator(device=DEV).manual_seed(2)
        return [[torch.rand(5000, generator=g, device=DEV)] for _ in range(4)]
    side = torch.cuda.Stream()
    a, b = tensors(), tensors()
    ta, tb = zc.AdamWTensors(*a), zc.AdamWTensors(*b)
    zc.adamw(ta, step=3, lr=1e-2, grad_scale=torch.full((1,), 0.5, device=DEV))
    m = torch.zeros(8192, 8192, dtype=torch.bfloat16, device=DEV)
    m2 = torch.zeros_like(m)
    torch.cuda.synchronize()
    factor = torch.full((1,), 0.5, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(50):
            torch.mm(m, m, out=m2)
    at = factor.data_ptr()
    zc.adamw(tb, step=3, lr=1e-2, grad_scale=factor, stream=side)
    del factor
    assert at not in {torch.full((1,), 8.0, device=DEV).data_ptr() for _ in range(40)}
    torch.cuda.synchronize()
    assert all(torch.equal(x[0], y[0]) for x, y in zip(a, b))
