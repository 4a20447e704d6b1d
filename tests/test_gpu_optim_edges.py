"""The optimizer's tensors as torch sees them: what autograd saved before a
step, and the memory that a list was made of."""
import pytest
import torch

from lossless_bf16_tensor_sign_amd import zc
from tests.test_gpu_optim import BF, F32, HYPER, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("views", [False, True])
def test_autograd_sees_that_a_step_writes_the_parameters(master, views):
    s = make([300, 50], BF, F32, master, False)
    if views:
        flat = torch.cat(s["params"])
        s["params"] = [flat[:300], flat[300:]]
    params = [p.requires_grad_() for p in s["params"]]
    t = zc.AdamWTensors(**s)
    assert len(t.counted) == (1 if views else 2) + (2 if master else 0)
    x = torch.ones(300, dtype=BF, device=DEV, requires_grad=True)
    loss = (params[0] * x).sum()                                # saves the parameter for x's gradient
    before = [p._version for p in params]
    zc.adamw(t, **HYPER)
    assert all(p._version > v for p, v in zip(params, before))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    if master:
        m = s["masters"][1]
        v = m._version
        zc.adamw(t, **HYPER)
        assert m._version > v


def test_step_of_tensors_made_in_inference_mode():
    with torch.inference_mode():
        s = make([300, 50], BF, F32, True, False)
        zc.adamw(zc.AdamWTensors(**s), **HYPER)
        want = [m.to(BF) for m in s["masters"]]
        assert all(torch.equal(a, b) for a, b in zip(want, s["params"]))


def test_lists_keep_the_memory_that_they_were_made_of():
    # a parameter's .data and .grad may be given other memory while a list
    # lives: the list's stays allocated, and is what the calls take
    s = make([70000], F32, F32, False, False)
    p = torch.nn.Parameter(s["params"][0].clone())
    p.grad = s["grads"][0].clone()
    twin = p.detach().clone()
    t, other = zc.AdamWTensors([p], [p.grad], s["avg"], s["sq"]), make([70000], F32, F32, False, False)
    norms = zc.TensorList([p.grad])
    old = p.detach()
    at = [x.data_ptr() for x in (p, p.grad)]
    p.data, p.grad.data = torch.zeros_like(p), torch.zeros_like(p)
    fresh = [torch.empty(70000, device=DEV) for _ in range(8)]
    assert not set(at) & {f.data_ptr() for f in fresh}
    zc.adamw(t, **HYPER)
    zc.adamw(zc.AdamWTensors([twin], other["grads"], other["avg"], other["sq"]), **HYPER)
    assert torch.equal(old, twin) and not p.any()
    assert torch.equal(zc.grad_norm(norms), zc.grad_norm(other["grads"]))
