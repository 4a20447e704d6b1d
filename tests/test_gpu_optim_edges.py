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
