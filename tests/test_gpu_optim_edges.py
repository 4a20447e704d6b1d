"""AdamW over lists that stream past the caches, the least code of an 8-bit
second state, and the tensors as torch sees them: what autograd saved before
a step, and the memory that a list was made of."""
import numpy as np
import pytest
import torch

from lossless_bf16_tensor_sign_amd import zc
from tests import ref_ops as ref
from tests.test_gpu_optim import BF, COMBOS, F32, HYPER, SIZES, U, f64, make, same, say, snapshot

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


# 60 tensors in two launches, 3.9 M values: at 10 bytes a value and more past
# the 32 MB from which loads and stores are streamed
LARGE = [1 + int(130000 * ((i * 0.6180339887) % 1.0)) for i in range(58)] + [1, 100003]


@pytest.mark.parametrize("param,grad,master,eight", COMBOS)
def test_adamw_of_a_list_that_streams_past_the_caches(param, grad, master, eight):
    # the bits of the same tensors stepped one at a time, which do not stream
    # (test_gpu_optim.py compares those with the definition); every tensor one
    # value off its allocation, so that no run of a wave is aligned
    say("adamw, streamed", param, grad, master, eight, sum(LARGE))
    assert 10 * sum(LARGE) > 33 << 20
    a, b = (make(LARGE, param, grad, master, eight, shift=1) for _ in range(2))
    before = snapshot(a)
    scale = torch.full((1,), 0.37, device=DEV)
    whole = zc.AdamWTensors(**a)
    alone = [zc.AdamWTensors(**{k: None if v is None else [v[i]] for k, v in b.items()}) for i in range(len(LARGE))]
    for step in (7, 8):
        zc.adamw(whole, grad_scale=scale, **{**HYPER, "step": step})
        for one in alone:
            zc.adamw(one, grad_scale=scale, **{**HYPER, "step": step})
    assert same(snapshot(a), snapshot(b))
    assert all(not torch.equal(x, y) for x, y in zip(before["params"], a["params"]) if x.numel() > 8)


def test_adamw_8bit_small_second_states_keep_the_least_code():
    # the first value's gradient is 1e7 times the others', whose square roots
    # of v are far below half the block's least code; its own first state
    # passes through 0, so that theirs are kept in full.  The next step then
    # divides m by the least code's value (without one, by eps = 1e-12)
    n, lr, eps, betas = 512, 1.0, 1e-12, (0.5, 0.75)
    s = make([n], F32, F32, False, True)
    for k in ("avg", "sq"):
        s[k][0].view(torch.uint8).zero_()
        s[k + "_scales"][0].zero_()
    s["avg"][0][::256] = -256.0
    s["avg_scales"][0][:] = 1.0 / 256.0                          # m = -1 there
    s["params"][0].zero_()
    g = s["grads"][0]
    g.fill_(1e-7)
    g[::256] = 1.0
    t = zc.AdamWTensors(**s)
    zc.adamw(t, step=1, lr=0.0, betas=betas, eps=eps, weight_decay=0.0)
    m, q = (s[k][0].view(torch.uint8).cpu().view(2, 256) for k in ("avg", "sq"))
    assert (m[:, 0] & 0x7F == 0).all() and (m[:, 1:] == 0x7E).all()          # 0 and 448
    assert (q[:, 0] == 0x7E).all() and (q[:, 1:] == 0x01).all()
    g.zero_()
    zc.adamw(t, step=2, lr=lr, betas=betas, eps=eps, weight_decay=0.0)
    m1 = 0.5 * 0.5 * float(np.float32(1e-7))
    v1 = 0.75 * (0.5 / 448 * 2.0 ** -9) ** 2
    want = -lr / (1 - 0.5 ** 2) * m1 / (np.sqrt(v1 / (1 - 0.75 ** 2)) + eps)
    p = f64(s["params"][0]).reshape(2, 256)
    # the scales carry 3 u, m 2 more, v twice those and 2, its root's product,
    # sum and reciprocal 5, rate and step 4: below 30 u
    assert (np.abs(p[:, 1:] - want) <= 30 * U * abs(want)).all() and not p[:, 0].any()


def f32(t):
    return t.detach().cpu().numpy().astype(np.float32)


@pytest.mark.parametrize("param,grad,master,eight", [c for c in COMBOS if c[0] is F32 or c[2]])
@pytest.mark.parametrize("sizes", SIZES[2:5])
def test_fp32_parameters_take_the_step_as_its_formulas_round_it(param, grad, master, eight, sizes):
    # every operation rounded to fp32 (numpy's are), the same bits
    s = make(sizes, param, grad, master, eight)
    key = "masters" if master else "params"
    one, b1, b2, lr, k = np.float32, *HYPER["betas"], HYPER["lr"], HYPER["step"]
    want = []
    for i in range(len(sizes)):
        x = s["grads"][i].float().cpu().numpy() * one(0.37)
        m, v = s["avg"][i], s["sq"][i]
        if eight:
            code = [ref.E4M3[c.view(torch.uint8).cpu().numpy()].astype(one) for c in (m, v)]
            m, v = (c * np.repeat(f32(s[n][i]), 256)[:sizes[i]] for c, n in zip(code, ("avg_scales", "sq_scales")))
            v = v * v
        else:
            m, v = f32(m), f32(v)
        m = one(b1) * m + one(1.0 - b1) * x
        v = one(b2) * v + one(1.0 - b2) * (x * x)
        den = np.sqrt(v) * one(1.0 / np.sqrt(1.0 - b2 ** k)) + one(HYPER["eps"])
        p = f32(s[key][i]) * one(1.0 - lr * HYPER["weight_decay"]) - one(lr / (1.0 - b1 ** k)) * (m / den)
        assert p.dtype == np.float32
        want.append((p, m, v))
    zc.adamw(zc.AdamWTensors(**s), grad_scale=torch.full((1,), 0.37, device=DEV), **HYPER)
    for i, (p, m, v) in enumerate(want):
        assert np.array_equal(f32(s[key][i]), p)
        assert eight or (np.array_equal(f32(s["avg"][i]), m) and np.array_equal(f32(s["sq"][i]), v))


def test_what_is_not_finite_in_an_8bit_block():
    # a NaN stays in its own value, an infinity leaves none finite in its block
    s = make([1024], BF, F32, True, True)
    s["grads"][0][300], s["grads"][0][700] = float("nan"), -float("inf")
    zc.adamw(zc.AdamWTensors(**s), **HYPER)
    for key in ("avg", "sq"):
        with np.errstate(invalid="ignore"):
            x = ref.decode_e4m3(s[key][0].view(torch.uint8).cpu().numpy(), f64(s[key + "_scales"][0]))
        assert np.isnan(x[300]) and np.isfinite(np.delete(x[:512], 300)).all()
        assert not np.isfinite(x[512:768]).any() and np.isfinite(x[768:]).all()
    p = s["masters"][0]
    assert torch.isfinite(p).sum() == 1022
