"""Routing and its gradient where the scores vanish and where a token without
experts holds values that are not finite, against the 64-bit references.

Tolerances (u = 2^-24, the fp32 rounding unit; k chosen experts):
  scores   a sigmoid of an exact logit near -88 carries 2 u of exp, 2 u of the
           sum and quotient and up to 4 u where it is a subnormal number (the
           smallest here, 3e-39, is 2^21 times the type's step): 8 u, so a
           normalised one 2 * 8 + k + 2 u; the softmax of exact logits up to
           50 apart the same without the 4 u
  gradient p (g - sum g p) with such p, of numbers up to max |g|: (18 + k) +
           (18 + 2 k) + 4 u twice, below (4 k + 60) 2 u of scale max |g|
"""
import numpy as np
import pytest
import torch

from lossless_bf16_tensor_sign_amd import zc
from tests import ref_ops as ref
from tests.test_gpu_moe import DEV, ROUND, TINY, U, f64, say

pytestmark = pytest.mark.gpu


def check_grad(xd, e, g, score, renorm, scale):
    d = zc.route_grad(xd, e, g, score=score, renorm=renorm, scale=scale)
    xs, es, gs, ds = f64(xd), e.cpu().numpy(), f64(g), f64(d)
    k = es.shape[1]
    for t in range(len(xs)):
        want = ref.route_grad(xs[t], es[t], gs[t], score, renorm, scale)
        tol = (4 * k + 60) * 2 * U * scale * np.abs(gs[t]).max() + np.abs(want) * ROUND[xd.dtype] + TINY[xd.dtype]
        assert (np.abs(ds[t] - want) <= tol).all(), (t, ds[t][es[t]], want[es[t]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,k", [(8, 2), (60, 6), (300, 8), (1000, 32)])
@pytest.mark.parametrize("low", [-80.0, -86.0, -88.5])
@pytest.mark.parametrize("size", [1.0, 300.0, 3e4])
def test_sigmoid_weights_of_tiny_scores_have_their_gradient(dtype, E, k, low, size):
    # the scores are 1e-35 to 3e-39, the weights ordinary, and so is the gradient
    say("route_grad of tiny sigmoids", dtype, E, k, low, size)
    rng = np.random.default_rng(E + k)
    x = np.full((9, E), low, np.float32)
    x[3:] += rng.integers(0, 13, size=(6, E)).astype(np.float32) / 2.0         # exact in bf16
    xd = torch.from_numpy(x).to(dtype).to(DEV)
    e, w = zc.route(xd, k, score="sigmoid")
    assert ((w.sum(1) - 1).abs() < (k + 20) * U).all()
    g = torch.from_numpy((size * rng.normal(size=(9, k))).astype(np.float32)).to(DEV)
    g[0] = size
    g[0, 1] = -size
    check_grad(xd, e, g, "sigmoid", True, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,k", [(16, 3), (64, 8), (200, 5), (400, 8), (1024, 32)])
def test_softmax_weights_of_experts_that_only_the_bias_chooses(dtype, E, k):
    # the upper half's logits lie 150 to 200 below the others': their softmax
    # is zero in fp32, their shares of each other are not
    say("route of vanishing softmax scores", dtype, E, k)
    rng = np.random.default_rng(E)
    h = E // 2
    x = rng.integers(-8, 9, size=(12, E)).astype(np.float32) / 4.0
    x[:, h:] = -200.0 + rng.integers(0, 51, size=(12, E - h))
    x[7:, 0] = 3.0                                                # ties with nothing: a number that counts
    b = np.zeros(E, np.float32)
    b[h:] = 2.0 + rng.permutation(E - h) / 8.0
    b[0] = 1e3 if k > 1 else 0.0                                  # and one of the lower half that always wins
    for bias, tokens in ((b, slice(7, 12)), (np.where(np.arange(E) == 0, 0.0, b).astype(np.float32), slice(0, 7))):
        xd = torch.from_numpy(x[tokens]).to(dtype).to(DEV)
        e, w = zc.route(xd, k, score="softmax", bias=torch.from_numpy(bias).to(DEV), scale=1.5)
        xs, bs = f64(xd), bias.astype(np.float64)
        for t in range(len(xs)):
            re, rw = ref.route(xs[t], k, "softmax", bs, renorm=True, scale=1.5)
            assert np.array_equal(e[t].cpu().numpy(), re)
            assert np.allclose(f64(w[t]), rw, rtol=2 * (k + 40) * U, atol=1e-37), (t, f64(w[t]), rw)
        g = torch.from_numpy(rng.normal(size=tuple(w.shape)).astype(np.float32)).to(DEV)
        check_grad(xd, e, g, "softmax", True, 1.5)


def test_softmax_weights_of_fewer_experts_than_choices():
    inf = float("inf")
    x = torch.full((3, 6), -inf)
    x[0, 2:4] = torch.tensor([-150.0, -151.0])
    x[1] = torch.tensor([0.0, 0.0, -150.0, -151.0, -inf, 0.0])
    b = torch.tensor([-inf, -inf, 0.0, 0.0, 0.0, -inf])
    e, w = zc.route(x.to(DEV), 4, bias=b.to(DEV))
    p = 1.0 / (1.0 + np.exp(-1.0))
    assert e.cpu().tolist() == [[2, 3, -1, -1], [2, 3, -1, -1], [-1] * 4]
    assert np.allclose(f64(w), [[p, 1 - p, 0, 0], [p, 1 - p, 0, 0], [0] * 4], rtol=88 * U, atol=0)


@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (300, 8), (1000, 20)])
def test_softmax_token_with_a_logit_that_is_not_finite_has_nan_weights(E, k):
    # also where the logit's own expert is not chosen
    x = torch.zeros(3, E)
    x[0, E - 1], x[1, E - 1] = float("nan"), float("inf")
    b = torch.zeros(E)
    b[E - 1] = -float("inf")
    for renorm in (False, True):
        e, w = zc.route(x.to(DEV), k, bias=b.to(DEV), renorm=renorm)
        assert torch.isnan(w[:2]).all() and torch.isfinite(w[2]).all() and (e == torch.arange(k, device=DEV)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (200, 8), (512, 3), (1000, 32)])
def test_token_without_experts_has_no_gradient_whatever_its_logits(dtype, score, renorm, E, k):
    # a padding token's row may hold anything
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(9, E, dtype=dtype)
    x[0], x[1], x[2], x[3] = nan, inf, -inf, torch.finfo(dtype).min
    x[4, E - 1], x[5, 0], x[6, E // 2] = nan, inf, -inf
    xd = x.to(DEV)
    valid = torch.zeros(9, dtype=torch.bool, device=DEV)
    valid[8] = True
    e, w = zc.route(xd, k, score=score, renorm=renorm, valid=valid)
    assert (e[:8] == -1).all() and not w[:8].any()
    g = torch.ones(9, k, device=DEV)
    g[8, 0] = 2.0
    g[:4] = nan                                                   # nor do the weights' gradients count
    d = zc.route_grad(xd, e, g, score=score, renorm=renorm)
    assert not d[:8].any()
    assert torch.isfinite(d[8]).all() and d[8].any()
