"""Routing and its gradient where the scores vanish, against the 64-bit
references.

Tolerances (u = 2^-24, the fp32 rounding unit; k chosen experts):
  scores   a sigmoid of an exact logit near -88 carries 2 u of exp, 2 u of the
           sum and quotient and up to 4 u where it is a subnormal number (the
           smallest here, 3e-39, is 2^21 times the type's step): 8 u, so a
           normalised one 2 * 8 + k + 2 u
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
