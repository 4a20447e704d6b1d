"""Routing at the limits between its kernel's forms.  Tolerances as in
test_gpu_moe.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_moe import check_route, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("E,groups,top,k", [(512, 2, 1, 8), (1024, 2, 1, 32), (512, 4, 1, 9), (256, 2, 1, 8),
                                            (128, 2, 1, 4), (16, 2, 1, 3), (1024, 8, 3, 12), (6, 2, 1, 3)])
def test_groups_of_many_lanes(group_score, E, groups, top, k):
    # one logit of a token is above the others, at any place of any group: a
    # group's score has to come from all of its lanes
    say("route, groups of", E // groups, group_score)
    rng = np.random.default_rng(E + groups)
    T = 16
    x = rng.integers(-3, 2, size=(T, E)).astype(np.float32)
    at = rng.integers(0, E, size=T)
    at[:4] = [0, E - 1, E // groups - 1, E // groups]
    x[np.arange(T), at] = 2.0
    x = torch.from_numpy(x)
    for score in ("sigmoid", "softmax"):
        e, _ = check_route(x, k, torch.float32, score, groups=groups, top_groups=top, group_score=group_score)
        # (two others may sum to more than it and its second)
        assert group_score == "top2" or np.array_equal(e[:, 0].cpu().numpy(), at)
        check_route(x, k, torch.bfloat16, score, groups=groups, top_groups=top, group_score=group_score, renorm=False)
