"""Experts that an infinite bias puts before all others, more of them than a token's
groups or slots take: the lower index wins, of groups and of experts."""
import numpy as np
import pytest
import torch

from test_gpu_block import INF, check_route, logits_of
from test_gpu_prompt import dev, rng  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [19, 4101])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(64, 8, 2, 8), (128, 16, 6, 8), (128, 4, 2, 6), (256, 8, 4, 8),
                                            (256, 4, 1, 8), (160, 8, 3, 6), (60, 4, 2, 6), (1024, 32, 3, 12)])
def test_groups_of_infinite_scores(dev, E, groups, top, k, score, T):  # noqa: F811
    r = rng(93, E, groups)
    z = logits_of(T, E, torch.float32, 94, masked=2)
    rows = np.arange(T) if T < 50 else np.concatenate([np.arange(12), [T - 1]])
    for share in (0.03, 0.1, 0.2, 0.25, 0.3, 0.4, 1.0):
        bias = 0.1 * r.standard_normal(E)
        bias[r.random(E) < share] = INF
        for dtype in (torch.float32, torch.bfloat16):
            for group_score in ("max", "top2"):
                check_route(dev, z.to(dtype), k, bias, rows, score=score, groups=groups, top_groups=top,
                            group_score=group_score)


def test_one_infinity_a_group_and_finite_ties(dev):  # noqa: F811
    # each group's largest is infinite, and so is the sum of two
    bias = np.zeros(64)
    bias[::8] = INF
    z = logits_of(9, 64, torch.float32, 95)
    for group_score in ("max", "top2"):
        ids, _ = check_route(dev, z, 3, bias, score="sigmoid", groups=8, top_groups=3, group_score=group_score)
        assert ids[:, :3].cpu().tolist() == [[0, 8, 16]] * 9
