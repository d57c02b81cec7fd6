"""The router's choice by score + bias where fp32 cannot tell two values apart:
it is the choice in 64 bits, whatever makes fp32 err: a sum of many
exponentials, a bias far larger than the sums that it cancels from, a tie
at the last slot."""
import pytest
import torch

import route_reference as ref
from test_gpu_route import check_route, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [256, 512, 1024, 2048])
@pytest.mark.parametrize("groups", [1, 8])
def test_one_expert_far_above_many(E, groups):
    """One logit of 0, the others near -16.7: what the others add to the largest one's exponential, one after another, is
    below its last place.  A bias sweeps another expert (of another group) through the first one's c."""
    l = torch.full((3, E), -16.7, device="cuda")
    l[:, 0] = 0.0
    l[1:, 1:] += (torch.rand((2, E - 1), generator=gen(E), device="cuda") - 0.5) * 0.2
    other = E // 8
    s = torch.softmax(l[:1].double(), 1)[0]
    for step in range(-60, 61):
        bias = torch.zeros(E, device="cuda")
        bias[other] = float(s[0] - s[other]) + step * 7e-8
        check_route(l, 2, "softmax", bias=bias, groups=groups, topk_groups=1)
