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


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("topk_groups", [1, 2, 3])
def test_groups_whose_large_biases_cancel(score, topk_groups):
    """Two experts of a group have biases of 1000 and -1000: c rounds by 3e-5, the group's sum is about the others'.  Their
    sums lie within 5e-5 of one another."""
    T, E, G = 600, 12, 4
    g = gen(topk_groups)
    l = torch.randn((T, E), generator=g, device="cuda") * 0.01
    l[:, 2::3] -= 6.0                                  # (the third of a group is far below)
    l[:, ::3] += (torch.rand((T, G), generator=g, device="cuda") - 0.5) * (2e-4 if score == "sigmoid" else 6e-4)
    # one value for both of a group's two best: their sum is what moves
    l[:, 1::3] = l[:, ::3].mean(1, keepdim=True)
    l[:, ::3] = l[:, 1::3] + (l[:, ::3] - l[:, 1::3]) * 0.01
    bias = torch.zeros(E, device="cuda")
    bias[3], bias[4], bias[5] = 1000.0, -1000.0, -2000.0
    check_route(l, 2, score, bias=bias, groups=G, topk_groups=topk_groups)
    check_route(l, 2, score, bias=bias + 0.125, groups=G, topk_groups=topk_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_a_tie_at_the_last_slot_and_a_third_value_next_to_it(score, groups):
    """The last slot's expert and the next are of one logit and one bias; a third one's c, of another logit and bias, lies
    within fp32's last places of theirs."""
    T, E, K = 4000, 40, 2
    g = gen(groups)
    l = torch.full((T, E), -9.0, device="cuda")
    l[:, 7] = 3.0
    tied = torch.rand(T, generator=g, device="cuda") * 0.5 + 1.0
    l[:, 11] = l[:, 12] = tied
    bias = torch.zeros(E, device="cuda")
    bias[33] = 0.0625
    # the third one's logit: c = that of the tied ones, within a few last places
    off = (torch.rand(T, generator=g, device="cuda", dtype=torch.float64) - 0.5) * 3e-7
    if score == "sigmoid":
        want = torch.sigmoid(tied.double()) - 0.0625 + off
        l[:, 33] = torch.logit(want).float()
    else:
        # e^x / (rest + e^x) = s of the tied ones - bias, which x changes too: to its fixed point
        rest = torch.exp(l.double()).sum(1) - torch.exp(l[:, 33].double())
        x = torch.exp(tied.double()) * 0.5
        for _ in range(200):
            x = (torch.exp(tied.double()) / (rest + x) - 0.0625 + off) * (rest + x)
        l[:, 33] = torch.log(x).float()
    check_route(l, K, score, bias=bias, groups=groups, topk_groups=groups)
    if groups > 1:
        check_route(l, K, score, bias=bias, groups=groups, topk_groups=groups - 1)


@pytest.mark.parametrize("E", [256, 512, 1024, 2048])
def test_a_value_behind_the_next_one_that_fp32_knows_less_well(E):
    """One logit of 0 among others near -16.6, each of which adds a whole last place to the largest one's exponential: its
    score comes out too small.  Two experts of small scores, known far better, lie next to one another at the last slot;
    the first one's c, by a bias, lies behind both in fp32 and sweeps through them in 64 bits."""
    l = torch.full((2, E), -16.6, device="cuda")
    l[:, 0] = 0.0
    l[1, 1:] += (torch.rand(E - 1, generator=gen(E), device="cuda") - 0.5) * 0.05
    s = torch.softmax(l[:1].double(), 1)[0]
    for gap in (1.2e-7, 2.4e-7, 5e-7, 1e-6):
        for step in range(-50, 51):
            bias = torch.zeros(E, device="cuda")
            bias[E // 3], bias[E // 2] = 0.5, 0.5 - gap
            bias[0] = float(0.5 - s[0]) + step * 6e-8
            for K in (1, 2):
                check_route(l, K, "softmax", bias=bias)
