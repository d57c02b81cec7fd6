"""The reference of the router's gradient against differences of its forward
reference, in 64 bits on the CPU."""
import pytest
import torch

import route_reference as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("part", ["weights", "loss", "both"])
def test_the_formula_against_differences(score, normalize, part):
    g = torch.Generator().manual_seed(3)
    T, E, K, S = 9, 7, 3, 3
    l = torch.randn((T, E), generator=g, dtype=torch.float64) * 1.5
    offset = torch.tensor([0, 4, 4, 8])      # an empty sequence, and one token behind the last
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 1, 1, 1], dtype=torch.bool)
    idx, _ = ref.route(l, K, score, mask=mask)
    idx[5, 1] = -1
    dw = torch.randn((T, K), generator=g, dtype=torch.float64)
    d_loss = torch.tensor([0.7], dtype=torch.float64)
    load = ref.balance(l, idx, score, offset, mask)[1]
    args = dict(d_weights=dw if part != "loss" else None, load=load if part != "weights" else None,
                d_loss=d_loss if part != "weights" else None)
    got, bound = ref.backward(l, idx, score, offset=offset, mask=mask, normalize=normalize, scale=2.5, **args)

    def value(l):
        out = 0.0
        if part != "weights":
            out = out + d_loss[0] * ref.balance(l, idx, score, offset, mask)[0]
        if part != "loss":
            there = (idx >= 0) & mask[:, None]
            s = ref.scores(l, score)[0].gather(1, idx.clamp_min(0)) * there
            w = s / s.sum(1, keepdim=True).clamp_min(1e-300) if normalize else s
            out = out + (w * 2.5 * dw).sum()
        return out

    step = 1e-5
    for t in range(T):
        for e in range(E):
            hi, lo = l.clone(), l.clone()
            hi[t, e] += step
            lo[t, e] -= step
            # differences: h^2 / 6 of a third derivative of order 1, and 2^-52 / h of values of order 10
            assert abs(float((value(hi) - value(lo)) / (2 * step) - got[t, e])) < 1e-8
    assert bool((got[2] == 0).all()) and bool((bound >= 0).all()) and bool((got != 0).any())


def test_the_choice_by_hand():
    l = torch.tensor([[0.0, 3.0, 3.0, -float("inf"), 1.0, 2.0]])
    idx, w = ref.route(l, 3, "softmax")
    assert idx.tolist() == [[1, 2, 5]] and abs(float(w.sum()) - 1.0) < 1e-12
    idx, _ = ref.route(l, 3, "sigmoid", groups=3, topk_groups=2)       # the closed one leaves its group one member
    assert idx.tolist() == [[1, 5, 4]]     # pairs add up to 0.5 + 0.95, 0.95, 0.73 + 0.88
    idx, w = ref.route(torch.full((1, 4), -float("inf")), 2, "softmax")
    assert idx.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]
