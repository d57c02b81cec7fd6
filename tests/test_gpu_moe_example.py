"""The example layer end to end: the few-token call, the rows path and its
backward pass against the plain layer in 64 bits with torch's autograd.

The norms of the differences are bounded by the roundings to bf16 on the way,
each at most 2^-8 of the value rounded: x, weights and saved pre-activations
are exact inputs or used as saved; the forward rounds h, each expert's output
and the sum (3); a gradient meets, beside those of the forward values it uses
(h, both z), the roundings of dy, dz and dh, its own and the combine's (at
most 8 in all, each passed on with a factor of order 1: slopes of silu and the
ratio of a value's norm to its gate's; 4 is allowed for it)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def plain(x, idx, tw, wu, wd):
    out = torch.zeros_like(x)
    for e in range(wu.shape[0]):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        g, u = (x[t] @ wu[e].T).chunk(2, dim=1)
        out = out.index_add(0, t, (torch.nn.functional.silu(g) * u) @ wd[e].T * tw[t, k][:, None])
    return out


def far(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk,ranks", [(200, 256, 192, 8, 3, 4), (777, 512, 136, 20, 5, 1)])
def test_layer_and_its_gradients(tokens, hidden, inner, experts, topk, ranks):
    import gpu_path  # noqa: F401  (builds the library)
    import moe_layer
    x, idx, tw, wu, wd = moe_layer.inputs(tokens, hidden, inner, experts, topk, seed=tokens)
    idx[::7, 0] = -1
    idx[5] = -1
    layer = moe_layer.MoeLayer(wu, wd, ranks)
    leaves = [t.double().requires_grad_() for t in (x, tw, wu, wd)]
    want = plain(leaves[0], idx, leaves[1], leaves[2], leaves[3])
    out, saved = layer.rows(x, idx, tw, train=True)
    assert far(out, want.detach()) <= 3 * 2.0 ** -8
    assert torch.equal(out, layer.rows(x, idx, tw))
    few = layer.few_tokens(x[:100], idx[:100], tw[:100])
    assert far(few, want.detach()[:100]) <= 2 * 2.0 ** -8
    d_out = torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    want.backward(d_out.double())
    got = layer.backward(d_out, saved)
    for name, a, leaf in zip(("x", "topk_weights", "w_up", "w_down"), got, leaves):
        assert far(a, leaf.grad) <= 4 * 8 * 2.0 ** -8, name
        assert far(a, leaf.grad) > 0
    assert bool((got[1][idx < 0] == 0).all())
    assert int(layer.status.item()) == 0


def test_example_runs():
    import gpu_path  # noqa: F401
    import moe_layer
    sys.argv = ["moe_layer.py", "--tokens", "300", "--hidden", "256", "--inner", "128", "--experts", "8"]
    assert moe_layer.main() == 0
