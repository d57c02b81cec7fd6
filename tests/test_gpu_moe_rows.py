"""The example layer's outputs and gradients row by row and expert by expert
against the plain layer in 64 bits: one row lost or mixed up shows, where a norm
over a whole tensor would hide it.

Bounds.  A result passes at most 8 roundings to bf16 (h, both z, dy, dz, dh, its
own, the combine's), each of an rms of at most 2^-8 / sqrt(3) of the value
rounded and independent of the others, so that they add in squares; each is
passed on with a factor of order 1, for which 4 is allowed, as in the test of
the whole tensors.  Norms over the 256 and more elements of a row, or of an
expert's matrix, then differ by at most 4 sqrt(8 / 3) 2^-8 = 2.6%.  The top-k
weights lie between 1 and 2, so that no entry is small: one that is lost changes
its row of x's gradient by 26% and its expert's matrices by 3.4% at least (the
64-bit layer with one entry masked, over 50 tokens of each case).  A top-k weight's gradient is a sum of products dy y of random signs: four
times that part of the root of their squares' sum."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

PART = 4 * math.sqrt(8 / 3) * 2.0 ** -8


def plain(x, idx, tw, wu, wd):
    """The layer's output and each entry's expert output, [T, K, H]."""
    T, K = idx.shape
    y = x.new_zeros((T * K, x.shape[1]))
    for e in range(wu.shape[0]):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        g, u = (x[t] @ wu[e].T).chunk(2, dim=1)
        y = y.index_copy(0, t * K + k, (torch.nn.functional.silu(g) * u) @ wd[e].T)
    y = y.view(T, K, -1)
    return (y * tw[:, :, None]).sum(1), y


def rows_close(got, want, what):
    off, size = (got.double() - want).flatten(1).norm(dim=1), want.flatten(1).norm(dim=1)
    bad = off > PART * size
    assert not bool(bad.any()), "%s: %d rows, first %d, %.3g of its norm" % (
        what, int(bad.sum()), int(bad.int().argmax()), float((off / size)[bad][0]))


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk,ranks", [(200, 256, 192, 8, 3, 4), (777, 512, 136, 20, 5, 1),
                                                                  (130, 264, 264, 3, 2, 1)])
def test_every_row_and_expert(tokens, hidden, inner, experts, topk, ranks):
    import gpu_path  # noqa: F401  (builds the library)
    import moe_layer
    x, idx, tw, wu, wd = moe_layer.inputs(tokens, hidden, inner, experts, topk, seed=tokens + 1)
    idx[::7, 0] = -1
    idx[5] = -1
    tw = tw + 1.0
    layer = moe_layer.MoeLayer(wu, wd, ranks)
    leaves = [t.double().requires_grad_() for t in (x, tw, wu, wd)]
    want, y = plain(leaves[0], idx, leaves[1], leaves[2], leaves[3])
    d_out = torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(torch.bfloat16)
    want.backward(d_out.double())
    out, saved = layer.rows(x, idx, tw, train=True)
    rows_close(out, want.detach(), "out")
    few = layer.few_tokens(x[-100:].clone(), idx[-100:].clone(), tw[-100:].clone())   # (16-byte alignment)
    rows_close(few, want.detach()[-100:], "few tokens")
    dx, d_topk, d_up, d_down = layer.backward(d_out, saved)
    rows_close(dx, leaves[0].grad, "x")
    rows_close(d_up, leaves[2].grad, "w_up")
    rows_close(d_down, leaves[3].grad, "w_down")
    size = (d_out.double()[:, None, :] * y.detach()).norm(dim=2)
    off = (d_topk.double() - leaves[1].grad).abs()
    assert bool((off <= 4 * PART * size).all()), "topk_weights: %.3g" % float((off / size).nan_to_num(0).max())
    assert int(layer.status.item()) == 0
