"""Router, balance loss, experts and all gradients together, as the example's
layer runs them, against the plain layer in 64 bits with torch's autograd.

The gradients of the logits meet the roundings of the top-k weights' gradients
(sums over rows rounded to bf16, see test_gpu_moe_example: 4 * 8 * 2^-8 of
their norm); the chain through softmax or sigmoid adds errors of fp32."""
import os
import sys

import pytest
import torch

from test_gpu_moe_example import far, plain

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk,score", [(300, 256, 128, 16, 4, "softmax"),
                                                                    (517, 384, 192, 24, 3, "sigmoid")])
def test_training_step(tokens, hidden, inner, experts, topk, score):
    import gpu_path  # noqa: F401  (builds the library)
    import combine_ep_get_gb300 as ep
    import moe_layer
    x, _, _, wu, wd = moe_layer.inputs(tokens, hidden, inner, experts, topk, seed=tokens)
    g = torch.Generator("cuda").manual_seed(2)
    wg = torch.randn((experts, hidden), device="cuda", generator=g) * hidden ** -0.5
    bias = torch.randn(experts, device="cuda", generator=g) * 0.05
    mask = torch.rand(tokens, device="cuda", generator=g) > 0.1
    logits = x.float() @ wg.T
    layer = moe_layer.MoeLayer(wu, wd)
    kind = ep.EP_SCORE_SOFTMAX if score == "softmax" else ep.EP_SCORE_SIGMOID
    idx, weights, loss, kept = layer.route(logits, topk, score=kind, bias=bias, token_mask=mask, coeff=0.3, scale=2.5,
                                           num_groups=4, topk_groups=2)
    out, saved = layer.rows(x, idx, weights, train=True)
    d_out = torch.randn(x.shape, device="cuda", generator=g).to(torch.bfloat16)
    d_loss = torch.full((1,), 2.0, device="cuda")
    d_topk = layer.backward(d_out, saved)[1]
    d_logits = layer.route_backward(d_topk.contiguous(), d_loss, kept)
    assert int(layer.status.item()) == 0

    l = logits.double().requires_grad_()
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    p = s / s.sum(1, keepdim=True)
    there = idx >= 0
    assert torch.equal(there, mask[:, None].expand_as(there))
    chosen = torch.where(there, s.gather(1, idx.clamp_min(0)), 0.0)
    w = 2.5 * chosen / torch.where(mask, chosen.sum(1), 1.0)[:, None]
    n = int(mask.sum())
    f = torch.bincount(idx[there], minlength=experts).double() * experts / (topk * n)
    want_loss = 0.3 * (f * p[mask].sum(0) / n).sum()
    want = plain(x.double(), idx, w, wu.double(), wd.double())
    (want * d_out.double()).sum().add(2.0 * want_loss).backward()
    assert far(out, want.detach()) <= 3 * 2.0 ** -8
    assert abs(float(loss) - float(want_loss)) <= 1e-5 * float(want_loss)
    assert bool((d_logits[~mask] == 0).all())
    assert 0 < far(d_logits[mask], l.grad[mask]) <= 4 * 8 * 2.0 ** -8
