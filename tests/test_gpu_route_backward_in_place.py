"""The router's gradient written over its logits: what slots read of a row by its
experts' numbers is read before other lanes write the row."""
import pytest
import torch

import route_reference as ref
from test_gpu_route import TYPES, gen, make_logits, offsets, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (700, 33, 32), (900, 256, 8), (5000, 64, 6), (60, 1000, 16), (30, 2048, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_in_place_gives_what_another_tensor_gets(T, E, K, score, normalize):
    from gpu_path import B
    for i, dtype in enumerate(TYPES):
        g = gen(T + E + i)
        pad = (0, 3, 8)[i]
        wide = torch.full((T + 1, E + pad), -77.0, dtype=TYPES[dtype], device="cuda")
        l = make_logits(g, T, E, dtype)
        wide[:T, :E] = l
        mask = torch.rand(T, generator=g, device="cuda") > 0.2
        idx = ref.route(l, K, score, mask=mask)[0].contiguous()
        idx[::7] = idx[::7, :1]          # one expert in every slot
        dw = torch.randn((T, K), generator=g, device="cuda")
        load, d_loss = torch.rand((2, E), generator=g, device="cuda"), torch.ones(1, device="cuda")
        off = offsets(0, T // 3, T - T // 5)
        kw = dict(score=B.EP_SCORE_SOFTMAX if score == "softmax" else B.EP_SCORE_SIGMOID, token_mask=mask,
                  normalize=normalize, d_topk_weights=dw, load=load, d_loss=d_loss, seq_offset=off)
        out, st = torch.empty((T, E), dtype=TYPES[dtype], device="cuda"), status()
        B.ep_route_backward(wide[:T, :E], idx, out, st, **kw)
        B.ep_route_backward(wide[:T, :E], idx, wide[:T, :E], st, **kw)
        assert int(st.item()) == 0
        assert torch.equal(wide[:T, :E], out)
        assert bool((wide[T:] == -77.0).all()) and bool((wide[:, E:] == -77.0).all())
