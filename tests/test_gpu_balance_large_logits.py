"""Balance loss and gradient where logits are large: rows of the type's lowest
value (a mask's), of values near its largest, and of 1e10 with a few last places
between them.

Bounds.  Normalised softmax scores see differences of logits alone, so `bound`
counts with them: u = 2^-24, l - max is rounded once (off by u R, R its size),
its product with log2(e) twice (the constant and the product), the hardware's
2^x is off by 2 units of its last place, and what is below 2^-126 is lost.  With
R at most 104 (2^-150 is nothing to a sum of 1 or more) a score is
good to (3 R + 4) u, a sum of E of them to (3 R + 4 + E / 32 + 8) u, the
reciprocal and the product to 4 u more: twice (3 R + E / 32 + 32) u holds a
ratio.  A sigmoid is shifted by its row's largest logit below -16 and has its
logit's size in the place of the difference above: R + 16.
"""
import pytest
import torch

import route_reference as ref
from test_gpu_route import TYPES, gen, run_balance, status

pytestmark = pytest.mark.gpu


def bound(l, score):
    l = l.double()
    gap = l.amax(1, keepdim=True) - l
    R = torch.where(gap < 104.0, gap, 0.0).amax(1) + (16.0 if score == "sigmoid" else 0.0)
    return 2 * (3 * R + l.shape[1] / 32 + 32) * ref.U


def rows(dtype, E):
    """Rows of large logits of either sign, and ordinary ones between them."""
    g, t = gen(E), TYPES[dtype]
    info = torch.finfo(t)
    low, high = info.min, info.max
    some = torch.rand((6, E), generator=g, device="cuda")
    out = [torch.full((E,), low), torch.full((E,), high), torch.full((E,), low / 2), torch.full((E,), high / 2)]
    for v in (low, high):        # two of them away from the rest
        r = torch.full((E,), v)
        r[E // 3] = r[E // 2] = v / 2
        out.append(r)
    r = torch.full((E,), low)    # all but a few masked
    r[::7] = torch.arange(0, E, 7).float() / E
    out.append(r)
    out = [r.to("cuda") for r in out]
    size = 1e10 if dtype != "fp16" else 3e4
    step = size * info.eps
    for sign in (1.0, -1.0):     # last places apart (in fp32 and bf16 many units)
        out.append(sign * size + step * torch.floor(some[0] * 3))
        out.append(sign * 1e4 * (1 + info.eps * torch.floor(some[1] * 8)))
    out += [some[2] * 4, -some[3] * 4]
    return torch.stack([r.to(t) for r in out])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E", [5, 64, 200, 256, 600, 2048])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_loss_of_large_logits(dtype, E, score):
    l = rows(dtype, E)
    T, K = l.shape[0], 3
    idx = ref.route(l, K, score)[0].contiguous()
    off = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    for o in (None, off):        # all tokens; a sequence each
        loss, load, counts = run_balance(l, idx, score, o, coeff=0.5)
        want, want_load, want_counts = ref.balance(l, idx, score, o, None, 0.5)
        assert torch.equal(counts.long(), want_counts)
        assert bool(((load.double() - want_load).abs() <= 16 * ref.U * want_load).all())
        # every term is positive; tiles, sequences and chunks add in fewer than 150 steps
        assert abs(float(loss) - float(want)) <= (float(bound(l, score).amax()) + 150 * 2 * ref.U) * float(want)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E", [5, 64, 200, 256, 600, 2048])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_large_logits(dtype, E, normalize, score):
    from gpu_path import B
    l = rows(dtype, E)
    T, K = l.shape[0], 4
    idx = ref.route(l, K, score)[0].contiguous()
    g = gen(E + 1)
    dw = torch.randn((T, K), generator=g, device="cuda")
    load, d_loss = torch.rand((1, E), generator=g, device="cuda"), torch.rand(1, generator=g, device="cuda") + 0.5
    for kw in (dict(d_weights=dw), dict(load=load, d_loss=d_loss), dict(d_weights=dw, load=load, d_loss=d_loss)):
        out, st = torch.empty_like(l), status()
        B.ep_route_backward(l, idx, out, st, d_topk_weights=kw.get("d_weights"), load=kw.get("load"), d_loss=kw.get("d_loss"),
                            score=B.EP_SCORE_SOFTMAX if score == "softmax" else B.EP_SCORE_SIGMOID, normalize=normalize,
                            scale=1.5)
        assert int(st.item()) == 0
        want, loose = ref.backward(l, idx, score, normalize=normalize, scale=1.5, **kw)
        # the same sums of absolute values, by the bound above; lost below 2^-126: at most 2^-124 of what it is multiplied by
        big = loose / (2 * ref.relative(l.double())[:, None])
        most = ref.rounded(want, big * 2 * bound(l, score)[:, None] + 2.0 ** -120, l.dtype)
        off = (out.double() - want).abs()
        assert bool((off <= most).all()), (off / most).amax(1)
