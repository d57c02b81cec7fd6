"""The router's calls on the GPU against their definitions in 64 bits: the
choice exactly, weights, loss and gradients within bounds of fp32 arithmetic."""
import math

import pytest
import torch

import route_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
INF = math.inf


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_logits(g, T, E, dtype, pad=0, std=1.5):
    wide = torch.randn((T, E + pad), generator=g, device="cuda") * std + torch.randn(E + pad, generator=g, device="cuda")
    return wide.to(TYPES[dtype])[:, pad // 2:pad // 2 + E]


def guarded(T, K, dtype, fill):
    """A [T, K] tensor with rows behind it that no call may touch."""
    whole = torch.full((T + 3, K), fill, dtype=dtype, device="cuda")
    return whole, whole[:T]


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def run_route(l, K, score, bias=None, mask=None, **kw):
    from gpu_path import B
    T = l.shape[0]
    idx_all, idx = guarded(T, K, torch.int64, -77)
    w_all, w = guarded(T, K, torch.float32, -77.0)
    st = status()
    B.ep_route(l, idx, w, st, score=B.EP_SCORE_SOFTMAX if score == "softmax" else B.EP_SCORE_SIGMOID, bias=bias,
               token_mask=mask, num_groups=kw.pop("groups", 1), **kw)
    assert bool((idx_all[T:] == -77).all()) and bool((w_all[T:] == -77.0).all())
    assert int(st.item()) == 0
    return idx, w


def check_route(l, K, score, bias=None, mask=None, **kw):
    idx, w = run_route(l, K, score, bias, mask, **kw)
    want_idx, want = ref.route(l, K, score, bias, mask, **kw)
    assert torch.equal(idx, want_idx)
    bound = ref.relative(l.double())[:, None] * want.abs()
    assert bool(((w.double() - want).abs() <= bound + 1e-43).all())
    return idx, w


SHAPES = [(1, 1, 1), (3, 2, 1), (5, 7, 7), (17, 32, 8), (129, 33, 4), (77, 60, 6), (128, 64, 8), (301, 96, 32),
          (64, 160, 6), (1000, 255, 8), (513, 256, 8), (40, 257, 16), (33, 512, 10), (9, 1000, 32), (6, 2048, 8)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_and_weights(T, E, K, score):
    for i, dtype in enumerate(TYPES):
        g = gen(T * 31 + E + i)
        l = make_logits(g, T, E, dtype, pad=(0, 1, 8)[i])
        check_route(l, K, score, normalize=True)
        check_route(l, K, score, normalize=False, scale=2.5)
        # steps of 0.001: many c that only the score's last bits tell apart, and exact ties
        bias = torch.round(torch.randn(E, generator=g, device="cuda") * 30) * 0.001
        mask = torch.rand(T, generator=g, device="cuda") > 0.3
        check_route(l, K, score, bias=bias, mask=mask, scale=1.7)
        check_route(l, K, score, bias=torch.zeros_like(bias), mask=mask.to(torch.uint8), normalize=False)


@pytest.mark.parametrize("T,E,K,groups,topk_groups", [(300, 256, 8, 8, 4), (300, 60, 6, 6, 3), (65, 96, 5, 32, 5),
                                                      (33, 8, 3, 8, 3), (50, 2048, 8, 16, 2), (31, 66, 1, 2, 1),
                                                      (20, 256, 8, 8, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(T, E, K, groups, topk_groups, score):
    for i, dtype in enumerate(TYPES):
        g = gen(E + i)
        l = make_logits(g, T, E, dtype)
        bias = torch.round(torch.randn(E, generator=g, device="cuda") * 30) * 0.001
        check_route(l, K, score, groups=groups, topk_groups=topk_groups)
        check_route(l, K, score, bias=bias, groups=groups, topk_groups=topk_groups, scale=2.5)
        # closed experts, whole groups of them
        l = l.clone()
        l[torch.rand((T, E), generator=g, device="cuda") < 0.6] = -INF
        l[::3, :E // groups] = -INF
        check_route(l, K, score, bias=bias, groups=groups, topk_groups=topk_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 3)])
def test_equal_and_nearly_equal_values(score, groups, topk_groups):
    E, K = 64, 8
    for biased in (False, True):
        # all equal; two values; values one step of fp32 apart, with a bias that nearly makes up for it
        g = gen(5)
        rows = [torch.zeros(E), torch.full((E,), -3.0), torch.arange(E) % 2 * 1.0, -(torch.arange(E) // 8) * 0.5]
        l = torch.stack(rows + [torch.nextafter(torch.full((E,), 0.5 + i), torch.tensor(9.0)) if i % 2 else
                                torch.full((E,), 0.5 + i) for i in range(8)]).cuda()
        near = torch.rand((200, E), generator=g, device="cuda") * 1e-6 + 0.25
        l = torch.cat([l, near])
        bias = torch.randint(-2, 3, (E,), generator=g, device="cuda") * 2.0 ** -24 if biased else None
        check_route(l, K, score, bias=bias, groups=groups, topk_groups=topk_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinities_and_nan(score):
    E, K = 40, 4
    l = make_logits(gen(1), 12, E, "fp32")
    l[0] = -INF                                  # nothing open
    l[1, 2:] = -INF                              # fewer open than slots
    l[2, 5] = l[2, 9] = float("nan")
    l[3, 7] = INF
    l[4] = -200.0                                # sigmoids below the least number
    l[4, 3] = -190.0
    l[5] = 3.0e38
    l[6, ::2] = -3.0e38
    idx, w = run_route(l, K, score)
    want_idx, want = ref.route(l, K, score)
    assert torch.equal(idx, want_idx)
    assert idx[2, :2].tolist() == [5, 9] and bool(torch.isnan(w[2]).all())
    assert (idx[3, 0] == 7) and bool(torch.isnan(w[3]).all()) == (score == "softmax")
    ok = [r for r in range(12) if r != 2 and not (r == 3 and score == "softmax")]
    assert bool((w[ok].double() - want[ok]).abs().max() < 1e-4)
    assert w[0].tolist() == [0.0] * K and w[1, 2:].tolist() == [0.0] * (K - 2)
    # a bias opens and closes: what is -inf is closed, +inf always chosen
    bias = torch.zeros(E, device="cuda")
    bias[11], bias[12] = -INF, INF
    idx, _ = run_route(l, K, score, bias=bias)
    assert bool((idx != 11).all()) and bool((idx[7:, 0] == 12).all())


def run_balance(l, idx, score, offset=None, mask=None, coeff=1.0, want_status=0):
    from gpu_path import B
    T, E = l.shape
    S = 1 if offset is None else offset.numel() - 1
    loss = torch.full((1,), -7.0, device="cuda")
    load = torch.full((S, E), -7.0, device="cuda")
    counts = torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((B.ep_balance_loss_workspace_bytes(T, E, S),), 0xA5, dtype=torch.uint8, device="cuda")
    st = status()
    B.ep_balance_loss(l, idx, ws, loss, load, st, score=B.EP_SCORE_SOFTMAX if score == "softmax" else B.EP_SCORE_SIGMOID,
                      token_mask=mask, seq_offset=offset, coeff=coeff, num_tokens_per_expert=counts)
    assert int(st.item()) == want_status
    return loss, load, counts


def check_balance(l, idx, score, offset=None, mask=None, coeff=0.01, want_status=0):
    loss, load, counts = run_balance(l, idx, score, offset, mask, coeff, want_status)
    want, want_load, want_counts = ref.balance(l, idx, score, offset, mask, coeff)
    assert torch.equal(counts.long(), want_counts)
    assert bool(((load.double() - want_load).abs() <= 16 * ref.U * want_load).all())
    # every term is positive: a sum of T of them, tile by tile, passes each through fewer than T / 2400 + 150 additions
    T = l.shape[0]
    rel = float(ref.relative(torch.where(torch.isfinite(l.double()), l.double(), 0.0)).amax()) if T else 0.0
    assert abs(float(loss) - float(want)) <= (rel + (T / 2400 + 150) * 2 * ref.U) * abs(float(want))
    return loss, load


def offsets(*at):
    return torch.tensor(at, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T,E,K", SHAPES + [(5000, 256, 8), (20000, 64, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_loss(T, E, K, score):
    for i, dtype in enumerate(TYPES):
        g = gen(T + E + i)
        l = make_logits(g, T, E, dtype, pad=(8, 0, 1)[i])
        mask = torch.rand(T, generator=g, device="cuda") > 0.2
        idx = ref.route(l, K, score, mask=mask)[0].contiguous()
        check_balance(l, idx, score)
        check_balance(l, idx, score, mask=mask, coeff=3.0)
        # ragged: an empty first one, one token, the rest in two, some tokens in none
        a, b = min(1, T), max(min(1, T), T // 2)
        check_balance(l, idx, score, offset=offsets(0, 0, a, b, T - T // 5 if T > 10 else T), mask=mask)
        if T > 10:
            check_balance(l, idx, score, offset=offsets(T // 4, T // 3, T // 3, T // 2))


def test_balance_many_short_sequences():
    g = gen(9)
    T, E, K = 900, 24, 3
    l = make_logits(g, T, E, "bf16")
    idx = ref.route(l, K, "softmax")[0].contiguous()
    cuts = torch.sort(torch.randint(0, T + 1, (400,), generator=g, device="cuda")).values.to(torch.int32)
    check_balance(l, idx, "softmax", offset=cuts)


def test_balance_without_tokens():
    E = 48
    l = torch.zeros((0, E), device="cuda")
    idx = torch.zeros((0, 2), dtype=torch.int64, device="cuda")
    for off in (None, offsets(0, 0, 0)):
        loss, load, counts = run_balance(l, idx, "softmax", off)
        assert float(loss) == 0.0 and not bool(load.any()) and not bool(counts.any())
    l = make_logits(gen(2), 50, E, "fp32")
    idx = ref.route(l, 2, "softmax")[0].contiguous()
    loss, load, counts = run_balance(l, idx, "softmax", mask=torch.zeros(50, dtype=torch.bool, device="cuda"))
    assert float(loss) == 0.0 and not bool(load.any()) and not bool(counts.any())
    l[3] = -INF
    check_balance(l, idx, "sigmoid")


def test_balance_flags_bad_indices_and_offsets():
    from gpu_path import B
    l = make_logits(gen(2), 50, 16, "fp32")
    idx = ref.route(l, 2, "softmax")[0].contiguous()
    idx[7, 1], idx[9, 0], idx[11] = 16, -2, -1
    check_balance(l, idx, "softmax", want_status=B.EP_ERR_INVALID_INDEX)
    for off in (offsets(0, 30, 20), offsets(-4, 20), offsets(0, 51), offsets(60, 70)):
        run_balance(l, ref.route(l, 2, "softmax")[0].contiguous(), "softmax", off,
                    want_status=B.EP_ERR_INVALID_INDEX)


def check_backward(l, idx, score, want_status=0, d_weights=None, load=None, d_loss=None, offset=None, mask=None,
                   normalize=True, scale=1.0, pad=0):
    from gpu_path import B
    T, E = l.shape
    wide = torch.full((T + 2, E + pad), -77.0, dtype=l.dtype, device="cuda")
    out = wide[:T, :E]
    st = status()
    B.ep_route_backward(l, idx, out, st, d_topk_weights=d_weights, load=load, d_loss=d_loss,
                        score=B.EP_SCORE_SOFTMAX if score == "softmax" else B.EP_SCORE_SIGMOID, token_mask=mask,
                        seq_offset=offset, normalize=normalize, scale=scale)
    assert int(st.item()) == want_status
    assert bool((wide[T:] == -77.0).all()) and bool((wide[:, E:] == -77.0).all())
    want, bound = ref.backward(l, idx, score, d_weights, load, d_loss, offset, mask, normalize, scale)
    off = (out.double() - want).abs()
    assert bool((off <= ref.rounded(want, bound, l.dtype)).all()), float((off / ref.rounded(want, bound, l.dtype)).max())
    return out


@pytest.mark.parametrize("T,E,K", SHAPES + [(3000, 256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward(T, E, K, score):
    for i, dtype in enumerate(TYPES):
        g = gen(T + 7 * E + i)
        l = make_logits(g, T, E, dtype, pad=(1, 8, 0)[i])
        mask = torch.rand(T, generator=g, device="cuda") > 0.2
        idx = ref.route(l, K, score, mask=mask)[0].contiguous()
        if K > 1:
            idx[::5, 1] = -1
        dw = torch.randn((T, K), generator=g, device="cuda")
        d_loss = torch.rand(1, generator=g, device="cuda") + 0.5
        load = torch.rand((1, E), generator=g, device="cuda")
        for normalize in (True, False):
            check_backward(l, idx, score, d_weights=dw, normalize=normalize, scale=2.5, pad=(0, 3, 8)[i])
            check_backward(l, idx, score, d_weights=dw, load=load, d_loss=d_loss, mask=mask, normalize=normalize)
        off = offsets(0, 0, min(1, T), T - T // 5 if T > 10 else T)
        check_backward(l, idx, score, load=torch.rand((3, E), generator=g, device="cuda"), d_loss=d_loss, offset=off)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_backward_of_closed_repeated_and_bad_entries(score, normalize):
    from gpu_path import B
    l = make_logits(gen(4), 30, 50, "fp32")
    l[2], l[3, 4:], l[4] = -INF, -INF, -150.0
    idx = ref.route(l, 5, score)[0].contiguous()
    idx[7] = idx[7, 0]                   # one expert in every slot
    idx[8, 3] = idx[8, 1]
    idx[9] = -1
    dw = torch.randn(idx.shape, generator=gen(5), device="cuda")
    load, d_loss = torch.rand((1, 50), generator=gen(6), device="cuda"), torch.ones(1, device="cuda")
    for kw in (dict(), dict(load=load, d_loss=d_loss)):
        out = check_backward(l, idx, score, d_weights=dw, normalize=normalize, **kw)
        assert bool((out[2] == 0).all()) and bool((out[3, 4:] == 0).all())
    idx[5, 0], idx[6, 2] = 50, -9
    check_backward(l, idx, score, d_weights=dw, normalize=normalize, want_status=B.EP_ERR_INVALID_INDEX)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_what_stands_in_masked_places_reaches_nothing(score, normalize):
    """Garbage in masked tokens' rows and slots, and NaN where a slot names no expert."""
    from gpu_path import B
    T, E, K = 80, 40, 4
    clean = make_logits(gen(4), T, E, "fp32").contiguous()
    mask = torch.rand(T, generator=gen(3), device="cuda") > 0.3
    l = clean.clone()
    l[~mask] = float("nan")
    idx, w = run_route(l, K, score, mask=mask, normalize=normalize)
    assert torch.equal(idx, ref.route(clean, K, score, mask=mask)[0]) and bool((w[~mask] == 0).all())
    idx[::3, 2] = -1
    loss, load, counts = run_balance(l, idx, score, mask=mask)
    want, want_load, want_counts = ref.balance(clean, idx, score, mask=mask)
    assert torch.equal(counts.long(), want_counts) and abs(float(loss) - float(want)) < 1e-5 * float(want)
    dw = torch.randn((T, K), generator=gen(5), device="cuda")
    dw[idx < 0] = float("nan")
    idx[~mask] = 99999
    out = torch.empty_like(l)
    st, d_loss = status(), torch.ones(1, device="cuda")
    B.ep_route_backward(l, idx, out, st, d_topk_weights=dw, load=load, d_loss=d_loss, token_mask=mask, normalize=normalize,
                        score=B.EP_SCORE_SOFTMAX if score == "softmax" else B.EP_SCORE_SIGMOID)
    assert int(st.item()) == 0
    want, bound = ref.backward(clean, torch.where(idx < E, idx, -1), score, torch.nan_to_num(dw), load, d_loss, None, mask,
                               normalize)
    assert bool(((out.double() - want).abs() <= ref.rounded(want, bound, out.dtype)).all())


def test_offsets_with_many_empty_sequences():
    l = make_logits(gen(6), 500, 32, "bf16")
    idx = ref.route(l, 2, "softmax")[0].contiguous()
    cuts = torch.cat([torch.zeros(3000), torch.full((3000,), 117.0), torch.full((2000,), 499.0), torch.full((1000,), 500.0)])
    check_balance(l, idx, "softmax", offset=cuts.to(torch.int32).cuda())


def test_backward_in_place():
    l = make_logits(gen(4), 100, 64, "bf16").contiguous()
    idx = ref.route(l, 5, "softmax")[0].contiguous()
    dw = torch.randn(idx.shape, generator=gen(5), device="cuda")
    want = check_backward(l, idx, "softmax", d_weights=dw)
    from gpu_path import B
    B.ep_route_backward(l, idx, l, status(), d_topk_weights=dw)
    assert torch.equal(l, want)


def test_no_tokens():
    from gpu_path import B
    l = torch.zeros((0, 16), device="cuda")
    idx, w = torch.zeros((0, 2), dtype=torch.int64, device="cuda"), torch.zeros((0, 2), device="cuda")
    B.ep_route(l, idx, w, status())
    B.ep_route_backward(l, idx, torch.zeros_like(l), status(), d_topk_weights=w)


def training_step(B, l, idx, w, ws, loss, load, dw, d_loss, dl, st, stream=None):
    B.ep_route(l, idx, w, st, score=B.EP_SCORE_SIGMOID, num_groups=4, topk_groups=2, stream=stream)
    B.ep_balance_loss(l, idx, ws, loss, load, st, score=B.EP_SCORE_SIGMOID, stream=stream)
    B.ep_route_backward(l, idx, dl, st, d_topk_weights=dw, load=load, d_loss=d_loss, score=B.EP_SCORE_SIGMOID,
                        stream=stream)


def buffers(B, T, E, K):
    return (torch.empty((T, K), dtype=torch.int64, device="cuda"), torch.empty((T, K), device="cuda"),
            torch.empty(B.ep_balance_loss_workspace_bytes(T, E), dtype=torch.uint8, device="cuda"),
            torch.empty(1, device="cuda"), torch.empty((1, E), device="cuda"))


def test_captured_replayed_and_on_two_streams():
    """A step in a graph gives what the calls give on their own, on every replay; two streams with their own
    buffers do not disturb each other; all bits are the same from run to run."""
    from gpu_path import B
    T, E, K = 2000, 64, 6
    inputs = [make_logits(gen(i), T, E, "fp32").contiguous() for i in range(4)]
    dw, d_loss = torch.randn((T, K), generator=gen(9), device="cuda"), torch.ones(1, device="cuda")
    want = []
    for l in inputs:
        b, dl, st = buffers(B, T, E, K), torch.empty_like(l), status()
        training_step(B, l, *b, dw, d_loss, dl, st)
        want.append([t.clone() for t in (b[0], b[1], b[3], b[4], dl)])
    l, b, dl, st = inputs[0].clone(), buffers(B, T, E, K), torch.empty_like(inputs[0]), status()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        training_step(B, l, *b, dw, d_loss, dl, st)
    for i in (0, 1, 2, 3, 1):
        l.copy_(inputs[i])
        graph.replay()
        for got, ok in zip((b[0], b[1], b[3], b[4], dl), want[i]):
            assert torch.equal(got, ok)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(buffers(B, T, E, K), torch.empty_like(l), status()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            training_step(B, inputs[i], *sets[i][0], dw, d_loss, sets[i][1], sets[i][2], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        b, dl, st = sets[i]
        for got, ok in zip((b[0], b[1], b[3], b[4], dl), want[i]):
            assert torch.equal(got, ok)
        assert int(st.item()) == 0


def test_calls_see_what_the_stream_wrote_before():
    from gpu_path import B
    T, E, K = 700, 96, 4
    inputs = [make_logits(gen(i), T, E, "bf16").contiguous() for i in range(3)]
    dw, d_loss = torch.randn((T, K), generator=gen(9), device="cuda"), torch.ones(1, device="cuda")
    l, b, dl, st = torch.empty_like(inputs[0]), buffers(B, T, E, K), torch.empty_like(inputs[0]), status()

    def one(i):
        l.copy_(inputs[i])
        training_step(B, l, *b, dw, d_loss, dl, st)
        return [t.clone() for t in (b[0], b[1], b[3], b[4], dl)]

    alone = []
    for i in range(3):
        torch.cuda.synchronize()
        alone.append(one(i))
    torch.cuda.synchronize()
    got = [(i % 3, one(i % 3)) for i in range(24)]
    for i, g in got:
        assert all(torch.equal(a, b) for a, b in zip(alone[i], g))
