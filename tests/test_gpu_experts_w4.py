"""The experts with 4-bit weights on the GPU against their definition in 64 bits."""
import pytest
import torch

import experts_w4_reference as ref
from experts_reference import ACTS, check

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SCALES = {"bf16": BF, "fp32": F32}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=BF, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def blocks(counts, align=1):
    at, first = 0, []
    for c in counts:
        first.append(at)
        at += -(-c // align) * align
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(first + [at], **i32), torch.tensor(counts, **i32), at


def norm_check(got, want, what=""):
    """Sums are good to far less than the output's rounding: the norm of all differences is within twice bf16's step."""
    if float(want.norm()) > 0:
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -8, what


def check_product(counts, K, N, act="none", form="int", zero=False, group=128, scales="bf16", bias=False, weight=False,
                  residual=False, align=1, extra=5, seed=0):
    from gpu_path import B
    g = gen(seed + K + N)
    E, Nw = len(counts), 2 * N if act == "swiglu" else N
    off, cnt, rows = blocks(counts, align)
    rows += extra
    x = normal(g, rows, K)
    w, sf, z = ref.make(g, E, Nw, K, group, form, zero, SCALES[scales])
    b = normal(g, E, Nw, dtype=F32, std=0.3) if bias else None
    rw = torch.rand(rows, generator=g, device="cuda") if weight else None
    res = normal(g, rows, N) if residual else None
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for a, c in zip(off.tolist(), counts):
        inside[a:a + c] = True
    x[~inside] = float("nan")       # what lies between the blocks reaches nothing
    y = torch.full((rows, N), -77.0, dtype=BF, device="cuda")
    st = status()
    B.ep_expert_gemm_w4(x, w, sf, off, cnt, y, st, w_zero=z, w_format=B.EP_W4_FP if form == "fp4" else B.EP_W4_INT,
                        bias=b, activation=ACTS[act], row_weight=rw, residual=res)
    assert int(st.item()) == 0
    assert bool((y[~inside] == -77.0).all())
    for e in range(E):
        r = slice(int(off[e]), int(off[e]) + counts[e])
        if counts[e] == 0:
            continue
        v, big = ref.values(w[e], sf[e], None if z is None else z[e], form)
        want, bound = ref.product_rows(x[r].double(), v, big, None if b is None else b[e].double(), act,
                                       None if rw is None else rw[r].double(), None if res is None else res[r].double())
        check(y[r], want, bound, "expert %d" % e)
        norm_check(y[r], want)
    return y


FORMS = [("int", False), ("int", True), ("fp4", False)]


@pytest.mark.parametrize("form,zero", FORMS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("scales", ["bf16", "fp32"])
def test_product_forms(form, zero, group, scales):
    check_product([3, 0, 8, 1], 512, 256, form=form, zero=zero, group=group, scales=scales, bias=True)
    check_product([5, 2], 384, 72, "swiglu", form=form, zero=zero, group=group, scales=scales)


@pytest.mark.parametrize("K", [128, 256, 384, 640, 1152, 2048, 2176])
@pytest.mark.parametrize("N", [8, 120, 136, 264])
def test_product_sizes(K, N):
    check_product([1, 7, 0, 9], K, N, "silu", group=128)
    check_product([2, 3], K, N, "swiglu", group=32, form="fp4", bias=True)


@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (96, 32), (64, 64), (192, 64), (160, 32), (544, 32)])
def test_product_short_sums(K, group):
    for form, zero in FORMS:
        check_product([4, 1, 17], K, 40, "gelu", form=form, zero=zero, group=group)


@pytest.mark.parametrize("counts", [[1], [8], [9], [16, 17], [31, 33, 0, 64], [65, 1], [130], [300, 2, 40]])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
def test_product_rows(counts, act):
    check_product(counts, 256, 128, act, bias=True, weight=True, residual=True, align=16)
    check_product(counts, 256, 48, act, zero=True, group=64)


def test_product_many_experts():
    counts = [(i * 7) % 5 for i in range(300)]
    check_product(counts, 128, 64, "swiglu")
    check_product([0] * 2047 + [3], 32, 8, group=32)


def test_product_long():
    check_product([1], 7168, 7168, bias=True, residual=True)
    check_product([2, 5], 7168, 136, "swiglu", zero=True)
    check_product([3], 16384 + 128, 64, form="fp4", group=32)


def test_product_extremes():
    """Scales at the ends of bf16's range, zero and infinite ones, rows of zeros and of large values."""
    from gpu_path import B
    g = gen(1)
    E, K, N = 2, 256, 64
    off, cnt, rows = blocks([4, 3])
    x = normal(g, rows, K)
    x[1] = 0.0
    x[2] *= 1e18
    w, sf, _ = ref.make(g, E, N, K, 128)
    sf[0, 0, 0] = 2.0 ** -126
    sf[0, :, 1] = 0.0
    sf[1, :, 2] = 2.0 ** 100
    for form in ("int", "fp4"):
        y = torch.empty((rows, N), dtype=BF, device="cuda")
        B.ep_expert_gemm_w4(x, w, sf, off, cnt, y, status(), w_format=B.EP_W4_FP if form == "fp4" else B.EP_W4_INT)
        for e, r in ((0, slice(0, 4)), (1, slice(4, 7))):
            v, big = ref.values(w[e], sf[e], None, form)
            want, bound = ref.product_rows(x[r].double(), v, big, None, "none", None, None)
            check(y[r], want, bound)
        assert bool((y[:4, 1] == 0).all()) and bool((y[1] == 0).all())


@pytest.mark.parametrize("rows", [1, 7, 16, 70])
@pytest.mark.parametrize("K,group", [(512, 32), (1024, 128), (416, 32)])
def test_fp4_rows_of_every_size(rows, K, group):
    """Rows whose 128 k's lie many powers of two apart, and apart from one another; subnormal ones, infinities, NaN.

    A row's values may be rounded to 2^-39 of the largest of their 128 k's (fp16 holds bf16's values to 2^-31 of it,
    and has a step of 2^-38 of it below), which counts where the largest meets a weight of zero."""
    from gpu_path import B
    g = gen(rows + K)
    N = 72
    x = normal(g, rows, K).float()
    blocks_ = -(-K // 128)
    far = torch.randint(-55, 56, (rows, blocks_), generator=g, device="cuda").repeat_interleave(128, 1)[:, :K]
    near = -torch.randint(0, 45, (rows, K), generator=g, device="cuda")
    near[rows // 2] = 0
    x = torch.ldexp(x, far + near)
    if rows > 3:
        x[0] = 0.0
        x[1] = torch.ldexp(normal(g, K).float(), torch.tensor(-132, device="cuda"))
    x = x.to(BF)
    w, sf, _ = ref.make(g, 1, N, K, group, "fp4")
    off, cnt, _ = blocks([rows])

    def call():
        y = torch.empty((rows, N), dtype=BF, device="cuda")
        B.ep_expert_gemm_w4(x, w, sf, off, cnt, y, status(), w_format=B.EP_W4_FP)
        return y

    y = call()
    v, big = ref.values(w[0], sf[0], None, "fp4")
    xd = x.double()
    largest = torch.stack([b.abs().amax(1) for b in xd.split(128, 1)], 1).repeat_interleave(128, 1)[:, :K]
    want, bound = ref.product_rows(xd, v, big, None, "none", None, None)
    check(y, want, bound + 2.0 ** -39 * (largest @ v.abs().T) + 2.0 ** -133)
    if rows > 3:
        x[2, 5], x[2, K - 1], x[3, 130] = float("inf"), 3e38, float("nan")
        # (a group's sum is fp32 before its scale: 3e38 times a code of 1.5 or more is beyond fp32's 3.4e38, and an
        # infinity there, which against the other one gives NaN)
        codes = ref.values(w[0], torch.ones_like(sf[0]), None, "fp4")[0].unflatten(1, (-1, group))
        sums = torch.einsum("rgk,fgk->rfg", x.double().unflatten(1, (-1, group)), codes).float().double()
        got, want = call(), (sums * sf[0].double().T).sum(-1)
        keep = [r for r in range(rows) if r not in (2, 3)]
        assert torch.equal(got[keep], y[keep]) and bool(got[3].isnan().all())
        assert torch.equal(got[2].isnan(), want[2].isnan())
        assert torch.equal(got[2].nan_to_num(0.0, 1.0, -1.0), want[2].nan_to_num(0.0, 1.0, -1.0).to(BF))


def test_product_skips_rows_beyond_and_overlapping_blocks():
    from gpu_path import B
    g = gen(3)
    E, K, N, rows = 3, 128, 64, 20
    x = normal(g, rows, K)
    w, sf, _ = ref.make(g, E, N, K, 128)
    i32 = dict(dtype=torch.int32, device="cuda")

    def call(off, cnt):
        y = torch.full((rows, N), -77.0, dtype=BF, device="cuda")
        st = status()
        B.ep_expert_gemm_w4(x, w, sf, torch.tensor(off, **i32), torch.tensor(cnt, **i32), y, st)
        assert int(st.item()) == B.EP_ERR_CAPACITY
        return y

    y = call([0, 8, 16, 26], [4, 4, 10])
    v, big = ref.values(w[2], sf[2], None, "int")
    check(y[16:], *ref.product_rows(x[16:].double(), v, big, None, "none", None, None))
    assert bool((y[4:8] == -77).all())
    y = call([0, 25, -3, 26], [4, 4, 2])
    assert bool((y[4:] == -77).all()) and bool((y[:4] != -77).all())
    assert bool((call([0, 0, 0, 20], [20, 20, 20]) == -77).all())


def make_few(T, H, I, E, K, act, form="int", zero=False, group=128, scales="bf16", bias=False, residual=False, seed=0,
             hot=False):
    g = gen(seed + T + H)
    Nw = 2 * I if act == "swiglu" else I
    idx = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), dim=1)[:, :K].contiguous()
    if hot:
        idx[:, 0] = E // 2
    idx[torch.rand((T, K), generator=g, device="cuda") < 0.1] = -1
    if T > 3:
        idx[T // 2] = -1
    return dict(x=normal(g, T, H), idx=idx, tw=torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1),
                up=ref.make(g, E, Nw, H, group, form, zero, SCALES[scales]),
                down=ref.make(g, E, H, I, group if I % group == 0 else 32, form, zero, SCALES[scales]),
                b_up=normal(g, E, Nw, dtype=F32, std=0.3) if bias else None,
                b_down=normal(g, E, H, dtype=F32, std=0.3) if bias else None,
                res=normal(g, T, H) if residual else None)


def run_few(d, act, form, ws=None, out=None, stream=None, st=None):
    from gpu_path import B
    T, H = d["x"].shape
    E, _, half = d["down"][0].shape
    K = d["idx"].shape[1]
    if ws is None:
        ws = torch.full((B.ep_moe_few_tokens_w4_workspace_bytes(T, K, H, 2 * half, E),), 0xA5, dtype=torch.uint8,
                        device="cuda")
    whole = torch.full((T + 1, H), -77.0, dtype=BF, device="cuda") if out is None else None
    out = whole[:T] if out is None else out
    st_ = status() if st is None else st
    B.ep_moe_few_tokens_w4(d["x"], d["idx"], d["tw"], d["up"][0], d["up"][1], d["down"][0], d["down"][1], ws, out, st_,
                           up_zero=d["up"][2], down_zero=d["down"][2],
                           w_format=B.EP_W4_FP if form == "fp4" else B.EP_W4_INT, bias_up=d["b_up"],
                           bias_down=d["b_down"], residual=d["res"], activation=ACTS[act], stream=stream)
    if st is None:
        assert int(st_.item()) == 0
    assert whole is None or bool((whole[T:] == -77.0).all())
    return out


def check_few(d, act, form):
    want, bound = ref.few_tokens(d["x"], d["idx"], d["tw"], d["up"], d["b_up"], act, d["down"], d["b_down"], d["res"],
                                 form)
    out = run_few(d, act, form)
    check(out, want, bound)
    norm_check(out, want)
    return out


@pytest.mark.parametrize("T,H,I,E,K", [(1, 256, 128, 4, 2), (1, 2048, 1024, 64, 8), (3, 128, 160, 5, 5), (8, 640, 384, 16, 4),
                                       (17, 1152, 256, 32, 8), (64, 256, 512, 8, 2), (128, 512, 256, 256, 8),
                                       (256, 128, 128, 3, 3), (256, 256, 64, 40, 16), (200, 128, 96, 1, 1)])
@pytest.mark.parametrize("form,zero", FORMS)
def test_few_tokens(T, H, I, E, K, form, zero):
    act = ("swiglu", "gelu", "silu")[(T + K) % 3]
    group = 64 if I % 64 == 0 else 32
    check_few(make_few(T, H, I, E, K, act, form, zero, group, "fp32" if T % 2 else "bf16", bias=T % 2 == 0,
                       residual=K % 2 == 0), act, form)
    check_few(make_few(T, H, I, E, K, "swiglu", form, zero, 32, hot=True, seed=3), "swiglu", form)


def test_few_tokens_wide():
    check_few(make_few(2, 7168, 2048, 6, 4, "swiglu", residual=True), "swiglu", "int")
    check_few(make_few(12, 2048, 7168, 3, 2, "none", "fp4", group=32, bias=True), "none", "fp4")


def test_few_tokens_masks_and_bad_indices():
    from gpu_path import B
    d = make_few(10, 256, 128, 6, 3, "swiglu", residual=True)
    d["idx"][:] = -1
    assert torch.equal(run_few(d, "swiglu", "int"), d["res"])
    d["res"] = None
    assert bool((run_few(d, "swiglu", "int") == 0).all())
    d = make_few(10, 256, 128, 6, 3, "swiglu")
    good = run_few(d, "swiglu", "int").clone()
    bad = dict(d, idx=d["idx"].clone())
    bad["idx"][d["idx"] < 0] = 6
    bad["idx"][0, 0], d["idx"][0, 0] = -5, -1
    st = status()
    got = run_few(bad, "swiglu", "int", st=st)
    assert int(st.item()) == B.EP_ERR_INVALID_INDEX
    assert torch.equal(got, run_few(d, "swiglu", "int")) and torch.equal(got[1:], good[1:])


def test_few_tokens_one_expert_twice():
    d = make_few(6, 256, 128, 4, 3, "silu", bias=True)
    d["idx"][:, 1] = d["idx"][:, 0]
    check_few(d, "silu", "int")


def test_few_tokens_residual_may_be_out():
    d = make_few(20, 512, 256, 8, 2, "swiglu", residual=True)
    want = run_few(d, "swiglu", "int").clone()
    got = d["res"].clone()
    run_few(dict(d, res=got), "swiglu", "int", out=got)
    assert torch.equal(got, want)


def test_captured_replayed_and_on_two_streams():
    from gpu_path import B
    T, H, I, E, K = 24, 512, 256, 16, 4
    ds = [make_few(T, H, I, E, K, "swiglu", residual=True, seed=s) for s in range(3)]
    want = [run_few(d, "swiglu", "int").clone() for d in ds]
    nbytes = B.ep_moe_few_tokens_w4_workspace_bytes(T, K, H, I, E)
    d = {k: tuple(t if t is None else t.clone() for t in v) if isinstance(v, tuple) else None if v is None else v.clone()
         for k, v in ds[0].items()}
    ws, out, st = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty_like(want[0]), status()
    run_few(d, "swiglu", "int", ws, out, st=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_few(d, "swiglu", "int", ws, out, st=st)
    for i in (1, 2, 0, 1):
        for k, v in ds[i].items():
            for a, b in zip(d[k] if isinstance(v, tuple) else (d[k],), v if isinstance(v, tuple) else (v,)):
                if b is not None:
                    a.copy_(b)
        graph.replay()
        assert torch.equal(out, want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty_like(want[0])) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            run_few(ds[i], "swiglu", "int", *sets[i], stream=s, st=st)
    torch.cuda.synchronize()
    assert torch.equal(sets[0][1], want[0]) and torch.equal(sets[1][1], want[1]) and int(st.item()) == 0


def test_calls_see_what_the_stream_wrote_before():
    ds = [make_few(9, 384, 256, 12, 4, "swiglu", seed=s) for s in range(3)]
    x, idx = torch.empty_like(ds[0]["x"]), torch.empty_like(ds[0]["idx"])
    ws = None

    def one(i):
        x.copy_(ds[i]["x"])
        idx.copy_(ds[i]["idx"])
        return run_few(dict(ds[0], x=x, idx=idx), "swiglu", "int", ws, torch.empty_like(x), st=st).clone()

    from gpu_path import B
    st = status()
    ws = torch.empty(B.ep_moe_few_tokens_w4_workspace_bytes(9, 4, 384, 256, 12), dtype=torch.uint8, device="cuda")
    alone = []
    for i in range(3):
        torch.cuda.synchronize()
        alone.append(one(i))
    torch.cuda.synchronize()
    got = [(i % 3, one(i % 3)) for i in range(24)]
    assert all(torch.equal(alone[i], o) for i, o in got)


def test_many_calls_in_flight():
    """A long queue of calls, so that the down product's kernel starts on the SMs that the up product leaves free and
    waits there with its first weights loaded: no wait runs out, and every call's answer is the same."""
    T, H, I, E, K = 1, 7168, 2048, 12, 8
    d = make_few(T, H, I, E, K, "swiglu")
    d["idx"] = torch.arange(K, device="cuda")[None, :].contiguous()
    from gpu_path import B
    ws = torch.empty(B.ep_moe_few_tokens_w4_workspace_bytes(T, K, H, I, E), dtype=torch.uint8, device="cuda")
    st, outs = status(), [torch.empty_like(d["x"]) for _ in range(40)]
    want = run_few(d, "swiglu", "int").clone()
    torch.cuda.synchronize()
    for out in outs:
        run_few(d, "swiglu", "int", ws, out, st=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert all(torch.equal(out, want) for out in outs)


def test_rows_of_a_dispatch():
    """Router, layout, dispatch, both products, combine: the rows path against the few-token call."""
    from gpu_path import B
    T, H, I, E, K, R = 60, 256, 128, 16, 4, 4
    d = make_few(T, H, I, E, K, "swiglu", group=64)
    logits = normal(gen(8), T, E)
    idx, tw, st = torch.empty_like(d["idx"]), torch.empty_like(d["tw"]), status()
    mask = torch.rand(T, generator=gen(9), device="cuda") > 0.2
    B.ep_route(logits, idx, tw, st, score=B.EP_SCORE_SIGMOID, token_mask=mask, num_groups=4, topk_groups=2)
    few = check_few(dict(d, idx=idx, tw=tw), "swiglu", "int")
    lay = B.alloc_layout(T, E, R, K=K)
    B.ep_get_layout(idx, E, R, lay, torch.empty(B.ep_layout_workspace_bytes(T, K, E, R), dtype=torch.uint8,
                                                device="cuda"), st, expert_alignment=8)
    n = B.ep_expanded_capacity_bound(T, K, E, 8)
    rx, rs, rw = torch.empty((n, H), dtype=BF, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda"), \
        torch.empty(n, device="cuda")
    B.ep_dispatch_expanded(d["x"], idx, tw, E, R, lay, rx, rs, rw, st)
    h, y = torch.empty((n, I), dtype=BF, device="cuda"), torch.empty((n, H), dtype=BF, device="cuda")
    first, count = lay.expert_offset, lay.num_tokens_per_expert
    B.ep_expert_gemm_w4(rx, *d["up"][:2], first, count, h, st, activation=B.EP_ACT_SWIGLU)
    B.ep_expert_gemm_w4(h, *d["down"][:2], first, count, y, st)
    out = torch.empty((T, H), dtype=BF, device="cuda")
    B.ep_combine_expanded(y, tw, K, E, R, lay, out, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # an expert's row is rounded once more here; 2^-8 of it each
    assert float((out.double() - few.double()).norm() / few.double().norm()) < 2 * 2.0 ** -8
    assert bool((out[~mask] == 0).all()) and bool((idx[mask] >= 0).all())
