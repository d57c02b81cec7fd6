"""GPU parity of the experts' operators against their definitions in 64 bits:
the grouped product with its epilogue (bf16 and FP8), its gradients, and the
whole layer for a few tokens; sizes around every tile edge, empty experts,
padding that holds NaN, masked and invalid entries, other streams, aliases,
rows beyond the arrays."""
import numpy as np
import pytest
import torch

import experts_reference as ref
from experts_reference import ACTS

pytestmark = pytest.mark.gpu

NAN = float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.bfloat16, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def blocks(counts, align=1, gap=0):
    """Offsets of the experts' blocks and the number of rows."""
    off, at = [], 0
    for c in counts:
        off.append(at)
        at += (c + align - 1) // align * align + gap
    off.append(at)
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(off, **i32), torch.tensor(counts, **i32), at


def owned(counts, off, rows):
    m = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e, c in enumerate(counts):
        m[int(off[e]):int(off[e]) + c] = True
    return m


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def run_product(counts, K, N, act="none", bias=False, rw=False, res=False, save=False, align=1, gap=0, seed=0,
                fp8=False, col_major=False, alias=False):
    from gpu_path import B
    g = gen(seed)
    off, cnt, rows = blocks(counts, align, gap)
    E, Nw = len(counts), 2 * N if act == "swiglu" else N
    mine = owned(counts, off, rows)
    x, w = normal(g, rows, K), normal(g, E, Nw, K, std=K ** -0.5)
    kw, x64, w64 = {}, x.double(), w.double()
    if fp8:
        x, xs = to_fp8(x, 1)
        w, ws = to_fp8(w, 128)
        x64 = x.double() * xs.double().repeat_interleave(128, 1)
        w64 = w.double() * ws.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        xs[~mine] = NAN
        if col_major:
            stride = (rows + 3) // 4 * 4
            buf = torch.full((K // 128, stride), NAN, device="cuda")
            buf[:, :rows] = xs.T
            xs = buf
        kw.update(x_sf=xs, w_sf=ws, sf_col_major=col_major)
    else:
        x[~mine] = NAN
    b = normal(g, E, Nw, dtype=torch.float32) if bias else None
    r = torch.rand(rows, generator=g, device="cuda") - 0.25 if rw else None
    s = normal(g, rows, N) if res else None
    for t in (r, s):
        if t is not None:
            t[~mine] = NAN
    s64 = s.double() if res else None
    y = s if alias else torch.full((rows, N), -7.0, dtype=torch.bfloat16, device="cuda")
    before = y.clone()
    z = torch.full((rows, Nw), -7.0, dtype=torch.bfloat16, device="cuda") if save else None
    st = status()
    B.ep_expert_gemm(x, w, off, cnt, y, st, bias=b, activation=ACTS[act], row_weight=r, residual=s, z=z, **kw)
    assert int(st.item()) == 0
    for e, c in enumerate(counts):
        d = slice(int(off[e]), int(off[e]) + c)
        yy, by, zz, bz = ref.product_rows(x64[d], w64[e], b[e].double() if bias else None, act,
                                          r[d].double() if rw else None, s64[d] if res else None)
        ref.check(y[d], yy, by, "y of expert %d" % e)
        if save:
            ref.check(z[d], zz, bz, "z of expert %d" % e)
    assert torch.equal(y[~mine].view(torch.int16), before[~mine].view(torch.int16))
    if save:
        assert bool((z[~mine] == -7.0).all())
    return y


def to_fp8(a, rows):
    *lead, n, k = a.shape
    v = a.float().reshape(*lead, n // rows, rows, k // 128, 128)
    amax = v.abs().amax(dim=(-3, -1), keepdim=True).clamp_min(1e-12)
    codes = (v * (448.0 / amax)).to(torch.float8_e4m3fn).reshape(a.shape)
    return codes, (amax / 448.0).reshape(*lead, n // rows, k // 128).contiguous()


EDGES = [1, 0, 7, 8, 9, 31, 33, 0, 64, 65, 127, 128, 129]


@pytest.mark.parametrize("act", list(ACTS))
def test_product_activations(act):
    run_product([5, 0, 130, 17], 72, 136, act, bias=True, rw=True, res=True, save=True, align=4, gap=3, seed=1)


@pytest.mark.parametrize("K,N", [(8, 8), (16, 24), (64, 64), (72, 40), (200, 136), (256, 512), (1000, 264)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_product_sizes(K, N, act):
    run_product(EDGES, K, N, act, seed=K + N)


@pytest.mark.parametrize("counts", [[1], [255], [256], [257], [511, 513], [1, 1, 1], [0, 0, 700, 0], [300] * 3])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_product_row_counts(counts, act):
    run_product(counts, 136, 200, act, bias=True, res=True, save=True, seed=sum(counts))


@pytest.mark.parametrize("counts", [[1], [3, 0, 40], [100], [300, 5]])
@pytest.mark.parametrize("K,N,act", [(2048, 136, "swiglu"), (1032, 200, "gelu"), (7168, 72, "none")])
def test_product_long_sums_of_few_tiles(counts, K, N, act):
    """A tile's sum shared by the CTAs of a cluster (2, 4 or 8 of them)."""
    run_product(counts, K, N, act, bias=True, rw=True, res=True, save=True, gap=1, seed=K + N)


def test_product_many_experts():
    rng = np.random.Generator(np.random.PCG64(5))
    counts = rng.integers(0, 9, size=2048).tolist()
    run_product(counts, 64, 72, "relu", bias=True, seed=5)


def test_product_larger():
    run_product([700, 0, 1300, 5, 2000, 129], 1024, 1408, "swiglu", rw=True, save=True, seed=9)


def test_product_residual_is_the_output():
    run_product([40, 0, 133], 96, 200, "gelu", res=True, alias=True, gap=2, seed=3)
    run_product([40, 0, 133], 96, 200, "swiglu", res=True, alias=True, gap=2, seed=3)


@pytest.mark.parametrize("counts", [EDGES, [600, 0, 3]])
@pytest.mark.parametrize("K,N,act,col", [(128, 128, "none", False), (384, 256, "swiglu", True), (896, 128, "silu", True)])
def test_product_fp8(counts, K, N, act, col):
    run_product(counts, K, N, act, bias=True, rw=True, res=True, save=True, fp8=True, col_major=col, gap=1, seed=K)


@pytest.mark.parametrize("K,N,act", [(384, 1024, "swiglu"), (256, 2176, "gelu")])
def test_product_fp8_full_experts(K, N, act):
    run_product([300, 0, 513, 257, 1000], K, N, act, bias=True, rw=True, res=True, save=True, fp8=True, gap=1, seed=N)


def test_product_fp8_many_experts():
    rng = np.random.Generator(np.random.PCG64(7))
    run_product(rng.integers(0, 4, size=2048).tolist(), 128, 128, "swiglu", fp8=True, seed=7)


@pytest.mark.parametrize("N,act", [(384, "gelu"), (256, "swiglu")])
@pytest.mark.parametrize("at", [(8, 0, 0), (0, 8, 0), (0, 0, 8), (8, 8, 8)])
def test_product_fp8_arrays_on_16_bytes(N, act, at):
    """y, z and the residual need 16-byte alignment alone; on 32 bytes they give the same bits."""
    from gpu_path import B
    g = gen(N)
    off, cnt, rows = blocks([5, 0, 140], gap=1)
    Nw = 2 * N if act == "swiglu" else N
    x, xs = to_fp8(normal(g, rows, 256), 1)
    w, ws = to_fp8(normal(g, 3, Nw, 256, std=1.0 / 16), 128)
    res = normal(g, rows, N)

    def put(shape, shift):
        n = shape[0] * shape[1]
        return torch.full((n + 16,), -7.0, dtype=torch.bfloat16, device="cuda")[shift:shift + n].view(shape)

    def run(ay, az, ar):
        y, z, r, st = put((rows, N), ay), put((rows, Nw), az), put((rows, N), ar), status()
        r.copy_(res)
        B.ep_expert_gemm(x, w, off, cnt, y, st, activation=ACTS[act], residual=r, z=z, x_sf=xs, w_sf=ws)
        assert int(st.item()) == 0
        return y, z

    for got, want in zip(run(*at), run(0, 0, 0)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("act", list(ACTS))
def test_nan_and_infinity_follow_the_activation(act):
    """NaN rows give NaN; +inf pre-activations give what the formula gives."""
    from gpu_path import B
    off, cnt, rows = blocks([3])
    x = torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = NAN, float("inf"), 2.0
    w = torch.zeros((1, 32 if act == "swiglu" else 16, 64), dtype=torch.bfloat16, device="cuda")
    w[:, :, 0] = 1.0
    y = torch.zeros((rows, 16), dtype=torch.bfloat16, device="cuda")
    st = status()
    B.ep_expert_gemm(x, w, off, cnt, y, st, activation=ACTS[act])
    assert int(st.item()) == 0
    assert bool(torch.isnan(y[0].float()).all()) and bool((y[1] == float("inf")).all())
    a, e = ref.activate(torch.full((1, w.shape[1]), 2.0, dtype=torch.float64, device="cuda"),
                        torch.zeros((1, w.shape[1]), dtype=torch.float64, device="cuda"), act)
    ref.check(y[2:], a, ref.bf16_bound(a, e))


def test_product_without_rows():
    from gpu_path import B
    off, cnt, _ = blocks([0, 0])
    st = status()
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = normal(gen(0), 2, 64, 64)
    y = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    B.ep_expert_gemm(x, w, off, cnt, y, st)
    y = torch.full((5, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    B.ep_expert_gemm(normal(gen(0), 5, 64), w, off, cnt, y, st)
    assert int(st.item()) == 0 and bool((y == -7.0).all())


def test_rows_beyond_the_arrays():
    """Offsets that promise more rows than there are: the ones inside are right, the bit is set."""
    from gpu_path import B
    g = gen(4)
    rows, K, N = 50, 64, 48
    off = torch.tensor([0, 20, 45, 60, 80], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([20, 25, 15, 9], dtype=torch.int32, device="cuda")
    x, w = normal(g, rows, K), normal(g, 4, N, K, std=K ** -0.5)
    y = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    st = status()
    B.ep_expert_gemm(x, w, off, cnt, y, st)
    assert int(st.item()) == B.EP_ERR_CAPACITY
    for e, (a, b) in enumerate(((0, 20), (20, 45), (45, 50))):
        yy, by, _, _ = ref.product_rows(x[a:b].double(), w[e].double(), None, "none", None, None)
        ref.check(y[a:b], yy, by)


def test_row_of_nan_stays_in_its_row():
    from gpu_path import B
    g = gen(6)
    off, cnt, rows = blocks([20, 13])
    x, w = normal(g, rows, 128), normal(g, 2, 64, 128)
    y = torch.empty((rows, 64), dtype=torch.bfloat16, device="cuda")
    clean = torch.empty_like(y)
    st = status()
    B.ep_expert_gemm(x, w, off, cnt, clean, st)
    x[7] = NAN
    x[25] = float("inf")
    B.ep_expert_gemm(x, w, off, cnt, y, st)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[7] = keep[25] = False
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[7].float()).all()) and not bool(torch.isfinite(y[25].float()).any())


def test_product_on_another_stream_repeats_exactly():
    from gpu_path import B
    g = gen(7)
    off, cnt, rows = blocks([300, 1, 0, 77])
    x, w = normal(g, rows, 256), normal(g, 4, 256, 256, std=1 / 16)
    a, b = (torch.empty((rows, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = status()
    B.ep_expert_gemm(x, w, off, cnt, a, st, activation=B.EP_ACT_SWIGLU)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    B.ep_expert_gemm(x, w, off, cnt, b, st, activation=B.EP_ACT_SWIGLU, stream=side)
    side.synchronize()
    assert torch.equal(a, b)


# ---------------------------------------------------------------- gradients

def run_backward(counts, K, N, act, rw=False, align=1, gap=0, seed=0, want=("dx", "dw", "dbias", "d_row_weight")):
    from gpu_path import B
    g = gen(seed)
    off, cnt, rows = blocks(counts, align, gap)
    E, Nw = len(counts), 2 * N if act == "swiglu" else N
    mine = owned(counts, off, rows)
    dy, x, z = normal(g, rows, N), normal(g, rows, K), normal(g, rows, Nw)
    w = normal(g, E, Nw, K, std=K ** -0.5)
    r = torch.rand(rows, generator=g, device="cuda") - 0.25 if rw else None
    for t in (dy, x, z, r):
        if t is not None:
            t[~mine] = NAN
    bf, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.float32, device="cuda")
    out = {"dx": torch.full((rows, K), -7.0, **bf), "dw": torch.full((E, Nw, K), NAN, **bf),
           "dbias": torch.full((E, Nw), NAN, **f32), "d_row_weight": torch.full((rows,), -7.0, **f32)}
    out = {k: v for k, v in out.items() if k in want}
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(rows, N, E, ACTS[act]), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0xFF)      # NaN everywhere
    st = status()
    B.ep_expert_gemm_backward(dy, x, w, z, off, cnt, ws, st, activation=ACTS[act], row_weight=r, **out)
    assert int(st.item()) == 0
    for e, c in enumerate(counts):
        d = slice(int(off[e]), int(off[e]) + c)
        R = ref.backward_rows(dy[d].double(), x[d].double(), w[e].double(), z[d].double(), act,
                              r[d].double() if rw else None)
        for name, v in out.items():
            got = v[e] if name in ("dw", "dbias") else v[d]
            ref.check(got, *R[name], what="%s of expert %d" % (name, e))
            if c == 0 and name in ("dw", "dbias"):
                assert bool((got == 0).all())
    for name in ("dx", "d_row_weight"):
        if name in out:
            assert bool((out[name][~mine] == -7.0).all())


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("rw", [False, True])
def test_backward_activations(act, rw):
    run_backward([5, 0, 130, 17], 72, 136, act, rw, align=4, gap=3, seed=11)


@pytest.mark.parametrize("K,N", [(8, 8), (24, 16), (64, 64), (72, 40), (200, 136), (512, 256), (264, 1000)])
@pytest.mark.parametrize("act", ["relu", "swiglu"])
def test_backward_sizes(K, N, act):
    run_backward(EDGES, K, N, act, True, seed=K + N)


@pytest.mark.parametrize("counts", [[1], [255], [256], [257], [511, 513], [1, 1, 1], [0, 0, 700, 0], [0]])
def test_backward_row_counts(counts):
    run_backward(counts, 136, 200, "swiglu", True, seed=sum(counts))


def test_backward_many_experts():
    rng = np.random.Generator(np.random.PCG64(6))
    run_backward(rng.integers(0, 9, size=2048).tolist(), 64, 72, "silu", True, seed=6)


def test_backward_larger():
    run_backward([700, 0, 1300, 5, 2000, 129], 1024, 704, "swiglu", True, seed=10)


@pytest.mark.parametrize("counts", [[1], [3, 0, 40], [300]])
def test_backward_long_sums_of_few_tiles(counts):
    run_backward(counts, 72, 2056, "silu", True, seed=sum(counts))


@pytest.mark.parametrize("counts", [[4200], [3000, 0, 129], [8192], [1030, 2000]])
@pytest.mark.parametrize("K,N", [(72, 200), (520, 264)])
def test_backward_many_rows_of_few_tiles(counts, K, N):
    """A weight gradient's rows shared by the CTAs of a cluster; some of them without any."""
    run_backward(counts, K, N, "gelu", True, gap=3, seed=sum(counts))


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dbias",), ("d_row_weight",), ("dx", "dbias")])
def test_backward_parts(want):
    run_backward([33, 0, 70], 80, 96, "gelu", True, want=want, seed=12)


def test_backward_without_activation_takes_no_z():
    from gpu_path import B
    g = gen(13)
    off, cnt, rows = blocks([9, 0, 70], gap=1)
    dy, x, w = normal(g, rows, 40), normal(g, rows, 48), normal(g, 3, 40, 48)
    dx, dw = torch.zeros_like(x), torch.empty_like(w)
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(rows, 40, 3), dtype=torch.uint8, device="cuda")
    st = status()
    B.ep_expert_gemm_backward(dy, x, w, None, off, cnt, ws, st, dx=dx, dw=dw)
    assert int(st.item()) == 0
    for e, (a, c) in enumerate(zip(off.tolist(), cnt.tolist())):
        R = ref.backward_rows(dy[a:a + c].double(), x[a:a + c].double(), w[e].double(), None, "none", None)
        ref.check(dx[a:a + c], *R["dx"])
        ref.check(dw[e], *R["dw"])


def test_backward_without_rows_writes_zeros():
    from gpu_path import B
    off, cnt, _ = blocks([0, 0])
    e = dict(dtype=torch.bfloat16, device="cuda")
    dw, db = torch.full((2, 64, 64), NAN, **e), torch.full((2, 64), NAN, device="cuda")
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(0, 64, 2), dtype=torch.uint8, device="cuda")
    st = status()
    none = torch.empty((0, 64), **e)
    B.ep_expert_gemm_backward(none, none, dw.clone(), none, off, cnt, ws, st, dx=none.clone(), dw=dw, dbias=db)
    assert int(st.item()) == 0 and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("act", ["gelu", "silu", "swiglu"])
def test_gradients_against_differences(act):
    """<gradient, v> against a central difference of the 64-bit forward along v.
    The kernel takes z rounded to bf16, so beside its own bound its slopes are
    off by 0.8 * |z| 2^-8 and, for the gated one, its factors by |z| 2^-8.  The
    difference's own error is of order step^2 times third derivatives (all
    at most a few units here), far below those."""
    from gpu_path import B
    g = gen(21)
    counts, K, N = [9, 4], 32, 24
    off, cnt, rows = blocks(counts)
    Nw = 2 * N if act == "swiglu" else N
    x, w, dy = normal(g, rows, K), normal(g, 2, Nw, K, std=K ** -0.5), normal(g, rows, N)
    bias = normal(g, 2, Nw, dtype=torch.float32)
    rw = torch.rand(rows, generator=g, device="cuda")
    y, z = torch.empty_like(dy), torch.empty((rows, Nw), dtype=torch.bfloat16, device="cuda")
    st = status()
    B.ep_expert_gemm(x, w, off, cnt, y, st, bias=bias, activation=ACTS[act], row_weight=rw, z=z)
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(rows, N, 2, ACTS[act]), dtype=torch.uint8,
                     device="cuda")
    dx, dw, db, drw = torch.empty_like(x), torch.empty_like(w), torch.empty_like(bias), torch.empty_like(rw)
    B.ep_expert_gemm_backward(dy, x, w, z, off, cnt, ws, st, dx=dx, dw=dw, dbias=db, d_row_weight=drw,
                              activation=ACTS[act], row_weight=rw)
    assert int(st.item()) == 0
    which = torch.tensor([0] * 9 + [1] * 4, device="cuda")

    def loss(x, w, b, r):
        zz = torch.einsum("rk,rnk->rn", x, w[which]) + b[which]
        a, _ = ref.activate(zz, torch.zeros_like(zz), act)
        return float((dy.double() * a * r[:, None]).sum())

    at = [t.double() for t in (x, w, bias, rw)]
    bounds = []
    for e, d in enumerate((slice(0, 9), slice(9, 13))):
        z64, dy64, r64 = z[d].double(), dy[d].double(), rw[d].double()
        R = ref.backward_rows(dy64, at[0][d], at[1][e], z64, act, r64)
        da = (dy64 * r64[:, None]).abs()
        q = 2.0 ** -8
        if act == "swiglu":
            gg, uu = z64[:, :N].abs(), z64[:, N:].abs()
            e_dz = torch.cat([da * q * (uu * 1.13 + 0.8 * uu * gg * 1.01), da * q * 1.13 * gg], 1)
            e_a = q * (1.13 * gg * uu + gg * uu * 1.01)
        else:
            e_dz, e_a = da * 0.8 * q * z64.abs(), 1.13 * q * z64.abs()
        bounds.append((R["dx"][1] + 1.01 * e_dz @ at[1][e].abs(), R["dw"][1] + 1.01 * e_dz.T @ at[0][d].abs(),
                       R["dbias"][1] + e_dz.sum(0), R["d_row_weight"][1] + (dy64.abs() * e_a).sum(1)))
    bound = [torch.cat([b[0] for b in bounds]), torch.stack([b[1] for b in bounds]),
             torch.stack([b[2] for b in bounds]), torch.cat([b[3] for b in bounds])]
    for i, grad in enumerate((dx, dw, db, drw)):
        v = torch.empty_like(at[i]).normal_(generator=g)
        step = 1e-4
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * v, at[i] - step * v
        diff = (loss(*up) - loss(*down)) / (2 * step)
        assert abs(float((grad.double() * v).sum()) - diff) <= float((bound[i] * v.abs()).sum()) + 1e-5


def test_offsets_beyond_32_bits():
    """More than 2^31 elements of y, z, dy and dz: the last expert's rows are right."""
    from gpu_path import B
    g = gen(33)
    rows, tail, K, N = 310_000, 77, 64, 7168
    off = torch.tensor([0, rows - tail, rows], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([rows - tail, tail], dtype=torch.int32, device="cuda")
    assert rows * N > 1 << 31
    x, w = normal(g, rows, K), normal(g, 2, N, K, std=K ** -0.5)
    y, z = (torch.empty((rows, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = status()
    B.ep_expert_gemm(x, w, off, cnt, y, st, activation=B.EP_ACT_SILU, z=z)
    last = slice(rows - tail, rows)
    yy, by, zz, bz = ref.product_rows(x[last].double(), w[1].double(), None, "silu", None, None)
    ref.check(y[last], yy, by)
    ref.check(z[last], zz, bz)
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(rows, N, 2, B.EP_ACT_SILU), dtype=torch.uint8,
                     device="cuda")
    dx, dw, drw = torch.empty_like(x), torch.empty_like(w), torch.empty(rows, device="cuda")
    B.ep_expert_gemm_backward(y, x, w, z, off, cnt, ws, st, dx=dx, dw=dw, d_row_weight=drw, activation=B.EP_ACT_SILU)
    assert int(st.item()) == 0
    R = ref.backward_rows(y[last].double(), x[last].double(), w[1].double(), z[last].double(), "silu", None)
    ref.check(dx[last], *R["dx"])
    ref.check(dw[1], *R["dw"])
    ref.check(drw[last], *R["d_row_weight"])


# ---------------------------------------------------------------- few tokens

def run_few(T, K, E, H, I, act="swiglu", bias=False, res=False, mode="distinct", mask=0.0, seed=0, alias=False,
            want_status=0, graph=False):
    from gpu_path import B, to_dev
    g = gen(seed)
    rng = np.random.Generator(np.random.PCG64(seed))
    if mode == "distinct":
        idx = np.argsort(rng.random((T, E)), axis=1)[:, :K]
    elif mode == "one":
        idx = np.full((T, K), E - 1)
    else:
        idx = rng.integers(-2 if mode == "invalid" else 0, E + (2 if mode == "invalid" else 0), size=(T, K))
    idx = idx.astype(np.int64)
    idx[rng.random((T, K)) < mask] = -1
    idx = to_dev(idx)
    Iw = 2 * I if act == "swiglu" else I
    x, tw = normal(g, T, H), torch.rand((T, K), generator=g, device="cuda") - 0.2
    tw[idx == -1] = NAN     # masked entries' weights are not read into anything
    wu, wd = normal(g, E, Iw, H, std=H ** -0.5), normal(g, E, H, I, std=I ** -0.5)
    named = torch.unique(idx)
    off = torch.ones(E, dtype=torch.bool, device="cuda")
    off[named[(named >= 0) & (named < E)]] = False
    wu[off] = NAN       # weights of experts nobody names are not read into anything
    wd[off] = NAN
    bu = normal(g, E, Iw, dtype=torch.float32) if bias else None
    bd = normal(g, E, H, dtype=torch.float32) if bias else None
    s = normal(g, T, H) if res else None
    want, bound = ref.few_tokens(x, idx, tw, wu, bu, act, wd, bd, s)
    out = s if alias else torch.full((T, H), NAN, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.ep_moe_few_tokens_workspace_bytes(T, K, H, I, E), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    st = status()

    def call():
        B.ep_moe_few_tokens(x, idx, tw, wu, wd, ws, out, st, bias_up=bu, bias_down=bd, residual=s,
                            activation=ACTS[act])
    call()
    assert int(st.item()) == want_status
    ref.check(out, want, bound, "out")
    if not alias:
        first = out.clone()
        call()              # the workspace now holds the first call's leavings
        assert torch.equal(first, out)
    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            call()
        for _ in range(3):
            out.fill_(NAN)
            cg.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)


@pytest.mark.parametrize("act", list(ACTS))
def test_few_activations(act):
    run_few(9, 3, 12, 136, 72, act, bias=True, res=True, mask=0.2, seed=31)


@pytest.mark.parametrize("T,K,E,H,I", [
    (1, 1, 1, 8, 8), (1, 8, 16, 256, 128), (2, 4, 7, 72, 200), (16, 8, 64, 512, 256), (17, 2, 3, 264, 1000),
    (128, 8, 32, 256, 192), (256, 16, 24, 128, 64), (256, 1, 2, 136, 72), (33, 16, 2048, 64, 64),
    (64, 4, 256, 1024, 384), (256, 16, 2048, 64, 64), (1, 1, 3, 2048, 1032), (3, 2, 2, 4096, 2048), (90, 1, 1, 1024, 1032),
])
def test_few_sizes(T, K, E, H, I):
    run_few(T, K, E, H, I, seed=T + K + E)
    run_few(T, K, E, H, I, "silu", bias=True, res=True, mask=0.3, seed=T + K + E + 1)


def test_few_one_expert_takes_everything():
    run_few(256, 16, 4, 64, 72, mode="one", seed=41)
    run_few(200, 3, 4, 128, 136, mode="one", bias=True, seed=42)


def test_few_repeated_experts():
    run_few(100, 8, 5, 128, 64, mode="random", bias=True, seed=43)


def test_few_invalid_entries():
    from gpu_path import B
    run_few(50, 6, 10, 128, 64, mode="invalid", bias=True, seed=44, want_status=B.EP_ERR_INVALID_INDEX)


def test_few_all_masked():
    run_few(5, 4, 8, 128, 64, mask=1.1, seed=45)
    run_few(5, 4, 8, 128, 64, mask=1.1, bias=True, res=True, seed=46)


def test_few_residual_is_the_output():
    run_few(12, 4, 8, 264, 64, res=True, alias=True, seed=47)


def test_few_in_a_graph():
    run_few(24, 4, 16, 512, 256, res=True, seed=48, graph=True)


def test_few_without_tokens():
    from gpu_path import B
    g = gen(0)
    st = status()
    none = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.ep_moe_few_tokens_workspace_bytes(0, 4, 64, 64, 8), dtype=torch.uint8, device="cuda")
    B.ep_moe_few_tokens(none, torch.empty((0, 4), dtype=torch.int64, device="cuda"),
                        torch.empty((0, 4), device="cuda"), normal(g, 8, 128, 64), normal(g, 8, 64, 64), ws,
                        none.clone(), st)
    assert int(st.item()) == 0


def test_few_tokens_equals_the_rows_path():
    """The same layer through layout, expanded dispatch, two products and the
    expanded combine: both within their bounds of the definition."""
    from gpu_path import B
    from combine_ep_get_gb300.inputs import make_inputs
    T, H, I, E, K, R = 100, 256, 192, 16, 4, 4
    d = make_inputs(T, H, E, K, R, seed=3, mask_frac=0.1)
    g = gen(50)
    idx, tw = torch.from_numpy(d["topk_idx"]).cuda(), torch.from_numpy(d["topk_weights"]).cuda()
    x = torch.from_numpy(d["x_bits"].view(np.int16)).cuda().view(torch.bfloat16)
    wu, wd = normal(g, E, 2 * I, H, std=H ** -0.5), normal(g, E, H, I, std=I ** -0.5)
    st = status()
    lay = B.alloc_layout(T, E, R, K=K)
    ws = torch.empty(B.ep_layout_workspace_bytes(T, K, E, R), dtype=torch.uint8, device="cuda")
    B.ep_get_layout(idx, E, R, lay, ws, st, expert_alignment=16)
    rows = B.ep_expanded_capacity_bound(T, K, E, 16)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    rx, src, rw = torch.full((rows, H), NAN, **bf), torch.empty(rows, dtype=torch.int32, device="cuda"), \
        torch.empty(rows, device="cuda")
    B.ep_dispatch_expanded(x, idx, tw, E, R, lay, rx, src, rw, st)
    h, y = torch.full((rows, I), NAN, **bf), torch.full((rows, H), NAN, **bf)
    B.ep_expert_gemm(rx, wu, lay.expert_offset, lay.num_tokens_per_expert, h, st, activation=B.EP_ACT_SWIGLU)
    B.ep_expert_gemm(h, wd, lay.expert_offset, lay.num_tokens_per_expert, y, st)
    a, b = torch.empty((T, H), **bf), torch.empty((T, H), **bf)
    B.ep_combine_expanded(y, tw, K, E, R, lay, a, st)
    fw = torch.empty(B.ep_moe_few_tokens_workspace_bytes(T, K, H, I, E), dtype=torch.uint8, device="cuda")
    B.ep_moe_few_tokens(x, idx, tw, wu, wd, fw, b, st)
    assert int(st.item()) == 0
    want, bound = ref.few_tokens(x, idx, tw, wu, None, "swiglu", wd, None, None)
    ref.check(b, want, bound, "few tokens")
    # the rows path rounds each expert's output to bf16 too
    extra = torch.zeros_like(want)
    for t, k in torch.nonzero(idx >= 0).tolist():
        extra[t] += tw[t, k].double() * y[lay.expanded_row[t, k]].double().abs() * ref.BF * 1.02
    ref.check(a, want, bound + extra, "rows path")
