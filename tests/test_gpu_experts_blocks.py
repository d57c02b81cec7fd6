"""Blocks of rows that the experts' calls have to bound by themselves: blocks
that overlap (more row tiles than disjoint ones can have) are flagged and count
as empty, nothing beyond the arrays or the workspace is written; rows beyond
the arrays are skipped; disjoint blocks may lie in any order."""
import pytest
import torch

import experts_reference as ref
from experts_reference import ACTS
from test_gpu_experts import gen, normal, status, to_fp8

pytestmark = pytest.mark.gpu


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp8,E,rows,K,N,act", [
    (False, 3, 40, 2048, 64, "none"),         # a cluster shares each tile's sum
    (False, 9, 300, 64, 64, "swiglu"),        # one CTA a tile
    (False, 40, 700, 64, 1024, "silu"),       # pairs of CTAs
    (False, 2048, (1 << 20) + 8, 8, 8, "none"),   # rows add up to more than 2^31
    (True, 7, 300, 256, 256, "gelu"),
])
def test_product_of_overlapping_blocks(fp8, E, rows, K, N, act):
    from gpu_path import B
    g = gen(E)
    Nw = 2 * N if act == "swiglu" else N
    x, w = normal(g, rows, K), normal(g, E, Nw, K)
    kw = {}
    if fp8:
        x, xs = to_fp8(x, 1)
        w, ws = to_fp8(w, 128)
        kw = dict(x_sf=xs, w_sf=ws)
    y = torch.full((rows, N), -7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((rows, Nw), -7.0, dtype=torch.bfloat16, device="cuda")
    st = status()
    B.ep_expert_gemm(x, w, i32([0] * (E + 1)), i32([rows] * E), y, st, activation=ACTS[act], z=z, **kw)
    assert int(st.item()) == B.EP_ERR_CAPACITY
    assert bool((y == -7.0).all()) and bool((z == -7.0).all())


@pytest.mark.parametrize("E,rows,K,N,act", [(64, 2000, 72, 136, "silu"), (5, 700, 512, 1024, "swiglu"), (3, 100, 64, 64, "none"),
                                            (2048, (1 << 20) + 8, 8, 8, "gelu")])
def test_gradients_of_overlapping_blocks(E, rows, K, N, act):
    """Nothing is written past the workspace, and no block's rows."""
    from gpu_path import B
    g = gen(E)
    Nw = 2 * N if act == "swiglu" else N
    dy, x, z, w = normal(g, rows, N), normal(g, rows, K), normal(g, rows, Nw), normal(g, E, Nw, K)
    dx = torch.full((rows, K), -7.0, dtype=torch.bfloat16, device="cuda")
    drw = torch.full((rows,), -7.0, device="cuda")
    dw, db = torch.full_like(w, -7.0), torch.full((E, Nw), -7.0, device="cuda")
    nbytes = B.ep_expert_gemm_backward_workspace_bytes(rows, N, E, ACTS[act])
    whole = torch.full((nbytes + (8 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    st = status()
    B.ep_expert_gemm_backward(dy, x, w, z, i32([0] * (E + 1)), i32([rows] * E), whole[:nbytes], st, dx=dx, dw=dw,
                              dbias=db, d_row_weight=drw, activation=ACTS[act], row_weight=torch.ones(rows, device="cuda"))
    assert int(st.item()) == B.EP_ERR_CAPACITY
    assert bool((whole[nbytes:] == 0x5A).all())
    assert bool((dx == -7.0).all()) and bool((drw == -7.0).all())
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_gradients_of_rows_beyond_the_arrays():
    """Offsets that promise more rows than there are: the ones inside are right, the bit is set."""
    from gpu_path import B
    g = gen(4)
    rows, K, N = 50, 64, 48
    off, cnt = i32([0, 20, 45, 60, 80]), i32([20, 25, 15, 9])
    dy, x, z, w = normal(g, rows, N), normal(g, rows, K), normal(g, rows, N), normal(g, 4, N, K, std=K ** -0.5)
    dx, dw, db, drw = torch.zeros_like(x), torch.empty_like(w), torch.empty((4, N), device="cuda"), \
        torch.zeros(rows, device="cuda")
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(rows, N, 4, B.EP_ACT_SILU), dtype=torch.uint8,
                     device="cuda")
    st = status()
    B.ep_expert_gemm_backward(dy, x, w, z, off, cnt, ws, st, dx=dx, dw=dw, dbias=db, d_row_weight=drw,
                              activation=B.EP_ACT_SILU)
    assert int(st.item()) == B.EP_ERR_CAPACITY
    for e, (a, b) in enumerate(((0, 20), (20, 45), (45, 50), (50, 50))):
        R = ref.backward_rows(dy[a:b].double(), x[a:b].double(), w[e].double(), z[a:b].double(), "silu", None)
        ref.check(dx[a:b], *R["dx"])
        ref.check(dw[e], *R["dw"])
        ref.check(db[e], *R["dbias"])
        ref.check(drw[a:b], *R["d_row_weight"])


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_disjoint_blocks_in_any_order(act):
    """Blocks need not ascend, and may fill the arrays to the last row."""
    from gpu_path import B
    g = gen(8)
    off, cnt, rows, K, N = [170, 0, 40, 41], [130, 40, 1, 129], 300, 64, 72
    Nw = 2 * N if act == "swiglu" else N
    x, w = normal(g, rows, K), normal(g, 4, Nw, K, std=K ** -0.5)
    y, z = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda"), torch.zeros((rows, Nw), dtype=torch.bfloat16,
                                                                                   device="cuda")
    st = status()
    B.ep_expert_gemm(x, w, i32(off + [0]), i32(cnt), y, st, activation=ACTS[act], z=z)
    dx, dw, db = torch.zeros_like(x), torch.empty_like(w), torch.empty((4, Nw), device="cuda")
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(rows, N, 4, ACTS[act]), dtype=torch.uint8, device="cuda")
    B.ep_expert_gemm_backward(y, x, w, z, i32(off + [0]), i32(cnt), ws, st, dx=dx, dw=dw, dbias=db, activation=ACTS[act])
    assert int(st.item()) == 0
    for e in range(4):
        d = slice(off[e], off[e] + cnt[e])
        yy, by, zz, bz = ref.product_rows(x[d].double(), w[e].double(), None, act, None, None)
        ref.check(y[d], yy, by)
        ref.check(z[d], zz, bz)
        R = ref.backward_rows(y[d].double(), x[d].double(), w[e].double(), z[d].double(), act, None)
        for name, got in (("dx", dx[d]), ("dw", dw[e]), ("dbias", db[e])):
            ref.check(got, *R[name], what=name)
