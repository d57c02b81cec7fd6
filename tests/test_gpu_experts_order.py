"""The experts' calls read what the stream wrote just before them: inputs are
overwritten by a kernel right ahead of every call, with no wait on the host,
and the results equal those of calls that were waited for, bit for bit.  Two of
the calls' kernels read inputs before the kernel ahead of them has ended."""
import pytest
import torch

from experts_reference import ACTS
from test_gpu_experts import gen, normal, status

pytestmark = pytest.mark.gpu

ROUNDS = 24


def back_to_back(versions, call, outputs):
    """call() on each version's values in the same buffers, waited for and not: both lists of outputs."""
    buffers = [torch.empty_like(t) for t in versions[0]]

    def one(v):
        for b, t in zip(buffers, v):
            b.copy_(t)
        call(*buffers)
        return [o.clone() for o in outputs]

    alone = []
    for v in versions:
        torch.cuda.synchronize()
        alone.append(one(v))
        torch.cuda.synchronize()
    order = [i % len(versions) for i in range(ROUNDS)]
    got = [one(versions[i]) for i in order]
    torch.cuda.synchronize()
    for i, g in zip(order, got):
        for a, b in zip(alone[i], g):
            assert torch.equal(a, b)
    assert not torch.equal(alone[0][0], alone[1][0])


def counts_of(g, E, rows):
    c = torch.rand(E, generator=g, device="cuda")
    c = (c / c.sum() * (rows - E)).int()
    off = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cumsum(c, 0).int()])
    return off, c


@pytest.mark.parametrize("rows,E,K,N,act", [(500, 6, 256, 512, "silu"), (3000, 20, 264, 520, "swiglu"),
                                            (700, 3, 64, 2056, "none")])
def test_gradients_see_what_the_stream_wrote_before(rows, E, K, N, act):
    from gpu_path import B
    Nw = 2 * N if act == "swiglu" else N
    versions = []
    for seed in range(3):
        g = gen(seed)
        versions.append([normal(g, rows, N), normal(g, rows, K), normal(g, E, Nw, K), normal(g, rows, Nw),
                         *counts_of(g, E, rows)])
    dx, dw = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda"), torch.empty_like(versions[0][2])
    db, drw = torch.empty((E, Nw), device="cuda"), torch.zeros(rows, device="cuda")
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(rows, N, E, ACTS[act]), dtype=torch.uint8, device="cuda")
    st = status()

    def call(dy, x, w, z, off, cnt):
        dx.zero_()      # rows of no block are not written
        drw.zero_()
        B.ep_expert_gemm_backward(dy, x, w, z, off, cnt, ws, st, dx=dx, dw=dw, dbias=db, d_row_weight=drw,
                                  activation=ACTS[act])

    back_to_back(versions, call, (dx, dw, db, drw))
    assert int(st.item()) == 0


@pytest.mark.parametrize("T,K,E,H,I", [(1, 4, 16, 512, 256), (40, 8, 32, 256, 512), (200, 2, 5, 1024, 136)])
def test_few_tokens_see_what_the_stream_wrote_before(T, K, E, H, I):
    from gpu_path import B
    versions = []
    for seed in range(3):
        g = gen(100 + seed)
        idx = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), dim=1)[:, :K].contiguous()
        versions.append([normal(g, T, H), idx, torch.rand((T, K), generator=g, device="cuda"),
                         normal(g, E, 2 * I, H, std=H ** -0.5), normal(g, E, H, I, std=I ** -0.5)])
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.ep_moe_few_tokens_workspace_bytes(T, K, H, I, E), dtype=torch.uint8, device="cuda")
    st = status()

    def call(x, idx, tw, wu, wd):
        B.ep_moe_few_tokens(x, idx, tw, wu, wd, ws, out, st)

    back_to_back(versions, call, (out,))
    assert int(st.item()) == 0


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
def test_product_and_gradients_in_a_graph(act):
    """Captured with the copies that bring their inputs, replayed with others: as outside a graph."""
    from gpu_path import B
    rows, E, K, N = 900, 7, 264, 520
    Nw = 2 * N if act == "swiglu" else N
    versions = []
    for seed in range(3):
        g = gen(200 + seed)
        versions.append([normal(g, rows, N), normal(g, rows, K), normal(g, E, Nw, K, std=K ** -0.5), *counts_of(g, E, rows)])
    source, buffers = ([torch.empty_like(t) for t in versions[0]] for _ in range(2))
    bf = dict(dtype=torch.bfloat16, device="cuda")
    out = [torch.empty((rows, N), **bf), torch.empty((rows, Nw), **bf), torch.empty((rows, K), **bf),
           torch.empty((E, Nw, K), **bf), torch.empty((E, Nw), device="cuda"), torch.empty(rows, device="cuda")]
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(rows, N, E, ACTS[act]), dtype=torch.uint8, device="cuda")
    st = status()

    def step():
        for b, s in zip(buffers, source):
            b.copy_(s)
        dy, x, w, off, cnt = buffers
        y, z, dx, dw, db, drw = out
        for t in (y, z, dx, drw):
            t.zero_()
        B.ep_expert_gemm(x, w, off, cnt, y, st, activation=ACTS[act], z=z)
        B.ep_expert_gemm_backward(dy, x, w, z, off, cnt, ws, st, dx=dx, dw=dw, dbias=db, d_row_weight=drw,
                                  activation=ACTS[act])

    want = []
    for v in versions:
        for s, t in zip(source, v):
            s.copy_(t)
        step()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(6):
        for s, t in zip(source, versions[i % 3]):
            s.copy_(t)
        graph.replay()
        for a, b in zip(want[i % 3], out):
            assert torch.equal(a, b)
    assert int(st.item()) == 0 and not torch.equal(want[0][0], want[1][0])


def test_two_streams_at_once():
    """Calls of two streams, each with its own buffers, overlap and keep their results."""
    from gpu_path import B
    sides = []
    for seed, (T, K, E, H, I) in enumerate([(30, 4, 16, 512, 520), (200, 2, 12, 776, 256)]):
        g = gen(300 + seed)
        idx = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), dim=1)[:, :K].contiguous()
        args = (normal(g, T, H), idx, torch.rand((T, K), generator=g, device="cuda"),
                normal(g, E, 2 * I, H, std=H ** -0.5), normal(g, E, H, I, std=I ** -0.5),
                torch.empty(B.ep_moe_few_tokens_workspace_bytes(T, K, H, I, E), dtype=torch.uint8, device="cuda"),
                torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), status())
        B.ep_moe_few_tokens(*args)
        rows = 500 + 300 * seed
        off, cnt = counts_of(g, E, rows)
        x, y = normal(g, rows, H), torch.zeros((rows, I), dtype=torch.bfloat16, device="cuda")
        B.ep_expert_gemm(x, args[3], off, cnt, y, args[7], activation=B.EP_ACT_SWIGLU)
        sides.append((args, (x, off, cnt, y), args[6].clone(), y.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for args, (x, off, cnt, y), _, _, stream in sides:
            B.ep_moe_few_tokens(*args, stream=stream)
            B.ep_expert_gemm(x, args[3], off, cnt, y, args[7], activation=B.EP_ACT_SWIGLU, stream=stream)
    torch.cuda.synchronize()
    for args, rest, out, y, _ in sides:
        assert torch.equal(args[6], out) and torch.equal(rest[3], y) and int(args[7].item()) == 0
