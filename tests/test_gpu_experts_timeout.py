"""The bounded waits of the experts' tensor-core kernels, without faulting or
hanging the GPU: a test-only copy of the library with a 1 ms wait limit, in
which the first CTA (or pair of CTAs) of every kernel announces its first rows
on a barrier and never loads them.  Nothing is in flight for that barrier and
every access stays in bounds; the waits on it run out, the kernel sets
EP_ERR_TIMEOUT, gives its tensor memory back and returns.  The same stream then
runs the product library, whose results are checked."""
import ctypes

import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def failing():
    from gpu_path import B
    from combine_ep_get_gb300 import build
    path = build.build_variant("expertswait", ["-DEP_WAIT_TIMEOUT_NS=1000000ull", "-DEP_TEST_DROP_FIRST_LOAD"],
                               recompile=("experts_mma.cu", "experts_fp8.cu"))
    lib = ctypes.CDLL(path)
    for name in ("ep_expert_gemm", "ep_expert_gemm_backward", "ep_moe_few_tokens"):
        f = getattr(lib, name)
        f.restype, f.argtypes = getattr(B.library(), name).restype, getattr(B.library(), name).argtypes
    return lib


def run(B, lib, call):
    """call(status) through `lib`; the status word it leaves."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = B._lib
    B._lib = lib
    try:
        call(st)
    finally:
        B._lib = keep
    torch.cuda.synchronize()
    return int(st.item())


@pytest.mark.parametrize("fp8,rows,n,k", [(False, 60, 128, 256), (False, 2100, 2048, 256), (False, 20, 64, 4096),
                                          (True, 300, 256, 256)])
def test_product_wait_runs_out_then_the_stream_works(failing, fp8, rows, n, k):
    """One CTA a tile, a pair of CTAs a tile, a cluster that shares a sum, FP8."""
    from gpu_path import B
    from test_gpu_experts import blocks, gen, normal, to_fp8
    g = gen(rows)
    off, cnt, total = blocks([rows, rows // 2])
    x, w = normal(g, total, k), normal(g, 2, n, k, std=k ** -0.5)
    kw, x64, w64 = {}, x.double(), w.double()
    if fp8:
        x, xs = to_fp8(x, 1)
        w, ws = to_fp8(w, 128)
        x64 = x.double() * xs.double().repeat_interleave(128, 1)
        w64 = w.double() * ws.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        kw = dict(x_sf=xs, w_sf=ws)
    y = torch.zeros((total, n), dtype=torch.bfloat16, device="cuda")

    def call(st):
        B.ep_expert_gemm(x, w, off, cnt, y, st, **kw)

    assert run(B, failing, call) == B.EP_ERR_TIMEOUT
    assert run(B, B.library(), call) == 0
    for e, d in enumerate((slice(0, rows), slice(rows, total))):
        want, bound, _, _ = ref.product_rows(x64[d], w64[e], None, "none", None, None)
        ref.check(y[d], want, bound)


@pytest.mark.parametrize("rows,k,n", [(60, 64, 64), (400, 2048, 1024), (2200, 64, 64)])
def test_backward_wait_runs_out_then_the_stream_works(failing, rows, k, n):
    from gpu_path import B
    from test_gpu_experts import blocks, gen, normal
    g = gen(rows)
    off, cnt, total = blocks([rows, rows + 3])
    dy, x, w = normal(g, total, n), normal(g, total, k), normal(g, 2, n, k, std=n ** -0.5)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(total, n, 2), dtype=torch.uint8, device="cuda")

    def call(st):
        B.ep_expert_gemm_backward(dy, x, w, None, off, cnt, ws, st, dx=dx, dw=dw)

    assert run(B, failing, call) == B.EP_ERR_TIMEOUT
    assert run(B, B.library(), call) == 0
    for e, d in enumerate((slice(0, rows), slice(rows, total))):
        r = ref.backward_rows(dy[d].double(), x[d].double(), w[e].double(), None, "none", None)
        ref.check(dx[d], *r["dx"])
        ref.check(dw[e], *r["dw"])


def test_few_tokens_wait_runs_out_then_the_stream_works(failing):
    from gpu_path import B
    from test_gpu_experts import gen, normal
    g = gen(3)
    T, K, E, H, I = 9, 2, 8, 256, 192
    idx = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), dim=1)[:, :K].contiguous()
    tw = torch.rand((T, K), generator=g, device="cuda")
    x, wu, wd = normal(g, T, H), normal(g, E, 2 * I, H, std=1 / 16), normal(g, E, H, I, std=I ** -0.5)
    out = torch.zeros_like(x)
    ws = torch.empty(B.ep_moe_few_tokens_workspace_bytes(T, K, H, I, E), dtype=torch.uint8, device="cuda")

    def call(st):
        B.ep_moe_few_tokens(x, idx, tw, wu, wd, ws, out, st)

    assert run(B, failing, call) == B.EP_ERR_TIMEOUT
    assert run(B, B.library(), call) == 0
    ref.check(out, *ref.few_tokens(x, idx, tw, wu, None, "swiglu", wd, None, None))
