"""The bounded waits of the experts' tensor-core kernels over sums longer than
their rings of stages: the first stage's rows never come while every other
stage's loads are under way, and the CTA (or pair) waits for each of them
before it ends.  The same test-only copy of the library as in
test_gpu_experts_timeout; every access stays in bounds.  The stream then runs
the product library, whose results are checked, and twice over, so that a
late load into a CTA's shared memory would show."""
import pytest
import torch

import experts_reference as ref
from test_gpu_experts_timeout import failing, run  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8,rows,n,k", [(False, 60, 128, 4096), (False, 2100, 512, 4096), (True, 300, 256, 4096)])
def test_product_of_a_long_sum(failing, fp8, rows, n, k):  # noqa: F811
    """One CTA a tile, a pair of CTAs a tile, FP8."""
    from gpu_path import B
    from test_gpu_experts import blocks, gen, normal, to_fp8
    g = gen(rows + k)
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

    for _ in range(2):
        assert run(B, failing, call) == B.EP_ERR_TIMEOUT
        y.zero_()
        assert run(B, B.library(), call) == 0
        for e, d in enumerate((slice(0, rows), slice(rows, total))):
            want, bound, _, _ = ref.product_rows(x64[d], w64[e], None, "none", None, None)
            ref.check(y[d], want, bound)


def test_gradients_of_long_sums(failing):  # noqa: F811
    """dx over 4096 features, dw over 4000 rows and a tail."""
    from gpu_path import B
    from test_gpu_experts import blocks, gen, normal
    g = gen(5)
    rows, k, n = 4003, 256, 4096
    off, cnt, total = blocks([rows, 50])
    dy, x, w = normal(g, total, n), normal(g, total, k), normal(g, 2, n, k, std=n ** -0.5)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(total, n, 2), dtype=torch.uint8, device="cuda")

    def call(st):
        B.ep_expert_gemm_backward(dy, x, w, None, off, cnt, ws, st, dx=dx, dw=dw)

    for _ in range(2):
        assert run(B, failing, call) == B.EP_ERR_TIMEOUT
        dx.zero_()
        dw.zero_()
        assert run(B, B.library(), call) == 0
        for e, d in enumerate((slice(0, rows), slice(rows, total))):
            r = ref.backward_rows(dy[d].double(), x[d].double(), w[e].double(), None, "none", None)
            ref.check(dx[d], *r["dx"])
            ref.check(dw[e], *r["dw"])
