"""The bounded waits of the 4-bit experts' kernels with FP4 codes, whose rows come
through registers, without faulting or hanging the GPU: a test-only copy of the
library with a 1 ms wait limit, in which the first CTA neither asks for its
first stage's codes nor arrives for its rows.  Every access stays in bounds; the
waits on that stage run out while later stages' loads are under way, the CTA
waits for each of those before it ends, sets EP_ERR_TIMEOUT and returns.  The
same stream then runs the product library, whose results are checked.  The
other CTAs' rows are those of the product library even in the failing call."""
import ctypes

import pytest
import torch

from test_gpu_experts_timeout import run
from test_gpu_experts_w4 import blocks, check_few, check_product, gen, make_few, normal, run_few

import experts_w4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def failing():
    from gpu_path import B
    from combine_ep_get_gb300 import build
    path = build.build_variant("w4fpwait", ["-DEP_WAIT_TIMEOUT_NS=1000000ull", "-DEP_TEST_DROP_FIRST_LOAD"],
                               recompile=("experts_w4_fp.cu", "experts_w4_zero.cu"))
    lib = ctypes.CDLL(path)
    for name in ("ep_expert_gemm_w4", "ep_moe_few_tokens_w4"):
        f = getattr(lib, name)
        f.restype, f.argtypes = getattr(B.library(), name).restype, getattr(B.library(), name).argtypes
    return lib


@pytest.mark.parametrize("rows", [1, 3, 11, 30])
@pytest.mark.parametrize("form,zero,group", [("fp4", False, 32), ("fp4", False, 128), ("int", True, 64)])
@pytest.mark.parametrize("K", [2048, 4096 + 128])
def test_product_wait_runs_out_then_the_stream_works(failing, rows, form, zero, group, K):
    """Up to 8, 16 and 32 rows of an expert; sums of which a ring of stages holds all, or a part."""
    from gpu_path import B
    g = gen(rows)
    off, cnt, total = blocks([rows, rows])
    x, y = normal(g, total, K), torch.full((total, 512), -77.0, dtype=torch.bfloat16, device="cuda")
    w, sf, z = ref.make(g, 2, 512, K, group, form, zero)
    good = torch.empty_like(y)

    def call(out):
        return lambda st: B.ep_expert_gemm_w4(x, w, sf, off, cnt, out, st, w_zero=z,
                                              w_format=B.EP_W4_FP if form == "fp4" else B.EP_W4_INT)

    assert run(B, failing, call(y)) == B.EP_ERR_TIMEOUT
    assert run(B, B.library(), call(good)) == 0
    written = y != -77.0
    assert torch.equal(y[written], good[written]) and bool((~written).any()) and bool(written.any())
    check_product([rows, rows], K, 512, form=form, zero=zero, group=group)


@pytest.mark.parametrize("form,zero", [("fp4", False), ("int", True)])
def test_few_tokens_wait_runs_out_then_the_stream_works(failing, form, zero):
    from gpu_path import B
    d = make_few(6, 2048, 512, 8, 4, "swiglu", form=form, zero=zero)
    out = torch.empty_like(d["x"])
    status = run(B, failing, lambda st: run_few(d, "swiglu", form, out=out, st=st))
    assert status == B.EP_ERR_TIMEOUT
    check_few(d, "swiglu", form)
