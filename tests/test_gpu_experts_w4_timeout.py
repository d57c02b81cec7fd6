"""The bounded waits of the 4-bit experts' kernels, without faulting or hanging
the GPU: a test-only copy of the library with a 1 ms wait limit, in which the
first CTA never arrives for its first rows.  Nothing is in flight for that
barrier and every access stays in bounds; the waits on it run out, the kernel
sets EP_ERR_TIMEOUT and returns.  The same stream then runs the product
library, whose results are checked."""
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
    path = build.build_variant("w4wait", ["-DEP_WAIT_TIMEOUT_NS=1000000ull", "-DEP_TEST_DROP_FIRST_LOAD"],
                               recompile=("experts_w4_int.cu",))
    lib = ctypes.CDLL(path)
    for name in ("ep_expert_gemm_w4", "ep_moe_few_tokens_w4"):
        f = getattr(lib, name)
        f.restype, f.argtypes = getattr(B.library(), name).restype, getattr(B.library(), name).argtypes
    return lib


@pytest.mark.parametrize("rows", [3, 11, 30])
def test_product_wait_runs_out_then_the_stream_works(failing, rows):
    """Up to 8, 16 and 32 rows of an expert: one or two teams of warps."""
    from gpu_path import B
    g = gen(rows)
    off, cnt, total = blocks([rows, rows])
    x, y = normal(g, total, 2048), torch.zeros((total, 512), dtype=torch.bfloat16, device="cuda")
    w, sf, _ = ref.make(g, 2, 512, 2048, 128)
    status = run(B, failing, lambda st: B.ep_expert_gemm_w4(x, w, sf, off, cnt, y, st))
    assert status & B.EP_ERR_TIMEOUT
    check_product([rows, rows], 2048, 512)


def test_few_tokens_wait_runs_out_then_the_stream_works(failing):
    from gpu_path import B
    d = make_few(6, 2048, 512, 8, 4, "swiglu")
    out = torch.empty_like(d["x"])
    status = run(B, failing, lambda st: run_few(d, "swiglu", "int", out=out, st=st))
    assert status & B.EP_ERR_TIMEOUT
    check_few(d, "swiglu", "int")
