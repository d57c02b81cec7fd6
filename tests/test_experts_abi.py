"""Refusals of the experts' entry points: host checks, before any CUDA call,
so they run on a machine without a GPU."""
import ctypes

import pytest

VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def B():
    from combine_ep_get_gb300 import build
    build.build()
    from combine_ep_get_gb300 import binding
    return binding


def change(args, **kw):
    return list({**args, **kw}.values())


def product_args():
    p = [VP(16 * (i + 1)) for i in range(12)]
    return dict(x=p[0], x_sf=None, col=0, w=p[1], w_sf=None, dtype=0, bias=p[2], act=0, rw=p[3], res=p[4], rows=100,
                K=64, N=64, E=4, off=p[5], cnt=p[6], y=p[7], z=p[8], st=p[9], stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(E=0), 1), (dict(K=60), 1), (dict(N=68), 1),
    (dict(act=5), 1), (dict(act=-1), 1), (dict(dtype=2), 1), (dict(dtype=1), 1),
    (dict(dtype=1, K=128, N=128), 1),                                  # FP8 without scales
    (dict(dtype=1, K=128, N=64, x_sf=VP(16), w_sf=VP(16)), 1),
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(off=None), 1), (dict(cnt=None), 1),
    (dict(st=None), 1), (dict(x=VP(24)), 1), (dict(w=VP(24)), 1), (dict(y=VP(18)), 1), (dict(z=VP(18)), 1),
    (dict(bias=VP(20)), 1), (dict(rw=VP(20)), 1), (dict(res=VP(18)), 1), (dict(off=VP(20)), 1),
    (dict(E=2049), 2), (dict(rows=1 << 31), 2), (dict(K=(1 << 20) + 8), 2), (dict(N=(1 << 20) + 8), 2),
])
def test_product_refusals(B, kw, code):
    assert B.library().ep_expert_gemm(*change(product_args(), **kw)) == code


def test_product_without_rows_launches_nothing(B):
    assert B.library().ep_expert_gemm(*change(product_args(), rows=0, x=None, y=None)) == 0


def backward_args():
    p = [VP(16 * (i + 1)) for i in range(14)]
    return dict(dy=p[0], x=p[1], w=p[2], z=p[3], act=3, rw=p[4], rows=100, K=64, N=64, E=4, off=p[5], cnt=p[6],
                dx=p[7], dw=p[8], db=p[9], drw=p[10], ws=p[11], ws_bytes=1 << 30, st=p[12], stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(K=12), 1), (dict(N=12), 1), (dict(act=9), 1), (dict(dy=None), 1), (dict(z=None), 1),
    (dict(x=None), 1), (dict(w=None), 1), (dict(ws=None), 1), (dict(ws_bytes=100), 1), (dict(st=None), 1),
    (dict(dx=VP(18)), 1), (dict(dw=VP(18)), 1), (dict(db=VP(20)), 1), (dict(drw=VP(20)), 1), (dict(dy=VP(18)), 1),
    (dict(act=0, z=None), 1),                                          # d_row_weight needs z
    (dict(E=4096), 2), (dict(rows=1 << 31), 2),
])
def test_backward_refusals(B, kw, code):
    assert B.library().ep_expert_gemm_backward(*change(backward_args(), **kw)) == code


def few_args():
    p = [VP(16 * (i + 1)) for i in range(12)]
    return dict(x=p[0], idx=p[1], tw=p[2], wu=p[3], bu=p[4], act=4, wd=p[5], bd=p[6], res=p[7], T=8, H=64, I=64, K=2,
                E=4, ws=p[8], ws_bytes=1 << 30, out=p[9], st=p[10], stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=12), 1), (dict(I=12), 1), (dict(K=0), 1), (dict(E=0), 1),
    (dict(act=7), 1), (dict(x=None), 1), (dict(idx=None), 1), (dict(tw=None), 1), (dict(wu=None), 1),
    (dict(wd=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(ws_bytes=64), 1), (dict(st=None), 1),
    (dict(x=VP(18)), 1), (dict(bu=VP(20)), 1), (dict(bd=VP(20)), 1), (dict(res=VP(18)), 1),
    (dict(T=257), 2), (dict(K=17), 2), (dict(E=2049), 2), (dict(H=(1 << 20) + 8), 2),
])
def test_few_refusals(B, kw, code):
    assert B.library().ep_moe_few_tokens(*change(few_args(), **kw)) == code


def test_workspace_sizes(B):
    assert B.ep_expert_gemm_backward_workspace_bytes(1000, 64, 4, B.EP_ACT_SWIGLU) >= 1000 * 128 * 2
    assert B.ep_expert_gemm_backward_workspace_bytes(0, 64, 4) >= 16
    assert B.ep_expert_gemm_backward_workspace_bytes(-1, 64, 4) == 16
    assert B.ep_moe_few_tokens_workspace_bytes(8, 2, 64, 32, 4) >= 16 * (32 * 2 + 64 * 4)
    assert B.ep_moe_few_tokens_workspace_bytes(-1, 2, 64, 32, 4) == 16
