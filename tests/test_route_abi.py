"""Refusals of the router's and the 4-bit experts' entry points: host checks,
before any CUDA call, so they run on a machine without a GPU."""
import ctypes

import pytest
import torch

from test_experts_abi import B, change  # noqa: F401  (a fixture)
from test_experts_binding import Library, OnGpu, Stream

VP = ctypes.c_void_p


def route_args():
    p = [VP(16 * (i + 1)) for i in range(6)]
    return dict(l=p[0], dt=3, stride=64, bias=p[1], mask=VP(33), T=10, E=64, K=4, score=1, G=8, TG=4, norm=1, scale=1.0,
                idx=p[2], w=p[3], st=p[4], stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(K=0), 1), (dict(K=65), 1), (dict(dt=1), 1), (dict(dt=4), 1), (dict(score=2), 1),
    (dict(stride=63), 1), (dict(l=None), 1), (dict(l=VP(18)), 1), (dict(dt=0, l=VP(17)), 1), (dict(idx=None), 1),
    (dict(idx=VP(24)), 1), (dict(w=None), 1), (dict(w=VP(24)), 1), (dict(bias=VP(20)), 1), (dict(st=None), 1),
    (dict(G=0), 1), (dict(G=7), 1), (dict(TG=0), 1), (dict(TG=9), 1), (dict(TG=1, K=9), 1),
    (dict(E=4096, stride=4096), 2), (dict(K=33), 2), (dict(T=1 << 26), 2), (dict(G=64, TG=64), 2),
    (dict(stride=1 << 62), 2),
])
def test_route_refusals(B, kw, code):  # noqa: F811
    assert B.library().ep_route(*change(route_args(), **kw)) == code


def test_route_without_tokens_launches_nothing(B):  # noqa: F811
    assert B.library().ep_route(*change(route_args(), T=0, l=None, idx=None, w=None)) == 0


def balance_args():
    p = [VP(16 * (i + 1)) for i in range(9)]
    return dict(l=p[0], dt=0, stride=64, idx=p[1], mask=None, off=p[2], T=10, E=64, K=4, S=2, score=0, coeff=1.0, loss=p[3],
                load=p[4], counts=p[5], ws=p[6], ws_bytes=1 << 30, st=p[7], stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(K=65), 1), (dict(dt=2, l=VP(33)), 1), (dict(S=0), 1), (dict(off=None), 1),
    (dict(off=VP(20)), 1), (dict(loss=None), 1), (dict(load=None), 1), (dict(counts=VP(20)), 1), (dict(ws=None), 1),
    (dict(ws_bytes=64), 1), (dict(idx=None), 1), (dict(score=-1), 1), (dict(st=None), 1), (dict(S=1 << 26), 2),
])
def test_balance_refusals(B, kw, code):  # noqa: F811
    assert B.library().ep_balance_loss(*change(balance_args(), **kw)) == code


def test_balance_workspace(B):  # noqa: F811
    assert B.ep_balance_loss_workspace_bytes(4096, 256) >= 256 * 8
    assert B.ep_balance_loss_workspace_bytes(-1, 256) == 16
    assert B.ep_balance_loss_workspace_bytes(0, 1) >= 16


def backward_args():
    p = [VP(16 * (i + 1)) for i in range(9)]
    return dict(l=p[0], dt=3, stride=64, idx=p[1], mask=None, dw=p[2], load=p[3], dl=p[4], off=p[5], T=10, E=64, K=4, S=2,
                score=0, norm=1, scale=1.0, out=p[6], ostride=64, st=p[7], stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(idx=None), 1), (dict(load=None), 1), (dict(dl=None), 1), (dict(S=0), 1),
    (dict(off=None), 1), (dict(dw=VP(20)), 1), (dict(load=VP(20)), 1), (dict(dl=VP(20)), 1), (dict(out=None), 1),
    (dict(out=VP(18)), 1), (dict(ostride=63), 1), (dict(st=None), 1), (dict(K=33), 2), (dict(ostride=1 << 62), 2),
])
def test_backward_refusals(B, kw, code):  # noqa: F811
    assert B.library().ep_route_backward(*change(backward_args(), **kw)) == code


def product_args():
    p = [VP(16 * (i + 1)) for i in range(10)]
    return dict(x=p[0], w=p[1], sf=p[2], zero=p[3], sdt=0, fmt=0, group=64, bias=p[4], act=0, rw=None, res=None, rows=100,
                K=128, N=64, E=4, off=p[5], cnt=p[6], y=p[7], st=p[8], stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(K=0), 1), (dict(K=96), 1), (dict(N=60), 1), (dict(E=0), 1), (dict(act=5), 1),
    (dict(group=16), 1), (dict(group=256, K=256), 1), (dict(fmt=1), 1), (dict(fmt=2), 1), (dict(sdt=1), 1), (dict(sdt=2), 1),
    (dict(x=None), 1), (dict(w=None), 1), (dict(sf=None), 1), (dict(y=None), 1), (dict(off=None), 1), (dict(st=None), 1),
    (dict(x=VP(24)), 1), (dict(w=VP(24)), 1), (dict(sf=VP(24)), 1), (dict(zero=VP(24)), 1), (dict(y=VP(24)), 1),
    (dict(bias=VP(20)), 1), (dict(rw=VP(20)), 1), (dict(res=VP(18)), 1), (dict(E=2049), 2), (dict(rows=1 << 31), 2),
    (dict(K=1 << 21), 2),
])
def test_w4_product_refusals(B, kw, code):  # noqa: F811
    assert B.library().ep_expert_gemm_w4(*change(product_args(), **kw)) == code


def test_w4_product_without_rows_launches_nothing(B):  # noqa: F811
    assert B.library().ep_expert_gemm_w4(*change(product_args(), rows=0, x=None, y=None)) == 0


def few_args():
    p = [VP(16 * (i + 1)) for i in range(14)]
    return dict(x=p[0], idx=p[1], tw=p[2], wu=p[3], us=p[4], uz=None, ug=32, bu=None, act=4, wd=p[5], ds=p[6], dz=None, dg=64,
                bd=None, sdt=0, fmt=0, res=p[7], T=8, H=96, I=64, K=2, E=4, ws=p[8], ws_bytes=1 << 30, out=p[9], st=p[10],
                stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=80), 1), (dict(I=96), 1), (dict(K=0), 1), (dict(act=7), 1), (dict(ug=16), 1),
    (dict(dg=256), 1), (dict(uz=VP(32)), 1), (dict(dz=VP(32)), 1), (dict(fmt=1, uz=VP(32), dz=VP(32)), 1), (dict(sdt=4), 1),
    (dict(x=None), 1), (dict(idx=None), 1), (dict(tw=None), 1), (dict(wu=None), 1), (dict(us=None), 1), (dict(wd=None), 1),
    (dict(ds=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(ws_bytes=64), 1), (dict(st=None), 1),
    (dict(bu=VP(20)), 1), (dict(bd=VP(20)), 1), (dict(res=VP(18)), 1), (dict(wu=VP(24)), 1), (dict(ds=VP(24)), 1),
    (dict(T=257), 2), (dict(K=17), 2), (dict(E=2049), 2), (dict(H=1 << 21), 2),
])
def test_w4_few_refusals(B, kw, code):  # noqa: F811
    assert B.library().ep_moe_few_tokens_w4(*change(few_args(), **kw)) == code


def test_w4_few_workspace(B):  # noqa: F811
    assert B.ep_moe_few_tokens_w4_workspace_bytes(8, 2, 64, 32, 4) >= 16 * (32 * 2 + 64 * 4)
    assert B.ep_moe_few_tokens_w4_workspace_bytes(-1, 2, 64, 32, 4) == 16


def calls(B):  # noqa: F811
    T, E, K, H, N, rows = 6, 8, 2, 128, 128, 24
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32

    def zeros(*shape, dtype=f32):
        return torch.zeros(shape, dtype=dtype)

    idx, st = dict(topk_idx=zeros(T, K, dtype=torch.int64)), dict(d_status=zeros(1, dtype=i32))
    route = dict(logits=zeros(T, E), topk_weights=zeros(T, K), bias=zeros(E), token_mask=zeros(T, dtype=torch.bool), **idx,
                 **st)
    balance = dict(logits=zeros(T, E, dtype=bf), workspace=zeros(4096, dtype=u8), loss=zeros(1), load=zeros(2, E),
                   token_mask=zeros(T, dtype=u8), seq_offset=zeros(3, dtype=i32),
                   num_tokens_per_expert=zeros(2, E, dtype=i32), **idx, **st)
    backward = dict(logits=zeros(T, E), d_logits=zeros(T, E), d_topk_weights=zeros(T, K), load=zeros(2, E), d_loss=zeros(1),
                    seq_offset=zeros(3, dtype=i32), **idx, **st)
    product = dict(x=zeros(rows, H, dtype=bf), w=zeros(E, N, H // 2, dtype=u8), w_sf=zeros(E, 2, N), w_zero=zeros(E, 2, N),
                   expert_offset=zeros(E + 1, dtype=i32), num_tokens_per_expert=zeros(E, dtype=i32),
                   y=zeros(rows, N, dtype=bf), bias=zeros(E, N), row_weight=zeros(rows), residual=zeros(rows, N, dtype=bf),
                   **st)
    few = dict(x=zeros(T, H, dtype=bf), topk_weights=zeros(T, K), w_up=zeros(E, 2 * N, H // 2, dtype=u8),
               up_sf=zeros(E, 1, 2 * N), w_down=zeros(E, H, N // 2, dtype=u8), down_sf=zeros(E, 2, H),
               workspace=zeros(64, dtype=u8), out=zeros(T, H, dtype=bf), up_zero=zeros(E, 1, 2 * N),
               down_zero=zeros(E, 2, H), bias_up=zeros(E, 2 * N), bias_down=zeros(E, H), residual=zeros(T, H, dtype=bf),
               **idx, **st)
    return {"route": (B.ep_route, route), "balance": (B.ep_balance_loss, balance),
            "backward": (B.ep_route_backward, backward), "product": (B.ep_expert_gemm_w4, product),
            "few": (B.ep_moe_few_tokens_w4, few)}


@pytest.mark.parametrize("which", ["route", "balance", "backward", "product", "few"])
def test_tensors_on_the_host_or_of_another_type_are_refused(B, which, monkeypatch):  # noqa: F811
    lib = Library()
    monkeypatch.setattr(B, "_lib", lib)
    f, args = calls(B)[which]
    on_gpu = {k: OnGpu(v) for k, v in args.items()}
    f(**on_gpu, stream=Stream)
    assert len(lib.calls) == 1
    for name in args:
        with pytest.raises(AssertionError):
            f(**{**on_gpu, name: args[name]}, stream=Stream)
        if name != "workspace":
            with pytest.raises(AssertionError):
                f(**{**on_gpu, name: OnGpu(args[name].to(torch.complex64))}, stream=Stream)
    assert len(lib.calls) == 1


def test_strided_logits(B, monkeypatch):  # noqa: F811
    lib = Library()
    monkeypatch.setattr(B, "_lib", lib)
    f, args = calls(B)["route"]
    on_gpu = {k: OnGpu(v) for k, v in args.items()}
    f(**{**on_gpu, "logits": OnGpu(torch.zeros(6, 20)[:, 3:11])}, stream=Stream)
    assert lib.calls[0][1][2] == 20
    for bad in (torch.zeros(8, 6).T, torch.zeros(6, 16)[:, ::2], torch.zeros(1, 8).expand(6, 8)):
        with pytest.raises(AssertionError):
            f(**{**on_gpu, "logits": OnGpu(bad)}, stream=Stream)
