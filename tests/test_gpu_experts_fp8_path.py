"""The FP8 rows and scales that the expanded dispatch leaves go straight into
the experts' product, in both layouts of the scales, with rows to spare."""
import numpy as np
import pytest
import torch

import experts_reference as ref
from experts_reference import ACTS
from test_gpu_experts import gen, normal, status, to_fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("col_major", [False, True])
@pytest.mark.parametrize("T,H,N,E,K,R,align,spare,act", [(150, 384, 256, 12, 3, 4, 16, 5, "swiglu"),
                                                         (77, 128, 384, 5, 2, 1, 1, 0, "gelu"),
                                                         (600, 896, 128, 32, 8, 8, 4, 3, "none")])
def test_dispatched_rows_through_the_product(T, H, N, E, K, R, align, spare, act, col_major):
    from gpu_path import B
    from combine_ep_get_gb300.inputs import make_inputs
    d = make_inputs(T, H, E, K, R, seed=T, mask_frac=0.1)
    idx, tw = torch.from_numpy(d["topk_idx"]).cuda(), torch.from_numpy(d["topk_weights"]).cuda()
    x = torch.from_numpy(d["x_bits"].view(np.int16)).cuda().view(torch.bfloat16)
    st = status()
    lay = B.alloc_layout(T, E, R, K=K)
    ws = torch.empty(B.ep_layout_workspace_bytes(T, K, E, R), dtype=torch.uint8, device="cuda")
    B.ep_get_layout(idx, E, R, lay, ws, st, expert_alignment=align)
    rows = B.ep_expanded_capacity_bound(T, K, E, align) + spare
    stride = (rows + 3) // 4 * 4 if col_major else rows
    codes = torch.full((rows, H), 0x7F, dtype=torch.uint8, device="cuda")      # NaN in padding
    sf = torch.full((stride * (H // 128),), float("nan"), device="cuda")
    src, rw = torch.full((rows,), -9, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
    B.ep_dispatch_expanded(x, idx, tw, E, R, lay, codes, src, rw, st, recv_sf=sf, out_dtype=B.EP_FP8_E4M3,
                           sf_col_major=col_major)
    Nw = 2 * N if act == "swiglu" else N
    w, w_sf = to_fp8(normal(gen(T), E, Nw, H, std=H ** -0.5), 128)
    y = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    B.ep_expert_gemm(codes, w.view(torch.uint8), lay.expert_offset, lay.num_tokens_per_expert, y, st,
                     activation=ACTS[act], row_weight=rw, x_sf=sf, w_sf=w_sf, sf_col_major=col_major)
    assert int(st.item()) == 0
    scales = sf.view(H // 128, stride)[:, :rows].T if col_major else sf.view(rows, H // 128)
    x64 = codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)
    w64 = w.double() * w_sf.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    first, count = lay.expert_offset.tolist(), lay.num_tokens_per_expert.tolist()
    assert sum(count) == int((idx >= 0).sum())
    for e in range(E):
        r = slice(first[e], first[e] + count[e])
        # e4m3 keeps 4 significant bits: a row is its token to within 2^-4 of each value and half the least code
        token = x[src[r].long()].double()
        assert bool(((x64[r] - token).abs() <= token.abs() / 16 + scales[r].double().repeat_interleave(128, 1) / 1024).all())
        yy, by, _, _ = ref.product_rows(x64[r], w64[e], None, act, rw[r].double(), None)
        ref.check(y[r], yy, by, "y of expert %d" % e)
