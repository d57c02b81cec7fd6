"""Gradients where only some are wanted and the inputs that the others need are
not given: the same bits as with all of them."""
import pytest
import torch

from experts_reference import ACTS
from test_gpu_experts import blocks, gen, normal, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("want,given", [
    (("dbias", "d_row_weight"), ()), (("dbias",), ()), (("d_row_weight",), ()), (("dbias", "d_row_weight"), ("x",)),
    (("dw", "dbias"), ("x",)), (("dx", "d_row_weight"), ("w",)),
])
def test_gradients_without_the_inputs_they_do_not_need(act, want, given):
    from gpu_path import B
    g = gen(len(want) + len(given))
    off, cnt, rows = blocks([33, 0, 70, 5], gap=2)
    K, N, E = 80, 136, 4
    Nw = 2 * N if act == "swiglu" else N
    dy, z = normal(g, rows, N), normal(g, rows, Nw)
    have = {"x": normal(g, rows, K), "w": normal(g, E, Nw, K)}
    ws = torch.empty(B.ep_expert_gemm_backward_workspace_bytes(rows, N, E, ACTS[act]), dtype=torch.uint8, device="cuda")

    def run(names, inputs):
        out = {"dx": torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda"), "dw": torch.zeros_like(have["w"]),
               "dbias": torch.zeros((E, Nw), device="cuda"), "d_row_weight": torch.zeros(rows, device="cuda")}
        out = {k: v for k, v in out.items() if k in names}
        st = status()
        B.ep_expert_gemm_backward(dy, inputs.get("x"), inputs.get("w"), z, off, cnt, ws, st, activation=ACTS[act], **out)
        assert int(st.item()) == 0
        return out

    whole = run(("dx", "dw", "dbias", "d_row_weight"), have)
    for name, got in run(want, {k: have[k] for k in given}).items():
        assert torch.equal(got, whole[name]) and bool((got != 0).any())
