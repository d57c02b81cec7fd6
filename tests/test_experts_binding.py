"""The experts' Python calls refuse tensors that are not on the GPU before the
library sees an address (a stand-in for it notes every call)."""
import pytest
import torch

from test_experts_abi import B  # noqa: F401  (a fixture)

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


class OnGpu:
    """A host tensor that says it is on the GPU."""

    def __init__(self, t):
        self.t = t
        self.is_cuda = True

    def __getattr__(self, name):
        return getattr(self.t, name)


class Stream:
    cuda_stream = 0


def calls(B):  # noqa: F811
    rows, K, N, E, T, TK = 24, 128, 128, 3, 5, 2

    def zeros(*shape, dtype=BF):
        return torch.zeros(shape, dtype=dtype)

    blocks = dict(expert_offset=zeros(E + 1, dtype=I32), num_tokens_per_expert=zeros(E, dtype=I32))
    st = dict(d_status=zeros(1, dtype=I32))
    product = dict(x=zeros(rows, K), w=zeros(E, N, K), y=zeros(rows, N), bias=zeros(E, N, dtype=F32),
                   row_weight=zeros(rows, dtype=F32), residual=zeros(rows, N), z=zeros(rows, N), **blocks, **st)
    codes = dict(x=zeros(rows, K, dtype=torch.uint8), w=zeros(E, N, K, dtype=torch.uint8), y=zeros(rows, N),
                 x_sf=zeros(rows, 1, dtype=F32), w_sf=zeros(E, 1, 1, dtype=F32), **blocks, **st)
    backward = dict(dy=zeros(rows, N), x=zeros(rows, K), w=zeros(E, N, K), z=zeros(rows, N), dx=zeros(rows, K),
                    dw=zeros(E, N, K), dbias=zeros(E, N, dtype=F32), d_row_weight=zeros(rows, dtype=F32),
                    row_weight=zeros(rows, dtype=F32), workspace=zeros(64, dtype=torch.uint8), **blocks, **st)
    few = dict(x=zeros(T, K), topk_idx=zeros(T, TK, dtype=torch.int64), topk_weights=zeros(T, TK, dtype=F32),
               w_up=zeros(E, 2 * N, K), w_down=zeros(E, K, N), workspace=zeros(64, dtype=torch.uint8), out=zeros(T, K),
               bias_up=zeros(E, 2 * N, dtype=F32), bias_down=zeros(E, K, dtype=F32), residual=zeros(T, K), **st)
    return {"product": (B.ep_expert_gemm, product), "fp8": (B.ep_expert_gemm, codes),
            "backward": (B.ep_expert_gemm_backward, backward), "few": (B.ep_moe_few_tokens, few)}


@pytest.mark.parametrize("which", ["product", "fp8", "backward", "few"])
def test_tensors_on_the_host_are_refused(B, which, monkeypatch):  # noqa: F811
    lib = Library()
    monkeypatch.setattr(B, "_lib", lib)
    f, args = calls(B)[which]
    on_gpu = {k: OnGpu(v) for k, v in args.items()}
    f(**on_gpu, stream=Stream)
    assert len(lib.calls) == 1
    for name in args:
        with pytest.raises(AssertionError):
            f(**{**on_gpu, name: args[name]}, stream=Stream)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("which", ["product", "backward", "few"])
def test_a_status_word_of_another_type_is_refused(B, which, monkeypatch):  # noqa: F811
    lib = Library()
    monkeypatch.setattr(B, "_lib", lib)
    f, args = calls(B)[which]
    on_gpu = {k: OnGpu(v) for k, v in args.items()}
    with pytest.raises(AssertionError):
        f(**{**on_gpu, "d_status": OnGpu(torch.zeros(1, dtype=torch.uint8))}, stream=Stream)
    assert not lib.calls
