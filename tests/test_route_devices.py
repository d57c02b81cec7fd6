"""The router's and the 4-bit experts' Python calls refuse a tensor of another
device than the current one before the library sees an address (a stand-in
for it notes every call; no kernel runs)."""
import pytest
import torch

from test_experts_abi import B  # noqa: F401  (a fixture)
from test_experts_binding import Library, OnGpu, Stream
from test_route_abi import calls


class On(OnGpu):
    """A host tensor that says it is on a GPU of this number."""

    def __init__(self, t, device):
        super().__init__(t)
        self.device = device

    def get_device(self):
        return self.device


class Pinned(OnGpu):
    """A host tensor that says it is pinned."""

    def __init__(self, t):
        super().__init__(t)
        self.is_cuda = False

    def is_pinned(self):
        return True


@pytest.mark.parametrize("which", ["route", "balance", "backward", "product", "few"])
def test_a_tensor_of_another_device_is_refused(B, which, monkeypatch):  # noqa: F811
    lib = Library()
    monkeypatch.setattr(B, "_lib", lib)
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    f, args = calls(B)[which]
    there = {k: On(v, 1) for k, v in args.items()}
    f(**there, stream=Stream)
    assert len(lib.calls) == 1
    for name in args:
        for device in (0, 2):
            with pytest.raises(AssertionError):
                f(**{**there, name: On(args[name], device)}, stream=Stream)
        with pytest.raises(AssertionError):      # all of them on one, but not the current one
            f(**{k: On(v, 0) for k, v in args.items()}, stream=Stream)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("which", ["route", "balance", "backward", "product", "few"])
def test_pinned_tensors_pass_and_hide_no_other_device(B, which, monkeypatch):  # noqa: F811
    lib = Library()
    monkeypatch.setattr(B, "_lib", lib)
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    f, args = calls(B)[which]
    for name in args:
        f(**{**{k: On(v, 1) for k, v in args.items()}, name: Pinned(args[name])}, stream=Stream)
    assert len(lib.calls) == len(args)
    # every tensor but one pinned, that one elsewhere
    for name in args:
        with pytest.raises(AssertionError):
            f(**{**{k: Pinned(v) for k, v in args.items()}, name: On(args[name], 0)}, stream=Stream)
    assert len(lib.calls) == len(args)
