"""The epilogue matmul and the mixture-of-experts operators have no backward
pass: tensors that require a gradient are refused while gradients are
recorded, where a detached result would train nothing without an error."""
import pytest
import torch

import mlp_matmul_amd as uw


class OnGpu:
    """As much of a GPU tensor as the checks look at."""
    device = torch.device("cuda", 0)

    def __init__(self, requires_grad=False):
        self.requires_grad = requires_grad


CALLS = {
    uw.linear: ("W", "X", "bias", "residual", "out"),
    uw.moe_route: ("logits",),
    uw.gemm_grouped: ("W", "X", "offsets", "order", "out"),
    uw.moe_gate_up: ("gate", "up", "X", "offsets", "order", "h"),
    uw.moe_combine: ("Y", "place", "weights", "residual", "out"),
    uw.moe_layer: ("gate", "up", "down", "X", "logits", "residual", "out"),
}


@pytest.mark.parametrize("call", list(CALLS), ids=lambda f: f.__name__)
def test_gradients_are_refused(call, monkeypatch):
    class Past(Exception):
        pass

    def past(*a):
        raise Past
    monkeypatch.setattr(uw, "_elsewhere", past)              # what follows the checks of the tensors
    extra = {"top_k": 2} if call in (uw.moe_route, uw.moe_layer) else {}
    for name in CALLS[call]:
        tensors = {n: OnGpu(n == name) for n in CALLS[call]}
        with pytest.raises(ValueError, match="gradient"):
            call(**tensors, **extra)
        with torch.no_grad(), pytest.raises(Past):
            call(**tensors, **extra)
        with pytest.raises(Past):
            call(**{n: OnGpu() for n in CALLS[call]}, **extra)
