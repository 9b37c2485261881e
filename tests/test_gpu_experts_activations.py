"""The activations of the epilogue matmul and the pair's SiLU over the whole
range of their arguments, relative to the result, against fp64."""
import math

import pytest

import mlp_matmul_amd as uw
from tests.gpu_util import print_case
from tests.test_gpu_experts import torch_cuda  # noqa: F401

pytestmark = pytest.mark.gpu

# The activations' own errors, relative to the result; 2^-24 is half a step.
#   SiLU: v / (1 + E), E = exp(-v) as 2^t.  t = -v log2(e) is rounded once and log2(e) itself is off by 0.225 half
#   steps: E is off by 1.225 |v| half steps of itself, by 2 more from the exponential (a unit), the sum by 1, the
#   reciprocal by 2, the product by 1.
#   tanh-GELU: v / (1 + exp(-2u)): the argument takes eight roundings (three products and a constant in the cube, the
#   sum, two constants' products, the last product), so E is off by 8 |2u| half steps, and 6 as above.
#   GELU: 1 + erff(x) is off by 6 half steps of 1 (the error function's two units, x's roundings times its slope, the
#   sum), and exactly 0 or 2 from |v| = 6 on, where the result is below 6e-9 or v.
# Results below 2^-126 |v| may be 0: exponentials are no denormal numbers.
H = 2.0 ** -24


def activation_bound(torch, v, want, act):
    small = v.abs() * 2.0 ** -125
    if act == "silu":
        return (1.225 * v.abs().clamp_max(200) + 6) * H * want.abs() + small.clamp_max(2.0 ** -100)
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        return (8 * (2 * u).abs().clamp_max(200) + 6) * H * want.abs() + small.clamp_max(2.0 ** -100)
    if act == "gelu":
        return 3 * v.abs().clamp_max(6) * H + 3 * H * want.abs()
    return torch.zeros_like(v)


def activation(torch, v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v.clamp_min(0) if act == "relu" else v


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_activation_tails(torch_cuda, act):  # noqa: F811
    """Exact arguments (through the identity) over the whole range, the far tails among them."""
    torch = torch_cuda
    cols = 1024
    x = torch.linspace(-110, 12, cols, dtype=torch.float64).bfloat16()
    x[::3] = torch.linspace(-14, 14, x[::3].numel(), dtype=torch.float64).bfloat16()
    for i, e in enumerate(range(-120, 127, 4)):
        x[5 * i], x[5 * i + 1] = 2.0 ** e, -2.0 ** e
    v = x.double().cuda()
    want = activation(torch, v, act)
    bound = activation_bound(torch, v, want, act)
    W = torch.eye(cols, dtype=torch.bfloat16, device="cuda")
    for batch in (1, 3, 40, 300):
        print_case(f"{act} tails, batch {batch}")
        out = uw.linear(W, x.cuda()[None].repeat(batch, 1), act=act)
        assert bool(out.isfinite().all())
        worst = ((out.double() - want).abs() / (bound + (want.abs() + bound) * H + 2.0 ** -148)).max(0)[0]
        assert float(worst.max()) <= 1, (float(worst.max()), float(v[worst.argmax()]))
    if act == "silu":
        off = torch.tensor([0, 40], dtype=torch.int32).cuda()
        for n in (1, 3, 40):                                 # the pair's: its argument times its SiLU
            out = uw.moe_gate_up(W[None], W[None], x.cuda()[None].repeat(40, 1)[:n], off.clamp_max(n))
            y = want * v
            keep = y.abs() < 2.0 ** 126
            limit = bound * v.abs() + y.abs() * 2.0 ** -23
            limit = limit + (y.abs() + limit) * 2.0 ** -8 + 2.0 ** -130
            worst = ((out.double() - y).abs() / limit)[:, keep].max()
            assert float(worst) <= 1, float(worst)
