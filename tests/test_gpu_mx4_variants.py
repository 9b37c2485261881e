"""Every kernel behind the products with 4-bit weights, at the sizes of
tests/mx4_cases.py, against the definitions in 64 bits.  Tolerances as derived
in tests/test_gpu_experts.py and tests/test_gpu_mx4.py."""
import pytest

import mlp_matmul_amd as uw
from tests.expert_cases import rows_of_experts
from tests.gpu_util import print_case
from tests.mx4_cases import GROUPED, LINEAR
from tests.test_gpu_experts import torch_cuda  # noqa: F401
from tests.test_gpu_experts_variants import check, products, silu

pytestmark = pytest.mark.gpu


def matrix(torch, seed, rows, cols):
    """(random Mx4Matrix, f(rows): its values there, fp64)."""
    g = torch.Generator("cuda").manual_seed(seed)
    ldc, lds = (cols // 2 + 15) // 16 * 16, (cols // 32 + 15) // 16 * 16
    codes = torch.randint(256, (rows, ldc), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((rows, lds), 255, dtype=torch.uint8, device="cuda")
    scales[:, :cols // 32] = torch.randint(117, 124, (rows, cols // 32), dtype=torch.uint8, device="cuda", generator=g)
    m = uw.Mx4Matrix(codes[:, :cols // 2], scales[:, :cols // 32])
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    table = torch.cat([grid, -grid])

    def values(at):
        c, s = m.codes[at], m.scales[at].double()
        v = table[torch.stack([c & 15, c >> 4], -1).view(c.shape[0], -1, 32).long()]
        return (v * torch.exp2(s - 127)[:, :, None]).view(c.shape[0], cols)
    return m, values


def rows_for(torch, seed, n, cols, x4):
    if x4:
        return matrix(torch, seed, n, cols)
    x = torch.randn(n, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).bfloat16()
    return x, lambda at: x[at].double()


def some(torch, lo, hi, most):
    """Rows lo .. hi - 1, or `most` of them with both ends."""
    if hi - lo <= most:
        return torch.arange(lo, hi, device="cuda")
    return torch.linspace(lo, hi - 1, most, device="cuda").round().long()


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(map(str, c)))
def test_linear(torch_cuda, case):  # noqa: F811
    torch = torch_cuda
    x4, rows, cols, batch = case
    print_case(f"mx4 linear x4={x4} {batch}x{rows}x{cols}")
    W, w = matrix(torch, rows + cols, rows, cols)
    X, x = rows_for(torch, batch, batch, cols, x4)
    g = torch.Generator("cuda").manual_seed(batch)
    bias = torch.randn(rows, device="cuda", generator=g)
    residual = torch.randn(batch, rows, device="cuda", generator=g).bfloat16()
    out = torch.full((batch + 1, rows + 3), 7.0, device="cuda")
    uw.linear(W, X, bias=bias, act="silu", residual=residual, out=out[:batch, :rows])
    assert bool((out[:, rows:] == 7).all()) and bool((out[batch:] == 7).all())
    assert bool(torch.isfinite(out).all())
    at = some(torch, 0, batch, 150)
    v, err = products(x(at), w(slice(None)))
    v = v + bias.double()
    err = err + v.abs() * 2.0 ** -23
    y, err = silu(torch, v, err)
    y = y + residual[at].double()
    check(torch, out[at, :rows], y, err + y.abs() * 2.0 ** -23, f"linear {case}")


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "-".join(map(str, c)))
def test_grouped(torch_cuda, case):  # noqa: F811
    torch = torch_cuda
    x4, pair, experts, rows, cols, n = case
    print_case(f"mx4 {'gate_up' if pair else 'grouped'} x4={x4} {experts} of {rows}x{cols}, {n} rows")
    ws = [matrix(torch, 5 * rows + i, experts * rows, cols) for i in range(2 if pair else 1)]
    X, x = rows_for(torch, n, n, cols, x4)
    counts = rows_of_experts(experts, n)
    offsets = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda")
    order = torch.randperm(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).int()
    if pair:
        out = torch.full((n + 2, rows + 3), 7.0, device="cuda", dtype=torch.bfloat16)
        uw.moe_gate_up(ws[0][0], ws[1][0], X, offsets, order, h=out[:n, :rows])
    else:
        out = torch.full((n + 2, rows + 3), 7.0, device="cuda")
        uw.gemm_grouped(ws[0][0], X, offsets, order, out=out[:n, :rows])
    assert bool((out[n:] == 7).all()) and bool((out[:, rows:] == 7).all())
    assert bool(torch.isfinite(out).all())
    at = offsets.tolist()
    for e in range(experts):
        if at[e] == at[e + 1]:
            continue
        pick = some(torch, at[e], at[e + 1], max(4, 150 // experts))
        xe, r = x(order[pick].long()), slice(e * rows, (e + 1) * rows)
        a, ea = products(xe, ws[0][1](r))
        if pair:
            u, eu = products(xe, ws[1][1](r))
            s, es = silu(torch, a, ea)
            a, ea = s * u, es * (u.abs() + eu) + s.abs() * eu + 2.0 ** -22 * (s * u).abs()
        check(torch, out[pick, :rows], a, ea, f"grouped {case} expert {e}")
