"""Every kernel behind the epilogue matmul and the products grouped by expert,
at the sizes of tests/expert_cases.py, against the definitions in 64 bits.
Tolerances as derived in tests/test_gpu_experts.py."""
import pytest

import mlp_matmul_amd as uw
from tests.expert_cases import GROUPED, LINEAR, rows_of_experts
from tests.gpu_util import print_case
from tests.test_gpu_experts import torch_cuda  # noqa: F401

pytestmark = pytest.mark.gpu


def matrix(torch, seed, pal, experts, rows, cols):
    """(what a call takes, its exact values bf16 [experts, rows, cols]); palette: random planes, one group in
    twenty verbatim."""
    g = torch.Generator("cuda").manual_seed(seed)
    if not pal:
        w = (torch.randn(experts, rows, cols, device="cuda", generator=g) * 0.02).bfloat16()
        return w, w

    def random(lo, hi, n):
        return torch.randint(lo, hi, (n,), device="cuda", generator=g, dtype=torch.uint8)
    n = experts * rows * cols
    groups, tiles = n // 64, -(-n // 4096)
    verbatim = torch.rand(groups, device="cuda", generator=g) < 0.05
    verbatim[-1] = True
    sm, index = random(0, 256, n), random(0, 16, n).view(groups, 64)
    index[verbatim] = 0
    count = int(verbatim.sum())
    vexp = random(100, 124, count * 64)
    flags = torch.zeros(tiles * 64, dtype=torch.int64, device="cuda")
    flags[:groups] = verbatim
    flags = flags.view(tiles, 64)
    base = torch.zeros(tiles + 1, dtype=torch.int32, device="cuda")
    base[1:] = flags.sum(1).cumsum(0)
    nib = index.view(-1, 2)
    W = uw.DeviceMatrix.from_sections(experts * rows, cols, range(106, 122), count, {
        "sm": sm, "nib": nib[:, 0] | (nib[:, 1] << 4), "vexp": vexp,
        "bitmap": (flags << torch.arange(64, device="cuda")).sum(1).view(torch.uint8), "tile_vbase": base.view(torch.uint8)})
    e = index + 106
    e[verbatim] = vexp.view(-1, 64)
    bits = ((sm.short() & 0x80) << 8) | (e.view(-1).short() << 7) | (sm.short() & 0x7F)
    return W, bits.view(torch.bfloat16).view(experts, rows, cols)


def products(x, w):
    """x . w^T in fp64 and the bound on an fp32 sum's error."""
    x, w = x.double(), w.double()
    return x @ w.t(), (x.shape[1] + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t())


def silu(torch, v, err):
    y = v * torch.sigmoid(v)
    return y, 1.13 * err + 2.0 ** -20 * (v.abs() + y.abs())


def check(torch, got, want, bound, what):
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    limit = bound + (want.abs() + bound) * (torch.finfo(got.dtype).eps / 2) + 1e-30
    worst = float(((got.double() - want).abs() / limit).max())
    assert worst <= 1, f"{what}: {worst:.2f} of the limit"


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(map(str, c)))
def test_linear(torch_cuda, case):  # noqa: F811
    torch = torch_cuda
    pal, rows, cols, batch, scratch = case
    print_case(f"linear palette={pal} {batch}x{rows}x{cols} scratch={scratch}")
    W, w = matrix(torch, rows + cols, pal, 1, rows, cols)
    g = torch.Generator("cuda").manual_seed(batch)
    X = torch.randn(batch, cols, device="cuda", generator=g).bfloat16()
    bias = torch.randn(rows, device="cuda", generator=g)
    residual = torch.randn(batch, rows, device="cuda", generator=g).bfloat16()
    out = torch.full((batch, rows + 3), 7.0, device="cuda")
    uw.linear(W if pal else W[0], X, bias=bias, act="silu", residual=residual, out=out[:, :rows],
              scratch=None if scratch else torch.empty(0, device="cuda"))
    v, err = products(X, w[0])
    v += bias.double()
    y, err = silu(torch, v, err + v.abs() * 2.0 ** -23)
    y += residual.double()
    check(torch, out[:, :rows], y, err + y.abs() * 2.0 ** -23, "linear")
    assert bool((out[:, rows:] == 7).all())


@pytest.mark.parametrize("case", GROUPED, ids=lambda c: "-".join(map(str, c)))
def test_grouped(torch_cuda, case):  # noqa: F811
    torch = torch_cuda
    pal, pair, experts, rows, cols, n, scratch = case
    print_case(f"grouped palette={pal} pair={pair} {n} rows of {experts} x {rows} x {cols} scratch={scratch}")
    W, w = matrix(torch, rows + cols, pal, experts, rows, cols)
    counts = rows_of_experts(experts, n)
    off = torch.tensor([0] + counts).cumsum(0).int().cuda()
    X = torch.randn(n, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(n)).bfloat16()
    s = None if scratch else torch.empty(0, device="cuda")
    if pair:
        U, u = matrix(torch, rows + cols + 1, pal, experts, rows, cols)
        out = torch.full((n, rows + 3), 7.0, device="cuda", dtype=torch.bfloat16)
        uw.moe_gate_up(W, U, X, off, h=out[:, :rows], scratch=s)
    else:
        out = torch.full((n, rows + 3), 7.0, device="cuda")
        uw.gemm_grouped(W, X, off, out=out[:, :rows], scratch=s)
    at = 0
    for e, k in enumerate(counts):
        if k == 0:
            continue
        x, got = X[at:at + k], out[at:at + k, :rows]
        v, err = products(x, w[e])
        if pair:
            q, err_q = products(x, u[e])
            y, err_y = silu(torch, v, err)
            v, err = y * q, err_y * (q.abs() + err_q) + y.abs() * err_q + (y * q).abs() * 2.0 ** -23
        check(torch, got, v, err, f"expert {e}")
        at += k
    assert bool((out[:, rows:] == 7).all())
