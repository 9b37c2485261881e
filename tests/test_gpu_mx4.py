"""GPU tests of the microscaled 4-bit operators against plain definitions in
64 bits.

Tolerances.  Codes and scales are whole numbers: equal.  A weight has two
significant bits, so its products with bf16 and 4-bit numbers are exact in
fp32; a sum of K of them in any order, each addition off by at most 2^-23 of the
sum of absolute values S, is within (K + 8) 2^-23 S.  Activations, residuals and
the rounding of the result as in tests/test_gpu_experts.py.
"""
import pytest

import mlp_matmul_amd as uw
from tests.expert_cases import rows_of_experts
from tests.gpu_util import print_case
from tests.mx4_util import quantize_ref, values_ref
from tests.test_gpu_experts import activate, check, f64, sum_bound, torch_cuda  # noqa: F401

pytestmark = pytest.mark.gpu


def normal(torch, seed, *shape, dtype=None, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype or torch.bfloat16).cuda()


def weight(torch, seed, rows, cols, pad=0):
    """(Mx4Matrix, its values fp64): random codes, scales over a few powers of two, rows `pad` units of 16 bytes further
    apart, with bytes between them that are no numbers."""
    g = torch.Generator().manual_seed(seed)
    ldc, lds = (cols // 2 + 15) // 16 * 16 + 16 * pad, (cols // 32 + 15) // 16 * 16 + 16 * pad
    codes = torch.randint(256, (rows, ldc), dtype=torch.uint8, generator=g)
    scales = torch.full((rows, lds), 255, dtype=torch.uint8)
    scales[:, :cols // 32] = torch.randint(117, 124, (rows, cols // 32), dtype=torch.uint8, generator=g)
    m = uw.Mx4Matrix(codes.cuda()[:, :cols // 2], scales.cuda()[:, :cols // 32])
    return m, values_ref(m.codes, m.scales)


def rows_for(torch, seed, n, cols, x4, pad=0):
    """(X as a call takes it, its values fp64)."""
    if x4:
        return weight(torch, seed, n, cols, pad // 8)
    x = normal(torch, seed, n, cols + pad)[:, :cols]
    return x, f64(x)


# ------------------------------------------------------------ the format
@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (7, 96), (5, 4096), (129, 1056), (1000, 512), (33, 14336)])
def test_quantize(torch_cuda, rows, cols, kind):
    torch = torch_cuda
    print_case(f"quantize {rows}x{cols} {kind}")
    for pad in (0, 8):
        x = normal(torch, rows + cols, rows, cols + pad, dtype=getattr(torch, kind))[:, :cols]
        x[:, ::5] *= 1e-3
        m = uw.mx4_quantize(x)
        codes, scales = quantize_ref(x)
        assert torch.equal(m.scales.cpu(), scales) and torch.equal(m.codes.cpu(), codes)
        want = values_ref(codes, scales)
        for t in (torch.float32, torch.bfloat16):
            room = torch.full((rows, cols + 3), 7.0, dtype=t, device="cuda")
            uw.mx4_dequantize(m, out=room[:, :cols])
            assert torch.equal(f64(room[:, :cols]), want) and bool((room[:, cols:] == 7).all())
        assert torch.equal(f64(uw.mx4_dequantize(m)), want)


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_quantize_ties_and_ends(torch_cuda, kind):
    """Every tie of the rounding at scales from the smallest to the largest, zeros of both signs, subnormals, and
    blocks that hold a NaN or an infinity."""
    torch = torch_cuda
    t = getattr(torch, kind)
    print_case(f"quantize ties {kind}")
    v = torch.tensor([4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.9, 0, 0.5, 1, 3, 0.1], dtype=torch.float64)
    blocks = [torch.ldexp(torch.cat([v, -v]), torch.tensor(e)) for e in list(range(-133, 126, 7)) + [-127, -126, 125]]
    blocks += [torch.zeros(32, dtype=torch.float64), -torch.zeros(32, dtype=torch.float64)]
    for i, bad in enumerate((float("nan"), float("inf"), -float("inf"))):
        b = blocks[3 + i].clone()
        b[11 * i] = bad
        blocks.append(b)
    x = torch.stack(blocks).to(t).cuda()
    m = uw.mx4_quantize(x)
    codes, scales = quantize_ref(x)
    assert torch.equal(m.scales.cpu(), scales)
    assert torch.equal(m.codes.cpu(), codes)
    got, want = f64(uw.mx4_dequantize(m)), values_ref(codes, scales)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(), want.nan_to_num())
    assert int(torch.isnan(want).sum()) == 3 * 32


def test_quantize_into(torch_cuda):
    """Into tensors of the caller's, rows further apart: the bytes between them stay."""
    torch = torch_cuda
    print_case("quantize into out")
    x = normal(torch, 4, 37, 160)
    codes = torch.full((37, 96), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((37, 32), 0xCD, dtype=torch.uint8, device="cuda")
    m = uw.Mx4Matrix(codes[:, :80], scales[:, :5])
    assert uw.mx4_quantize(x, out=m) is m
    want = quantize_ref(x)
    assert torch.equal(codes[:, :80].cpu(), want[0]) and torch.equal(scales[:, :5].cpu(), want[1])
    assert bool((codes[:, 80:] == 0xAB).all()) and bool((scales[:, 5:] == 0xCD).all())


# ------------------------------------------------------------ linear
def linear_case(torch, rows, cols, batch, x4, act="none", bias=None, residual=None, out_dtype=None, pad=0, seed=0):
    what = f"mx4 linear {batch}x{rows}x{cols} x4={x4} {act} bias={bias} residual={residual} out={out_dtype} pad={pad}"
    print_case(what)
    W, w = weight(torch, seed + rows + cols, rows, cols, pad // 8)
    X, x = rows_for(torch, seed + batch, batch, cols, x4, pad)
    g = torch.Generator().manual_seed(seed + 5)
    b = None if bias is None else torch.randn(rows, generator=g).to(bias).cuda()
    r = None if residual is None else torch.randn(batch, rows + pad, generator=g).to(residual).cuda()[:, :rows]
    room = torch.full((batch, rows + pad + 1), 7.0, dtype=out_dtype or torch.float32, device="cuda")
    out = uw.linear(W, X, bias=b, act=act, residual=r, out=room[:, :rows])
    assert bool((room[:, rows:] == 7).all()), what
    v, err = x @ w.t(), sum_bound(torch, x, w)
    if b is not None:
        v = v + f64(b)
        err = err + v.abs() * 2.0 ** -23
    y = activate(torch, v, act)
    if act != "none":
        err = 1.13 * err + 2.0 ** -20 * (v.abs() + y.abs())
    if r is not None:
        y = y + f64(r)
        err = err + y.abs() * 2.0 ** -23
    check(torch, out, y, err, what)


@pytest.mark.parametrize("x4", [False, True])
@pytest.mark.parametrize("batch", [1, 2, 3, 4, 5, 16, 17, 32, 33, 64, 65, 130, 257, 400])
def test_linear_batches(torch_cuda, batch, x4):
    torch = torch_cuda
    linear_case(torch, 300, 1088, batch, x4, seed=batch)
    linear_case(torch, 129, 4096, batch, x4, "silu", torch.float32, torch.bfloat16, torch.bfloat16, seed=batch)


@pytest.mark.parametrize("x4", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 32), (15, 64), (16, 96), (17, 128), (63, 160), (64, 224), (65, 4096),
                                       (1000, 14336), (4099, 128), (257, 2080), (130, 544)])
def test_linear_shapes(torch_cuda, rows, cols, x4):
    torch = torch_cuda
    for batch in (1, 7, 40, 70, 300):
        linear_case(torch, rows, cols, batch, x4, "none", torch.bfloat16, torch.float32, torch.float32)


@pytest.mark.parametrize("x4", [False, True])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_linear_epilogues(torch_cuda, act, x4):
    torch = torch_cuda
    f, h = torch.float32, torch.bfloat16
    for bias, residual, out in ((None, None, h), (f, None, f), (h, f, h), (f, h, h), (None, h, f), (h, None, f)):
        for batch in (1, 9, 70, 140, 300):
            linear_case(torch, 132, 256, batch, x4, act, bias, residual, out, pad=8)


@pytest.mark.parametrize("x4", [False, True])
def test_linear_every_weight(torch_cuda, x4):
    """One-hot rows give the weights themselves: every code at every place of a block, and scales of both ends."""
    torch = torch_cuda
    rows, cols = 80, 352
    W, _ = weight(torch, 9, rows, cols)
    W.scales[:, 3] = 0
    W.scales[:, 5] = 250
    W.scales[7, 2] = 255                                      # no numbers in one block of one row
    w = values_ref(W.codes, W.scales)
    for batch in (1, 3, 16, 40, 352):
        print_case(f"mx4 one-hot {batch} x4={x4}")
        at = torch.arange(batch) * 37 % cols
        X = torch.zeros(batch, cols, dtype=torch.bfloat16)
        X[torch.arange(batch), at] = 1.0
        X = X.cuda()
        got = f64(uw.linear(W, uw.mx4_quantize(X) if x4 else X))
        bad = torch.isnan(w).any(1)
        assert torch.isnan(got[:, bad]).all() and bool(torch.isfinite(got[:, ~bad]).all())
        # products below 2^-126 may be flushed by the matrix units
        assert bool(((got - w[:, at].t()).abs()[:, ~bad] <= 2.0 ** -125).all())


@pytest.mark.parametrize("x4", [False, True])
def test_linear_smallest_weights(torch_cuda, x4):
    """One-hot rows on scale bytes 0 to 3: weights of 2^-126 and above come back as they are; those below, which fp32 holds
    as subnormal numbers, as they are or as zero."""
    torch = torch_cuda
    rows, cols = 80, 352
    W, _ = weight(torch, 12, rows, cols)
    W.scales[:] = torch.arange(11, dtype=torch.uint8, device="cuda") % 4
    w = values_ref(W.codes, W.scales)
    for batch in (1, 3, 16, 40, 352):
        print_case(f"mx4 one-hot, smallest scales, {batch} x4={x4}")
        at = torch.arange(batch) * 37 % cols
        X = torch.zeros(batch, cols, dtype=torch.bfloat16)
        X[torch.arange(batch), at] = 1.0
        X = X.cuda()
        got, want = f64(uw.linear(W, uw.mx4_quantize(X) if x4 else X)), w[:, at].t()
        small = want.abs() < 2.0 ** -126
        assert 0 < int(small.sum()) < small.numel()
        assert bool(((got == want) | (small & (got == 0))).all())


def test_linear_numbers_that_are_none(torch_cuda):
    """A NaN or an infinity of a row of X stays in that row."""
    torch = torch_cuda
    W, w = weight(torch, 21, 70, 288)
    for batch in (1, 5, 20, 70, 300):
        for v in (float("nan"), float("inf")):
            print_case(f"mx4 linear {batch} rows with {v}")
            X = normal(torch, batch, batch, 288)
            X[batch // 2, 287] = v
            for x in (X, uw.mx4_quantize(X)):
                out = uw.linear(W, x)
                rest = torch.arange(batch) != batch // 2
                assert not bool(torch.isfinite(out[batch // 2]).all())
                assert bool(torch.isfinite(out[rest.cuda()]).all())


# ------------------------------------------------------------ grouped by expert
def grouped_case(torch, experts, rows, cols, counts, x4, pair, ordered, seed=0, pad=0):
    n = sum(counts)
    what = f"mx4 {'gate_up' if pair else 'grouped'} {experts} of {rows}x{cols} rows {counts} x4={x4} ordered={ordered}"
    print_case(what)
    ws = [weight(torch, seed + i, experts * rows, cols, pad // 8) for i in range(2 if pair else 1)]
    extra, top_k = 3, 3 if ordered else 1
    g = torch.Generator().manual_seed(seed + 7)
    offsets = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)
    slots = n + extra
    order = torch.randperm(slots, generator=g).to(torch.int32) if ordered else None
    X, x = rows_for(torch, seed + 3, -(-slots // top_k), cols, x4, pad)
    at = order.long() // top_k if ordered else torch.arange(slots)
    o = None if order is None else order.cuda()
    if pair:
        out = torch.full((slots, rows + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        uw.moe_gate_up(ws[0][0], ws[1][0], X, offsets.cuda(), o, top_k, h=out[:, :rows])
    else:
        out = torch.full((slots, rows + pad), 7.0, device="cuda")
        uw.gemm_grouped(ws[0][0], X, offsets.cuda(), o, top_k, out=out[:, :rows])
    assert bool((out[n:] == 7).all()) and bool((out[:, rows:] == 7).all()), f"{what}: written outside"
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        xe = x[at[lo:hi]]
        w = [v[1].view(experts, rows, cols)[e] for v in ws]
        if pair:
            a, u = xe @ w[0].t(), xe @ w[1].t()
            ea, eu = sum_bound(torch, xe, w[0]), sum_bound(torch, xe, w[1])
            s = activate(torch, a, "silu")
            es = 1.13 * ea + 2.0 ** -20 * (a.abs() + s.abs())
            want, err = s * u, es * (u.abs() + eu) + s.abs() * eu + 2.0 ** -22 * (s * u).abs()
        else:
            want, err = xe @ w[0].t(), sum_bound(torch, xe, w[0])
        check(torch, out[lo:hi, :rows], want, err, f"{what} expert {e}")


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("x4", [False, True])
@pytest.mark.parametrize("experts,rows,cols,n", [(1, 33, 64, 2), (4, 64, 256, 4), (5, 48, 96, 40), (8, 200, 544, 333),
                                                 (3, 300, 160, 700), (70, 40, 128, 150), (130, 16, 32, 260),
                                                 (16, 64, 2080, 9), (2, 520, 1056, 900)])
def test_grouped(torch_cuda, experts, rows, cols, n, x4, pair):
    torch = torch_cuda
    for ordered in (False, True):
        grouped_case(torch, experts, rows, cols, rows_of_experts(experts, n), x4, pair, ordered, seed=n,
                     pad=16 if ordered else 0)


@pytest.mark.parametrize("x4", [False, True])
def test_grouped_offsets_out_of_range(torch_cuda, x4):
    """Offsets that descend or pass the rows, and an order outside X: nothing outside is read or written, experts whose
    offsets are sound are computed."""
    torch = torch_cuda
    print_case(f"mx4 grouped bad offsets x4={x4}")
    W, w = weight(torch, 3, 4 * 40, 96)
    X, x = rows_for(torch, 4, 50, 96, x4)
    out = torch.full((50, 40), 7.0, device="cuda")
    uw.gemm_grouped(W, X, torch.tensor([0, 10, 5, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda"),
                    torch.tensor([2 ** 30, -5] + list(range(48)), dtype=torch.int32, device="cuda"), out=out)
    at = torch.tensor([0, 0] + list(range(48)))
    xe, we = x[at[:5]], w.view(4, 40, 96)[0]
    check(torch, out[:5], xe @ we.t(), sum_bound(torch, xe, we), "expert 0")
    xe, we = x[at[10:]], w.view(4, 40, 96)[3]
    check(torch, out[10:], xe @ we.t(), sum_bound(torch, xe, we), "expert 3")
