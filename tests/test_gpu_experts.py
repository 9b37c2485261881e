"""GPU tests of the epilogue matmul and the mixture-of-experts operators
against plain definitions in 64 bits, and of a run of them together.

Tolerances.  Products of two bf16 numbers are exact in fp32; a sum of K of
them in any order, each addition off by at most 2^-23 of the sum of absolute
values S, is within (K + 8) 2^-23 S.  An activation's slope is at most 1.13;
its own evaluation (an exponential or erff, and a division, a few fp32 steps each)
adds at most 2^-20 |v| + 2^-20 |act(v)|.  A residual's addition is one fp32 rounding.
The final rounding to a type t is half a step, finfo(t).eps / 2 of the value.
"""
import math

import numpy as np
import pytest

import mlp_matmul_amd as uw
import workloads
from tests.gpu_util import print_case, to_dev_bf16

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    uw.lib()
    return torch


def f64(t):
    return t.detach().double().cpu()


def make_weight(torch, seed, experts, rows, cols, pal, p_out=0.004):
    """(what the call takes, the exact values [experts, rows, cols] in fp64)."""
    w = workloads.gaussian_weights(np.random.default_rng(seed), experts * rows, cols, 0.02, p_out, 1.0)
    exact = f64(torch.from_numpy(w.view(np.int16)).view(torch.bfloat16)).view(experts, rows, cols)
    if pal:
        return uw.compress(w).to_device(uw.DIRECT_SECTIONS), exact
    return to_dev_bf16(w).view(experts, rows, cols), exact


def rows_of(torch, seed, n, cols, pad=0):
    """bf16 [n, cols] with a row stride of cols + pad."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, cols + pad, generator=g).to(torch.bfloat16).cuda()[:, :cols]


def activate(torch, v, act):
    if act == "relu":
        return v.clamp_min(0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def sum_bound(torch, x, w):
    """Bound on the fp32 sum's error, [rows of x, rows of w]."""
    return (x.shape[1] + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t())


def check(torch, got, want, bound, what):
    g, half = f64(got), torch.finfo(got.dtype).eps / 2
    assert g.shape == want.shape, (what, g.shape, want.shape)
    limit = bound + (want.abs() + bound) * half + 1e-30
    off = (g - want).abs() > limit
    assert bool(torch.isfinite(g).all()), f"{what}: not finite"
    assert not bool(off.any()), (f"{what}: {int(off.sum())} of {off.numel()} off; worst "
                                 f"{float(((g - want).abs() / limit).max()):.2f} of the limit")


def linear_case(torch, rows, cols, batch, pal, act="none", bias=None, residual=None, out_dtype=None, pad=0, seed=0):
    what = f"linear {batch}x{rows}x{cols} pal={pal} {act} bias={bias} residual={residual} out={out_dtype} pad={pad}"
    print_case(what)
    W, w = make_weight(torch, seed + rows + cols, 1, rows, cols, pal)
    X = rows_of(torch, seed + batch, batch, cols, pad)
    g = torch.Generator().manual_seed(seed + 5)
    b = None if bias is None else torch.randn(rows, generator=g).to(bias).cuda()
    r = None if residual is None else torch.randn(batch, rows + pad, generator=g).to(residual).cuda()[:, :rows]
    out = uw.linear(W if pal else W[0], X, bias=b, act=act, residual=r, out_dtype=out_dtype)
    x = f64(X)
    v, err = x @ w[0].t(), sum_bound(torch, x, w[0])
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
    return W, X, out


@pytest.mark.parametrize("pal", [False, True])
@pytest.mark.parametrize("batch", [1, 2, 3, 5, 16, 17, 33, 64, 65, 130, 257])
def test_linear_batches(torch_cuda, batch, pal):
    torch = torch_cuda
    linear_case(torch, 300, 1088, batch, pal, seed=batch)
    linear_case(torch, 129, 4096, batch, pal, "silu", torch.float32, torch.bfloat16, torch.bfloat16, seed=batch)


@pytest.mark.parametrize("pal", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 64), (15, 128), (16, 192), (17, 64), (63, 320), (64, 64), (65, 4096),
                                       (1000, 14336), (4099, 128)])
def test_linear_shapes(torch_cuda, rows, cols, pal):
    torch = torch_cuda
    for batch in (1, 7, 40, 70):
        linear_case(torch, rows, cols, batch, pal, "none", torch.bfloat16, torch.float32, torch.float32)


@pytest.mark.parametrize("act", ACTS)
def test_linear_epilogues(torch_cuda, act):
    """Every activation with each type of bias, residual and output, strided."""
    torch = torch_cuda
    f, h = torch.float32, torch.bfloat16
    for bias, residual, out in ((None, None, h), (f, None, f), (h, f, h), (f, h, h), (None, h, f), (h, None, f)):
        for pal, batch in ((False, 1), (True, 1), (True, 9), (False, 70), (True, 140)):
            linear_case(torch, 132, 256, batch, pal, act, bias, residual, out, pad=8)


def test_linear_weights_exact(torch_cuda):
    """One-hot inputs give the weights themselves, verbatim groups among them, in both forms."""
    torch = torch_cuda
    rows, cols = 200, 576
    for batch in (1, 12, 40, 96):
        print_case(f"linear one-hot batch {batch}")
        at = torch.arange(batch) * 37 % cols
        X = torch.zeros(batch, cols, dtype=torch.bfloat16)
        X[torch.arange(batch), at] = 1.0
        for pal in (False, True):
            W, w = make_weight(torch, 3, 1, rows, cols, pal, 0.02)
            out = uw.linear(W if pal else W[0], X.cuda())
            assert torch.equal(f64(out), w[0][:, at].t())


def test_linear_in_place_residual_and_gaps(torch_cuda):
    """out may be the residual; what lies between the rows of out stays."""
    torch = torch_cuda
    for batch, rows in ((1, 100), (5, 130), (40, 131), (100, 64)):
        print_case(f"linear in place {batch}x{rows}")
        W, w = make_weight(torch, 1, 1, rows, 256, True)
        X = rows_of(torch, 2, batch, 256)
        base = torch.randn(batch, rows + 12, dtype=torch.float32).cuda()
        keep = base.clone()
        separate = uw.linear(W, X, residual=keep[:, :rows])
        got = uw.linear(W, X, residual=base[:, :rows], out=base[:, :rows])
        assert got.data_ptr() == base.data_ptr()
        assert torch.equal(base[:, :rows], separate) and torch.equal(base[:, rows:], keep[:, rows:])


@pytest.mark.parametrize("act", ACTS)
def test_linear_activation_extremes(torch_cuda, act):
    """The activations from the smallest to the largest numbers, through the identity: every product but one is 0."""
    torch = torch_cuda
    x = torch.zeros(128, dtype=torch.bfloat16)
    big = torch.tensor([2.0 ** e for e in (-100, -20, -3, 0, 2, 4, 5, 6, 6.5, 7, 8, 13, 40, 60, 100, 127)]).bfloat16()
    x[:16], x[16:32] = big, -big
    x[32:] = torch.linspace(-12, 12, 96).bfloat16()
    W = torch.eye(128, dtype=torch.bfloat16).cuda()
    want = activate(torch, f64(x), act)
    for batch in (1, 3, 40, 300):
        print_case(f"{act} extremes, batch {batch}")
        out = uw.linear(W, x[None].repeat(batch, 1).cuda(), act=act)
        check(torch, out, want[None].expand(batch, -1), (2.0 ** -20 * (f64(x).abs() + want.abs()))[None].expand(batch, -1),
              "extremes")


def test_linear_infinities(torch_cuda):
    """Infinite and NaN inputs reach exactly the outputs of their own row."""
    torch = torch_cuda
    for batch in (1, 6, 40, 100):
        for pal in (False, True):
            print_case(f"linear nan rows batch {batch} pal {pal}")
            W, _ = make_weight(torch, 1, 1, 70, 192, pal)
            X = rows_of(torch, 3, batch, 192)
            clean = uw.linear(W if pal else W[0], X, act="relu")
            X[0, 5] = math.nan
            X[batch - 1, 190] = math.inf if batch > 1 else math.nan
            out = uw.linear(W if pal else W[0], X, act="relu")
            assert bool(out[0].isnan().all())
            assert torch.equal(out[1:-1], clean[1:-1])
            assert not bool(out[-1].isfinite().logical_and(out[-1] != 0).any())


def scratches(torch, need):
    """None (the call takes its own), none at all, too little and exactly enough, full of NaN."""
    return [None] + [torch.full((k,), 255, dtype=torch.uint8).cuda() for k in sorted({0, max(need - 16, 0), need})]


@pytest.mark.parametrize("pal", [False, True])
@pytest.mark.parametrize("rows,cols,batch", [(130, 4096, 40), (4099, 1024, 100), (1000, 14336, 130), (260, 128, 70),
                                             (300, 2048, 600), (516, 4096, 1300), (4096, 576, 2050)])
def test_linear_scratch(torch_cuda, rows, cols, batch, pal):
    """Slices of K, tails and expanded weights: any scratch gives the result; rows are checked at both ends."""
    torch = torch_cuda
    W, w = make_weight(torch, rows, 1, rows, cols, pal)
    need = uw.lib().uw_linear_scratch_bytes(int(pal), rows, cols, batch)
    g = torch.Generator().manual_seed(batch)
    bias = torch.randn(rows, generator=g).cuda()
    at = torch.arange(batch) if batch <= 200 else torch.cat([torch.arange(70), torch.arange(batch - 70, batch)])
    for pad in (0, 8):
        X = rows_of(torch, batch, batch, cols, pad)
        res = torch.randn(batch, rows + pad, generator=g).bfloat16().cuda()[:, :rows]
        x = f64(X)[at]
        v, err = x @ w[0].t() + f64(bias), sum_bound(torch, x, w[0])
        y = activate(torch, v, "gelu")
        want = y + f64(res)[at]
        err = 1.13 * (err + v.abs() * 2.0 ** -23) + 2.0 ** -20 * (v.abs() + y.abs()) + want.abs() * 2.0 ** -23
        for s in scratches(torch, need):
            what = f"linear scratch {batch}x{rows}x{cols} pal={pal} pad={pad} {None if s is None else s.numel()} of {need}"
            print_case(what)
            out = torch.full((batch, rows + 4), 7.0).cuda()
            uw.linear(W if pal else W[0], X, bias=bias, act="gelu", residual=res, out=out[:, :rows], scratch=s)
            check(torch, out[at.cuda(), :rows], want, err, what)
            assert bool(out.isfinite().all()) and bool((out[:, rows:] == 7).all())


# ------------------------------------------------------------------- routing
def plain_route(logits, top_k, renorm):
    l = logits.astype(np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, np.finfo(np.float32).max)
    t, e = l.shape
    ids = np.argsort(-l, axis=1, kind="stable")[:, :top_k]
    v = np.take_along_axis(l, ids, 1)
    dead = np.isneginf(v)
    top = np.where(dead[:, :1], 0.0, v[:, :1])
    p = np.exp(v - top)
    s = p.sum(1, keepdims=True) if renorm else np.exp(l - top).sum(1, keepdims=True)
    w = np.where(dead, 0.0, p / np.where(s > 0, s, 1))
    ids = np.where(dead, -1, ids)
    flat = ids.reshape(-1)
    key = np.where(flat < 0, e, flat)
    order = np.argsort(key, kind="stable")
    place = np.empty(t * top_k, dtype=np.int64)
    place[order] = np.arange(t * top_k)
    place[flat < 0] = -1
    offsets = np.searchsorted(np.sort(key), np.arange(e + 1))
    order = np.where(key[order] == e, -1, order)
    return ids, w, offsets, order, place.reshape(t, top_k)


def check_route(torch, logits, top_k, renorm, what):
    print_case(what)
    got = uw.moe_route(logits, top_k, renormalize=renorm)
    want = plain_route(logits.float().cpu().numpy(), top_k, renorm)
    for name, g, w in zip(("ids", "offsets", "order", "place"), (got.ids, got.offsets, got.order, got.place),
                          (want[0], want[2], want[3], want[4])):
        assert np.array_equal(g.cpu().numpy(), w), f"{what}: {name}"
    # expf, the sum of up to 512 terms and the division
    err = np.abs(got.weights.cpu().numpy() - want[1])
    assert (err <= 520 * 2.0 ** -23 * np.abs(want[1]) + 1e-37).all(), f"{what}: weights"
    return got


@pytest.mark.parametrize("tokens", [0, 1, 3, 63, 64, 65, 200, 1000, 4100, 9001, 16390])
def test_route(torch_cuda, tokens):
    torch = torch_cuda
    g = torch.Generator().manual_seed(tokens)
    for experts, top_k in ((1, 1), (5, 5), (8, 2), (16, 4), (17, 3), (64, 6), (100, 1), (128, 8), (256, 8), (512, 16),
                           (300, 16)):
        l = torch.randn(tokens, experts, generator=g)
        check_route(torch, l.cuda(), top_k, True, f"route {tokens} of {experts} top {top_k}")
        check_route(torch, l.bfloat16().cuda(), top_k, False, f"route bf16 {tokens} of {experts} top {top_k}")


def test_route_many_tokens(torch_cuda):
    """More tokens than fit 256 blocks whose counts have 16 bits; a padded one among them."""
    torch = torch_cuda
    tokens = (1 << 24) + 777
    print_case(f"route {tokens} tokens")
    l = torch.randn(tokens, 2, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    l[tokens // 2] = -math.inf
    l[:70000, 1] = -100.0                                    # a block's tokens all on one expert
    r = uw.moe_route(l, 1)
    ids = torch.where(l[:, 1] > l[:, 0], 1, 0)
    ids[tokens // 2] = 2
    order = torch.sort(ids, stable=True).indices
    n0, n1 = int((ids == 0).sum()), int((ids == 1).sum())
    assert r.offsets.tolist() == [0, n0, n0 + n1] and n0 + n1 == tokens - 1
    assert torch.equal(r.ids[:, 0], torch.where(ids == 2, -1, ids).int())
    order[-1] = -1
    assert torch.equal(r.order, order.int())
    place = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    place[order[:-1]] = torch.arange(tokens - 1, dtype=torch.int32, device="cuda")
    assert torch.equal(r.place[:, 0], place)


def test_route_ties_masks_and_strides(torch_cuda):
    torch = torch_cuda
    for tokens in (7, 300):
        l = torch.zeros(tokens, 40 + 3).cuda()[:, :40]                 # all equal: the lowest indexes
        assert np.array_equal(check_route(torch, l, 4, True, "route ties").ids.cpu().numpy(),
                              np.tile(np.arange(4), (tokens, 1)))
        l = torch.randint(-2, 3, (tokens, 40)).float().cuda()
        l[l == 0] = -0.0                                               # -0 and +0 are equal
        l[::3, ::2] = 0.0
        check_route(torch, l, 8, False, "route small integers")
        l = torch.randn(tokens, 40).cuda()
        l[::2] = -math.inf                                             # padded tokens
        l[1, 3:] = -math.inf                                           # fewer than top_k
        l[3, :] = torch.finfo(torch.float32).min                       # a mask of the type's lowest value is finite
        l[5, 7] = math.inf
        l[5, 9] = math.inf
        l[5, 11] = math.nan
        l[-1] = math.nan
        for k in (1, 6):
            for renorm in (True, False):
                check_route(torch, l, k, renorm, "route masked")
        check_route(torch, torch.full((tokens, 9), -math.inf).cuda(), 3, True, "route nothing")


# ------------------------------------------------------------ grouped products
def grouping(torch, seed, counts, top_k=1, tokens=None):
    """Offsets of the given counts and an order of that many slots."""
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    n = int(off[-1])
    g = torch.Generator().manual_seed(seed)
    order = torch.randint(0, (tokens or max(n, 1)) * top_k, (n,), generator=g, dtype=torch.int32)
    return off.cuda(), order.cuda(), n


COUNTS = {
    "one": [0, 1, 0, 0],
    "few": [3, 0, 1, 5, 0, 0, 16, 2],
    "empty ends": [0, 0, 40, 17, 0],
    "uneven": [1, 300, 0, 7, 64, 65, 2],
    "large": [257, 130, 511],
    "many": [int(c) for c in np.random.default_rng(1).integers(0, 9, 150)],
    "none": [0, 0, 0],
    "all in one": [0] * 63 + [100] + [0] * 40,
}


@pytest.mark.parametrize("pal", [False, True])
@pytest.mark.parametrize("name", list(COUNTS))
def test_grouped(torch_cuda, name, pal):
    """gemm_grouped and moe_gate_up over ragged groups, with and without an
    order; rows of out behind the last group stay."""
    torch = torch_cuda
    counts = COUNTS[name]
    experts = len(counts)
    rows, cols = (70, 192) if experts > 50 else (200, 1088)
    W, w = make_weight(torch, 11, experts, rows, cols, pal)
    U, u = make_weight(torch, 12, experts, rows, cols, pal)
    off, order, n = grouping(torch, 3, counts, 3, 50)
    e = np.repeat(np.arange(experts), counts)
    for ordered in (True, False):
        what = f"grouped {name} pal={pal} ordered={ordered}"
        print_case(what)
        X = rows_of(torch, 5, 50 if ordered else n + 4, cols, 8)
        spare = torch.full((order.shape[0] + 4,), -1, dtype=torch.int32).cuda()
        spare[:n] = order
        o, k = (spare, 3) if ordered else (None, 1)
        xs = f64(X)[(order.cpu().long() // 3)] if ordered else f64(X)[:n]
        v = torch.stack([xs[s] @ w[e[s]].t() for s in range(n)]) if n else torch.zeros(0, rows, dtype=torch.float64)
        gu = torch.stack([xs[s] @ u[e[s]].t() for s in range(n)]) if n else v
        scale = torch.stack([xs[s].abs() @ w[e[s]].abs().t() for s in range(n)]) if n else v
        scale_u = torch.stack([xs[s].abs() @ u[e[s]].abs().t() for s in range(n)]) if n else v
        err, err_u = [(cols + 8) * 2.0 ** -23 * s for s in (scale, scale_u)]
        out = torch.full((n + 4, rows + 4), 7.0).cuda()[:, :rows]
        uw.gemm_grouped(W, X, off, o, k, out=out)
        check(torch, out[:n], v, err, what)
        assert bool((out[n:] == 7).all())
        check(torch, uw.gemm_grouped(W, X, off, o, k, out_dtype=torch.bfloat16)[:n], v, err, what + " bf16")
        h = torch.full((n + 4, rows), 7.0, dtype=torch.bfloat16).cuda()
        uw.moe_gate_up(W, U, X, off, o, k, h=h)
        s = activate(torch, v, "silu")
        err_s = 1.13 * err + 2.0 ** -20 * (v.abs() + s.abs())
        check(torch, h[:n], s * gu, err_s * (gu.abs() + err_u) + s.abs() * err_u + (s * gu).abs() * 2.0 ** -23,
              what + " pair")
        assert bool((h[n:] == 7).all())


def test_grouped_weights_exact(torch_cuda):
    """One-hot rows pick single weights of their own expert, verbatim groups among them; expert matrices that
    start inside a tile of 64 groups."""
    torch = torch_cuda
    experts, rows, cols = 5, 37, 320
    for per in (1, 9, 70):
        for pal in (False, True):
            print_case(f"grouped one-hot {per} rows an expert pal={pal}")
            W, w = make_weight(torch, 21, experts, rows, cols, pal, 0.02)
            n = experts * per
            at = torch.arange(n) * 41 % cols
            X = torch.zeros(n, cols, dtype=torch.bfloat16)
            X[torch.arange(n), at] = 1.0
            off = torch.arange(experts + 1, dtype=torch.int32).cuda() * per
            out = f64(uw.gemm_grouped(W, X.cuda(), off))
            e = torch.arange(n) // per
            assert torch.equal(out, w[e, :, at])


def test_grouped_verbatim_in_the_first_expert_only(torch_cuda):
    """Experts behind the last verbatim group, with every number of rows an expert."""
    torch = torch_cuda
    experts, rows, cols = 4, 64, 256
    w = workloads.gaussian_weights(np.random.default_rng(5), experts * rows, cols, 0.02, 0.05, 1.0)
    w[rows:] = 0x3F00 | (w[rows:] & 0x807F)                # one exponent: all of these groups are palette groups
    c = uw.compress(w)
    assert c.info().verbatim_groups > 0
    W = c.to_device(uw.DIRECT_SECTIONS)
    exact = f64(torch.from_numpy(w.view(np.int16)).view(torch.bfloat16)).view(experts, rows, cols)
    for per in (1, 3, 9, 30, 70):
        print_case(f"grouped without verbatim groups at the end, {per} rows an expert")
        X = rows_of(torch, per, experts * per, cols)
        off = torch.arange(experts + 1, dtype=torch.int32).cuda() * per
        x = f64(X).view(experts, per, cols)
        want = torch.bmm(x, exact.transpose(1, 2).contiguous()).view(-1, rows)
        bound = (cols + 8) * 2.0 ** -23 * torch.bmm(x.abs(), exact.abs().transpose(1, 2).contiguous()).view(-1, rows)
        check(torch, uw.gemm_grouped(W, X, off), want, bound, "products")
        if per == 1:
            logits = torch.tensor([[0.0, 1.0, 2.0, 3.0]]).cuda()
            r = uw.moe_route(logits, 2)
            h = rows_of(torch, 9, 2, cols)
            y = uw.gemm_grouped(W, h, r.offsets)
            e = r.ids[0].cpu().long()
            hx = f64(h)[r.place[0].cpu().long()]
            check(torch, y[r.place[0].long()], torch.stack([hx[j] @ exact[e[j]].t() for j in range(2)]),
                  torch.stack([(cols + 8) * 2.0 ** -23 * (hx[j].abs() @ exact[e[j]].abs().t()) for j in range(2)]), "routed")


@pytest.mark.parametrize("pal", [False, True])
def test_grouped_past_32_bits(torch_cuda, pal):
    """The last expert of a stack of more than 2^31 weights gives what its own matrix gives.  The bound on either
    sum is that of fp32 sums, with the sum of absolute products from the same matrix without its signs."""
    torch = torch_cuda
    E, R, C = 36, 8192, 8192
    one, tiles = R * C, R * C // 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    if pal:
        sm = torch.randint(0, 256, (E * one,), generator=g, dtype=torch.uint8, device="cuda")
        nib = torch.randint(0, 256, (E * one // 2,), generator=g, dtype=torch.uint8, device="cuda")
        vexp = torch.randint(108, 122, (E * tiles * 64,), generator=g, dtype=torch.uint8, device="cuda")

        def handle(lo, hi, mask=255):                        # the first group of every tile is verbatim
            n = (hi - lo) * tiles
            return uw.DeviceMatrix.from_sections((hi - lo) * R, C, range(106, 122), n, {
                "sm": sm[lo * one:hi * one] if mask == 255 else sm[lo * one:hi * one] & mask,
                "nib": nib[lo * one // 2:hi * one // 2], "vexp": vexp[lo * tiles * 64:hi * tiles * 64],
                "bitmap": torch.ones(n, dtype=torch.int64, device="cuda").view(torch.uint8),
                "tile_vbase": torch.arange(n + 1, dtype=torch.int32, device="cuda").view(torch.uint8)})
        whole, last, size = handle(0, E), handle(E - 1, E), handle(E - 1, E, 0x7F)
    else:
        whole = torch.empty(E, R, C, dtype=torch.bfloat16, device="cuda")
        for e in range(E):
            whole[e] = torch.randn(R, C, generator=g, device="cuda") * 0.02
        last, size = whole[E - 1], whole[E - 1].abs()
    for n in (1, 3, 40, 700):
        print_case(f"last of {E} experts, {n} rows, pal={pal}")
        X = rows_of(torch, n, n, C)
        off = torch.zeros(E + 1, dtype=torch.int32).cuda()
        off[E] = n
        bound = 2 * (C + 8) * 2.0 ** -23 * f64(uw.linear(size, X.abs())) * 1.01
        want = uw.linear(last, X)
        assert bool(want.isfinite().all())
        check(torch, uw.gemm_grouped(whole, X, off), f64(want), bound, "products")
        h, q = uw.moe_gate_up(whole, whole, X, off), f64(want)
        y = activate(torch, q, "silu")
        check(torch, h, y * q, (1.13 * bound + 2.0 ** -20 * (q.abs() + y.abs())) * (q.abs() + bound) + y.abs() * bound +
              (y * q).abs() * 2.0 ** -23, "pair")


def test_grouped_scratch(torch_cuda):
    """Experts with hundreds of rows: any scratch gives the result, an expert without rows is not expanded."""
    torch = torch_cuda
    counts, rows, cols = [2900, 0, 1600, 2701], 1020, 1088
    (W, w), (U, u) = (make_weight(torch, 50 + i, 4, rows, cols, True, 0.02) for i in range(2))
    off, order, n = grouping(torch, 8, counts, 2, 1000)
    X = rows_of(torch, 5, 1000, cols, 8)
    at = torch.cat([torch.arange(0, n, 211), off[1:].cpu().long() - 1])
    e = torch.from_numpy(np.repeat(np.arange(4), counts))[at]
    x = f64(X)[order.cpu().long()[at] // 2]
    v, q = [torch.bmm(m[e], x[:, :, None])[:, :, 0] for m in (w, u)]
    err, err_q = [(cols + 8) * 2.0 ** -23 * torch.bmm(m[e].abs(), x.abs()[:, :, None])[:, :, 0] for m in (w, u)]
    s = activate(torch, v, "silu")
    err_s = 1.13 * err + 2.0 ** -20 * (v.abs() + s.abs())
    L = uw.lib()
    for pair in (0, 1):
        need = L.uw_grouped_scratch_bytes(1, pair, 4, rows, cols, n)
        assert need >= (1 + pair) * 4 * rows * cols * 2 and L.uw_grouped_scratch_bytes(0, pair, 4, rows, cols, n) == 0
        for t in scratches(torch, need):
            what = f"grouped scratch pair={pair} {None if t is None else t.numel()} of {need}"
            print_case(what)
            if pair:
                h = uw.moe_gate_up(W, U, X, off, order, 2, scratch=t)
                check(torch, h[at.cuda()], s * q, err_s * (q.abs() + err_q) + s.abs() * err_q +
                      (s * q).abs() * 2.0 ** -23, what)
            else:
                check(torch, uw.gemm_grouped(W, X, off, order, 2, scratch=t)[at.cuda()], v, err, what)


def test_no_room_for_scratch(torch_cuda, monkeypatch):
    """Where memory has no room for what would make a call faster, it runs with what it needs."""
    torch = torch_cuda
    print_case("no room for scratch")
    E, F, H, tokens = 2, 1024, 1088, 8000
    G, U = (make_weight(torch, i, E, F, H, True)[0] for i in range(2))
    D, _ = make_weight(torch, 2, E, H, F, True)
    X = rows_of(torch, 1, tokens, H)
    logits = torch.randn(tokens, E).cuda()
    least = uw.moe_scratch_bytes(tokens, E, 1, F, H)
    assert uw.moe_scratch_bytes(tokens, E, 1, F, H, True) > least
    assert uw.lib().uw_linear_scratch_bytes(1, E * F, H, tokens) > 0
    r = uw.moe_route(logits, 1)
    calls = (lambda: uw.moe_layer(G, U, D, X, logits, 1), lambda: uw.moe_gate_up(G, U, X, r.offsets, r.order, 1),
             lambda: uw.linear(G, X))
    want = [f() for f in calls]
    empty = torch.empty

    def small(*a, dtype=None, **kw):
        if dtype == torch.uint8 and a[0] > least:
            raise torch.cuda.OutOfMemoryError("no room")
        return empty(*a, dtype=dtype, **kw)
    monkeypatch.setattr(torch, "empty", small)
    least_linear, least = least, 0
    for f, w in zip(calls[1:], want[1:]):
        got = f()
        assert float((got.float() - w.float()).norm() / w.float().norm()) < 2 ** -8      # half a step of bf16 each
    least = least_linear
    got = calls[0]()
    assert float((got - want[0]).norm() / want[0].norm()) < 2 ** -8


def test_grouped_bad_offsets_stay_inside(torch_cuda):
    """Offsets out of order or out of range and indexes outside X: rows outside the output's are untouched."""
    torch = torch_cuda
    for pal in (False, True):
        W, _ = make_weight(torch, 31, 4, 48, 128, pal)
        X = rows_of(torch, 1, 20, 128)
        for off in ([0, 5, 3, 30, 25], [-7, 4, 4, 900, 2 ** 31 - 1], [20, 10, 5, 0, 0], [3, 3, 3, 3, 3]):
            print_case(f"grouped offsets {off} pal={pal}")
            o = torch.tensor(off, dtype=torch.int32).cuda()
            buf = torch.full((30, 48), 7.0).cuda()
            order = torch.randint(-50, 90, (20,), dtype=torch.int32).cuda()
            uw.gemm_grouped(W, X, o, order, 2, out=buf[5:25])
            uw.moe_gate_up(W, W, X, o, order, 2)
            torch.cuda.synchronize()
            assert bool((buf[:5] == 7).all()) and bool((buf[25:] == 7).all())


def test_combine(torch_cuda):
    torch = torch_cuda
    g = torch.Generator().manual_seed(4)
    for tokens, top_k, cols, n in ((1, 1, 64, 1), (5, 2, 130, 10), (40, 8, 1000, 250), (3, 16, 7, 0)):
        print_case(f"combine {tokens} x {top_k} x {cols}")
        Y = torch.randn(n, cols, generator=g).cuda()
        place = torch.randint(-2, n + 3, (tokens, top_k), generator=g, dtype=torch.int32).cuda()
        weights = torch.rand(tokens, top_k, generator=g).cuda()
        for res, out in ((None, torch.float32), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
            r = None if res is None else torch.randn(tokens, cols + 3, generator=g).to(res).cuda()[:, :cols]
            got = uw.moe_combine(Y, place, weights, residual=r, out_dtype=out)
            p = place.cpu().long()
            ok = (p >= 0) & (p < n)
            terms = f64(torch.cat([Y, Y.new_zeros(1, cols)]))[torch.where(ok, p, n)] * (f64(weights) * ok)[:, :, None]
            want, size = terms.sum(1), terms.abs().sum(1)
            if r is not None:
                want, size = want + f64(r), size + f64(r).abs()
            check(torch, got, want, 18 * 2.0 ** -23 * size, "combine")


def layer_reference(torch, g, u, d, x, logits, top_k, renorm, residual):
    """The layer in 64 bits, and a bound: h rounded to bf16 (half a step of each), fp32 sums."""
    ids, w, _, _, _ = plain_route(logits.float().cpu().numpy(), top_k, renorm)
    y = torch.zeros(x.shape[0], d.shape[1], dtype=torch.float64)
    err = torch.zeros_like(y)
    F, H = g.shape[1], g.shape[2]
    for t in range(x.shape[0]):
        for j in range(top_k):
            e = ids[t, j]
            if e < 0:
                continue
            v, q = g[e] @ x[t], u[e] @ x[t]
            ev, eq = [(H + 8) * 2.0 ** -23 * (m[e].abs() @ x[t].abs()) for m in (g, u)]
            s = v * torch.sigmoid(v)
            es = 1.13 * ev + 2.0 ** -20 * (v.abs() + s.abs())
            h = s * q
            eh = es * (q.abs() + eq) + s.abs() * eq + h.abs() * 2.0 ** -8 * 1.01
            ey = d[e].abs() @ eh + (F + 8) * 2.0 ** -23 * (d[e].abs() @ h.abs())
            y[t] += w[t, j] * (d[e] @ h)
            err[t] += w[t, j] * (ey + 600 * 2.0 ** -23 * (d[e] @ h).abs())
    if residual is not None:
        y = y + f64(residual)
    return y, err + y.abs() * 2.0 ** -22


@pytest.mark.parametrize("pal", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 8, 2), (2, 4, 4), (7, 16, 3), (33, 8, 2), (70, 100, 2),
                                                  (150, 5, 1), (1100, 2, 1)])
def test_layer(torch_cuda, tokens, experts, top_k, pal):
    """The whole layer, padded tokens among the others, with and without a
    residual; the single calls in a row give the same result."""
    torch = torch_cuda
    F, H = 192, 256
    print_case(f"layer {tokens} of {experts} top {top_k} pal={pal}")
    (G, g), (U, u), (D, d) = (make_weight(torch, 40 + i, experts, r, c, pal) for i, (r, c) in
                              enumerate(((F, H), (F, H), (H, F))))
    X = rows_of(torch, 6, tokens, H, 8)
    logits = torch.randn(tokens, experts, generator=torch.Generator().manual_seed(9)).cuda()
    if tokens > 2:
        logits[tokens // 2] = -math.inf
    for renorm, res, out_dtype in ((True, None, torch.float32), (False, X, torch.bfloat16)):
        y, err = layer_reference(torch, g, u, d, f64(X), logits, top_k, renorm, res)
        out = uw.moe_layer(G, U, D, X, logits, top_k, renormalize=renorm, residual=res, out_dtype=out_dtype)
        check(torch, out, y, err, "layer")
        r = uw.moe_route(logits, top_k, renormalize=renorm)
        h = uw.moe_gate_up(G, U, X, r.offsets, r.order, top_k)
        Y = uw.gemm_grouped(D, h, r.offsets)
        check(torch, uw.moe_combine(Y, r.place, r.weights, residual=res, out_dtype=out_dtype), y, err, "calls in a row")
        again = uw.moe_layer(G, U, D, X, logits, top_k, renormalize=renorm, residual=res, out_dtype=out_dtype)
        assert torch.equal(out, again)


@pytest.mark.parametrize("pal", [False, True])
def test_layer_single_token(torch_cuda, pal):
    """One token: more experts than it can have, masked ones among them, none
    at all, rows of several tiles of 64 groups and of parts of one."""
    torch = torch_cuda
    for experts, top_k, F, H in ((8, 8, 64, 64), (5, 3, 1088, 320), (20, 16, 192, 128), (3, 2, 8256, 64), (6, 4, 64, 4160)):
        print_case(f"layer of one token, {experts} experts, top {top_k}, F={F} H={H} pal={pal}")
        (G, g), (U, u), (D, d) = (make_weight(torch, 80 + i, experts, r, c, pal, 0.01) for i, (r, c) in
                                  enumerate(((F, H), (F, H), (H, F))))
        X = rows_of(torch, 6, 1, H)
        for masked in (0, 2, experts):
            logits = torch.randn(1, experts, generator=torch.Generator().manual_seed(masked)).cuda()
            logits[0, :masked] = -math.inf
            for res, out_dtype in ((None, torch.float32), (X, torch.bfloat16), (X.float(), torch.float32)):
                y, err = layer_reference(torch, g, u, d, f64(X), logits, top_k, True, res)
                out = uw.moe_layer(G, U, D, X, logits, top_k, residual=res, out_dtype=out_dtype)
                check(torch, out, y, err, f"layer of one token, masked {masked}")


def test_block_together(torch_cuda):
    """Router projection with its bias, routing, the layer added to the
    residual stream in place, then a projection on it, as a model would."""
    torch = torch_cuda
    print_case("projection, layer, projection")
    tokens, experts, top_k, F, H = 45, 12, 3, 128, 256
    (R, r), (G, g), (U, u), (D, d), (O, o) = (
        make_weight(torch, 60 + i, e, a, b, pal) for i, (e, a, b, pal) in
        enumerate(((1, experts, H, False), (experts, F, H, True), (experts, F, H, True), (experts, H, F, False),
                   (1, 200, H, True))))
    x = rows_of(torch, 8, tokens, H)
    bias = torch.randn(experts, generator=torch.Generator().manual_seed(2)).cuda()
    logits = uw.linear(R[0], x, bias=bias)
    check(torch, logits, f64(x) @ r[0].t() + f64(bias), sum_bound(torch, f64(x), r[0]) + 2.0 ** -21, "router")
    y, err = layer_reference(torch, g, u, d, f64(x), logits, top_k, True, x)
    out = uw.moe_layer(G, U, D, x, logits, top_k, residual=x, out=x)
    assert out.data_ptr() == x.data_ptr()
    check(torch, x, y, err, "layer in place")
    z = uw.linear(O, x, act="gelu")
    v = f64(x) @ o[0].t()
    w = activate(torch, v, "gelu")
    check(torch, z, w, 1.13 * sum_bound(torch, f64(x), o[0]) + 2.0 ** -20 * (v.abs() + w.abs()), "last projection")


def test_graphs_streams_and_scratch(torch_cuda):
    """Captured with its own scratch, replayed several times on new inputs with
    eager work between: every replay equals the eager call.  A raw stream
    handle gives the same results."""
    torch = torch_cuda
    print_case("layer in a graph")
    experts, top_k, F, H = 8, 2, 128, 192
    G, U, D = (make_weight(torch, 70 + i, experts, r, c, True)[0] for i, (r, c) in enumerate(((F, H), (F, H), (H, F))))
    P, _ = make_weight(torch, 75, 1, 300, H, False)
    for tokens in (1, 5, 90):
        X = rows_of(torch, 1, tokens, H)
        L = torch.randn(tokens, experts).cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            uw.linear(P[0], uw.moe_layer(G, U, D, X, L, top_k, out_dtype=torch.bfloat16), act="silu")
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mid = uw.moe_layer(G, U, D, X, L, top_k, out_dtype=torch.bfloat16)
            out = uw.linear(P[0], mid, act="silu")
        for i in range(4):
            X.copy_(rows_of(torch, 10 + i, tokens, H))
            L.copy_(torch.randn(tokens, experts))
            graph.replay()
            torch.cuda.synchronize()
            m = uw.moe_layer(G, U, D, X, L, top_k, out_dtype=torch.bfloat16)
            assert torch.equal(mid, m) and torch.equal(out, uw.linear(P[0], m, act="silu")), (tokens, i)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        m2 = uw.moe_layer(G, U, D, X, L, top_k, out_dtype=torch.bfloat16, stream=s.cuda_stream)
        o2 = uw.linear(P[0], m2, act="silu", stream=s.cuda_stream)
        s.synchronize()
        assert torch.equal(m, m2) and torch.equal(out, o2)


def test_from_sections(torch_cuda):
    """A handle on sections that are on the device already reads the same matrix."""
    torch = torch_cuda
    print_case("from_sections")
    w = workloads.gaussian_weights(np.random.default_rng(2), 96, 256, 0.02, 0.004, 1.0)
    b = uw.compress(w)
    a = b.to_device(uw.DIRECT_SECTIONS)
    inf = b.info()
    m = uw.DeviceMatrix.from_sections(96, 256, bytes(inf.palette), inf.verbatim_groups,
                                      {k: a.buffers[k] for k in uw.DIRECT_SECTIONS})
    X = rows_of(torch, 4, 9, 256)
    assert torch.equal(uw.linear(a, X), uw.linear(m, X)) and m.device_bytes() == a.device_bytes()
    assert torch.equal(uw.gemm_recon_pal(m, None, X), uw.gemm_recon_pal(a, None, X))
    with pytest.raises(ValueError, match="at least"):
        uw.DeviceMatrix.from_sections(96, 512, bytes(inf.palette), inf.verbatim_groups, dict(a.buffers))
    with pytest.raises(ValueError, match="missing"):
        uw.DeviceMatrix.from_sections(96, 256, bytes(inf.palette), inf.verbatim_groups, {"sm": a.buffers["sm"]})


def test_python_refusals(torch_cuda):
    torch = torch_cuda
    print_case("refusals")
    W, _ = make_weight(torch, 1, 1, 64, 128, False)
    X = rows_of(torch, 2, 6, 128)
    off = torch.tensor([0, 6], dtype=torch.int32).cuda()
    bad = [lambda: uw.linear(W[0], X.float()), lambda: uw.linear(W[0], X[:, :64]), lambda: uw.linear(W[0].t(), X),
           lambda: uw.linear(W, X), lambda: uw.linear(W[0].float(), X), lambda: uw.linear(W[0], X, act="tanh"),
           lambda: uw.linear(W[0], X, bias=torch.zeros(63).cuda()), lambda: uw.linear(W[0], X.cpu()),
           lambda: uw.linear(W[0], X, bias=torch.zeros(64)), lambda: uw.linear(W[0], X, residual=X),
           lambda: uw.linear(W[0], X, out=torch.zeros(6, 64).cuda().half()),
           lambda: uw.linear(W[0], X, bias=torch.zeros(64).cuda().half()),
           lambda: uw.gemm_grouped(W, X, off.long()), lambda: uw.gemm_grouped(W, X, off, off.float()),
           lambda: uw.gemm_grouped(W, X, off[:1]), lambda: uw.gemm_grouped(W[0], X, off),
           lambda: uw.moe_gate_up(W, W[:, :32].contiguous(), X, off),
           lambda: uw.moe_route(torch.zeros(3, 4).cuda().half(), 2),
           lambda: uw.moe_combine(torch.zeros(3, 4).cuda(), off, torch.zeros(2).cuda()),
           lambda: uw.moe_layer(W, W, W, X, torch.zeros(6, 1).cuda(), 1)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
    refused = [lambda: uw.linear(W[0], X.as_strided((3, 128), (132, 1))),
               lambda: uw.linear(W[0], X, residual=torch.zeros(1, 64).cuda().expand(6, 64)),
               lambda: uw.linear(W[0], X, out=X.view(torch.float32)),
               lambda: uw.moe_route(torch.zeros(3, 4).cuda(), 5), lambda: uw.moe_route(torch.zeros(3, 40).cuda(), 17),
               lambda: uw.moe_route(torch.zeros(3, 513).cuda(), 2),
               lambda: uw.gemm_grouped(W, X[:3], torch.tensor([0, 6], dtype=torch.int32).cuda(), None, 1,
                                       out=torch.zeros(3, 64).cuda()[:, :64].as_strided((3, 64), (32, 1))),
               lambda: uw.moe_layer(W[:, :, :64].contiguous(), W[:, :, :64].contiguous(), W[:, :, :64].contiguous(),
                                    X[:, :64], torch.zeros(6, 1).cuda(), 1, scratch=torch.zeros(64).cuda())]
    for i, f in enumerate(refused):
        with pytest.raises(uw.UnweightError):
            f()
