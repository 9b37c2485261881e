"""GPU tests of what unweight.h promises of the microscaled 4-bit operators, of
the scored router and of the experts on a routing, beyond single calls: a run of
them together, graphs, streams, scratch, far apart rows.  Tolerances and helpers
of tests/test_gpu_mx4.py and tests/test_gpu_route_scored.py."""
import pytest

import mlp_matmul_amd as uw
from tests.gpu_util import print_case
from tests.mx4_util import quantize_ref, route_ref, values_ref
from tests.test_gpu_experts import activate, check, f64, sum_bound, torch_cuda  # noqa: F401
from tests.test_gpu_mx4 import normal, weight
from tests.test_gpu_route_scored import experts_ref, logits_of, three_weights

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ together
@pytest.mark.parametrize("tokens", [1, 5, 77, 300])
def test_block_together(torch_cuda, tokens):  # noqa: F811
    """Router projection, routing, the experts on 4-bit rows step by step, their sum on the residual in place, and the
    projection behind it: each against the definition on what the step before gave."""
    torch = torch_cuda
    print_case(f"block of 4-bit weights, {tokens} tokens")
    E, k, F, H = 12, 3, 160, 288
    (R, r), (O, o) = weight(torch, 60, E, H), weight(torch, 61, 200, H)
    (G, U, D), (g, u, d) = three_weights(torch, "mx4", E, F, H, 62)
    x = normal(torch, 8, tokens, H)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(2)).cuda() * 0.1
    logits = uw.linear(R, x)
    check(torch, logits, f64(x) @ r.t(), sum_bound(torch, f64(x), r), "router")
    routing = uw.moe_route_scored(logits, k, bias=bias, groups=4, top_groups=2, scale=1.5)
    ids = route_ref(logits, k, "sigmoid", bias, 4, 2, 2, True, 1.5)[0]
    assert (routing.ids.cpu().numpy() == ids).all()

    x4 = uw.mx4_quantize(x)
    assert torch.equal(x4.codes.cpu(), quantize_ref(x)[0])
    h = uw.moe_gate_up(G, U, x4, routing.offsets, routing.order, k)
    h4 = uw.mx4_quantize(h)
    y = uw.gemm_grouped(D, h4, routing.offsets)
    off, order = routing.offsets.tolist(), routing.order.cpu().long()
    xv, hv = values_ref(x4.codes, x4.scales), values_ref(h4.codes, h4.scales)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        xe = xv[order[lo:hi] // k]
        a, b = xe @ g[e].t(), xe @ u[e].t()
        ea, eb = sum_bound(torch, xe, g[e]), sum_bound(torch, xe, u[e])
        s = activate(torch, a, "silu")
        es = 1.13 * ea + 2.0 ** -20 * (a.abs() + s.abs())
        check(torch, h[lo:hi], s * b, es * (b.abs() + eb) + s.abs() * eb + 2.0 ** -22 * (s * b).abs(), f"h of {e}")
        check(torch, y[lo:hi], hv[lo:hi] @ d[e].t(), sum_bound(torch, hv[lo:hi], d[e]), f"y of {e}")
    out = uw.moe_combine(y, routing.place, routing.weights, residual=x, out_dtype=torch.float32)
    w, place = f64(routing.weights), routing.place.cpu().long()
    terms = w[:, :, None] * f64(y)[place]
    want = terms.sum(1) + f64(x)
    check(torch, out, want, (k + 2) * 2.0 ** -23 * (terms.abs().sum(1) + f64(x).abs()), "sum")

    # on bf16 rows in one call, in place of the residual
    z, err = experts_ref(torch, f64(x), (g, u, d), routing.ids.cpu(), w, x)
    stream = x.clone()
    assert uw.moe_experts(G, U, D, stream, routing, residual=stream, out=stream) is stream
    off_ = (f64(stream) - z).abs() > err + (z.abs() + err) * 2.0 ** -8
    assert not bool(off_.any())
    p = uw.linear(O, stream, act="gelu")
    v = f64(stream) @ o.t()
    q = activate(torch, v, "gelu")
    check(torch, p, q, 1.13 * sum_bound(torch, f64(stream), o) + 2.0 ** -20 * (v.abs() + q.abs()), "last projection")


def test_a_padded_batch(torch_cuda):  # noqa: F811
    """Tokens of -inf logits behind the batch's last: routed nowhere, their residual comes back, and the others' results
    are those of the batch without them."""
    torch = torch_cuda
    print_case("padded batch")
    E, k, F, H = 8, 2, 96, 160
    ws, _ = three_weights(torch, "mx4", E, F, H, 5)
    x, l = normal(torch, 1, 90, H), logits_of(torch, 2, 90, E)
    l[70:] = -float("inf")
    x[80:] = float("nan")
    r = uw.moe_route_scored(l, k, groups=2, top_groups=1)
    assert int(r.offsets[-1]) == 70 * k and bool((r.ids[70:] == -1).all())
    out = uw.moe_experts(*ws, x, r, residual=x)
    alone = uw.moe_route_scored(l[:70], k, groups=2, top_groups=1)
    assert torch.equal(alone.offsets, r.offsets) and torch.equal(alone.weights, r.weights[:70])
    assert torch.equal(out[:70], uw.moe_experts(*ws, x[:70], alone, residual=x[:70]))
    assert torch.equal(out[70:80], x[70:80].float()) and bool(torch.isnan(out[80:]).all())
    # nobody at all
    l[:] = -float("inf")
    none = uw.moe_route_scored(l, k)
    assert torch.equal(uw.moe_experts(*ws, x[:80], uw.moe_route_scored(l[:80], k), residual=x[:80]), x[:80].float())
    room = torch.full((90 * k, F), 7.0, dtype=torch.bfloat16, device="cuda")
    uw.moe_gate_up(ws[0], ws[1], x, none.offsets, none.order, k, h=room)
    assert bool((room == 7).all())


@pytest.mark.parametrize("x4", [False, True])
def test_one_row_many_times(torch_cuda, x4):  # noqa: F811
    """An order that names one row again and again: every place has that row's product."""
    torch = torch_cuda
    print_case(f"one row many times x4={x4}")
    W, w = weight(torch, 3, 3 * 48, 160)
    x = normal(torch, 4, 6, 160)
    X = uw.mx4_quantize(x) if x4 else x
    v = values_ref(X.codes, X.scales) if x4 else f64(x)
    for n in (3, 40, 200):
        order = torch.full((n,), 4, dtype=torch.int32, device="cuda")
        out = uw.gemm_grouped(W, X, torch.tensor([0, n // 3, n // 3, n], dtype=torch.int32, device="cuda"), order)
        for e, lo, hi in ((0, 0, n // 3), (2, n // 3, n)):
            we = w.view(3, 48, 160)[e]
            check(torch, out[lo:hi], (v[4:5] @ we.t()).expand(hi - lo, -1), sum_bound(torch, v[4:5], we).expand(hi - lo, -1), "row")


# ------------------------------------------------------------ graphs, streams, scratch
def calls(torch, seed, scratch=None):
    """Calls of every kind: (their inputs, the call).  Several launches: rows behind the last tile, a routing of more
    than 64 tokens.  scratch: (of the routing, of the experts), shared."""
    E, k, F, H = 8, 2, 160, 224
    (G, U, D), _ = three_weights(torch, "mx4", E, F, H, 62)
    W, _ = weight(torch, 7, 300, 1056)
    T, _ = weight(torch, 8, 7085, 1696)
    x, l = normal(torch, seed, 150, H), logits_of(torch, seed, 150, E)
    X = normal(torch, seed + 1, 37, 1056)
    Y = normal(torch, seed + 2, 1164, 1696)
    one, ol = normal(torch, seed + 3, 1, H), logits_of(torch, seed, 1, E)
    route_room, room = scratch or (None, None)

    def layer(x, l):
        r = uw.moe_route_scored(l, k, score="softmax", groups=4, top_groups=2, scratch=route_room)
        h = uw.moe_gate_up(G, U, uw.mx4_quantize(x), r.offsets, r.order, k)
        y = uw.gemm_grouped(D, uw.mx4_quantize(h), r.offsets)
        return (uw.moe_combine(y, r.place, r.weights, residual=x),
                uw.moe_experts(G, U, D, x, r, residual=x, scratch=room))

    return [((x, l), lambda: layer(x, l)), ((one, ol), lambda: layer(one, ol)),
            ((X,), lambda: (uw.linear(W, X, act="silu"), uw.mx4_dequantize(uw.mx4_quantize(X)))),
            ((Y,), lambda: (uw.linear(T, uw.mx4_quantize(Y), residual=None),))]


def renew(torch, inputs, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    for t in inputs:
        t.copy_(torch.randn(t.shape, device="cuda", generator=g))


def same(torch, a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_graphs(torch_cuda):  # noqa: F811
    """All of them in two graphs that share their scratch, replayed in turn on new inputs with eager work between: as the
    eager calls."""
    torch = torch_cuda
    print_case("graphs of 4-bit calls")
    scratch = (torch.empty(1 << 16, dtype=torch.uint8, device="cuda"), torch.empty(1 << 21, dtype=torch.uint8, device="cuda"))
    both = [calls(torch, 1, scratch), calls(torch, 50, scratch)]
    graphs = []
    for made in both:
        for _, f in made:
            f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [f() for _, f in made]
        graphs.append((g, out))
    for i in range(6):
        for made in both:
            for inputs, _ in made:
                renew(torch, inputs, i)
        for (g, _) in graphs:
            g.replay()
        if i % 3 == 0:
            torch.cuda.synchronize()
        for made, (_, out) in zip(both, graphs):
            for j, (_, f) in enumerate(made):
                assert same(torch, out[j], f()), (i, j)


def test_streams_at_once(torch_cuda):  # noqa: F811
    """The same calls on two streams at once, on inputs of their own; and on a raw handle."""
    torch = torch_cuda
    print_case("4-bit calls on two streams at once")
    sides = [calls(torch, 1), calls(torch, 90)]
    want = [[f() for _, f in made] for made in sides]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for s, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[s].append([f() for _, f in sides[s]])
    torch.cuda.synchronize()
    for s in (0, 1):
        for run in got[s]:
            for k, out in enumerate(run):
                assert same(torch, out, want[s][k]), (s, k)
    raw = streams[0].cuda_stream
    W, _ = weight(torch, 7, 300, 96)
    X, l = normal(torch, 3, 70, 96), logits_of(torch, 4, 70, 12)
    a, b = uw.moe_route_scored(l, 3), uw.moe_route_scored(l, 3, stream=raw)
    m, n = uw.mx4_quantize(X), uw.mx4_quantize(X, stream=raw)
    p, q = uw.linear(W, m), uw.linear(W, n, stream=raw)
    v, u = uw.mx4_dequantize(m), uw.mx4_dequantize(n, stream=raw)
    streams[0].synchronize()
    assert same(torch, a, b) and torch.equal(m.codes, n.codes) and torch.equal(m.scales, n.scales)
    assert torch.equal(p, q) and torch.equal(v, u)


# ------------------------------------------------------------ rows far apart
def far(torch, rows, cols, stride, dtype):
    """A view [rows, cols] of rows `stride` elements apart."""
    return torch.empty(rows * stride, dtype=dtype, device="cuda").as_strided((rows, cols), (stride, 1))


def test_rows_past_32_bits(torch_cuda):  # noqa: F811
    """Inputs and outputs whose offsets pass 2^32 bytes: as on the same rows close together."""
    torch = torch_cuda
    rows, cols = 70000, 64
    print_case("rows past 2^32 bytes")
    x = normal(torch, 1, rows, cols)
    X = far(torch, rows, cols, 40000, torch.bfloat16)
    X.copy_(x)
    m = uw.mx4_quantize(x)
    # 4-bit rows, both codes and scales
    M = uw.Mx4Matrix(far(torch, rows, cols // 2, 1 << 16, torch.uint8), far(torch, rows, cols // 32, 1 << 16, torch.uint8))
    uw.mx4_quantize(X, out=M)
    assert torch.equal(M.codes, m.codes) and torch.equal(M.scales, m.scales)
    out = far(torch, rows, cols, 32000, torch.float32)
    uw.mx4_dequantize(M, out=out)
    assert torch.equal(out, uw.mx4_dequantize(m))
    W, _ = weight(torch, 2, 40, cols)
    res = torch.randn(rows, 40, device="cuda")
    for near, apart in ((x, X), (m, M)):
        got = far(torch, rows, 40, 32000, torch.float32)
        got.copy_(res)
        want = uw.linear(W, near, residual=res)
        uw.linear(W, apart, residual=got, out=got)
        assert torch.equal(got, want)
        # few rows far out, by an order
        order = torch.arange(rows - 9, rows, dtype=torch.int32, device="cuda")
        off = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
        assert torch.equal(uw.gemm_grouped(W, apart, off, order), uw.gemm_grouped(W, near, off, order))


@pytest.mark.parametrize("x4", [False, True])
def test_experts_past_32_bits(torch_cuda, x4):  # noqa: F811
    """Weights of experts whose codes and scales pass 2^32 bytes."""
    torch = torch_cuda
    E, rows, cols = 300, 500, 64
    print_case(f"experts past 2^32 bytes x4={x4}")
    near, _ = weight(torch, 4, E * rows, cols)
    apart = uw.Mx4Matrix(far(torch, E * rows, cols // 2, 1 << 15, torch.uint8), far(torch, E * rows, cols // 32, 1 << 15, torch.uint8))
    apart.codes.copy_(near.codes)
    apart.scales.copy_(near.scales)
    for per in (1, 3, 70):
        n = E * per
        x = normal(torch, 5, n, cols)
        X = uw.mx4_quantize(x) if x4 else x
        off = torch.arange(0, n + 1, per, dtype=torch.int32, device="cuda")
        assert torch.equal(uw.gemm_grouped(apart, X, off), uw.gemm_grouped(near, X, off))
        assert torch.equal(uw.moe_gate_up(apart, near, X, off), uw.moe_gate_up(near, apart, X, off))


def test_many_numbers(torch_cuda):  # noqa: F811
    """More than 2^32 numbers in one matrix."""
    torch = torch_cuda
    rows, cols = 140000, 32768
    print_case("quantise 4.6e9 numbers")
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    some = [0, 1, 65535, 65536, 131071, 131072, rows - 1]
    for i in some:
        x[i].copy_(torch.randn(cols, generator=torch.Generator().manual_seed(i)))
    m = uw.mx4_quantize(x)
    codes, scales = quantize_ref(x[some])
    assert torch.equal(m.codes[some].cpu(), codes) and torch.equal(m.scales[some].cpu(), scales)
    assert int((m.scales != 0).any(1).sum()) == len(some)
    back = uw.mx4_dequantize(m, out=x)
    assert torch.equal(f64(back[some]), values_ref(codes, scales))


def test_nothing_to_do(torch_cuda):  # noqa: F811
    """No rows, no weights, no tokens."""
    torch = torch_cuda
    print_case("empty calls")
    W, _ = weight(torch, 1, 48, 96)
    none = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    m = uw.mx4_quantize(none)
    assert m.shape == (0, 96) and uw.mx4_dequantize(m).shape == (0, 96)
    for x in (none, m):
        assert uw.linear(W, x).shape == (0, 48)
        assert uw.gemm_grouped(W, x, torch.zeros(4, dtype=torch.int32, device="cuda")[:4]).shape == (0, 16)
    x = normal(torch, 2, 5, 96)
    assert uw.linear(m, x).shape == uw.linear(m, uw.mx4_quantize(x)).shape == (5, 0)
    narrow = uw.mx4_quantize(x[:, :0])
    assert narrow.shape == (5, 0) and uw.mx4_dequantize(narrow).shape == (5, 0)
    r = uw.moe_route_scored(torch.empty(0, 3, device="cuda"), 2)
    assert r.ids.shape == (0, 2) and bool((r.offsets == 0).all())
    D, _ = weight(torch, 3, 3 * 96, 32)
    G, _ = weight(torch, 4, 3 * 32, 96)
    assert uw.moe_experts(G, G, D, none, r).shape == (0, 96)
