"""GPU tests of what unweight.h promises of the epilogue matmul and of the
mixture-of-experts operators, beyond tests/test_gpu_experts.py (whose
tolerances and helpers they share)."""
import numpy as np
import pytest

import mlp_matmul_amd as uw
import workloads
from tests.gpu_util import print_case
from tests.test_gpu_experts import check, f64, rows_of, sum_bound, torch_cuda  # noqa: F401
from tests.test_gpu_experts_variants import matrix

pytestmark = pytest.mark.gpu


def test_palette_without_verbatim_groups(torch_cuda):  # noqa: F811
    """A matrix without verbatim groups whose VEXP section is there all the same, with nothing in it."""
    torch = torch_cuda
    experts, rows, cols = 4, 200, 256
    w = workloads.gaussian_weights(np.random.default_rng(5), experts * rows, cols, 0.02, 0.05, 1.0)
    w = 0x3C00 | (w & 0x83FF)                              # eight exponents
    c = uw.compress(w)
    inf = c.info()
    assert inf.verbatim_groups == 0
    a = c.to_device(uw.DIRECT_SECTIONS)
    W = uw.DeviceMatrix.from_sections(experts * rows, cols, bytes(inf.palette), 0,
                                      {**a.buffers, "vexp": torch.zeros(16, dtype=torch.uint8).cuda()})
    exact = f64(torch.from_numpy(w.view(np.int16)).view(torch.bfloat16))
    for batch in (1, 2, 3, 9, 40, 300):
        print_case(f"no verbatim groups, {batch} rows")
        X = rows_of(torch, batch, batch, cols)
        check(torch, uw.linear(W, X), f64(X) @ exact.t(), sum_bound(torch, f64(X), exact), "linear")
        check(torch, uw.gemm_recon_pal(W, None, X), f64(X) @ exact.t(), sum_bound(torch, f64(X), exact), "matmul")
        off = torch.tensor([0, 0, 0, batch, batch], dtype=torch.int32).cuda()
        e = exact[2 * rows:3 * rows]
        check(torch, uw.gemm_grouped(W, X, off), f64(X) @ e.t(), sum_bound(torch, f64(X), e), "grouped")


def scratch_calls(torch):
    """Calls that take scratch: K-slices of a bf16 matrix, sums of a palette matrix in scratch, an expanded one, a layer
    whose routing takes two launches and whose weights are expanded.  Each: (its inputs, the call)."""
    calls = []
    for i, (pal, rows, cols, batch) in enumerate(((0, 355, 2240, 611), (1, 2177, 1024, 99), (1, 721, 704, 354))):
        assert uw.lib().uw_linear_scratch_bytes(pal, rows, cols, batch) > 0
        W, _ = matrix(torch, i, pal, 1, rows, cols)
        X = rows_of(torch, i, batch, cols)
        calls.append(((X,), lambda W=W if pal else W[0], X=X: uw.linear(W, X, act="silu")))
    E, F, H, tokens = 3, 1024, 1088, 3000
    assert uw.moe_scratch_bytes(tokens, E, 2, F, H, True) > uw.moe_scratch_bytes(tokens, E, 2, F, H)
    assert uw.lib().uw_moe_route_scratch_bytes(tokens, E, 2) > 0
    G, U = (matrix(torch, 10 + i, True, E, F, H)[0] for i in range(2))
    D, _ = matrix(torch, 12, True, E, H, F)
    X, logits = rows_of(torch, 5, tokens, H), torch.randn(tokens, E, device="cuda")
    calls.append(((X, logits), lambda: uw.moe_layer(G, U, D, X, logits, 2, residual=X)))
    return calls


def renew(torch, inputs, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    for t in inputs:
        t.copy_(torch.randn(t.shape, device="cuda", generator=g))


def test_graphs_of_calls_with_scratch(torch_cuda):  # noqa: F811
    """All of them in two graphs, replayed in turn on new inputs with eager work between: as the eager calls."""
    torch = torch_cuda
    print_case("graphs of calls with scratch")
    calls = scratch_calls(torch)
    for _, f in calls:
        f()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [f() for _, f in calls]
        graphs.append((g, out))
    for i in range(6):
        for inputs, _ in calls:
            renew(torch, inputs, i)
        g, out = graphs[i % 2]
        g.replay()
        if i % 3 == 0:
            torch.cuda.synchronize()
        for k, (_, f) in enumerate(calls):
            assert torch.equal(out[k], f()), (i, k)


def test_streams_at_once(torch_cuda):  # noqa: F811
    """The same calls on two streams at once, on inputs of their own."""
    torch = torch_cuda
    print_case("calls on two streams at once")
    sides = [scratch_calls(torch), scratch_calls(torch)]
    want = []
    for s, calls in enumerate(sides):
        for inputs, _ in calls:
            renew(torch, inputs, 100 + s)
        want.append([f() for _, f in calls])
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
                assert torch.equal(out, want[s][k]), (s, k)


def test_inference_on_parameters(torch_cuda):  # noqa: F811
    """A module's weights run under no_grad and are refused where a gradient would be lost."""
    torch = torch_cuda
    print_case("parameters")
    layer = torch.nn.Linear(192, 100, device="cuda", dtype=torch.bfloat16)
    X = rows_of(torch, 3, 7, 192)
    with pytest.raises(ValueError, match="gradient"):
        uw.linear(layer.weight, X, bias=layer.bias)
    with torch.no_grad():
        out = uw.linear(layer.weight, X, bias=layer.bias)
    w = f64(layer.weight)
    v = f64(X) @ w.t() + f64(layer.bias)
    check(torch, out, v, sum_bound(torch, f64(X), w) + v.abs() * 2.0 ** -23, "linear")
