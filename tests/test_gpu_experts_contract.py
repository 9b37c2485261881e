"""GPU tests of what unweight.h promises of the epilogue matmul and of the
mixture-of-experts operators, beyond tests/test_gpu_experts.py (whose
tolerances and helpers they share)."""
import numpy as np
import pytest

import mlp_matmul_amd as uw
import workloads
from tests.gpu_util import print_case
from tests.test_gpu_experts import check, f64, rows_of, sum_bound, torch_cuda  # noqa: F401

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
