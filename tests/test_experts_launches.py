"""What the calls launch, seen from the host (tests/launch_util.py): no GPU."""
import ctypes as ct
import shutil

import numpy as np
import pytest

import mlp_matmul_amd as uw
import workloads
from mlp_matmul_amd import _capi
from tests.launch_util import Recorder

P, BIG = 0x1000000, 1 << 32            # placeholder device addresses, far apart


def at(i):
    return P + i * BIG


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    return Recorder(tmp_path_factory.mktemp("recorder"))


def dmat(recorder, info, **over):
    """A descriptor whose sections are placeholder addresses."""
    ptrs = (ct.c_void_p * _capi.UW_NUM_SECTIONS)()
    for i in range(len(_capi.SECTION_NAMES)):
        ptrs[i] = at(20 + i)
    d = _capi.uw_dmat()
    assert recorder.lib.uw_dmat_init(ct.byref(d), ct.byref(info), ptrs) == 0
    for k, v in over.items():
        setattr(d, k, v)
    return d


def info_of(rows, cols, verbatim):
    inf = _capi.uw_info(rows=rows, cols=cols, groups=rows * cols // 64, verbatim_groups=verbatim, palette_size=16,
                        has_palette=1)
    inf.tiles = (inf.groups + 63) // 64
    return inf


VEXP, SM = at(20 + _capi.SECTION_NAMES.index("vexp")), at(20 + _capi.SECTION_NAMES.index("sm"))


def palette_calls(L, d, batch):
    """Every call that takes a palette matrix [4096, 256] (4 experts of 1024 rows for the grouped ones)."""
    down = info_of(1024, 1024, d.verbatim_groups)
    X, off, out, scratch = at(1), at(2), at(3), at(9)
    p = ct.byref(d)
    yield "linear", lambda: L.uw_linear(None, p, 4096, 256, X, 256, batch, None, 0, 0, None, 0, 0, out, 0, 4096, scratch,
                                        1 << 31, None)
    yield "linear without scratch", lambda: L.uw_linear(None, p, 4096, 256, X, 256, batch, None, 0, 0, None, 0, 0, out, 0,
                                                        4096, None, 0, None)
    yield "grouped", lambda: L.uw_gemm_grouped(None, p, 4, 1024, 256, X, batch, 256, off, None, 1, batch, out, 0, 1024,
                                               scratch, 1 << 31, None)
    yield "gate_up", lambda: L.uw_moe_gate_up(None, p, None, p, 4, 1024, 256, X, batch, 256, off, None, 1, batch, out, 1024,
                                              None, 0, None)
    yield "recon_pal", lambda: L.uw_gemm_recon_pal(p, d.nib, X, batch, out, 0, 1, None, 0, None)


def qwords(raw):
    return set(np.frombuffer(raw[:len(raw) // 8 * 8], dtype=np.uint64).tolist())


@pytest.mark.parametrize("batch", [1, 2, 3, 9, 20, 40, 100, 300, 3000])
def test_an_empty_vexp_is_not_read(recorder, batch):
    """Lanes without a verbatim group load from VEXP's start.  Without any such group the section is empty: what they
    are given is SM, or no address (the kernels then take SM), whatever the descriptor's pointer is."""
    for verbatim in (0, 40):
        d = dmat(recorder, info_of(4096, 256, verbatim))
        for name, call in palette_calls(recorder.lib, d, batch):
            rcs = []
            seen = recorder.launches(lambda: rcs.append(call()), 56)      # a weight's pointers come first
            assert rcs == [0], (name, recorder.lib.uw_last_error())
            reads = [k for k, _, _, raw in seen if SM in qwords(raw)]
            assert reads, (name, [k for k, *_ in seen])
            for kernel, _, _, raw in seen:
                assert (VEXP in qwords(raw)) == (verbatim > 0 and SM in qwords(raw)), (name, kernel, verbatim)
