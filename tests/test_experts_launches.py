"""What the calls launch, seen from the host (tests/launch_util.py): no GPU."""
import ctypes as ct
import shutil

import numpy as np
import pytest

import mlp_matmul_amd as uw
from mlp_matmul_amd import _capi
from tests.expert_cases import GROUPED, LINEAR
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


# ------------------------------------------------------- which kernels the sizes of the GPU tests run
OWN = ("skinny_kernel", "tile_kernel", "tile_pal_kernel", "gemv_rows_kernel", "expand_kernel", "sums_epilogue_kernel")


def of_case(recorder, linear, case):
    """The kernels that a case of tests/expert_cases.py launches, in order."""
    L, rcs = recorder.lib, []
    if linear:
        pal, rows, cols, n, scratch = case
        pair, experts = 0, 1
    else:
        pal, pair, experts, rows, cols, n, scratch = case
    d = ct.byref(dmat(recorder, info_of(experts * rows, cols, 40))) if pal else None
    w, s = None if pal else at(1), (at(60), 1 << 40) if scratch else (None, 0)
    if linear:
        call = lambda: rcs.append(L.uw_linear(w, d, rows, cols, at(2), cols, n, at(3), 0, 2, at(4), 1, rows, at(5), 0,  # noqa: E731
                                              rows, *s, None))
    elif pair:
        call = lambda: rcs.append(L.uw_moe_gate_up(w, d, w, d, experts, rows, cols, at(2), n, cols, at(3), None, 1, n,  # noqa: E731
                                                   at(5), rows, *s, None))
    else:
        call = lambda: rcs.append(L.uw_gemm_grouped(w, d, experts, rows, cols, at(2), n, cols, at(3), None, 1, n, at(5),  # noqa: E731
                                                    0, rows, *s, None))
    names = [k for k, *_ in recorder.launches(call)]
    assert rcs == [0], recorder.lib.uw_last_error()
    return names


def test_the_gpu_tests_reach_every_kernel(recorder):
    runs = [(True, c, of_case(recorder, True, c)) for c in LINEAR] + [(False, c, of_case(recorder, False, c)) for c in GROUPED]
    kernels = [k for k in recorder.kernels() if k.split("<")[0] in OWN]
    assert len(kernels) > 50
    reached = {k for _, _, names in runs for k in names}
    assert not set(kernels) - reached, sorted(set(kernels) - reached)
    tiles = [k for k in kernels if k.startswith("tile_kernel<false")]
    pairs = [k for k in kernels if k.startswith("tile_kernel<true")]
    assert len(tiles) == 4 and len(pairs) == 3
    chains = {(linear, *names) for linear, _, names in runs}
    for t in tiles:
        assert (True, t, "sums_epilogue_kernel") in chains, f"slices of K: {t}"
        assert (True, "expand_kernel", t) in chains and (False, "expand_kernel", t) in chains, f"expanded: {t}"
        assert (True, "expand_kernel", t, "sums_epilogue_kernel") in chains, f"expanded, slices of K: {t}"
    for t in pairs:
        assert (False, "expand_kernel", "expand_kernel", t) in chains, f"expanded: {t}"
    assert len({c[1] for c in chains if c[1].startswith("lds_gemm") and c[2] == "sums_epilogue_kernel"}) == 3
    # rows behind the last whole tile
    for expanded in ((), ("expand_kernel",)):
        for tail in ("gemv_rows_kernel", "skinny_kernel"):
            k = len(expanded)
            assert any(c[1:1 + k] == expanded and len(c) == 3 + k and c[1 + k] in tiles and c[2 + k].startswith(tail)
                       for c in chains), (expanded, tail)
    # tables of more than 64 groups of a row: reloaded by the palette tiles, in segments of a wave's K-slice by the skinny kernel
    long = {k for linear, c, names in runs for k in names if c[2 if linear else 4] > 4096}
    assert not [k for k in kernels if k.startswith("tile_pal_kernel") and k not in long]
    for pair in ("false", "true"):
        assert any(k.startswith(f"skinny_kernel<true, {pair}") and c[2 if linear else 4] // 128 // int(k[:-1].split()[-1]) > 32
                   and c[2 if linear else 4] % 128 for linear, c, names in runs for k in names), pair
