"""What the C entries of the epilogue matmul and of the mixture-of-experts
operators refuse before any launch: placeholder device pointers, no GPU."""
import ctypes as ct

import numpy as np
import pytest

import mlp_matmul_amd as uw
import workloads
from mlp_matmul_amd import _capi

P = 0x1000000          # placeholder device addresses, far apart
BIG = 1 << 32


def at(i):
    return P + i * BIG


def linear(**kw):
    a = dict(w=at(1), d=None, rows=128, cols=256, X=at(2), ldx=256, batch=4, bias=at(3), bt=0, act=0, res=at(4), rt=0,
             ldr=128, out=at(5), ot=0, ldo=128, scratch=None, sb=0, stream=None)
    a.update(kw)
    return uw.lib().uw_linear(*a.values())


def route(**kw):
    a = dict(logits=at(1), lt=0, ld=8, tokens=100, experts=8, top_k=2, renorm=1, ids=at(2), weights=at(3), off=at(4),
             order=at(5), place=at(6), scratch=at(7), sb=1 << 20, stream=None)
    a.update(kw)
    return uw.lib().uw_moe_route(*a.values())


def grouped(**kw):
    a = dict(w=at(1), d=None, experts=4, rows=64, cols=128, X=at(2), xr=20, ldx=128, off=at(3), order=at(4), top_k=2,
             n=40, out=at(5), ot=0, ldo=64, scratch=None, sb=0, stream=None)
    a.update(kw)
    return uw.lib().uw_gemm_grouped(*a.values())


def gate_up(**kw):
    a = dict(gw=at(1), gd=None, uw_=at(2), ud=None, experts=4, rows=64, cols=128, X=at(3), xr=20, ldx=128, off=at(4),
             order=at(5), top_k=2, n=40, h=at(6), ldh=64, scratch=None, sb=0, stream=None)
    a.update(kw)
    return uw.lib().uw_moe_gate_up(*a.values())


def combine(**kw):
    a = dict(Y=at(1), n=40, cols=64, place=at(2), weights=at(3), tokens=20, top_k=2, res=at(4), rt=1, ldr=64,
             out=at(5), ot=1, ldo=64, stream=None)
    a.update(kw)
    return uw.lib().uw_moe_combine(*a.values())


def layer(**kw):
    a = dict(gw=at(1), gd=None, uw_=at(2), ud=None, dw=at(3), dd=None, experts=4, rows=64, cols=128, X=at(4), ldx=128,
             tokens=20, logits=at(5), lt=0, ldl=4, top_k=2, renorm=1, res=at(6), rt=1, ldr=128, out=at(7), ot=1,
             ldo=128, scratch=at(8), sb=1 << 28, stream=None)
    a.update(kw)
    return uw.lib().uw_moe_layer(*a.values())


BAD = {
    linear: [dict(w=None), dict(w=at(1) + 2), dict(cols=100), dict(cols=0), dict(rows=-1), dict(batch=-1),
             dict(ldx=255), dict(ldx=260), dict(X=None), dict(X=at(2) + 4), dict(bt=2), dict(bias=at(3) + 2),
             dict(act=5), dict(act=-1), dict(rt=7), dict(ldr=127), dict(ot=2), dict(out=None), dict(out=at(5) + 4),
             dict(ldo=127), dict(scratch=at(9) + 4, sb=64), dict(scratch=at(5), sb=1 << 20), dict(out=at(2) + 256), dict(out=at(3)), dict(out=at(4) + 16), dict(out=at(4), ot=1),
             dict(out=at(4), ldo=130), dict(batch=1 << 31)],
    route: [dict(tokens=-1), dict(experts=0), dict(experts=513), dict(top_k=0), dict(top_k=9), dict(lt=3),
            dict(ld=7), dict(logits=None), dict(ids=None), dict(weights=at(3) + 4), dict(off=None), dict(order=None),
            dict(place=None), dict(scratch=None), dict(sb=16), dict(scratch=at(7) + 8), dict(experts=40, ld=40, top_k=17),
            dict(tokens=1 << 30)],
    grouped: [dict(w=None), dict(experts=0), dict(experts=513), dict(n=-1), dict(off=None), dict(off=at(3) + 4),
              dict(order=at(4) + 4), dict(top_k=0), dict(xr=0), dict(xr=39, order=None), dict(ldx=120), dict(ldx=132),
              dict(cols=96), dict(out=None), dict(ldo=63), dict(ot=4), dict(out=at(2)), dict(n=1 << 31)],
    gate_up: [dict(gw=None), dict(uw_=None), dict(h=None), dict(h=at(6) + 8), dict(ldh=60), dict(h=at(3)),
              dict(experts=-3), dict(cols=32), dict(X=None)],
    combine: [dict(Y=None), dict(place=None), dict(weights=None), dict(top_k=0), dict(top_k=17), dict(n=-1),
              dict(out=at(1)), dict(rt=2), dict(ot=-1), dict(ldo=63), dict(res=at(5) + 16), dict(tokens=-1)],
    layer: [dict(gw=None), dict(uw_=None), dict(dw=None), dict(rows=0), dict(rows=96), dict(cols=0), dict(X=None),
            dict(ldx=130), dict(logits=None), dict(ldl=3), dict(lt=2), dict(top_k=5), dict(scratch=None), dict(sb=100),
            dict(scratch=at(8) + 8), dict(out=None), dict(ldo=100), dict(out=at(8)), dict(tokens=-5), dict(experts=600)],
}


@pytest.mark.parametrize("call", list(BAD), ids=lambda f: f.__name__)
def test_refused(call):
    for kw in BAD[call]:
        assert call(**kw) == _capi.UW_EINVAL, (call.__name__, kw, uw.lib().uw_last_error())
        assert uw.lib().uw_last_error()


def test_nothing_to_do():
    """Empty calls succeed without reading a pointer."""
    assert linear(batch=0, X=None, out=None) == 0
    assert linear(rows=0, w=None) == 0
    assert grouped(n=0, off=None, X=None, out=None) == 0
    assert grouped(rows=0, w=None) == 0
    assert gate_up(n=0, off=None, X=None, h=None) == 0
    assert combine(tokens=0, place=None, out=None) == 0
    assert layer(tokens=0, X=None, logits=None, out=None, scratch=None) == 0


def test_too_large():
    assert linear(rows=1 << 20, cols=1 << 11) == _capi.UW_EUNSUPPORTED
    assert grouped(rows=1 << 16, cols=1 << 15) == _capi.UW_EUNSUPPORTED


def test_compressed_weights():
    """A descriptor of another shape or without its sections, and both forms at once, are refused."""
    b = uw.compress(workloads.gaussian_weights(np.random.default_rng(1), 256, 128, 0.02, 0.01, 1.0))
    inf = b.info()

    def dmat(drop=(), **over):
        ptrs = (ct.c_void_p * _capi.UW_NUM_SECTIONS)()
        for i, name in enumerate(_capi.SECTION_NAMES):
            if name not in drop:
                ptrs[i] = at(20 + i) + over.pop(name, 0)
        d = _capi.uw_dmat()
        assert uw.lib().uw_dmat_init(ct.byref(d), ct.byref(inf), ptrs) == 0
        for k, v in over.items():
            setattr(d, k, v)
        return d

    for kw in (dict(rows=64, cols=256), dict(rows=32), dict(w=at(1))):
        assert grouped(**{"w": None, "d": ct.byref(dmat()), **kw}) == _capi.UW_EINVAL, kw
    for drop in ("nib", "sm", "bitmap", "tile_vbase", "vexp"):
        assert grouped(w=None, d=ct.byref(dmat(drop=(drop,)))) == _capi.UW_EINVAL, drop
    assert grouped(w=None, d=ct.byref(dmat(nib=8))) == _capi.UW_EINVAL
    assert grouped(w=None, d=ct.byref(dmat(groups=3))) == _capi.UW_EINVAL
    assert gate_up(gw=None, gd=ct.byref(dmat())) == _capi.UW_EINVAL
    assert b"both" in uw.lib().uw_last_error()


def test_scratch_sizes():
    L = uw.lib()
    assert L.uw_moe_route_scratch_bytes(64, 256, 8) == 0
    assert L.uw_moe_route_scratch_bytes(65, 256, 8) == 5 * 256 * 2
    assert L.uw_moe_route_scratch_bytes(1 << 24, 16, 8) == 8448          # 257 blocks of 32 bytes, up to 256
    assert L.uw_moe_route_scratch_bytes(1, 0, 1) == _capi.UW_EINVAL
    assert L.uw_moe_scratch_bytes(0, 3, 8, 2, 64, 128) == 256 * 5 + 6 * 64 * 2 + 6 * 128 * 4
    assert L.uw_moe_scratch_bytes(0, 3, 8, 2, 60, 128) == _capi.UW_EINVAL
    assert L.uw_moe_scratch_bytes(1, 3, 8, 2, 64, 128) == L.uw_moe_scratch_bytes(0, 3, 8, 2, 64, 128)
    assert (L.uw_moe_scratch_bytes(1, 9000, 2, 1, 1024, 2048) ==
            L.uw_moe_scratch_bytes(0, 9000, 2, 1, 1024, 2048) + 2 * 2 * 1024 * 2048 * 2)
    assert L.uw_grouped_scratch_bytes(1, 1, 4, 1024, 2048, 20 * 4) == 0
    assert L.uw_grouped_scratch_bytes(1, 1, 4, 1024, 2048, 5000 * 4) == 2 * 4 * 1024 * 2048 * 2
    assert L.uw_grouped_scratch_bytes(1, 0, 4, 1024, 2048, 5000 * 4) == 4 * 1024 * 2048 * 2
    assert L.uw_grouped_scratch_bytes(0, 1, 4, 1024, 2048, 5000 * 4) == 0
    assert L.uw_grouped_scratch_bytes(1, 0, 0, 64, 128, 5) == _capi.UW_EINVAL
    assert L.uw_grouped_scratch_bytes(1, 0, 4, 64, 100, 5) == _capi.UW_EINVAL
    assert L.uw_grouped_scratch_bytes(1, 0, 4, 1 << 20, 1 << 11, 5) == _capi.UW_EUNSUPPORTED
    assert L.uw_linear_scratch_bytes(1, 64, 100, 4) == _capi.UW_EINVAL
    assert L.uw_linear_scratch_bytes(1, 1 << 20, 1 << 11, 4) == _capi.UW_EUNSUPPORTED
    assert L.uw_linear_scratch_bytes(1, 4096, 4096, 2) == 0
    assert L.uw_linear_scratch_bytes(0, 4096, 4096, 2) == 0
    assert L.uw_linear_scratch_bytes(0, 8192, 8192, 8192) == 0
    assert L.uw_linear_scratch_bytes(1, 8192, 8192, 8192) == 2 * 8192 * 8192
    assert L.uw_linear_scratch_bytes(0, 4096, 14336, 64) % (64 * 4096 * 4) == 0
    assert L.uw_linear_scratch_bytes(0, 4096, 14336, 64) > 0


def test_scratch_refusals():
    """Scratch that is misaligned or lies in an input or the output."""
    for f, x, out in ((linear, 2, 5), (grouped, 2, 5), (gate_up, 3, 6)):
        for kw in (dict(scratch=at(9) + 8, sb=1 << 10), dict(scratch=at(x), sb=1 << 10), dict(scratch=at(out), sb=1 << 10)):
            assert f(**kw) == _capi.UW_EINVAL, (f, kw)
            assert b"scratch" in uw.lib().uw_last_error()
    assert linear(scratch=at(3), sb=16) == linear(scratch=at(4), sb=16) == _capi.UW_EINVAL


def test_from_sections_refusals():
    for args in ((64, 100, b"", 0, {}), (-1, 64, b"", 0, {}), (64, 64, b"x" * 17, 0, {}), (64, 64, b"", 65, {}),
                 (64, 64, b"", 0, {"huff": None}), (64, 64, b"", 0, {})):
        with pytest.raises(ValueError):
            uw.DeviceMatrix.from_sections(*args)
