"""What the entries of the microscaled 4-bit operators, of the scored router and
of the experts' part of a layer refuse before any launch, from C and from
Python: placeholder device pointers, no GPU."""
import ctypes as ct

import numpy as np
import pytest
import torch

import mlp_matmul_amd as uw
import workloads
from mlp_matmul_amd import _capi
from tests.test_experts_gradients import OnGpu
from tests.test_experts_launches import dmat, info_of
from tests.test_experts_overlap import inside
from tests.test_experts_refusals import at


class _Library:
    lib = uw.lib()


def matrix(i, rows, cols, **kw):
    """A descriptor with codes at place i and scales at i + 1."""
    a = dict(rows=rows, cols=cols, codes=at(i), scales=at(i + 1), ldc=(cols // 2 + 15) // 16 * 16,
             lds=(cols // 32 + 15) // 16 * 16)
    a.update(kw)
    return ct.byref(_capi.uw_mx4(*a.values()))


def quantize(**kw):
    a = dict(X=at(1), type=1, ldx=96, rows=20, cols=96, codes=at(2), ldc=48, scales=at(3), lds=16, stream=None)
    a.update(kw)
    return uw.lib().uw_mx4_quantize(*a.values())


def dequantize(**kw):
    a = dict(m=matrix(1, 20, 96), out=at(5), ot=0, ldo=96, stream=None)
    a.update(kw)
    return uw.lib().uw_mx4_dequantize(*a.values())


def linear(**kw):
    a = dict(w=matrix(1, 128, 96), X=at(5), ldx=96, x4=None, batch=4, bias=at(7), bt=0, act=0, res=at(8), rt=0, ldr=128,
             out=at(9), ot=0, ldo=128, stream=None)
    a.update(kw)
    return uw.lib().uw_mx4_linear(*a.values())


def linear4(**kw):
    return linear(**{"X": None, "x4": matrix(5, 4, 96), **kw})


def grouped(**kw):
    a = dict(w=matrix(1, 4 * 64, 96), experts=4, X=at(5), xr=20, ldx=96, x4=None, off=at(7), order=at(8), top_k=2, n=40,
             out=at(9), ot=0, ldo=64, stream=None)
    a.update(kw)
    return uw.lib().uw_mx4_gemm_grouped(*a.values())


def grouped4(**kw):
    return grouped(**{"X": None, "x4": matrix(5, 20, 96), **kw})


def gate_up(**kw):
    a = dict(g=matrix(1, 4 * 64, 96), u=matrix(3, 4 * 64, 96), experts=4, X=at(5), xr=20, ldx=96, x4=None, off=at(7),
             order=at(8), top_k=2, n=40, h=at(9), ldh=64, stream=None)
    a.update(kw)
    return uw.lib().uw_mx4_gate_up(*a.values())


def route(**kw):
    a = dict(logits=at(1), lt=0, ld=12, tokens=100, experts=12, top_k=2, score=1, bias=at(8), groups=4, top_groups=2,
             group_top=2, renorm=1, scale=1.0, ids=at(2), weights=at(3), off=at(4), order=at(5), place=at(6),
             scratch=at(7), sb=1 << 20, stream=None)
    a.update(kw)
    return uw.lib().uw_moe_route_scored(*a.values())


def experts(**kw):
    a = dict(form=2, g=matrix(1, 4 * 64, 96), u=matrix(3, 4 * 64, 96), d=matrix(5, 4 * 96, 64), experts=4, rows=64, cols=96,
             X=at(7), ldx=96, tokens=20, top_k=2, weights=at(8), off=at(9), order=at(10), place=at(11), res=at(12), rt=1,
             ldr=96, out=at(13), ot=1, ldo=96, scratch=at(14), sb=1 << 24, stream=None)
    a.update(kw)
    return uw.lib().uw_moe_experts(*a.values())


def bf16_experts(**kw):
    return experts(**{"form": 0, "g": at(1), "u": at(3), "d": at(5), "cols": 128, "ldx": 128, "ldr": 128, "ldo": 128, **kw})


MATRIX = [dict(codes=None), dict(codes=at(1) + 8), dict(scales=None), dict(scales=at(2) + 4), dict(ldc=32), dict(ldc=56),
          dict(ldc=1 << 40), dict(lds=0), dict(lds=24), dict(lds=1 << 40)]
ROWS4 = [dict(x4=matrix(5, 4, 96, **m)) for m in MATRIX]
BAD = {
    quantize: [dict(type=2), dict(rows=-1), dict(rows=1 << 31), dict(cols=-32), dict(cols=48), dict(cols=1 << 31),
               dict(X=None), dict(X=at(1) + 8), dict(ldx=88), dict(ldx=100), dict(type=0, ldx=98), dict(codes=None),
               dict(codes=at(2) + 4), dict(ldc=32), dict(ldc=56), dict(scales=None), dict(scales=at(3) + 8),
               dict(lds=8), dict(lds=0), dict(codes=at(1)), dict(scales=at(1) + 16), dict(scales=at(2) + 32),
               dict(ldx=1 << 40)],
    dequantize: [dict(m=None), dict(ot=2), dict(out=None), dict(out=at(5) + 8), dict(ldo=95), dict(out=at(1)),
                 dict(out=at(2)), dict(m=matrix(1, -1, 96)), dict(m=matrix(1, 20, 48)), dict(m=matrix(1, 1 << 31, 32))]
    + [dict(m=matrix(1, 20, 96, **m)) for m in MATRIX],
    linear: [dict(w=None), dict(w=matrix(1, -2, 96)), dict(w=matrix(1, 128, 0)), dict(w=matrix(1, 128, 80)),
             dict(batch=-1), dict(batch=1 << 31), dict(X=None), dict(X=at(5) + 4), dict(ldx=88), dict(ldx=100),
             dict(x4=matrix(5, 4, 96)), dict(bt=2), dict(bias=at(7) + 2), dict(act=5), dict(act=-1), dict(rt=7),
             dict(ldr=127), dict(res=at(8) + 8), dict(out=None), dict(out=at(9) + 4), dict(ot=2), dict(ldo=127),
             dict(out=at(1)), dict(out=at(2)), dict(out=at(5)), dict(out=at(7)), dict(out=at(8) + 16),
             dict(out=at(8), ot=1), dict(out=at(8), ldo=130)] + [dict(w=matrix(1, 128, 96, **m)) for m in MATRIX],
    linear4: [dict(X=at(20)), dict(x4=None), dict(x4=matrix(5, 5, 96)), dict(x4=matrix(5, 4, 64)), dict(out=at(5)),
              dict(out=at(6))] + ROWS4,
    grouped: [dict(w=None), dict(experts=0), dict(experts=513), dict(experts=3), dict(n=-1), dict(n=1 << 31), dict(off=None),
              dict(off=at(7) + 4), dict(order=at(8) + 4), dict(top_k=0), dict(xr=0), dict(xr=39, order=None), dict(xr=-1),
              dict(X=None), dict(ldx=88), dict(ldx=100), dict(w=matrix(1, 256, 80)), dict(out=None), dict(ldo=63), dict(ot=4),
              dict(out=at(1)), dict(out=at(2)), dict(out=at(5)), dict(out=at(7)), dict(out=at(8)),
              dict(x4=matrix(5, 20, 96))] + [dict(w=matrix(1, 256, 96, **m)) for m in MATRIX],
    grouped4: [dict(x4=matrix(5, 19, 96)), dict(x4=matrix(5, 20, 128)), dict(out=at(6)), dict(X=at(20))],
    gate_up: [dict(g=None), dict(u=None), dict(u=matrix(3, 4 * 32, 96)), dict(u=matrix(3, 4 * 64, 64)), dict(h=None),
              dict(h=at(9) + 8), dict(ldh=60), dict(h=at(3)), dict(h=at(4)), dict(h=at(7)), dict(experts=-3), dict(X=None),
              dict(x4=matrix(5, 20, 96)), dict(X=None, x4=matrix(5, 21, 96)), dict(off=None), dict(n=-1)]
    + [dict(g=matrix(1, 256, 96, **m)) for m in MATRIX],
    route: [dict(tokens=-1), dict(experts=0), dict(experts=513, ld=600), dict(top_k=0), dict(top_k=13), dict(lt=3),
            dict(ld=11), dict(logits=None), dict(ids=None), dict(weights=at(3) + 4), dict(off=None), dict(order=None),
            dict(place=None), dict(scratch=None), dict(sb=16), dict(scratch=at(7) + 8), dict(score=0), dict(score=3),
            dict(bias=at(8) + 4), dict(groups=0), dict(groups=17), dict(groups=5), dict(top_groups=0), dict(top_groups=5),
            dict(group_top=0), dict(group_top=3), dict(top_groups=1, top_k=4), dict(scale=float("nan")),
            dict(scale=float("inf")), dict(ids=at(1)), dict(weights=at(8)), dict(place=at(5)), dict(off=at(8)),
            dict(tokens=1 << 30)],
    experts: [dict(form=3), dict(form=-1), dict(g=None), dict(u=None), dict(d=None), dict(d=matrix(5, 4 * 64, 96)),
              dict(u=matrix(3, 4 * 64, 64)), dict(rows=0), dict(rows=48), dict(cols=0), dict(cols=80), dict(experts=0),
              dict(experts=513), dict(top_k=0), dict(top_k=5), dict(tokens=-1), dict(X=None), dict(ldx=88), dict(ldx=100),
              dict(weights=None), dict(off=None), dict(order=None), dict(place=None), dict(place=at(11) + 4), dict(rt=2),
              dict(ldr=95), dict(out=None), dict(ldo=95), dict(ot=2), dict(scratch=None), dict(sb=256),
              dict(scratch=at(14) + 8)] + [dict(out=at(i)) for i in (1, 2, 3, 4, 5, 6, 8, 9, 10, 11, 14)]
    + [dict(scratch=at(i)) for i in (1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12)],
    bf16_experts: [dict(g=None), dict(d=None), dict(u=at(3) + 2), dict(rows=96), dict(cols=96), dict(out=at(5)),
                   dict(scratch=at(3))],
}


@pytest.mark.parametrize("call", list(BAD), ids=lambda f: f.__name__)
def test_refused(call):
    for kw in BAD[call]:
        shown = {k: (v._obj.rows, v._obj.cols, v._obj.codes, v._obj.scales, v._obj.ldc, v._obj.lds) if hasattr(v, "_obj") else v
                 for k, v in kw.items()}
        assert call(**kw) == _capi.UW_EINVAL, (call.__name__, shown, uw.lib().uw_last_error())
        assert uw.lib().uw_last_error()


def test_nothing_to_do():
    """Empty calls succeed without reading a pointer."""
    none = dict(codes=None, scales=None)
    assert quantize(rows=0, X=None, codes=None, scales=None) == 0
    assert quantize(cols=0, X=None, codes=None, scales=None) == 0
    assert dequantize(m=matrix(1, 0, 96, **none), out=None) == 0
    assert dequantize(m=matrix(1, 20, 0, **none), out=None) == 0
    assert linear(batch=0, X=None, out=None) == linear4(batch=0, x4=None, out=None) == 0
    assert linear(w=matrix(1, 0, 96, **none), out=None) == 0
    assert grouped(n=0, off=None, X=None, out=None) == grouped4(n=0, off=None, x4=None, out=None) == 0
    assert grouped(w=matrix(1, 0, 96, **none), out=None) == 0
    assert gate_up(n=0, off=None, X=None, h=None) == 0
    assert experts(tokens=0, X=None, weights=None, off=None, order=None, place=None, out=None, scratch=None) == 0


def test_too_large():
    big = matrix(1, 1 << 20, 1 << 11)
    assert linear(w=big) == _capi.UW_EUNSUPPORTED
    assert grouped(w=matrix(1, 4 << 16, 1 << 15)) == _capi.UW_EUNSUPPORTED
    # rows so far apart that one matrix spans 2^31 bytes
    for far in (dict(ldc=1 << 24), dict(lds=1 << 24)):
        assert linear(w=matrix(1, 128, 96, **far)) == _capi.UW_EUNSUPPORTED
        assert gate_up(u=matrix(3, 256, 96, **{k: v << 1 for k, v in far.items()})) == _capi.UW_EUNSUPPORTED
    assert experts(rows=1 << 16, cols=1 << 15) == _capi.UW_EUNSUPPORTED


def test_out_and_scratch_in_an_input():
    """Over an input's first and last 16 bytes."""
    codes, scales = 128 * 48, 127 * 16 + 3
    for p in (*inside(at(1), codes), *inside(at(2), scales), *inside(at(5), 4 * 96 * 2), *inside(at(7), 128 * 4)):
        assert linear(out=p) == _capi.UW_EINVAL and b"overlaps" in uw.lib().uw_last_error()
    for p in (*inside(at(5), 4 * 48), *inside(at(6), 3 * 16 + 3)):
        assert linear4(out=p) == _capi.UW_EINVAL and b"overlaps" in uw.lib().uw_last_error()
    codes, scales = 256 * 48, 255 * 16 + 3
    for p in (*inside(at(1), codes), *inside(at(2), scales), *inside(at(3), codes), *inside(at(4), scales),
              *inside(at(5), 20 * 96 * 2), *inside(at(7), 5 * 4), *inside(at(8), 40 * 4)):
        assert gate_up(h=p) == _capi.UW_EINVAL and b"overlaps" in uw.lib().uw_last_error()
    need = uw.lib().uw_moe_experts_scratch_bytes(2, 20, 4, 2, 64, 96)
    for i, size in ((1, codes), (3, codes), (5, 4 * 96 * 32), (6, (4 * 96 - 1) * 16 + 2), (7, 20 * 96 * 2), (8, 160), (9, 20),
                    (10, 160), (11, 160), (12, 20 * 96 * 2)):
        for p in (at(i) + 16 - need, inside(at(i), size)[1]):
            assert experts(scratch=p, sb=need) == _capi.UW_EINVAL, i
            assert b"scratch overlaps" in uw.lib().uw_last_error()
    # every section of compressed weights
    d, u = (ct.byref(dmat(_Library, info_of(256, 128, 40))) for _ in range(2))
    down = ct.byref(dmat(_Library, info_of(512, 64, 40)))
    for name in ("nib", "sm", "vexp", "bitmap", "tile_vbase"):
        p = at(20 + _capi.SECTION_NAMES.index(name))
        kw = dict(form=1, g=d, u=u, d=down, cols=128, ldx=128, ldr=128, ldo=128)
        assert experts(**kw, out=p) == experts(**kw, scratch=p) == _capi.UW_EINVAL, name


def test_routing_outputs_share_nothing():
    slots, offsets, experts_ = 100 * 2 * 4, 13 * 4, 12
    need = uw.lib().uw_moe_route_scratch_bytes(100, experts_, 2)
    spans = {"ids": (at(2), slots), "weights": (at(3), slots), "off": (at(4), offsets), "order": (at(5), slots),
             "place": (at(6), slots), "scratch": (at(7), need)}
    read = {"logits": (at(1), 100 * 12 * 4), "bias": (at(8), 48)}
    for name, (_, size) in spans.items():
        for other, (address, length) in {**spans, **read}.items():
            if other != name:
                for p in (inside(address, length)[1], address + 16 - -(-size // 16) * 16):
                    assert route(**{name: p}) == _capi.UW_EINVAL, (name, other)
                    assert b"overlaps" in uw.lib().uw_last_error()


def test_scratch_sizes():
    L = uw.lib()
    assert L.uw_moe_experts_scratch_bytes(2, 3, 8, 2, 32, 96) == 6 * 32 * 2 + 128 + 6 * 96 * 4
    assert L.uw_moe_experts_scratch_bytes(0, 3, 8, 2, 64, 128) == 6 * 64 * 2 + 6 * 128 * 4
    assert L.uw_moe_experts_scratch_bytes(1, 3, 8, 2, 64, 128) == L.uw_moe_experts_scratch_bytes(0, 3, 8, 2, 64, 128)
    assert (L.uw_moe_experts_scratch_bytes(1, 9000, 2, 1, 1024, 2048) ==
            L.uw_moe_experts_scratch_bytes(0, 9000, 2, 1, 1024, 2048) + 2 * 2 * 1024 * 2048 * 2)
    assert L.uw_moe_experts_scratch_bytes(0, 3, 8, 2, 96, 128) == _capi.UW_EINVAL
    assert L.uw_moe_experts_scratch_bytes(3, 3, 8, 2, 64, 128) == _capi.UW_EINVAL
    assert L.uw_moe_experts_scratch_bytes(2, -1, 8, 2, 64, 128) == _capi.UW_EINVAL
    for form in range(3):
        assert L.uw_moe_experts_scratch_bytes(form, 1, 8, 1, 1 << 16, 1 << 15) == _capi.UW_EUNSUPPORTED


# ------------------------------------------------------------ from Python
def bytes_(rows, cols, stride=None):
    stride = stride or (cols + 15) // 16 * 16
    return torch.zeros(max(rows, 1) * stride + 16, dtype=torch.uint8).as_strided((rows, cols), (stride, 1))


def test_the_matrix():
    m = uw.Mx4Matrix(bytes_(5, 48), bytes_(5, 3))
    assert m.shape == (5, 96) and (m.mx4.ldc, m.mx4.lds) == (48, 16) and m.device_bytes() == 5 * 51
    one = uw.Mx4Matrix(bytes_(1, 16).contiguous(), bytes_(1, 1).contiguous())
    assert (one.mx4.ldc, one.mx4.lds) == (16, 16)
    good = bytes_(5, 48), bytes_(5, 3)
    for codes, scales in ((good[0].to(torch.int8), good[1]), (good[0], good[1].float()), (good[0][0], good[1]),
                          (good[0], bytes_(4, 3)), (good[0], bytes_(5, 2)), (bytes_(5, 40), good[1]),
                          (bytes_(5, 48, 56), good[1]), (good[0], bytes_(5, 3, 17)), (bytes_(48, 5, 16).t(), good[1]),
                          (bytes_(5, 64)[:, 8:56], good[1])):
        with pytest.raises(ValueError):
            uw.Mx4Matrix(codes, scales)


class Bf16(OnGpu):
    """A GPU tensor of any shape that is not there."""

    def __init__(self, *shape, dtype=torch.bfloat16, requires_grad=False):
        super().__init__(requires_grad)
        self.meta = torch.empty(shape, dtype=dtype, device="meta")

    def __getattr__(self, name):
        return getattr(self.meta, name)


@pytest.fixture
def on_gpu(monkeypatch):
    """Mx4Matrix objects and tensors as if they were on a GPU; no call reaches the library."""
    def no(*a):
        raise AssertionError("the library was called")

    monkeypatch.setattr(uw, "_elsewhere", lambda dev, stream: None)
    monkeypatch.setattr(uw, "lib", no)
    monkeypatch.setattr(uw, "_new_matrix", lambda rows, cols, dtype, dev: Bf16(rows, cols, dtype=dtype))

    def make(rows, cols):
        m = uw.Mx4Matrix(bytes_(rows, cols // 2), bytes_(rows, cols // 32))
        m.device = OnGpu.device
        return m
    return make


def test_python_refusals(on_gpu):
    W, X = on_gpu(128, 96), Bf16(4, 96)
    i32 = torch.int32
    off, order = Bf16(5, dtype=i32), Bf16(40, dtype=i32)
    with torch.no_grad():
        for call, match in (
                (lambda: uw.linear(W, Bf16(4, 64)), "X must be"),
                (lambda: uw.linear(W, on_gpu(4, 64)), "X must be"),
                (lambda: uw.linear(W, Bf16(4, 96, dtype=torch.float32)), "bfloat16"),
                (lambda: uw.linear(W, X, act="tanh"), "act must be"),
                (lambda: uw.linear(W, X, bias=Bf16(96)), "bias must be"),
                (lambda: uw.linear(W, X, residual=Bf16(4, 96)), "residual"),
                (lambda: uw.linear(Bf16(128, 96), on_gpu(4, 96)), "Mx4Matrix"),
                (lambda: uw.gemm_grouped(on_gpu(126, 96), X, off), "4 experts"),
                (lambda: uw.gemm_grouped(Bf16(4, 64, 96), on_gpu(40, 96), off), "Mx4Matrix"),
                (lambda: uw.moe_gate_up(W, Bf16(4, 32, 96), X, off, order, 2), "Mx4Matrix"),
                (lambda: uw.moe_gate_up(Bf16(4, 32, 64), W, Bf16(4, 64), off, order, 2), "Mx4Matrix"),
                (lambda: uw.moe_gate_up(W, on_gpu(128, 64), X, off, order, 2), "same shape"),
                (lambda: uw.moe_layer(W, W, on_gpu(384, 32), X, Bf16(4, 4), 2), "moe_experts"),
                (lambda: uw.moe_route_scored(Bf16(4, 8, dtype=torch.float32), 2, score="tanh"), "score must be"),
                (lambda: uw.moe_route_scored(Bf16(4, 8, dtype=torch.float32), 2, bias=Bf16(8)), "bias must be"),
                (lambda: uw.moe_route_scored(Bf16(4, 8, dtype=torch.float32), 2, bias=Bf16(7, dtype=torch.float32)), "bias must be"),
                (lambda: uw.moe_route_scored(Bf16(4, 8, dtype=torch.float16), 2), "float32 or bfloat16"),
                (lambda: uw.mx4_quantize(Bf16(4, 48)), "32 columns"),
                (lambda: uw.mx4_quantize(Bf16(4, 64, dtype=torch.float16)), "float32 or bfloat16"),
                (lambda: uw.mx4_quantize(X, out=on_gpu(4, 64)), "out must be"),
                (lambda: uw.mx4_quantize(on_gpu(4, 96)), "X"),
                (lambda: uw.mx4_dequantize(W, out_dtype=torch.float16), "float32 or bfloat16"),
                (lambda: uw.mx4_dequantize(X), "Mx4Matrix")):
            with pytest.raises(ValueError, match=match):
                call()


def test_a_matrix_in_the_place_of_a_tensor(on_gpu):
    """A 4-bit matrix where a call takes a tensor, and a tensor where it takes a 4-bit matrix to write, are refused as
    other arguments of a wrong type are."""
    W, X, M = on_gpu(128, 96), Bf16(4, 96), on_gpu(4, 128)
    f32, i32 = torch.float32, torch.int32
    off, order = Bf16(5, dtype=i32), Bf16(40, dtype=i32)
    D = uw.DeviceMatrix.__new__(uw.DeviceMatrix)
    D.info, D.buffers = uw.uw_info(rows=4, cols=96), {"nib": OnGpu()}
    with torch.no_grad():
        for call, match in (
                (lambda: uw.mx4_quantize(X, out=Bf16(4, 96)), "out must be an Mx4Matrix"),
                (lambda: uw.mx4_quantize(X, out=D), "out must be an Mx4Matrix"),
                (lambda: uw.mx4_quantize(D), "X"),
                (lambda: uw.mx4_dequantize(M, out=M), "out"),
                (lambda: uw.mx4_dequantize(M, out=M, out_dtype=f32), "out"),
                (lambda: uw.linear(W, X, out=M), "out"),
                (lambda: uw.linear(W, X, out=M, out_dtype=f32), "out"),
                (lambda: uw.linear(W, X, residual=M), "residual"),
                (lambda: uw.linear(W, X, residual=D), "residual"),
                (lambda: uw.linear(W, X, bias=M), "bias"),
                (lambda: uw.linear(W, D), "X"),
                (lambda: uw.gemm_grouped(W, X, off, order, 2, out=on_gpu(40, 32)), "out"),
                (lambda: uw.gemm_grouped(W, X, off, order, 2, out=on_gpu(40, 32), out_dtype=f32), "out"),
                (lambda: uw.moe_gate_up(W, W, X, off, order, 2, h=on_gpu(40, 32)), "out|h "),
                (lambda: uw.moe_combine(M, Bf16(4, 2, dtype=i32), Bf16(4, 2, dtype=f32)), "Y must be"),
                (lambda: uw.moe_combine(Bf16(8, 96, dtype=f32), Bf16(4, 2, dtype=i32), Bf16(4, 2, dtype=f32), residual=M),
                 "residual"),
                (lambda: uw.moe_route_scored(Bf16(4, 8, dtype=f32), 2, bias=M), "bias must be"),
                (lambda: uw.moe_route_scored(M, 2), "logits must be"),
                (lambda: uw.moe_route(M, 2), "logits must be"),
                (lambda: uw.moe_layer(Bf16(4, 32, 64), W, Bf16(4, 64, 32), Bf16(4, 64), Bf16(4, 4), 2), "up is an Mx4Matrix"),
                (lambda: uw.moe_layer(Bf16(4, 32, 64), Bf16(4, 32, 64), W, Bf16(4, 64), Bf16(4, 4), 2), "down is an Mx4Matrix"),
                (lambda: uw.moe_layer(Bf16(4, 32, 64), Bf16(4, 32, 64), Bf16(4, 64, 32), Bf16(4, 64), M, 2), "logits must be")):
            with pytest.raises(ValueError, match=match):
                call()


def test_moe_experts_refusals(on_gpu):
    i32 = torch.int32

    def routing(tokens=20, top_k=2, experts_=4, **kw):
        a = dict(ids=Bf16(tokens, top_k, dtype=i32), weights=Bf16(tokens, top_k, dtype=torch.float32),
                 offsets=Bf16(experts_ + 1, dtype=i32), order=Bf16(tokens * top_k, dtype=i32), place=Bf16(tokens, top_k, dtype=i32))
        a.update(kw)
        return uw.Routing(**a)

    W, D, X = on_gpu(4 * 64, 96), on_gpu(4 * 96, 64), Bf16(20, 96)
    with torch.no_grad():
        for args, match in (
                ((W, W, W, X, routing()), "gate and up must be"),
                ((W, on_gpu(4 * 64, 64), D, X, routing()), "gate and up must be"),
                ((W, W, Bf16(4, 96, 64), X, routing()), "Mx4Matrix"),
                ((Bf16(4, 64, 128), W, D, X, routing()), "Mx4Matrix"),
                ((W, W, D, Bf16(20, 128), routing()), "X must be"),
                ((W, W, D, Bf16(19, 96), routing()), "place must be"),
                ((W, W, D, on_gpu(20, 96), routing()), "bfloat16"),
                ((W, W, D, X, routing(weights=Bf16(20, 2))), "weights must be"),
                ((W, W, D, X, routing(weights=Bf16(20, 3, dtype=torch.float32))), "weights must be"),
                ((W, W, D, X, routing(order=Bf16(39, dtype=i32))), "order must be"),
                ((W, W, D, X, routing(offsets=Bf16(1, dtype=i32))), "offsets"),
                ((W, W, D, X, routing(place=Bf16(20, 2, dtype=torch.int64))), "place must be"),
                ((on_gpu(4 * 64 + 1, 96), W, D, X, routing()), "4 experts")):
            with pytest.raises(ValueError, match=match):
                uw.moe_experts(*args)


CALLS = {
    uw.mx4_quantize: ("X",),
    uw.moe_route_scored: ("logits", "bias"),
    uw.moe_experts: ("gate", "up", "down", "X", "residual", "out"),
}


@pytest.mark.parametrize("call", list(CALLS), ids=lambda f: f.__name__)
def test_gradients_are_refused(call, monkeypatch):
    class Past(Exception):
        pass

    def past(*a):
        raise Past
    monkeypatch.setattr(uw, "_elsewhere", past)              # what follows the checks of the tensors
    extra = {"top_k": 2} if call is uw.moe_route_scored else {}
    if call is uw.moe_experts:
        extra["routing"] = uw.Routing(*(OnGpu() for _ in range(5)))
    for name in CALLS[call]:
        tensors = {n: OnGpu(n == name) for n in CALLS[call]}
        with pytest.raises(ValueError, match="gradient"):
            call(**tensors, **extra)
        with torch.no_grad(), pytest.raises(Past):
            call(**tensors, **extra)
    if call is uw.moe_experts:
        with pytest.raises(ValueError, match="gradient"):
            call(**{n: OnGpu() for n in CALLS[call]}, routing=uw.Routing(OnGpu(), OnGpu(True), *(OnGpu() for _ in range(3))))
    with pytest.raises(ValueError, match="on a GPU"):
        uw.mx4_dequantize(uw.Mx4Matrix(bytes_(5, 48), bytes_(5, 3)))


def test_reference_of_the_format():
    """The plain definition that the GPU tests compare with, on a matrix of a compressed weight's numbers: values are
    the nearest of the block's grid, and dequantised numbers quantise to themselves."""
    from tests.mx4_util import GRID, quantize_ref, values_ref
    w = workloads.gaussian_weights(np.random.default_rng(2), 8, 96, 0.02, 0.01, 1.0)
    x = torch.from_numpy(w.view(np.int16)).view(torch.bfloat16)
    codes, scales = quantize_ref(x)
    v = values_ref(codes, scales)
    f = torch.ldexp(torch.ones(scales.shape, dtype=torch.float64), scales.long() - 127).repeat_interleave(32, 1)
    off = (x.double() - v).abs() / f
    best = ((x.double() / f).abs()[..., None] - GRID).abs().amin(-1)
    assert torch.equal(off, best)
    again = quantize_ref(v.float())
    assert torch.equal(values_ref(*again), v)
