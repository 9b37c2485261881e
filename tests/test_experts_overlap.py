"""Scratch and outputs that lie in what a call reads are refused before any
launch: placeholder device pointers, no GPU."""
import ctypes as ct

import mlp_matmul_amd as uw
from mlp_matmul_amd import _capi
from tests.test_experts_launches import dmat, info_of
from tests.test_experts_refusals import at, combine, gate_up, grouped, layer, linear, route


class _Library:
    lib = uw.lib()


def planes(rows, cols, verbatim=40):
    """A descriptor of placeholder sections, and {section: (address, bytes)}."""
    d = dmat(_Library, info_of(rows, cols, verbatim))
    n = rows * cols
    sizes = {"sm": n, "nib": n // 2, "vexp": 64 * verbatim, "bitmap": 8 * d.tiles, "tile_vbase": 4 * (d.tiles + 1)}
    return d, {k: (at(20 + _capi.SECTION_NAMES.index(k)), v) for k, v in sizes.items()}


def inside(address, size):
    """Its first 16 bytes and those that hold its last byte."""
    return address, address + (size - 1) // 16 * 16


def test_scratch_in_an_input():
    def refused(f, address, size, **kw):
        for p in inside(address, size):
            assert f(**{"scratch": p, "sb": 16, **kw}) == _capi.UW_EINVAL, (f.__name__, hex(address), size)
            assert b"scratch overlaps" in uw.lib().uw_last_error()

    # weights [128, 256] and experts' [4, 64, 128] (down [4, 128, 64]) in bf16
    refused(linear, at(1), 128 * 256 * 2)
    refused(grouped, at(1), 4 * 64 * 128 * 2)
    for i in (1, 2):
        refused(gate_up, at(i), 4 * 64 * 128 * 2)
    # the groups: offsets of 4 experts, an order of 40 rows
    refused(grouped, at(3), 5 * 4)
    refused(grouped, at(4), 40 * 4)
    refused(gate_up, at(4), 5 * 4)
    refused(gate_up, at(5), 40 * 4)
    # a layer's needs its scratch whole: it ends behind the input's first bytes, or starts in its last ones
    need = uw.lib().uw_moe_scratch_bytes(0, 20, 4, 2, 64, 128)
    for i, size in ((1, 4 * 64 * 128 * 2), (2, 4 * 64 * 128 * 2), (3, 4 * 64 * 128 * 2), (4, 20 * 128 * 2), (5, 20 * 4 * 4)):
        for p in (at(i) + 16 - need, inside(at(i), size)[1]):
            assert layer(scratch=p, sb=need) == _capi.UW_EINVAL, i
            assert b"scratch overlaps" in uw.lib().uw_last_error()
    # compressed weights: every section
    d, sections = planes(256, 128)
    for address, size in sections.values():
        refused(grouped, address, size, w=None, d=ct.byref(d))
        refused(gate_up, address, size, gw=None, gd=ct.byref(d), uw_=None, ud=ct.byref(d))
    d, sections = planes(128, 256)
    for address, size in sections.values():
        refused(linear, address, size, w=None, d=ct.byref(d))


def test_out_in_an_input():
    def refused(f, address, size, out="out", **kw):
        for p in inside(address, size):
            assert f(**{out: p, **kw}) == _capi.UW_EINVAL, (f.__name__, hex(address), size)
            assert b"out overlaps" in uw.lib().uw_last_error()

    refused(linear, at(1), 128 * 256 * 2)
    refused(linear, at(2), 4 * 256 * 2)
    refused(linear, at(3), 128 * 4)
    refused(grouped, at(1), 4 * 64 * 128 * 2)
    refused(grouped, at(2), 20 * 128 * 2)
    refused(grouped, at(3), 5 * 4)
    refused(grouped, at(4), 40 * 4)
    for i, size in ((1, 4 * 64 * 128 * 2), (2, 4 * 64 * 128 * 2), (3, 20 * 128 * 2), (4, 5 * 4), (5, 40 * 4)):
        refused(gate_up, at(i), size, "h")
    refused(combine, at(1), 40 * 64 * 4)
    refused(combine, at(2), 20 * 2 * 4)
    refused(combine, at(3), 20 * 2 * 4)
    for i in (1, 2, 3):
        refused(layer, at(i), 4 * 64 * 128 * 2)
    d, sections = planes(256, 128)
    for address, size in sections.values():
        refused(grouped, address, size, w=None, d=ct.byref(d))
        refused(gate_up, address, size, "h", gw=None, gd=ct.byref(d), uw_=None, ud=ct.byref(d))


def test_routing_outputs_share_nothing():
    slots, offsets = 100 * 2 * 4, 9 * 4
    need = uw.lib().uw_moe_route_scratch_bytes(100, 8, 2)
    spans = {"ids": (at(2), slots), "weights": (at(3), slots), "off": (at(4), offsets), "order": (at(5), slots),
             "place": (at(6), slots), "scratch": (at(7), need)}
    for name, (_, size) in spans.items():
        for other, (address, length) in {**spans, "logits": (at(1), 100 * 8 * 4)}.items():
            if other != name:
                # over its last bytes, and ending in its first ones
                for p in (inside(address, length)[1], address + 16 - -(-size // 16) * 16):
                    assert route(**{name: p}) == _capi.UW_EINVAL, (name, other)
                    assert b"overlaps" in uw.lib().uw_last_error()


def test_layer_scratch_of_matrices_that_no_call_takes():
    """2^31 weights or more in a matrix: an error code, as the layer itself gives, and no wrapped size."""
    for rows, cols in ((1 << 16, 1 << 15), (64, (1 << 31) - 64), ((1 << 31) - 64, (1 << 31) - 64)):
        for tokens in (1, (1 << 31) - 1):
            assert uw.lib().uw_moe_scratch_bytes(0, tokens, 8, 1, rows, cols) == _capi.UW_EUNSUPPORTED, (rows, cols)
    assert uw.lib().uw_moe_scratch_bytes(0, (1 << 31) - 1, 8, 1, 64, (1 << 25) - 64) > 1 << 57
