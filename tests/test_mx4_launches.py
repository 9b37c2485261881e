"""What the calls of the microscaled 4-bit operators and of the scored router
launch, seen from the host (tests/launch_util.py): no GPU."""
import ctypes as ct

from mlp_matmul_amd import _capi
from tests.mx4_cases import GROUPED, LINEAR, ROUTES
from tests.test_experts_launches import at, recorder  # noqa: F401


def matrix(i, rows, cols):
    return ct.byref(_capi.uw_mx4(rows, cols, at(i), at(i + 1), (cols // 2 + 15) // 16 * 16, (cols // 32 + 15) // 16 * 16))


def of_case(recorder, linear, case):  # noqa: F811
    """The kernels that a case of tests/mx4_cases.py launches, in order."""
    L, rcs = recorder.lib, []
    if linear:
        x4, rows, cols, n = case
        pair, experts = 0, 1
    else:
        x4, pair, experts, rows, cols, n = case
    X, x = (None, matrix(5, n, cols)) if x4 else (at(5), None)
    w = matrix(1, experts * rows, cols)
    if linear:
        call = lambda: rcs.append(L.uw_mx4_linear(w, X, cols, x, n, None, 0, 0, None, 0, 0, at(9), 0, rows, None))  # noqa: E731
    elif pair:
        call = lambda: rcs.append(L.uw_mx4_gate_up(w, matrix(3, experts * rows, cols), experts, X, n, cols, x, at(7), None,  # noqa: E731
                                                   1, n, at(9), rows, None))
    else:
        call = lambda: rcs.append(L.uw_mx4_gemm_grouped(w, experts, X, n, cols, x, at(7), None, 1, n, at(9), 0, rows, None))  # noqa: E731
    names = [k for k, *_ in recorder.launches(call)]
    assert rcs == [0], recorder.lib.uw_last_error()
    return names


def test_the_gpu_tests_reach_every_product(recorder):  # noqa: F811
    runs = [(True, c, of_case(recorder, True, c)) for c in LINEAR] + [(False, c, of_case(recorder, False, c)) for c in GROUPED]
    kernels = [k for k in recorder.kernels() if k.startswith(("mx4_skinny", "mx4_tile"))]
    assert len(kernels) == 50
    reached = {k for _, _, names in runs for k in names}
    assert not set(kernels) - reached, sorted(set(kernels) - reached)
    # the single product on tiles, alone and by expert
    for linear in (True, False):
        single = {k for lin, _, names in runs if lin == linear for k in names}
        lost = [k for k in kernels if k.startswith("mx4_tile") and k.split(", ")[1] == "false" and k not in single]
        assert not lost, (linear, lost)
    # rows behind the last whole tile
    chains = {tuple(names) for _, _, names in runs if len(names) > 1}
    for x4 in ("true", "false"):
        assert any(c[0].startswith(f"mx4_tile_kernel<{x4}") and c[1].startswith(f"mx4_skinny_kernel<{x4}") for c in chains), chains


def test_the_gpu_tests_reach_every_router(recorder):  # noqa: F811
    L = recorder.lib
    reached = set()
    for tokens, experts, top_k, groups, top_groups in ROUTES:
        rcs = []
        for k, *_ in recorder.launches(lambda: rcs.append(L.uw_moe_route_scored(
                at(1), 0, experts, tokens, experts, top_k, 1, at(8), groups, top_groups, 1, 1, 1.0, at(2), at(3), at(4), at(5),
                at(6), at(7), 1 << 30, None))):
            reached.add(k)
        assert rcs == [0], L.uw_last_error()
    kernels = [k for k in recorder.kernels() if k.startswith("route_kernel") and (k.endswith("true>") or k.startswith("route_kernel<2"))]
    assert len(kernels) >= 12
    assert not set(kernels) - reached, (sorted(set(kernels) - reached), reached)


def test_the_experts_are_three_products_and_a_sum(recorder):  # noqa: F811
    L = recorder.lib
    rcs = []
    names = [k for k, *_ in recorder.launches(lambda: rcs.append(L.uw_moe_experts(
        2, matrix(1, 4 * 64, 96), matrix(3, 4 * 64, 96), matrix(5, 4 * 96, 64), 4, 64, 96, at(7), 96, 20, 2, at(8), at(9),
        at(10), at(11), None, 0, 0, at(13), 1, 96, at(14), 1 << 24, None)))]
    assert rcs == [0] and len(names) == 3, (rcs, names)
    assert names[0].startswith("mx4_") and names[1].startswith("mx4_") and names[2].startswith("combine_kernel"), names


def test_one_token_sums_its_experts_in_one_kernel(recorder):  # noqa: F811
    """Where sums are not too long for the rows."""
    L = recorder.lib

    def names(rows, cols):
        rcs = []
        seen = recorder.launches(lambda: rcs.append(L.uw_moe_experts(
            2, matrix(1, 4 * rows, cols), matrix(3, 4 * rows, cols), matrix(5, 4 * cols, rows), 4, rows, cols, at(7), cols, 1, 2,
            at(8), at(9), at(10), at(11), None, 0, 0, at(13), 1, cols, at(14), 1 << 24, None)))
        assert rcs == [0], L.uw_last_error()
        return [k.split("<")[0] for k, *_ in seen]

    assert names(160, 64) == names(32, 96) == ["mx4_skinny_kernel", "mx4_one_kernel"]
    assert names(192, 64) == ["mx4_skinny_kernel", "mx4_skinny_kernel", "combine_kernel"]


def test_more_numbers_than_a_launch_takes(recorder):  # noqa: F811
    """2^32 - 1 eights of numbers a launch: the rest of the rows follow, where the first ones end."""
    L, rows, cols = recorder.lib, (1 << 21) + 5, 1 << 15
    rcs = []
    seen = recorder.launches(lambda: rcs.append(L.uw_mx4_quantize(1 << 40, 1, cols, rows, cols, 1 << 50, cols // 2, 1 << 55,
                                                                  cols // 32, None)), 72)
    assert rcs == [0] and [k for k, *_ in seen] == ["mx4_quantize_kernel<false>"] * 3
    at, left = 0, rows
    for _, grid, block, raw in seen:
        X, _, codes, scales, ld, ldc, lds = (int.from_bytes(raw[8 * i:8 * i + 8], "little") for i in range(7))
        eights, total = (int.from_bytes(raw[56 + 4 * i:60 + 4 * i], "little") for i in range(2))
        n = total // eights
        assert total == n * eights and eights == cols // 8 and grid[0] * block[0] * 4 >= total
        assert (X, codes, scales) == ((1 << 40) + at * cols * 2, (1 << 50) + at * cols // 2, (1 << 55) + at * cols // 32)
        assert (ld, ldc, lds) == (cols, cols // 2, cols // 32)
        at, left = at + n, left - n
    assert left == 0
