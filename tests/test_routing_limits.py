"""Sizes beside what a launch can hold: a grid has fewer than 2^32 threads, and
a call that needs more is refused before anything is enqueued (no GPU needed:
a misaligned pointer ends the calls that fit)."""
import ctypes
import os

import pytest

import fine_grained_block_e4m3_amd as fp8

OK, INVALID, SHAPE, ALIGN, UNSUP = range(5)
P = ctypes.c_void_p
A, ODD = P(4096), P(4097)
GRID = (2 ** 32 - 1) // 256          # workgroups of 256 threads


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fp8.LIB_PATH):
        from fine_grained_block_e4m3_amd import build
        build.build()
    return fp8.load_library()


def test_router(L):
    """Four rows a workgroup."""
    for T, want in ((4 * GRID, ALIGN), (4 * GRID + 1, UNSUP), ((1 << 31) - 1, UNSUP)):
        assert L.fp8_route_topk(A, T, 8, 2, 0, 1, 1.0, A, ODD, None) == want, T
        assert L.fp8_route_topk_grad(A, A, ODD, T, 8, 2, 0, 1, 1.0, A, None) == want, T


def test_moving_rows(L):
    """A wave per token and run of its row, and one per 8 rows that may be cleared; four waves a workgroup."""
    for T, rows, src, want in ((4 * GRID, 8, None, ALIGN), (4 * GRID + 1, 8, None, UNSUP), (4 * GRID - 1, 8, A, ALIGN),
                               (4 * GRID - 1, 9, A, UNSUP), (4 * GRID, 1, A, UNSUP)):
        assert L.fp8_expert_dispatch(A, ODD, src, A, T, 1, rows, 16, 1, None) == want, (T, rows)
    # runs of 2048 BF16 or 1024 FP32 elements
    for kind, run in ((1, 2048), (0, 1024)):
        for T, K, want in ((2 * GRID, 2 * run, ALIGN), (2 * GRID + 1, 2 * run, UNSUP), (2 * GRID, 2 * run + 1, UNSUP)):
            assert L.fp8_expert_dispatch(A, ODD, None, A, T, 1, 8, K, kind, None) == want, (T, K)
    # the combine's of half as many
    for kind, run in ((1, 1024), (0, 512)):
        for T, N, want in ((4 * GRID, run, ALIGN), (4 * GRID + 1, run, UNSUP), (4 * GRID, run + 1, UNSUP)):
            assert L.fp8_expert_combine(A, ODD, None, A, T, 1, 8, N, kind, None) == want, (T, N)


def test_quantizing_dispatch(L):
    """Runs of 1024, and workgroups in whole 8s."""
    most = 4 * (GRID // 8 * 8)
    for T, K, want in ((most, 1024, ALIGN), (most + 1, 1024, UNSUP), (most // 2, 1152, ALIGN), (most // 2 + 1, 1152, UNSUP)):
        assert L.fp8_expert_dispatch_quant(A, ODD, A, A, T, 1, 8, K, 1, 0, None) == want, (T, K)


def test_combine_gradient(L):
    """A workgroup per token, and one per 32 rows that may be cleared."""
    for T, rows, src, want in ((GRID, 8, None, ALIGN), (GRID + 1, 8, None, UNSUP), (GRID - 1, 32, A, ALIGN),
                               (GRID - 1, 33, A, UNSUP), (GRID, 1, A, UNSUP)):
        assert L.fp8_expert_combine_grad(A, A, ODD, None, src, A, A, T, 1, rows, 16, 1, None) == want, (T, rows)
    # without dy nothing is cleared
    assert L.fp8_expert_combine_grad(A, A, ODD, None, A, None, A, GRID, 1, 1 << 30, 16, 1, None) == ALIGN


def test_adapters(L):
    """Tiles times parts of K or of N, of either kernel."""
    def plan(T, n, rows, N, K, R):
        return L.fp8_adapters_plan(T, n, rows, N, K, R, 256, ctypes.byref(fp8.AdaptersPlan()))
    # single tiles take parts of 1024 of N: 2^20 tiles are 16 times as many workgroups
    rows = 16 << 20
    assert plan(rows, 1 << 30, rows, 15 * 1024, 128, 8) == OK
    assert plan(rows, 1 << 30, rows, 16 * 1024, 128, 8) == UNSUP
    assert L.fp8_adapters_workspace_size(rows, 1 << 30, rows, 16 * 1024, 128, 8) == 0
    # groups of four: a part of N each, however wide
    assert plan(rows, 8, rows, 1 << 20, 128, 8) == OK
    with pytest.raises(fp8.Fp8GemmError):
        fp8.adapters_plan(rows, 1 << 30, 16 * 1024, 128, 8)
