"""Host-side checks of clipping's sizes (no GPU needed)."""
import ctypes

import pytest

import fine_grained_block_e4m3_amd as fp8

UNSUP, SCRATCH = 4, 7


def _call(sizes, ws_bytes=1 << 40):
    n = len(sizes)
    ptrs, types = (ctypes.c_void_p * n)(*[4096] * n), (ctypes.c_int32 * n)(*[0] * n)
    a = ctypes.c_void_p(4096)
    return fp8.load_library().fp8_clip_grad_norm(ptrs, ptrs, (ctypes.c_int64 * n)(*sizes), types, n, 1.0, a, a,
                                                 ws_bytes, None)


def _size(sizes):
    return fp8.load_library().fp8_clip_workspace_size((ctypes.c_int64 * len(sizes))(*sizes), len(sizes))


@pytest.mark.parametrize("large", [1 << 44, (1 << 61) + 5, (1 << 63) - 1])
@pytest.mark.parametrize("at", [0, 130, 249])
def test_too_many_elements_are_refused_before_any_launch(large, at):
    """Also where the tensors before them would fill whole launches."""
    sizes = [8192 * 3] * 250
    sizes[at] = large
    assert _call(sizes) == UNSUP and _size(sizes) == 0


def test_a_batch_of_too_many_elements():
    sizes = [100] * 130 + [1 << 43, 1 << 43, 5]
    assert _call(sizes) == UNSUP and _size(sizes) == 0


def test_workspace_size():
    assert _size([1, 0, 20000]) == 8 * 4
    assert _size([0, 0]) == 8
    assert _size([8192] * 250) == 8 * 250
    assert _size([1 << 43]) == 8 * 2048
    assert _call([1 << 43], 8 * 2048 - 1) == SCRATCH
