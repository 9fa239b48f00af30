"""Host-side checks of the feed-forward entry points (no GPU needed): bad
arguments are refused before any device call."""
import ctypes
import os

import pytest

import fine_grained_block_e4m3_amd as fp8

OK, INVALID, SHAPE, ALIGN, UNSUP, NODEV, LAUNCH, SCRATCH = range(8)
P = ctypes.c_void_p
A = P(4096)
MIS = P(4100)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fp8.LIB_PATH):
        from fine_grained_block_e4m3_amd import build
        build.build()
    return fp8.load_library()


def test_gated_validation(L):
    def call(xq=A, h=A, g=None, u=None, M=4, N=8, K=128, act=0, flags=0, ws=None, ws_bytes=0):
        return L.fp8_gated_nt(xq, A, A, A, A, A, h, g, u, M, N, K, act, flags, ws, ws_bytes, None)
    assert call(xq=None) == INVALID
    assert call(h=None) == INVALID
    assert call(g=A) == INVALID              # g without u
    assert call(act=2) == INVALID
    assert call(act=-1) == INVALID
    assert call(flags=fp8.FLAG_FAST_ACCUM) == INVALID
    assert call(M=-1) == INVALID
    assert call(N=1 << 31) == INVALID
    assert call(ws_bytes=16) == INVALID
    assert call(K=100) == SHAPE
    assert call(K=0) == SHAPE
    assert call(K=(1 << 22) + 128) == UNSUP
    assert call(xq=MIS) == ALIGN
    assert call(g=MIS, u=A) == ALIGN
    assert call(M=0, xq=None) == OK
    assert call(N=0) == OK


def test_gated_quantized_validation(L):
    def call(hq=A, sh=A, M=4, N=128, K=128, act=1, flags=1):
        return L.fp8_gated_nt_qout(A, A, A, A, A, A, hq, sh, M, N, K, act, flags, None, 0, None)
    assert call(N=100) == SHAPE
    assert call(K=64) == SHAPE
    assert call(hq=None) == INVALID
    assert call(sh=MIS) == ALIGN
    assert call(flags=4) == INVALID
    assert call(M=0, hq=None) == OK
    assert L.fp8_gated_workspace_size(4, 8, 100, 0) == 0
    assert L.fp8_gated_workspace_size(4, 8, 128, 3) == 0
    assert L.fp8_gated_workspace_size(-1, 8, 128, 0) == 0


def test_grad_validation(L):
    def call(dh=A, x=A, wg=A, dx=A, dwg=A, dwu=A, M=4, N=8, K=128, act=0, ws=None, ws_bytes=0):
        return L.fp8_gated_nt_grad(dh, A, A, x, wg, A, dx, dwg, dwu, M, N, K, act, ws, ws_bytes, None)
    assert call(dh=None) == INVALID
    assert call(x=None) == INVALID
    assert call(wg=None) == INVALID
    assert call(dwu=None) == INVALID         # one weight gradient without the other
    assert call(act=7) == INVALID
    assert call(ws_bytes=1) == INVALID
    assert call(K=130) == SHAPE
    assert call(N=1 << 22) == UNSUP
    assert call(dx=P(4098)) == ALIGN
    assert call(K=0) == OK
    assert call(dx=None, dwg=None, dwu=None) == OK
    assert call(M=0, N=0, dh=None, x=None, wg=None) == OK
    assert L.fp8_gated_grad_workspace_size(-1, 4, 128) == 0


def test_gemv_validation(L):
    def call(x=A, w=A, s=A, z=None, y=A, M=1, N=8, K=128, group=64):
        return L.fp8_gemv_w4(x, w, s, z, y, M, N, K, group, None)
    assert call(group=16) == INVALID
    assert call(group=-1) == INVALID
    assert call(x=None) == INVALID
    assert call(s=None) == INVALID
    assert call(z=A, group=fp8.W4_MXFP4) == INVALID
    assert call(M=17) == SHAPE
    assert call(K=64) == SHAPE
    assert call(K=0) == SHAPE
    assert call(N=3) == call()               # a row's scales are read one by one
    assert call(y=MIS) == ALIGN
    assert call(M=0, x=None) == OK
    assert call(N=0) == OK

    def gated(zg=None, zu=None, act=0, group=128, M=1):
        return L.fp8_gated_gemv_w4(A, A, A, zg, A, A, zu, A, M, 8, 128, group, act, None)
    assert gated(zg=A) == INVALID
    assert gated(act=2) == INVALID
    assert gated(zu=MIS, zg=A) == ALIGN
    assert gated(M=20) == SHAPE
    assert gated(M=0) == OK
    assert L.fp8_quant_int4(A, 4, 128, 48, A, A, None, None) == INVALID
    assert L.fp8_quant_int4(A, 4, 100, 64, A, A, None, None) == SHAPE
    assert L.fp8_quant_int4(A, 4, 128, 64, A, None, None, None) == INVALID
    assert L.fp8_quant_int4(MIS, 4, 128, 64, A, A, None, None) == ALIGN
    assert L.fp8_quant_int4(None, 0, 128, 64, None, None, None, None) == OK


def _clip(L, ptrs=(4096, 8192), outs=None, sizes=(10, 20), types=(0, 1), max_norm=1.0, norm=A, ws=A, ws_bytes=1 << 20):
    n = len(sizes)
    gp = (P * n)(*ptrs)
    return L.fp8_clip_grad_norm(gp, (P * n)(*outs) if outs else gp, (ctypes.c_int64 * n)(*sizes),
                                (ctypes.c_int32 * n)(*types), n, max_norm, norm, ws, ws_bytes, None)


def test_clip_validation(L):
    assert _clip(L, max_norm=-1.0) == INVALID
    assert _clip(L, max_norm=float("nan")) == INVALID
    assert _clip(L, norm=None) == INVALID
    assert _clip(L, ws=None) == INVALID
    assert _clip(L, ptrs=(4096, None)) == INVALID
    assert _clip(L, types=(0, 3)) == INVALID
    assert _clip(L, sizes=(-1, 2)) == INVALID
    assert _clip(L, ptrs=(4098, 8192)) == ALIGN          # FP32 off its elements
    assert _clip(L, outs=(4096, 8193)) == ALIGN
    assert _clip(L, ws_bytes=8) == SCRATCH
    assert L.fp8_clip_grad_norm(None, None, None, None, 1, 1.0, A, A, 8, None) == INVALID
    assert L.fp8_clip_workspace_size(None, 3) == 0
    sizes = (ctypes.c_int64 * 3)(1, 0, 20000)
    assert L.fp8_clip_workspace_size(sizes, 3) == 8 * 4  # one slot per chunk of 8192


def test_binding_refuses_cpu_tensors():
    import torch
    x, w = torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((8, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        fp8.gemv_w4(x, w, torch.zeros((1, 8), dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU tensor"):
        fp8.gated_nt_grad(*[torch.zeros((2, 2), dtype=torch.bfloat16)] * 6)
    with pytest.raises(ValueError, match="GPU tensor"):
        fp8.quant_int4(torch.zeros((2, 128)))
    with pytest.raises(ValueError, match="GPU tensors"):
        fp8.clip_grad_norm([torch.zeros(3)], 1.0)
