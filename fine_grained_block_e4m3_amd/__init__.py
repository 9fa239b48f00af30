"""Fine-grained block-scaled E4M3 GEMM for AMD MI355X (gfx950).

Thin ctypes binding over ``libfp8gemm.so`` (C ABI in ``include/fp8gemm.h``).
Every function below only checks tensor shapes/dtypes/devices, allocates the
outputs through torch and passes raw device pointers plus the current HIP
stream to the library; all arithmetic runs in the library's HIP kernels.  If
the library is not built, or no GPU is visible, calls raise -- there is no
CPU fallback.

Names follow the C ABI: ``quant_1x128``, ``quant_128x128``, ``gemm_nt``,
``grouped_gemm_contiguous``, ``grouped_gemm_masked``,
``get_mk_alignment_for_contiguous_layout``; the feed-forward operators
``gated_nt``, ``gated_nt_qout``, ``gated_nt_grad``, ``gemv_w4``,
``gated_gemv_w4``, ``quant_int4``, ``clip_grad_norm``.
"""
from __future__ import annotations

import ctypes
import os
from array import array

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8gemm.so")

FLAG_UE8M0 = 1
FLAG_FAST_ACCUM = 2
PLAN_MX = 0x100
PLAN_QOUT = 0x200
ACT = {"silu": 0, "gelu": 1}
GATED_OUTPUTS = {"h": 0, "save": 1, "quant": 2}
W4_MXFP4 = 0
CLIP_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
LAYOUT = {"dense": 0, "contiguous": 1, "masked": 2}

STATUS = {
    0: "FP8_OK",
    1: "FP8_ERR_INVALID_ARG",
    2: "FP8_ERR_SHAPE",
    3: "FP8_ERR_ALIGNMENT",
    4: "FP8_ERR_UNSUPPORTED",
    5: "FP8_ERR_NO_DEVICE",
    6: "FP8_ERR_LAUNCH",
    7: "FP8_ERR_SCRATCH",
}

# Exported C symbols (kept in step with include/fp8gemm.h by the tests).
SYMBOLS = (
    "fp8_quant_1x128",
    "fp8_quant_128x128",
    "fp8_gemm_nt",
    "fp8_gemm_nt_ws",
    "fp8_gemm_nt_noalloc",
    "fp8_gemm_workspace_size",
    "fp8_gemm_plan",
    "fp8_gemm_nt_qout",
    "fp8_grouped_gemm_contiguous",
    "fp8_grouped_gemm_masked",
    "fp8_quant_mx",
    "fp8_gemm_nt_mx",
    "fp8_quant_mxfp4",
    "fp8_gemm_nt_mx_w4",
    "fp8_gated_nt",
    "fp8_gated_nt_qout",
    "fp8_gated_workspace_size",
    "fp8_gated_plan",
    "fp8_gated_nt_grad",
    "fp8_gated_grad_workspace_size",
    "fp8_gated_grad_plan",
    "fp8_gemv_w4",
    "fp8_gated_gemv_w4",
    "fp8_quant_int4",
    "fp8_clip_grad_norm",
    "fp8_clip_workspace_size",
    "fp8_get_mk_alignment_for_contiguous_layout",
    "fp8_status_string",
)


class GemmPlan(ctypes.Structure):
    """fp8_gemm_plan_t: the kernel instances a GEMM call launches."""
    _fields_ = [("exact", ctypes.c_int32), ("kernel", ctypes.c_int32), ("tile_m", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("waves", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("tiles", ctypes.c_int64), ("main_rows", ctypes.c_int64), ("tail_tile_m", ctypes.c_int32),
                ("tail_tile_n", ctypes.c_int32), ("tail_tiles", ctypes.c_int64), ("k_splits", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_size_t), ("main_cols", ctypes.c_int64),
                ("paired", ctypes.c_int32), ("mid_tile_m", ctypes.c_int32), ("mid_tile_n", ctypes.c_int32),
                ("mid_tiles", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class GatedPlan(ctypes.Structure):
    """fp8_gated_plan_t: the kernels a call of the gated block launches."""
    _fields_ = [("few_tokens", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("k_splits", ctypes.c_int32), ("joined", ctypes.c_int32), ("tiles", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_size_t)]
    as_dict = GemmPlan.as_dict


class GatedGradPlan(ctypes.Structure):
    """fp8_gated_grad_plan_t: the products a call of the gated block's gradient launches."""
    _fields_ = [("dx_tile_n", ctypes.c_int32), ("dw_tile_n", ctypes.c_int32), ("dx_splits", ctypes.c_int32),
                ("dw_splits", ctypes.c_int32), ("dw_first", ctypes.c_int32), ("dx_tiles", ctypes.c_int64),
                ("dw_tiles", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t)]
    as_dict = GemmPlan.as_dict


class Fp8GemmError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({msg})")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfp8gemm.so (no GPU needed to load it).  Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is not built; run `python -m fine_grained_block_e4m3_amd.build` "
            "(hipcc, gfx950). There is no CPU fallback.")
    L = ctypes.CDLL(path)
    P, I64, I32, U32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
    L.fp8_quant_1x128.argtypes = [P, I64, I64, P, P, U32, P]
    L.fp8_quant_128x128.argtypes = [P, I64, I64, P, P, U32, P]
    L.fp8_gemm_nt.argtypes = [P, P, P, P, P, I64, I64, I64, U32, P]
    L.fp8_gemm_nt_ws.argtypes = [P, P, P, P, P, I64, I64, I64, U32, P, ctypes.c_size_t, P]
    L.fp8_gemm_nt_noalloc.argtypes = [P, P, P, P, P, I64, I64, I64, U32, P]
    L.fp8_gemm_workspace_size.argtypes = [I64, I64, I64, U32]
    L.fp8_gemm_workspace_size.restype = ctypes.c_size_t
    L.fp8_gemm_plan.argtypes = [I32, I64, I64, I64, U32, I32, ctypes.c_size_t, ctypes.POINTER(GemmPlan)]
    L.fp8_gemm_nt_qout.argtypes = [P, P, P, P, P, P, I64, I64, I64, U32, P]
    L.fp8_grouped_gemm_contiguous.argtypes = [P, P, P, P, P, P, I64, I64, I64, I32, U32, P]
    L.fp8_grouped_gemm_masked.argtypes = [P, P, P, P, P, P, I32, I64, I64, I64, U32, P]
    L.fp8_quant_mx.argtypes = [P, I64, I64, P, P, P]
    L.fp8_gemm_nt_mx.argtypes = [P, P, P, P, P, I64, I64, I64, U32, P]
    L.fp8_quant_mxfp4.argtypes = [P, I64, I64, P, P, P]
    L.fp8_gemm_nt_mx_w4.argtypes = [P, P, P, P, P, I64, I64, I64, U32, P]
    L.fp8_gated_nt.argtypes = [P] * 9 + [I64, I64, I64, I32, U32, P, ctypes.c_size_t, P]
    L.fp8_gated_nt_qout.argtypes = [P] * 8 + [I64, I64, I64, I32, U32, P, ctypes.c_size_t, P]
    L.fp8_gated_workspace_size.argtypes = [I64, I64, I64, I32]
    L.fp8_gated_workspace_size.restype = ctypes.c_size_t
    L.fp8_gated_plan.argtypes = [I64, I64, I64, I32, I32, ctypes.c_size_t, ctypes.POINTER(GatedPlan)]
    L.fp8_gated_nt_grad.argtypes = [P] * 9 + [I64, I64, I64, I32, P, ctypes.c_size_t, P]
    L.fp8_gated_grad_workspace_size.argtypes = [I64, I64, I64]
    L.fp8_gated_grad_workspace_size.restype = ctypes.c_size_t
    L.fp8_gated_grad_plan.argtypes = [I64, I64, I64, I32, I32, I32, ctypes.POINTER(GatedGradPlan)]
    L.fp8_gemv_w4.argtypes = [P] * 5 + [I64, I64, I64, I32, P]
    L.fp8_gated_gemv_w4.argtypes = [P] * 8 + [I64, I64, I64, I32, I32, P]
    L.fp8_quant_int4.argtypes = [P, I64, I64, I32, P, P, P, P]
    # (host arrays of pointers, counts and types)
    L.fp8_clip_grad_norm.argtypes = [P, P, P, P, I32, ctypes.c_float, P, P, ctypes.c_size_t, P]
    L.fp8_clip_workspace_size.argtypes = [P, I32]
    L.fp8_clip_workspace_size.restype = ctypes.c_size_t
    for fn in ("fp8_quant_1x128", "fp8_quant_128x128", "fp8_gemm_nt", "fp8_gemm_nt_ws", "fp8_gemm_nt_noalloc",
               "fp8_gemm_plan",
               "fp8_gemm_nt_qout",
               "fp8_grouped_gemm_contiguous", "fp8_grouped_gemm_masked", "fp8_quant_mx",
               "fp8_gemm_nt_mx", "fp8_quant_mxfp4", "fp8_gemm_nt_mx_w4", "fp8_gated_nt", "fp8_gated_nt_qout", "fp8_gated_plan",
               "fp8_gated_grad_plan", "fp8_gated_nt_grad", "fp8_gemv_w4", "fp8_gated_gemv_w4", "fp8_quant_int4",
               "fp8_clip_grad_norm"):
        getattr(L, fn).restype = ctypes.c_int
    L.fp8_get_mk_alignment_for_contiguous_layout.argtypes = []
    L.fp8_get_mk_alignment_for_contiguous_layout.restype = I32
    L.fp8_status_string.argtypes = [ctypes.c_int]
    L.fp8_status_string.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(fn: str, status: int) -> None:
    if status != 0:
        msg = load_library().fp8_status_string(status).decode()
        raise Fp8GemmError(fn, status, msg)


# The raw handle of a device's current stream, without building a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor) -> int:
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch_stream(t: torch.Tensor) -> int:
    """The current stream of t's device, which has to be the current device:
    kernels are launched there."""
    if t.get_device() != _current_device():
        raise ValueError(f"operands on {t.device}, but the current device is cuda:{_current_device()}: "
                         f"call within torch.cuda.device({t.get_device()})")
    return _stream(t)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int) -> None:
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.dim() == ndim and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out(t, name: str, dtype: torch.dtype, shape, like: torch.Tensor) -> torch.Tensor:
    """A caller's output buffer: the kernels write exactly this shape, so any
    other shape, type, layout or device is refused before a launch."""
    _need(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the inputs on {like.device}")
    return t


def _same_device(*ts: torch.Tensor) -> None:
    d = ts[0].get_device()
    for t in ts[1:]:
        if t.get_device() != d:
            raise ValueError(f"operands on different devices: {ts[0].device} and {t.device}")


def _ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


def _flags(ue8m0: bool, fast_accum: bool = False) -> int:
    return (FLAG_UE8M0 if ue8m0 else 0) | (FLAG_FAST_ACCUM if fast_accum else 0)


def gemm_plan(layout: str, M: int, N: int, K: int, ue8m0: bool = False, fast_accum: bool = False,
              mx: bool = False, qout: bool = False, compute_units: int = 256,
              workspace_bytes: int = 0) -> dict:
    """The kernel instances a GEMM call of this shape launches (host-side
    arithmetic only; no GPU needed).  layout: dense, contiguous or masked
    (max_m as M)."""
    L = load_library()
    flags = _flags(ue8m0, fast_accum) | (PLAN_MX if mx else 0) | (PLAN_QOUT if qout else 0)
    plan = GemmPlan()
    _check("fp8_gemm_plan", L.fp8_gemm_plan(LAYOUT[layout], M, N, K, flags, compute_units, workspace_bytes,
                                            ctypes.byref(plan)))
    return plan.as_dict()


def get_mk_alignment_for_contiguous_layout() -> int:
    return int(load_library().fp8_get_mk_alignment_for_contiguous_layout())


def quant_1x128(x: torch.Tensor, ue8m0: bool = False, out=None):
    """x fp32 (M, K) -> (xq uint8 (M, K), sa fp32 (K/128, M))."""
    L = load_library()
    _need(x, "x", torch.float32, 2)
    M, K = x.shape
    if out is None:
        xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
        sa = torch.empty((K // 128, M), dtype=torch.float32, device=x.device)
    else:
        xq = _out(out[0], "out[0]", torch.uint8, (M, K), x)
        sa = _out(out[1], "out[1]", torch.float32, (K // 128, M), x)
    _check("fp8_quant_1x128", L.fp8_quant_1x128(_ptr(x), M, K, _ptr(xq), _ptr(sa),
                                                _flags(ue8m0), _stream(x)))
    return xq, sa


def quant_128x128(w: torch.Tensor, ue8m0: bool = False, out=None):
    """w fp32 (N, K) -> (wq uint8 (N, K), sb fp32 (ceil(N/128), K/128))."""
    L = load_library()
    _need(w, "w", torch.float32, 2)
    N, K = w.shape
    if out is None:
        wq = torch.empty((N, K), dtype=torch.uint8, device=w.device)
        sb = torch.empty(((N + 127) // 128, K // 128), dtype=torch.float32, device=w.device)
    else:
        wq = _out(out[0], "out[0]", torch.uint8, (N, K), w)
        sb = _out(out[1], "out[1]", torch.float32, ((N + 127) // 128, K // 128), w)
    _check("fp8_quant_128x128", L.fp8_quant_128x128(_ptr(w), N, K, _ptr(wq), _ptr(sb),
                                                    _flags(ue8m0), _stream(w)))
    return wq, sb


def gemm_nt(xq, sa, wq, sb, ue8m0: bool = False, fast_accum: bool = False, out=None,
            workspace=None) -> torch.Tensor:
    """Y (M, N) bf16 = block-scaled X * W^T.  fast_accum: block partials from
    the FP8 matrix instruction (see FP8_FLAG_FAST_ACCUM).  With fast_accum and
    a decode-sized M the library splits K when given a workspace: a uint8
    device tensor of at least fp8_gemm_workspace_size() bytes, allocated here
    through torch when not passed."""
    L = load_library()
    _need(xq, "xq", torch.uint8, 2)
    _need(wq, "wq", torch.uint8, 2)
    _need(sa, "sa", torch.float32, 2)
    _need(sb, "sb", torch.float32, 2)
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K or sa.shape != (K // 128, M) or sb.shape != ((N + 127) // 128, K // 128):
        raise ValueError("gemm_nt: inconsistent operand shapes")
    _same_device(xq, sa, wq, sb)
    y = _out(out, "out", torch.bfloat16, (M, N), xq) if out is not None \
        else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    flags = _flags(ue8m0, fast_accum)
    if workspace is None and M and N and K:
        nbytes = int(L.fp8_gemm_workspace_size(M, N, K, flags))
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=xq.device)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1)
        _same_device(xq, workspace)
        ws, ws_bytes = _ptr(workspace), workspace.numel()
    else:
        ws, ws_bytes = None, 0
    _check("fp8_gemm_nt_ws", L.fp8_gemm_nt_ws(_ptr(xq), _ptr(sa), _ptr(wq), _ptr(sb), _ptr(y),
                                              M, N, K, flags, ws, ws_bytes, _stream(xq)))
    return y


def gemm_nt_qout(xq, sa, wq, sb, ue8m0: bool = False, fast_accum: bool = False, out=None):
    """Block-scaled X * W^T written quantized for the next GEMM: (yq uint8
    (M, N) E4M3 codes, sy fp32 (N/128, M) 1x128 scales); N % 128 == 0."""
    L = load_library()
    _need(xq, "xq", torch.uint8, 2)
    _need(wq, "wq", torch.uint8, 2)
    _need(sa, "sa", torch.float32, 2)
    _need(sb, "sb", torch.float32, 2)
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K or sa.shape != (K // 128, M) or sb.shape != ((N + 127) // 128, K // 128):
        raise ValueError("gemm_nt_qout: inconsistent operand shapes")
    _same_device(xq, sa, wq, sb)
    if out is None:
        yq = torch.empty((M, N), dtype=torch.uint8, device=xq.device)
        sy = torch.empty((N // 128, M), dtype=torch.float32, device=xq.device)
    else:
        yq = _out(out[0], "out[0]", torch.uint8, (M, N), xq)
        sy = _out(out[1], "out[1]", torch.float32, (N // 128, M), xq)
    _check("fp8_gemm_nt_qout", L.fp8_gemm_nt_qout(_ptr(xq), _ptr(sa), _ptr(wq), _ptr(sb), _ptr(yq),
                                                  _ptr(sy), M, N, K, _flags(ue8m0, fast_accum),
                                                  _stream(xq)))
    return yq, sy


def grouped_gemm_contiguous(xq, sa, wq, sb, m_indices, ue8m0: bool = False, fast_accum: bool = False,
                            out=None) -> torch.Tensor:
    """xq (M, K), sa (K/128, M), wq (E, N, K), sb (E, N/128, K/128), m_indices int32 (M)."""
    L = load_library()
    _need(xq, "xq", torch.uint8, 2)
    _need(wq, "wq", torch.uint8, 3)
    _need(sa, "sa", torch.float32, 2)
    _need(sb, "sb", torch.float32, 3)
    _need(m_indices, "m_indices", torch.int32, 1)
    M, K = xq.shape
    E, N, _ = wq.shape
    if wq.shape[2] != K or sa.shape != (K // 128, M) or sb.shape != (E, N // 128, K // 128) \
            or m_indices.shape[0] != M:
        raise ValueError("grouped_gemm_contiguous: inconsistent operand shapes")
    _same_device(xq, sa, wq, sb, m_indices)
    y = _out(out, "out", torch.bfloat16, (M, N), xq) if out is not None \
        else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    _check("fp8_grouped_gemm_contiguous",
           L.fp8_grouped_gemm_contiguous(_ptr(xq), _ptr(sa), _ptr(wq), _ptr(sb), _ptr(m_indices),
                                         _ptr(y), M, N, K, E, _flags(ue8m0, fast_accum), _stream(xq)))
    return y


def grouped_gemm_masked(xq, sa, wq, sb, masked_m, ue8m0: bool = False, fast_accum: bool = False,
                        out=None) -> torch.Tensor:
    """xq (E, max_m, K), sa (K/128, E*max_m), wq (E, N, K), sb (E, N/128, K/128),
    masked_m int32 (E).  Returns y (E, max_m, N) bf16 (rows past masked_m untouched)."""
    L = load_library()
    _need(xq, "xq", torch.uint8, 3)
    _need(wq, "wq", torch.uint8, 3)
    _need(sa, "sa", torch.float32, 2)
    _need(sb, "sb", torch.float32, 3)
    _need(masked_m, "masked_m", torch.int32, 1)
    E, max_m, K = xq.shape
    N = wq.shape[1]
    if wq.shape != (E, N, K) or sa.shape != (K // 128, E * max_m) \
            or sb.shape != (E, N // 128, K // 128) or masked_m.shape[0] != E:
        raise ValueError("grouped_gemm_masked: inconsistent operand shapes")
    _same_device(xq, sa, wq, sb, masked_m)
    y = _out(out, "out", torch.bfloat16, (E, max_m, N), xq) if out is not None \
        else torch.empty((E, max_m, N), dtype=torch.bfloat16, device=xq.device)
    _check("fp8_grouped_gemm_masked",
           L.fp8_grouped_gemm_masked(_ptr(xq), _ptr(sa), _ptr(wq), _ptr(sb), _ptr(masked_m),
                                     _ptr(y), E, max_m, N, K, _flags(ue8m0, fast_accum), _stream(xq)))
    return y


def quant_mx(x: torch.Tensor, out=None):
    """MXFP8: x fp32 (R, K) -> (q uint8 (R, K), e int32 (K/128, R)).  e holds the
    packed scale bytes: byte t of e[kb, r] is the exponent byte b of 1x32 group
    4*kb + t of row r, whose scale is 2^(b - 127)."""
    L = load_library()
    _need(x, "x", torch.float32, 2)
    R, K = x.shape
    if out is None:
        q = torch.empty((R, K), dtype=torch.uint8, device=x.device)
        e = torch.empty((K // 128, R), dtype=torch.int32, device=x.device)
    else:
        q = _out(out[0], "out[0]", torch.uint8, (R, K), x)
        e = _out(out[1], "out[1]", torch.int32, (K // 128, R), x)
    _check("fp8_quant_mx", L.fp8_quant_mx(_ptr(x), R, K, _ptr(q), _ptr(e), _stream(x)))
    return q, e


def gemm_nt_mx(xq, ea, wq, eb, out=None) -> torch.Tensor:
    """Y (M, N) bf16 = MXFP8 X * W^T; ea (K/128, M) and eb (K/128, N) are the
    packed scale tables that quant_mx writes."""
    L = load_library()
    _need(xq, "xq", torch.uint8, 2)
    _need(wq, "wq", torch.uint8, 2)
    _need(ea, "ea", torch.int32, 2)
    _need(eb, "eb", torch.int32, 2)
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K or ea.shape != (K // 128, M) or eb.shape != (K // 128, N):
        raise ValueError("gemm_nt_mx: inconsistent operand shapes")
    _same_device(xq, ea, wq, eb)
    y = _out(out, "out", torch.bfloat16, (M, N), xq) if out is not None \
        else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    _check("fp8_gemm_nt_mx", L.fp8_gemm_nt_mx(_ptr(xq), _ptr(ea), _ptr(wq), _ptr(eb), _ptr(y),
                                              M, N, K, 0, _stream(xq)))
    return y


def quant_mxfp4(w: torch.Tensor, out=None):
    """MXFP4 weights: w fp32 (R, K) -> (q uint8 (R, K/2), two E2M1 nibbles per
    byte, the even element low; e int32 (K/128, R) packed scale bytes)."""
    L = load_library()
    _need(w, "w", torch.float32, 2)
    R, K = w.shape
    if out is None:
        q = torch.empty((R, K // 2), dtype=torch.uint8, device=w.device)
        e = torch.empty((K // 128, R), dtype=torch.int32, device=w.device)
    else:
        q = _out(out[0], "out[0]", torch.uint8, (R, K // 2), w)
        e = _out(out[1], "out[1]", torch.int32, (K // 128, R), w)
    _check("fp8_quant_mxfp4", L.fp8_quant_mxfp4(_ptr(w), R, K, _ptr(q), _ptr(e), _stream(w)))
    return q, e


def gemm_nt_mx_w4(xq, ea, wq, eb, out=None) -> torch.Tensor:
    """Y (M, N) bf16 = MXFP8 X * (MXFP4 W)^T; wq (N, K/2) packed nibbles."""
    L = load_library()
    _need(xq, "xq", torch.uint8, 2)
    _need(wq, "wq", torch.uint8, 2)
    _need(ea, "ea", torch.int32, 2)
    _need(eb, "eb", torch.int32, 2)
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] * 2 != K or ea.shape != (K // 128, M) or eb.shape != (K // 128, N):
        raise ValueError("gemm_nt_mx_w4: inconsistent operand shapes")
    _same_device(xq, ea, wq, eb)
    y = _out(out, "out", torch.bfloat16, (M, N), xq) if out is not None \
        else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    _check("fp8_gemm_nt_mx_w4", L.fp8_gemm_nt_mx_w4(_ptr(xq), _ptr(ea), _ptr(wq), _ptr(eb), _ptr(y),
                                                    M, N, K, 0, _stream(xq)))
    return y


def _act(act: str) -> int:
    if act not in ACT:
        raise ValueError(f"act must be one of {sorted(ACT)}, got {act!r}")
    return ACT[act]


def _workspace(workspace, nbytes: int, like: torch.Tensor):
    """(pointer, bytes) of the caller's workspace, or of one of nbytes allocated
    through torch, and the tensor that holds it."""
    if workspace is None:
        if not nbytes:
            return None, 0, None
        workspace = like.new_empty(nbytes, dtype=torch.uint8)
    else:
        _need(workspace, "workspace", torch.uint8, 1)
        _same_device(like, workspace)
    return _ptr(workspace), workspace.numel(), workspace


_U8, _F32, _BF16 = torch.uint8, torch.float32, torch.bfloat16


def _gated_operands(xq, sa, wgq, sbg, wuq, sbu, fn: str):
    # A decode-sized call spends more time here than on the device: operands
    # that fit pass one expression, and what follows finds the fault in others.
    try:
        M, K = xq.shape
        N = len(wgq)
        blocks = ((N + 127) // 128, K // 128)
        if (xq.dtype is _U8 and wgq.dtype is _U8 and wuq.dtype is _U8
                and sa.dtype is _F32 and sbg.dtype is _F32 and sbu.dtype is _F32
                and wgq.shape == wuq.shape == (N, K) and sa.shape == (K // 128, M) and sbg.shape == sbu.shape == blocks
                and xq.is_contiguous() and wgq.is_contiguous() and wuq.is_contiguous()
                and sa.is_contiguous() and sbg.is_contiguous() and sbu.is_contiguous()
                and (0 <= xq.get_device() == wgq.get_device() == wuq.get_device()
                     == sa.get_device() == sbg.get_device() == sbu.get_device())):
            return M, N, K
    except (AttributeError, TypeError, ValueError):
        pass
    for t, name, dtype in ((xq, "xq", torch.uint8), (sa, "sa", torch.float32), (wgq, "wgq", torch.uint8),
                           (sbg, "sbg", torch.float32), (wuq, "wuq", torch.uint8), (sbu, "sbu", torch.float32)):
        _need(t, name, dtype, 2)
    M, K = xq.shape
    N = wgq.shape[0]
    blocks = ((N + 127) // 128, K // 128)
    if wgq.shape[1] != K or wuq.shape != (N, K) or sa.shape != (K // 128, M) or sbg.shape != blocks \
            or sbu.shape != blocks:
        raise ValueError(f"{fn}: inconsistent operand shapes")
    _same_device(xq, sa, wgq, sbg, wuq, sbu)
    return M, N, K


def _gated_workspace_size(M: int, N: int, K: int, outputs: int) -> int:
    if M <= 16 and outputs != 2:
        return 0            # one kernel, K split inside its workgroups
    return int(load_library().fp8_gated_workspace_size(M, N, K, outputs))


def gated_plan(M: int, N: int, K: int, outputs: str = "h", compute_units: int = 256,
               workspace_bytes: int | None = None) -> dict:
    """The kernels gated_nt (outputs "h", or "save" with g and u) or
    gated_nt_qout ("quant") launches for this shape (host-side arithmetic only;
    no GPU needed), by default with all the workspace it can use."""
    plan = GatedPlan()
    nbytes = ctypes.c_size_t(-1).value if workspace_bytes is None else workspace_bytes
    _check("fp8_gated_plan", load_library().fp8_gated_plan(M, N, K, GATED_OUTPUTS[outputs], compute_units, nbytes,
                                                           ctypes.byref(plan)))
    return plan.as_dict()


def gated_nt(xq, sa, wgq, sbg, wuq, sbu, act: str = "silu", ue8m0: bool = False, save: bool = False, out=None,
             workspace=None):
    """Gated feed-forward block on block-scaled E4M3 operands: h (M, N) bf16 =
    act(X Wg^T) * (X Wu^T), act "silu" or "gelu" (tanh form).  With save the
    projections are returned too: (h, g, u), which gated_nt_grad takes.  out:
    h, or (h, g, u).  workspace: as for gemm_nt, where the output has too few
    tiles to fill the device."""
    L = load_library()
    a = _act(act)
    M, N, K = _gated_operands(xq, sa, wgq, sbg, wuq, sbu, "gated_nt")
    if out is None:
        ys = [xq.new_empty((M, N), dtype=_BF16)]
        if save:
            ys += [torch.empty_like(ys[0]), torch.empty_like(ys[0])]
    else:
        ys = list(out) if save else [out]
        if len(ys) != (3 if save else 1):
            raise ValueError("gated_nt: out must be (h, g, u) with save")
        ys = [_out(t, f"out[{i}]", torch.bfloat16, (M, N), xq) for i, t in enumerate(ys)]
    ws, ws_bytes, keep = _workspace(workspace, _gated_workspace_size(M, N, K, 1 if save else 0), xq)
    _check("fp8_gated_nt", L.fp8_gated_nt(
        xq.data_ptr(), sa.data_ptr(), wgq.data_ptr(), sbg.data_ptr(), wuq.data_ptr(), sbu.data_ptr(), ys[0].data_ptr(),
        _ptr(ys[1]) if save else None, _ptr(ys[2]) if save else None, M, N, K, a, _flags(ue8m0), ws, ws_bytes,
        _launch_stream(xq)))
    return tuple(ys) if save else ys[0]


def gated_nt_qout(xq, sa, wgq, sbg, wuq, sbu, act: str = "silu", ue8m0: bool = False, out=None, workspace=None):
    """gated_nt with h quantized for the down projection: (hq uint8 (M, N) E4M3
    codes, sh fp32 (N/128, M) 1x128 scales); N % 128 == 0."""
    L = load_library()
    a = _act(act)
    M, N, K = _gated_operands(xq, sa, wgq, sbg, wuq, sbu, "gated_nt_qout")
    if out is None:
        hq = torch.empty((M, N), dtype=torch.uint8, device=xq.device)
        sh = torch.empty((N // 128, M), dtype=torch.float32, device=xq.device)
    else:
        hq = _out(out[0], "out[0]", torch.uint8, (M, N), xq)
        sh = _out(out[1], "out[1]", torch.float32, (N // 128, M), xq)
    ws, ws_bytes, keep = _workspace(workspace, _gated_workspace_size(M, N, K, 2), xq)
    _check("fp8_gated_nt_qout", L.fp8_gated_nt_qout(
        _ptr(xq), _ptr(sa), _ptr(wgq), _ptr(sbg), _ptr(wuq), _ptr(sbu), _ptr(hq), _ptr(sh), M, N, K, a,
        _flags(ue8m0), ws, ws_bytes, _launch_stream(xq)))
    return hq, sh


def _grad_operands(dh, g, u, x, wg, wu):
    # (one expression for operands that fit, as in _gated_operands)
    try:
        M, N = dh.shape
        K = x.shape[1]
        if (dh.dtype is _BF16 and g.dtype is _BF16 and u.dtype is _BF16 and x.dtype is _BF16 and wg.dtype is _BF16
                and wu.dtype is _BF16 and g.shape == u.shape == (M, N) and x.shape == (M, K)
                and wg.shape == wu.shape == (N, K) and dh.is_contiguous() and g.is_contiguous() and u.is_contiguous()
                and x.is_contiguous() and wg.is_contiguous() and wu.is_contiguous()
                and (0 <= dh.get_device() == g.get_device() == u.get_device() == x.get_device()
                     == wg.get_device() == wu.get_device())):
            return M, N, K
    except (AttributeError, TypeError, ValueError, IndexError):
        pass
    for t, name in ((dh, "dh"), (g, "g"), (u, "u"), (x, "x"), (wg, "wg"), (wu, "wu")):
        _need(t, name, torch.bfloat16, 2)
    M, N = dh.shape
    K = x.shape[1]
    if g.shape != (M, N) or u.shape != (M, N) or x.shape[0] != M or wg.shape != (N, K) or wu.shape != (N, K):
        raise ValueError("gated_nt_grad: inconsistent operand shapes")
    _same_device(dh, g, u, x, wg, wu)
    return M, N, K


def gated_grad_plan(M: int, N: int, K: int, need_dx: bool = True, need_dw: bool = True,
                    compute_units: int = 256) -> dict:
    """The products gated_nt_grad launches for this shape (host-side arithmetic
    only; no GPU needed)."""
    plan = GatedGradPlan()
    _check("fp8_gated_grad_plan", load_library().fp8_gated_grad_plan(M, N, K, need_dx, need_dw, compute_units,
                                                                     ctypes.byref(plan)))
    return plan.as_dict()


def gated_nt_grad(dh, g, u, x, wg, wu, act: str = "silu", need_dx: bool = True, need_dw: bool = True, out=None,
                  workspace=None):
    """Gradient of the gated block, BF16: dh, g, u (M, N), x (M, K), wg, wu
    (N, K) -> (dx (M, K), dwg (N, K), dwu (N, K)); dx is None without need_dx,
    dwg and dwu without need_dw.  out: (dx, dwg, dwu) buffers."""
    L = load_library()
    a = _act(act)
    M, N, K = _grad_operands(dh, g, u, x, wg, wu)
    shapes, wanted = ((M, K), (N, K), (N, K)), (need_dx, need_dw, need_dw)
    if out is None:
        ys = [dh.new_empty(shape) if w else None for shape, w in zip(shapes, wanted)]
    else:
        ys = [_out(t, f"out[{i}]", torch.bfloat16, shape, dh) if w else None
              for i, (t, shape, w) in enumerate(zip(out, shapes, wanted))]
    ws, ws_bytes, keep = _workspace(workspace, int(L.fp8_gated_grad_workspace_size(M, N, K)), dh)
    _check("fp8_gated_nt_grad", L.fp8_gated_nt_grad(
        _ptr(dh), _ptr(g), _ptr(u), _ptr(x), _ptr(wg), _ptr(wu), *[_ptr(t) if t is not None else None for t in ys],
        M, N, K, a, ws, ws_bytes, _launch_stream(dh)))
    return tuple(ys)


def _w4(w, s, z, N: int, K: int, name: str, x) -> int:
    """Checks one 4-bit weight for the activations x and returns its `group`
    (W4_MXFP4 for packed E8M0 scales)."""
    # (one expression for weights that fit, as in _gated_operands)
    try:
        groups, cols = s.shape
        if (w.dtype is _U8 and w.shape == (N, K // 2) and cols == N and w.is_contiguous() and s.is_contiguous()
                and x.get_device() == w.get_device() == s.get_device()):
            if s.dtype is torch.int32 and z is None and groups == K // 128:
                return W4_MXFP4
            if s.dtype is _BF16 and groups and K in (32 * groups, 64 * groups, 128 * groups) and (
                    z is None or (z.dtype is _U8 and z.shape == s.shape and z.is_contiguous()
                                  and z.get_device() == s.get_device())):
                return K // groups
    except (AttributeError, TypeError, ValueError):
        pass
    _need(w, name, torch.uint8, 2)
    _same_device(x, w)
    if w.shape != (N, K // 2):
        raise ValueError(f"{name} must have shape {(N, K // 2)}, got {tuple(w.shape)}")
    if isinstance(s, torch.Tensor) and s.dtype == torch.int32:
        _need(s, f"scales of {name}", torch.int32, 2)
        _same_device(x, s)
        if s.shape != (K // 128, N) or z is not None:
            raise ValueError(f"MXFP4 {name}: scales must be (K/128, N), without zeros")
        return W4_MXFP4
    _need(s, f"scales of {name}", torch.bfloat16, 2)
    _same_device(x, s)
    groups = s.shape[0]
    if s.shape[1] != N or groups == 0 or K % groups or K // groups not in (32, 64, 128):
        raise ValueError(f"scales of {name} must be (K/group, N) with a group of 32, 64 or 128")
    if z is not None:
        _need(z, f"zeros of {name}", torch.uint8, 2)
        if z.shape != s.shape:
            raise ValueError(f"zeros of {name} must have the scales' shape")
        _same_device(s, z)
    return K // groups


def gemv_w4(x, w, scales, zeros=None, out=None) -> torch.Tensor:
    """y (M, N) bf16 = x (M, K) bf16 * W^T for up to 16 tokens, W in 4 bits:
    w uint8 (N, K/2) with either the int32 (K/128, N) scales of quant_mxfp4, or
    the bf16 (K/group, N) scales (and uint8 zeros, else 8) of quant_int4."""
    L = load_library()
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    N = w.shape[0]
    group = _w4(w, scales, zeros, N, K, "w", x)
    y = _out(out, "out", torch.bfloat16, (M, N), x) if out is not None \
        else x.new_empty((M, N))
    _check("fp8_gemv_w4", L.fp8_gemv_w4(
        x.data_ptr(), w.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(), y.data_ptr(),
        M, N, K, group, _launch_stream(x)))
    return y


def gated_gemv_w4(x, wg, scales_g, wu, scales_u, zeros_g=None, zeros_u=None, act: str = "silu",
                  out=None) -> torch.Tensor:
    """The gated block on 4-bit weights for up to 16 tokens: y (M, N) bf16 =
    act(x Wg^T) * (x Wu^T); weights as for gemv_w4, both of one format."""
    L = load_library()
    a = _act(act)
    _need(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    N = wg.shape[0]
    group = _w4(wg, scales_g, zeros_g, N, K, "wg", x)
    if _w4(wu, scales_u, zeros_u, N, K, "wu", x) != group or (zeros_g is None) != (zeros_u is None):
        raise ValueError("gated_gemv_w4: both weights must have one format")
    y = _out(out, "out", torch.bfloat16, (M, N), x) if out is not None \
        else x.new_empty((M, N))
    _check("fp8_gated_gemv_w4", L.fp8_gated_gemv_w4(
        x.data_ptr(), wg.data_ptr(), scales_g.data_ptr(), None if zeros_g is None else zeros_g.data_ptr(),
        wu.data_ptr(), scales_u.data_ptr(), None if zeros_u is None else zeros_u.data_ptr(), y.data_ptr(),
        M, N, K, group, a, _launch_stream(x)))
    return y


def quant_int4(w: torch.Tensor, group: int = 128, symmetric: bool = False, out=None):
    """4-bit integer weights: w fp32 (N, K) -> (q uint8 (N, K/2), scales bf16
    (K/group, N), zeros uint8 (K/group, N), or None when symmetric)."""
    L = load_library()
    _need(w, "w", torch.float32, 2)
    N, K = w.shape
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    if out is None:
        q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
        s = torch.empty((K // group, N), dtype=torch.bfloat16, device=w.device)
        z = None if symmetric else torch.empty((K // group, N), dtype=torch.uint8, device=w.device)
    else:
        q = _out(out[0], "out[0]", torch.uint8, (N, K // 2), w)
        s = _out(out[1], "out[1]", torch.bfloat16, (K // group, N), w)
        z = None if symmetric else _out(out[2], "out[2]", torch.uint8, (K // group, N), w)
    _check("fp8_quant_int4", L.fp8_quant_int4(_ptr(w), N, K, group, _ptr(q), _ptr(s),
                                              _ptr(z) if z is not None else None, _launch_stream(w)))
    return q, s, z


def _dims(t: torch.Tensor) -> list:
    return [(stride, size) for stride, size in zip(t.stride(), t.shape) if size != 1]


def _is_dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill a run of memory, in any order of its dimensions."""
    if t.is_contiguous():
        return True
    run = 1
    for stride, size in sorted(_dims(t)):
        if stride != run:
            return False
        run *= size
    return True


def _same_order(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two dense tensors hold their elements in one order."""
    return a.is_contiguous() and b.is_contiguous() or _dims(a) == _dims(b)


def clip_grad_norm(grads, max_norm: float, out=None, workspace=None) -> torch.Tensor:
    """Scales the tensors of `grads` (fp32, bf16 or fp16, any mix; dense, with
    their dimensions in any order of memory) by min(1, max_norm / (norm +
    1e-6)), norm being the 2-norm over all of them, and returns norm (0-dim
    fp32, on the device).  In place unless `out` gives one tensor of the same
    type, size and order of memory per gradient."""
    L = load_library()
    grads = list(grads)
    outs = grads if out is None else list(out)
    n = len(grads)
    if not n:
        raise ValueError("clip_grad_norm: no gradients")
    if len(outs) != n:
        raise ValueError("clip_grad_norm: out must hold one tensor per gradient")
    T = torch.Tensor
    both = grads if outs is grads else grads + outs
    # one pass per property: the calls that matter here hold hundreds of tensors
    try:
        types = [CLIP_TYPES[t.dtype] for t in both]
    except KeyError as e:
        raise TypeError(f"clip_grad_norm: gradients must be fp32, bf16 or fp16, got {e.args[0]}") from None
    counts, devices = list(map(T.numel, both)), set(map(T.get_device, both))
    if len(devices) != 1 or -1 in devices:
        raise ValueError("clip_grad_norm: gradients must be GPU tensors of one device (no CPU path exists)")
    if outs is not grads and (types[:n] != types[n:] or counts[:n] != counts[n:]):
        raise ValueError("clip_grad_norm: out[i] must have the type and size of grads[i]")
    if not all(map(T.is_contiguous, both)):
        # any order of the dimensions, as long as out has the same
        if not all(map(_is_dense, both)):
            raise ValueError("clip_grad_norm: gradients must be dense (every element of their memory once)")
        if outs is not grads and not all(map(_same_order, grads, outs)):
            raise ValueError("clip_grad_norm: out[i] must have the strides of grads[i]")
    ptrs = array("q", map(T.data_ptr, both))
    sizes, kinds = array("q", counts), array("i", types)
    gp, sp, kp = ptrs.buffer_info()[0], sizes.buffer_info()[0], kinds.buffer_info()[0]
    op = gp if outs is grads else gp + n * ptrs.itemsize
    norm = grads[0].new_empty((), dtype=torch.float32)
    ws, ws_bytes, keep = _workspace(workspace, int(L.fp8_clip_workspace_size(sp, n)), grads[0])
    _check("fp8_clip_grad_norm", L.fp8_clip_grad_norm(gp, op, sp, kp, n, float(max_norm), norm.data_ptr(), ws,
                                                      ws_bytes, _launch_stream(grads[0])))
    return norm
