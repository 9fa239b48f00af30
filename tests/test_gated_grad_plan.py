"""Which products the gradient of the gated block launches, and every
combination of them against 64 bits: tile widths, splits of either contraction
and of both, and each result by itself."""
import ctypes
import random

import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import check_guards, guarded, say

OK, INVALID, SHAPE, UNSUP = 0, 1, 2, 4
CUS = 256

# M, N, K, then dX's and dW's tile columns, their splits, and whether dW's tiles come first
SHAPES = [(65, 1, 128, 128, 128, 1, 1, 1), (130, 129, 256, 128, 128, 1, 1, 0), (1, 482, 128, 128, 128, 2, 1, 0),
          (1001, 1, 128, 128, 128, 1, 2, 1), (1002, 543, 128, 128, 128, 2, 2, 0), (1052, 511, 128, 128, 128, 2, 2, 1),
          (1024, 512, 128, 128, 128, 2, 2, 0), (2048, 1024, 128, 128, 128, 4, 4, 0),
          (268, 1285, 6400, 128, 256, 1, 1, 0), (2927, 1410, 5632, 128, 256, 1, 1, 1),
          (1, 8217, 896, 128, 256, 8, 1, 0), (256, 4096, 7168, 128, 256, 2, 1, 0),
          (3259, 130, 5120, 256, 128, 1, 1, 1), (8161, 1, 1920, 256, 128, 1, 8, 1),
          (8192, 130, 2048, 256, 128, 1, 4, 1), (8192, 300, 1024, 128, 128, 1, 8, 1),
          (2364, 1331, 6784, 256, 256, 1, 1, 0), (2521, 1212, 7168, 256, 256, 1, 1, 1)]


@pytest.mark.parametrize("M,N,K,dx,dw,sx,sw,first", SHAPES)
def test_plan(M, N, K, dx, dw, sx, sw, first):
    p = fp8.gated_grad_plan(M, N, K, compute_units=CUS)
    assert (p["dx_tile_n"], p["dw_tile_n"], p["dx_splits"], p["dw_splits"], p["dw_first"]) == (dx, dw, sx, sw, first), p
    rows, padded = -(-M // 128), -(-N // 64) * 64
    assert p["dx_tiles"] == rows * -(-K // dx) and p["dw_tiles"] == 2 * -(-N // 128) * -(-K // dw)
    split = [(t, s) for t, s in ((p["dx_tiles"], sx), (p["dw_tiles"], sw)) if s > 1]
    assert p["workspace_bytes"] == 4 * M * padded + sum(4 * t * (s * 128 * 128 + 1) for t, s in split)


def test_the_shapes_above_reach_every_combination():
    assert {s[3:5] for s in SHAPES} == {(a, b) for a in (128, 256) for b in (128, 256)}
    assert {(s[5] > 1, s[6] > 1) for s in SHAPES} == {(a, b) for a in (False, True) for b in (False, True)}
    assert {(s[3], s[4], s[7]) for s in SHAPES} >= {(a, a, f) for a in (128, 256) for f in (0, 1)}


def test_wide_tiles_are_not_split():
    r = random.Random(1)

    def size(hi):
        return int(2 ** r.uniform(0, hi))
    for _ in range(20000):
        M, N, K, cus = size(18), size(16), 128 * size(7), r.choice([1, 64, 256, 304])
        p = fp8.gated_grad_plan(M, N, K, r.random() < 0.8, r.random() < 0.8, cus)
        assert p["dx_tile_n"] != 256 or p["dx_splits"] == 1
        assert p["dw_tile_n"] != 256 or p["dw_splits"] == 1
        assert max(p["dx_splits"], p["dw_splits"]) <= 8


def test_plan_validation():
    L = fp8.load_library()

    def call(M=4, N=8, K=128, dx=1, dw=1, cus=CUS, plan=fp8.GatedGradPlan()):
        return L.fp8_gated_grad_plan(M, N, K, dx, dw, cus, ctypes.byref(plan) if plan else None)
    assert call() == OK and call(K=0) == OK and call(M=0, N=0) == OK
    assert call(plan=None) == INVALID
    assert call(N=-1) == INVALID and call(M=1 << 31) == INVALID
    assert call(cus=0) == INVALID
    assert call(K=130) == SHAPE
    assert call(N=1 << 22) == UNSUP
    nothing = fp8.gated_grad_plan(4, 8, 128, False, False)
    assert nothing["dx_tiles"] == nothing["dw_tiles"] == nothing["workspace_bytes"] == 0


# --------------------------------------------------------------------------
# The same shapes on the GPU, against 64 bits there.
# --------------------------------------------------------------------------
def _case(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + 5 * N + K)

    def rand(r, c, s):
        return torch.randn((r, c), generator=g, device="cuda").mul_(s).bfloat16()
    return [rand(M, N, 0.1), rand(M, N, 1.5), rand(M, N, 1.5), rand(M, K, 1.0), rand(N, K, 0.05), rand(N, K, 0.05)]


def _exact(ops, act):
    """(dx, dwg, dwu) in 64 bits, and their sums of magnitudes."""
    dh, g, u, x, wg, wu = (t.double() for t in ops)
    c = 2.0 * (2.0 / torch.pi) ** 0.5
    t, dt = (g, 1.0) if act == "silu" else (c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g))
    p = torch.sigmoid(t)
    dg, du = dh * u * (p + g * dt * p * (1 - p)), dh * g * p

    def three(dg, du, x, wg, wu):
        return (torch.matmul(dg, wg) + torch.matmul(du, wu), torch.matmul(dg.t().contiguous(), x),
                torch.matmul(du.t().contiguous(), x))
    return three(dg, du, x, wg, wu), three(dg.abs(), du.abs(), x.abs(), wg.abs(), wu.abs())


def _check(got, want, mag, M, N, K):
    for t, w, m, name in zip(got, want, mag, ("dx", "dwg", "dwu")):
        if t is None:
            continue
        diff = (t.double() - w).abs()
        # dg and du off by one rounding each and by their FP32 evaluation, sums of
        # at most 2^-24 (n / 16 + 64), one rounding
        n = 2 * N if name == "dx" else M
        bound = (1.02 * ref.U_BF16 + (n / 16 + 64) * ref.U_F32 + 2 ** -18) * m + 1.01 * ref.U_BF16 * w.abs()
        assert bool((diff <= bound).all()), name
        if min(M, N, K) >= 64:
            # two independent roundings, in the 2-norm each below 2^-9 of the values
            assert float(torch.linalg.norm(diff)) <= 2.0 ** -8 * float(torch.linalg.norm(w)), name


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [s[:3] for s in SHAPES])
def test_products(M, N, K):
    """All results, then each alone (whose plan and bits may differ)."""
    assert torch.cuda.get_device_properties(0).multi_processor_count == CUS
    act = "gelu" if N % 2 else "silu"
    say(f"grad plan M={M} N={N} K={K} {act}")
    ops = _case(M, N, K)
    want, mag = _exact(ops, act)
    bufs = [guarded(s) for s in ((M, K), (N, K), (N, K))]
    _check(fp8.gated_nt_grad(*ops, act=act, out=[b[1] for b in bufs]), want, mag, M, N, K)
    for full, out in bufs:
        check_guards(full, out.numel())
    for part in ({"need_dw": False}, {"need_dx": False}):
        got = fp8.gated_nt_grad(*ops, act=act, **part)
        assert [t is None for t in got] == ([False, True, True] if "need_dw" in part else [True, False, False])
        _check(got, want, mag, M, N, K)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [s[:3] for s in SHAPES if max(s[5:7]) > 1])
def test_joined_splits_are_repeatable(M, N, K):
    """Sums joined by whichever split comes last: the same bits in every call, in
    a workspace of the exact size that holds other values each time, eagerly
    and replayed."""
    ops = _case(M, N, K)
    size = fp8.load_library().fp8_gated_grad_workspace_size(M, N, K)
    say(f"grad splits M={M} N={N} K={K} workspace={size}")
    full, ws = guarded((size // 2,))
    ws = ws.view(torch.uint8)
    want = [t.clone() for t in fp8.gated_nt_grad(*ops)]
    for i in range(6):
        ws.fill_(37 * i)
        assert all(torch.equal(a, b) for a, b in zip(fp8.gated_nt_grad(*ops, workspace=ws), want))
    outs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.gated_nt_grad(*ops, out=outs, workspace=ws)
    for i in range(4):
        for t in outs:
            t.zero_()
        ws.fill_(83 * i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        fp8.gated_nt_grad(*ops)
        torch.cuda.synchronize()
    check_guards(full, size // 2)
