"""Which kernels the gated block launches, and every one of them against the
64-bit form: each tile in one round and in several rounds per workgroup, with K
split and joined, for h alone, with g and u, and quantized."""
import ctypes

import numpy as np
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
import oracle
from gpu_helpers import say

OK, INVALID, SHAPE, UNSUP = 0, 1, 2, 4
CUS = 256

# M, N, K and the tile, its splits along K, and whether a workgroup takes several tiles
PLAIN = [(65, 130, 128, (64, 64), 1, False), (4623, 411, 2304, (64, 64), 1, True),
         (100, 500, 1664, (64, 64), 3, False), (8264, 65, 128, (64, 128), 1, False),
         (388, 8359, 384, (64, 128), 1, True), (2143, 68, 2048, (64, 128), 4, False),
         (8271, 131, 128, (128, 64), 1, False), (8219, 417, 384, (128, 64), 1, True),
         (5467, 1, 1536, (128, 64), 3, False), (193, 8201, 128, (128, 128), 1, False),
         (774, 8257, 128, (128, 128), 1, True), (67, 5708, 3712, (128, 128), 5, False),
         (390, 8319, 128, (256, 128), 1, False), (901, 8358, 128, (256, 128), 1, True),
         (129, 5709, 6656, (256, 128), 5, False)]
QUANT = [(100, 128, 2048, (64, 64), 4, False), (300, 640, 256, (64, 128), 1, False),
         (388, 8320, 384, (64, 128), 1, True), (130, 2048, 2048, (64, 128), 4, False),
         (202, 8448, 128, (128, 128), 1, False), (771, 8448, 128, (128, 128), 1, True),
         (68, 6016, 3200, (128, 128), 5, False), (2100, 2048, 128, (256, 128), 1, False),
         (7900, 2048, 384, (256, 128), 1, True), (129, 5632, 6656, (256, 128), 5, False)]
# ... and the kernel for few tokens: M, N, K, its rows, its columns
FEW = [(1, 2048, 256, 16, 8), (16, 3000, 384, 16, 16), (9, 7000, 128, 16, 32), (20, 130, 640, 32, 8),
       (30, 2093, 256, 32, 16), (17, 6156, 128, 32, 32), (40, 1000, 640, 48, 8), (37, 2112, 1536, 48, 16),
       (64, 500, 1664, 64, 8), (64, 3001, 256, 64, 16)]


def _is(plan, tile, splits, rounds):
    return (not plan["few_tokens"] and (plan["tile_m"], plan["tile_n"]) == tile and plan["k_splits"] == splits
            and (plan["tiles"] > CUS) == rounds and plan["joined"] == (splits > 1))


@pytest.mark.parametrize("M,N,K,tile,splits,rounds", PLAIN)
def test_plan_of_the_projections(M, N, K, tile, splits, rounds):
    for outputs in ("h", "save"):
        plan = fp8.gated_plan(M, N, K, outputs, CUS)
        assert _is(plan, tile, splits, rounds), plan
        assert plan["workspace_bytes"] == (8 * splits * M * N if splits > 1 else 0)
        assert fp8.gated_plan(M, N, K, outputs, CUS, plan["workspace_bytes"]) == plan
        if splits > 1:
            less = fp8.gated_plan(M, N, K, outputs, CUS, plan["workspace_bytes"] - 1)
            assert less["k_splits"] == 1 and less["workspace_bytes"] == 0


@pytest.mark.parametrize("M,N,K,tile,splits,rounds", QUANT)
def test_plan_of_the_quantized_block(M, N, K, tile, splits, rounds):
    plan = fp8.gated_plan(M, N, K, "quant", CUS)
    assert _is(plan, tile, splits, rounds), plan
    less = fp8.gated_plan(M, N, K, "quant", CUS, 0)
    assert less["k_splits"] == 1 and not less["joined"] and less["tile_n"] == 128


@pytest.mark.parametrize("M,N,K,rows,cols", FEW)
def test_plan_of_few_tokens(M, N, K, rows, cols):
    plan = fp8.gated_plan(M, N, K, "save", CUS)
    assert plan["few_tokens"] and (plan["tile_m"], plan["tile_n"]) == (rows, cols) and not plan["joined"], plan


def test_the_shapes_above_reach_every_instance():
    tiles = {(64, 64), (64, 128), (128, 64), (128, 128), (256, 128)}
    assert {(t, s > 1, r) for *_, t, s, r in PLAIN} == {(t, s, r) for t in tiles
                                                        for s, r in ((False, False), (False, True), (True, False))}
    wide = {t for t in tiles if t[1] == 128}            # (a quantization group per tile where unsplit)
    assert {(t, s > 1, r) for *_, t, s, r in QUANT} == {((64, 64), True, False)} | {
        (t, s, r) for t in wide for s, r in ((False, False), (False, True), (True, False))}
    assert {(r, c) for *_, r, c in FEW} == {(16 * b, c) for b in (1, 2) for c in (8, 16, 32)} | {
        (16 * b, c) for b in (3, 4) for c in (8, 16)}


def test_plan_validation():
    L = fp8.load_library()

    def call(M=4, N=128, K=128, outputs=0, cus=CUS, plan=fp8.GatedPlan()):
        return L.fp8_gated_plan(M, N, K, outputs, cus, 0, ctypes.byref(plan) if plan else None)
    assert call() == OK and call(M=0) == OK and call(N=0) == OK
    assert call(plan=None) == INVALID
    assert call(M=-1) == INVALID
    assert call(outputs=3) == INVALID
    assert call(outputs=-1) == INVALID
    assert call(cus=0) == INVALID
    assert call(K=100) == SHAPE and call(K=0) == SHAPE
    assert call(N=100, outputs=2) == SHAPE and call(N=100) == OK
    assert call(K=(1 << 22) + 128) == UNSUP


# --------------------------------------------------------------------------
# The same shapes on the GPU, against 64 bits there.
# --------------------------------------------------------------------------
def _decoded(q, s_rows):
    values = torch.from_numpy(oracle.e4m3_decode(np.arange(256)).astype(np.float64)).cuda()
    R, K = q.shape
    return (values[q.long()].view(R, K // 128, 128) * s_rows.double()[..., None]).view(R, K)


def _case(M, N, K, act, pow2):
    """Device operands, and (h, g, u) in 64 bits with the bounds of their FP32
    errors, as in ffn_reference.gated."""
    gen = torch.Generator(device="cuda").manual_seed(M + 3 * N + K + pow2)
    x = torch.randn((M, K), generator=gen, device="cuda")
    x *= 1.0 + 30.0 * (torch.rand((M, K), generator=gen, device="cuda") < 0.005)
    xq, sa = fp8.quant_1x128(x, ue8m0=pow2)
    ws = [fp8.quant_128x128(torch.randn((N, K), generator=gen, device="cuda") * 1.5 / K ** 0.5, ue8m0=pow2)
          for _ in range(2)]
    xd, rows = _decoded(xq, sa.t()), torch.arange(N, device="cuda") // 128
    wd = [_decoded(q, s[rows]) for q, s in ws]
    g, u = (torch.matmul(xd, w.t()) for w in wd)
    steps = K / 16 + 2 * K / 128 + 32
    eg, eu = (steps * ref.U_F32 * torch.matmul(xd.abs(), w.t().abs()) for w in wd)
    t = g if act == "silu" else 2.0 * (2.0 / np.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    a = g * torch.sigmoid(t)
    eh = 1.13 * u.abs() * eg + a.abs() * eu + 1.13 * eg * eu + (8 + 4 * t.abs()) * ref.U_F32 * (a * u).abs()
    return (xq, sa, *ws[0], *ws[1]), (a * u, g, u), (eh, eg, eu)


def _assert_bf16(got, want, err, what):
    got = got.double()
    assert bool(torch.isfinite(got).all()), what
    _, e = torch.frexp(want.abs() + 1.01 * err)
    bound = 1.01 * err + torch.ldexp(torch.ones_like(want), e.clamp_min(-125) - 9)
    bad = (got - want).abs() > bound
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound"


def _guarded(M, N):
    full = torch.full((M * N + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    return full, full[2048:2048 + M * N].view(M, N)


def _check_guards(full):
    assert bool((full[:2048] == 7).all()) and bool((full[-2048:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [s[:3] for s in PLAIN + FEW])
@pytest.mark.parametrize("act,pow2", [("silu", False), ("gelu", True)])
def test_projections(M, N, K, act, pow2):
    assert torch.cuda.get_device_properties(0).multi_processor_count == CUS
    say(f"gated plan M={M} N={N} K={K} {act} pow2={pow2}")
    ops, refs, errs = _case(M, N, K, act, pow2)
    full, h = _guarded(M, N)
    fp8.gated_nt(*ops, act=act, ue8m0=pow2, out=h)
    _assert_bf16(h, refs[0], errs[0], "h")
    bufs = [_guarded(M, N) for _ in range(3)]
    outs = fp8.gated_nt(*ops, act=act, ue8m0=pow2, save=True, out=[b[1] for b in bufs])
    for name, got, r, e in zip("hgu", outs, refs, errs):
        _assert_bf16(got, r, e, name)
    for f, _ in bufs + [(full, h)]:
        _check_guards(f)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [s[:3] for s in QUANT])
@pytest.mark.parametrize("act,pow2", [("silu", True), ("gelu", False)])
def test_quantized(M, N, K, act, pow2):
    say(f"gated plan quantized M={M} N={N} K={K} {act} pow2={pow2}")
    ops, (h, _, _), (e, _, _) = _case(M, N, K, act, pow2)
    hq, sh = fp8.gated_nt_qout(*ops, act=act, ue8m0=pow2)
    h, e, s = h.view(M, N // 128, 128), e.view(M, N // 128, 128), sh.t().double()
    amax = h.abs().amax(2)
    lo, hi = ((m.clamp_min(1e-4) / 448) for m in (amax - e.amax(2), amax + e.amax(2)))
    if pow2:
        lo, hi = (torch.exp2(torch.ceil(torch.log2(v))) for v in (lo, hi))
    assert bool(((s >= lo * (1 - 2 ** -22)) & (s <= hi * (1 + 2 ** -22))).all())
    pair = _decoded(hq, s).view(h.shape)
    # nearest E4M3: half a unit of 3 fraction bits, or of the subnormals
    bound = 1.01 * e + 2.0 ** -4 * (h.abs() + e) * (1 + 2 ** -20) + 2.0 ** -10 * s[..., None] * (1 + 2 ** -20)
    assert bool(((pair - h).abs() <= bound).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(130, 2048, 2048), (100, 128, 2048), (33, 384, 2560)])
def test_joined_calls_replay(M, N, K):
    """Calls of two kernels in a graph: every replay gives the eager bits."""
    ops, _, _ = _case(M, N, K, "silu", True)
    say(f"gated joined graph M={M} N={N} K={K}")
    size = max(fp8.gated_plan(M, N, K, o, CUS)["workspace_bytes"] for o in ("save", "quant"))
    assert fp8.gated_plan(M, N, K, "quant", CUS)["joined"] and size
    want = [t.clone() for t in (*fp8.gated_nt(*ops, save=True, ue8m0=True), *fp8.gated_nt_qout(*ops, ue8m0=True))]
    outs, ws = [torch.empty_like(t) for t in want], torch.empty(size, dtype=torch.uint8, device="cuda")

    def calls():
        fp8.gated_nt(*ops, save=True, ue8m0=True, out=outs[:3], workspace=ws)
        fp8.gated_nt_qout(*ops, ue8m0=True, out=outs[3:], workspace=ws)
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in range(4):
        for t in outs:
            t.zero_()
        ws.fill_(17 * i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        fp8.gated_nt(*ops, ue8m0=True)
        torch.cuda.synchronize()
