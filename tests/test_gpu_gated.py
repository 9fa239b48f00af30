"""The gated feed-forward block on E4M3 operands against its 64-bit form:
every kernel it is made of (up to 16 tokens, decode-sized with K split, the
four tile sizes), odd sizes, saved projections, quantized outputs, guards
around every output, side streams and graph replays."""
import ctypes

import numpy as np
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
import oracle
import workloads
from gpu_helpers import bf16_bits, bf16_to_f64, check_guards, dev, guarded, host, say

pytestmark = pytest.mark.gpu


def _case(M, N, K, seed, pow2=False):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[rng.random((M, K)) < 0.005] *= 30.0
    ws = [(rng.standard_normal((N, K)) * 1.5 / np.sqrt(K)).astype(np.float32) for _ in range(2)]
    flags = oracle.FLAG_UE8M0 if pow2 else 0
    xq, sa = oracle.quant_1x128(x, flags)
    (gq, sg), (uq, su) = (oracle.quant_128x128(w, flags) for w in ws)
    return (xq, sa, gq, sg, uq, su), (ref.decode_x(xq, sa), ref.decode_w(gq, sg), ref.decode_w(uq, su))


def _values(t):
    return bf16_to_f64(bf16_bits(t))


# one to four blocks of 16 tokens, with one to six weight tiles per workgroup;
# then the tiles of every size, with and without K split (256 compute units)
SHAPES = [(1, 1, 128), (1, 96, 384), (2, 100, 640), (15, 37, 1152), (16, 2112, 256), (7, 4103, 128),
          (17, 1, 128), (33, 130, 640), (64, 500, 1664), (20, 12300, 3200), (40, 6200, 1664),
          (65, 31, 128), (130, 333, 384), (300, 96, 640), (600, 3300, 128), (1100, 3700, 256), (2100, 3700, 128), (100, 500, 1664), (500, 1000, 384), (700, 4160, 128)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act,pow2", [("silu", False), ("gelu", True)])
def test_gated_matches_the_64_bit_form(M, N, K, act, pow2):
    say(f"gated M={M} N={N} K={K} act={act} pow2={pow2}")
    ops, (x, wg, wu) = _case(M, N, K, M + N + K, pow2)
    full, out = guarded((M, N))
    got = fp8.gated_nt(*[dev(a) for a in ops], act=act, ue8m0=pow2, out=out)
    assert got is out
    (h, _, _), (eh, _, _) = ref.gated(x, wg, wu, act)
    ref.assert_bf16(_values(out), h, eh, "h")
    check_guards(full, M * N)


@pytest.mark.parametrize("M,N,K", [(1, 5, 128), (16, 200, 384), (40, 1000, 640), (65, 31, 128), (300, 500, 256),
                                   (1100, 3700, 128), (2100, 3700, 128)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_saved_projections(M, N, K, act):
    say(f"gated save M={M} N={N} K={K} act={act}")
    ops, (x, wg, wu) = _case(M, N, K, 3 * M + N)
    bufs = [guarded((M, N)) for _ in range(3)]
    outs = fp8.gated_nt(*[dev(a) for a in ops], act=act, save=True, out=[b[1] for b in bufs])
    refs, errs = ref.gated(x, wg, wu, act)
    for (full, _), got, r, e, name in zip(bufs, outs, refs, errs, "hgu"):
        ref.assert_bf16(_values(got), r, e, name)
        check_guards(full, M * N)


@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (16, 256, 384), (33, 640, 640), (64, 1024, 1664), (65, 128, 128),
                                   (300, 640, 256), (2100, 3712, 128)])
@pytest.mark.parametrize("act,pow2", [("silu", True), ("gelu", False)])
def test_quantized_output(M, N, K, act, pow2):
    say(f"gated quantized M={M} N={N} K={K} act={act} pow2={pow2}")
    _check_quantized(M, N, K, act, pow2)


def _check_quantized(M, N, K, act, pow2, workspace=None):
    ops, (x, wg, wu) = _case(M, N, K, 7 * M + N, pow2)
    hq, sh = fp8.gated_nt_qout(*[dev(a) for a in ops], act=act, ue8m0=pow2, workspace=workspace)
    (h, _, _), (eh, _, _) = ref.gated(x, wg, wu, act)
    s = host(sh).astype(np.float64)
    groups = h.reshape(M, N // 128, 128)
    e = eh.reshape(M, N // 128, 128)
    amax = np.abs(groups).max(2)
    lo, hi = (np.maximum(a, 1e-4) / 448.0 for a in (amax - e.max(2), amax + e.max(2)))
    if pow2:
        lo, hi = np.exp2(np.ceil(np.log2(lo) - 1e-6)), np.exp2(np.ceil(np.log2(hi) + 1e-6))
    assert np.all(s.T >= lo * (1 - 2 ** -22)) and np.all(s.T <= hi * (1 + 2 ** -22))
    got = oracle.e4m3_decode(np.arange(256))[host(hq)].reshape(groups.shape) * s.T[..., None]
    # nearest E4M3: half a unit of 3 fraction bits, or of the subnormals
    bound = 1.01 * e + 2.0 ** -4 * (np.abs(groups) + e) * (1 + 2 ** -20) + 2.0 ** -10 * s.T[..., None] * (1 + 2 ** -20)
    assert np.all(np.abs(got - groups) <= bound)


# Up to 64 tokens, each number of token blocks and weight tiles, and shapes that
# the tiles take; then the same without a workspace.
FEW = [(1, 3, 256), (16, 2000, 384), (9, 5002, 128), (20, 7001, 384), (30, 1300, 256), (48, 2100, 640), (40, 401, 1664),
       (64, 3001, 256), (50, 260, 896), (64, 24704, 128), (17, 12300, 3200)]


@pytest.mark.parametrize("M,N,K", FEW)
@pytest.mark.parametrize("workspace", [True, False])
def test_few_tokens(M, N, K, workspace):
    say(f"gated few tokens M={M} N={N} K={K} workspace={workspace}")
    ops, (x, wg, wu) = _case(M, N, K, M * 5 + N)
    a = [dev(t) for t in ops]
    ws = None if workspace else torch.empty(0, dtype=torch.uint8, device="cuda")
    refs, errs = ref.gated(x, wg, wu, "silu")
    full, out = guarded((M, N))
    fp8.gated_nt(*a, out=out, workspace=ws)
    ref.assert_bf16(_values(out), refs[0], errs[0], "h")
    check_guards(full, M * N)
    bufs = [guarded((M, N)) for _ in range(3)]
    outs = fp8.gated_nt(*a, save=True, out=[b[1] for b in bufs], workspace=ws)
    for (full, _), got, r, e, name in zip(bufs, outs, refs, errs, "hgu"):
        ref.assert_bf16(_values(got), r, e, name)
        check_guards(full, M * N)


@pytest.mark.parametrize("M,N,K", [(1, 2048, 640), (5, 128, 1664), (16, 5120, 128), (17, 7168, 384), (48, 2176, 256),
                                   (64, 3200, 256), (64, 24704, 128), (33, 384, 2560)])
@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantized_few_tokens(M, N, K, workspace, pow2):
    say(f"gated quantized few tokens M={M} N={N} K={K} workspace={workspace} pow2={pow2}")
    _check_quantized(M, N, K, "gelu" if pow2 else "silu", pow2,
                     None if workspace else torch.empty(0, dtype=torch.uint8, device="cuda"))


def test_without_workspace_takes_unsplit_tiles():
    L = fp8.load_library()
    M, N, K = 100, 300, 1664
    ops, (x, wg, wu) = _case(M, N, K, 5)
    a = [dev(t) for t in ops]
    need = L.fp8_gated_workspace_size(M, N, K, 0)
    assert need > 0 and L.fp8_gated_workspace_size(64, N, K, 0) == 0
    (h, _, _), (eh, _, _) = ref.gated(x, wg, wu, "silu")
    s = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for nbytes in (0, need - 1, need):
        say(f"gated with {nbytes} bytes of workspace")
        full, out = guarded((M, N))
        assert L.fp8_gated_nt(*[t.data_ptr() for t in a], out.data_ptr(), None, None, M, N, K, 0, 0,
                              ws.data_ptr() if nbytes else None, nbytes, s) == 0
        ref.assert_bf16(_values(out), h, eh, "h")
        check_guards(full, M * N)


def test_extreme_gates():
    """Gates far beyond where the exponential overflows or vanishes."""
    M, N, K = 4, 64, 128
    xq = np.zeros((M, K), np.uint8)
    xq[:, 0] = 0x38                                   # 1.0
    gq = np.zeros((N, K), np.uint8)
    gq[:, 0] = np.where(np.arange(N) % 2, 0x7E, 0xFE)  # +-448
    uq = np.zeros((N, K), np.uint8)
    uq[:, 0] = 0x38
    for act in ("silu", "gelu"):
        for scale in (1.0, 1e-3, 1e30):
            sa = np.ones((1, M), np.float32)
            sg, su = np.full((1, 1), scale, np.float32), np.ones((1, 1), np.float32)
            say(f"gated extreme {act} {scale}")
            got = _values(fp8.gated_nt(*[dev(a) for a in (xq, sa, gq, sg, uq, su)], act=act))
            with np.errstate(over="ignore"):
                want = ref.act_value(act, ref.decode_x(xq, sa) @ ref.decode_w(gq, sg).T)
            assert np.all(np.isfinite(got))
            assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 1e-30)


def test_empty_and_refused():
    ops, _ = _case(8, 256, 128, 1)
    a = [dev(t) for t in ops]
    say("gated refusals")
    with pytest.raises(ValueError, match="act"):
        fp8.gated_nt(*a, act="relu")
    with pytest.raises(ValueError):
        fp8.gated_nt(*a[:4], dev(ops[4][:255].copy()), a[5])
    with pytest.raises(ValueError):
        fp8.gated_nt(*a, save=True, out=[torch.empty((8, 256), dtype=torch.bfloat16, device="cuda")] * 2)
    with pytest.raises(TypeError):
        fp8.gated_nt(*a, out=torch.empty((8, 256), dtype=torch.float32, device="cuda"))
    with pytest.raises(ValueError):
        fp8.gated_nt(a[0].t().contiguous().t(), *a[1:])
    ragged, _ = _case(8, 100, 128, 1)
    with pytest.raises(fp8.Fp8GemmError) as e:
        fp8.gated_nt_qout(*[dev(t) for t in ragged])
    assert e.value.status == 2
    empty = fp8.gated_nt(a[0][:0], a[1][:, :0].contiguous(), *a[2:])
    assert empty.shape == (0, 256)


def test_side_stream_and_graph():
    """On a stream of its own, and captured: every replay equals the eager call."""
    for M in (3, 40, 200):
        ops, _ = _case(M, 384, 640, M)
        a = [dev(t) for t in ops]
        want = fp8.gated_nt(*a).clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        say(f"gated on a side stream M={M}")
        with torch.cuda.stream(side):
            got = fp8.gated_nt(*a)
        side.synchronize()
        assert torch.equal(got, want)
        out = torch.empty_like(want)
        ws = torch.empty(max(1, fp8.load_library().fp8_gated_workspace_size(M, 384, 640, 0)), dtype=torch.uint8,
                         device="cuda")
        fp8.gated_nt(*a, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        say(f"gated graph M={M}")
        with torch.cuda.graph(graph):
            fp8.gated_nt(*a, out=out, workspace=ws)
        for _ in range(4):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            fp8.gated_nt(*a)
            torch.cuda.synchronize()
