"""4-bit matrix-vector products (MXFP4 and integer codes with group scales,
plain and gated) against their 64-bit forms, and the integer quantizer
bit-exact against its definition."""
import numpy as np
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
import oracle
from gpu_helpers import bf16_bits, bf16_to_f64, check_guards, dev, guarded, host, say

pytestmark = pytest.mark.gpu

FORMATS = [("mxfp4", 32, False), ("int4", 32, True), ("int4", 64, False), ("int4", 64, True), ("int4", 128, True),
           ("int4", 128, False), ("int4", 32, False)]


def _bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _weight(rng, N, K, fmt, group, zeros):
    """Device operands (codes, scales, zeros), the weight and the magnitudes it
    is formed from, in 64 bits."""
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        e = rng.integers(100, 140, (K // 128, N, 4), dtype=np.uint8)
        packed = np.ascontiguousarray(e).view(np.uint32).reshape(K // 128, N)
        w = ref.decode_mxfp4(q, packed)
        return (dev(q), dev(packed.view(np.int32)), None), w, np.abs(w)
    s = ref.to_bf16(np.exp(rng.uniform(-6, 1, (K // group, N))))
    z = rng.integers(0, 16, (K // group, N), dtype=np.uint8) if zeros else None
    w, mag = ref.decode_int4(q, s, z, group)
    return (dev(q), _bf16(ref.bf16_bits_of(s)), dev(z) if zeros else None), w, mag


def _sum_error(K, x, mag):
    # sums of 32 products at a time (within a group first), 8 waves joined
    return (K / 32 * 3 + 64) * ref.U_F32 * (np.abs(x) @ mag.T)


# N from one tile of rows to the widths that take 2, 3, 4 and 6 tiles per
# workgroup on 256 compute units; K with and without a lone last block
SHAPES = [(1, 4, 128), (1, 5, 384), (2, 16, 256), (3, 17, 1152), (16, 33, 128), (15, 130, 640), (8, 1000, 2048),
          (4, 4803, 128), (5, 10000, 128), (16, 14336, 128), (9, 24570, 128)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
def test_gemv_matches_the_64_bit_form(M, N, K, fmt, group, zeros):
    say(f"gemv {fmt} group={group} zeros={zeros} M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K + group)
    x = ref.to_bf16(rng.standard_normal((M, K)))
    (q, s, z), w, mag = _weight(rng, N, K, fmt, group, zeros)
    full, out = guarded((M, N))
    assert fp8.gemv_w4(_bf16(ref.bf16_bits_of(x)), q, s, zeros=z, out=out) is out
    ref.assert_bf16(bf16_to_f64(bf16_bits(out)), x @ w.T, _sum_error(K, x, mag), "y")
    check_guards(full, M * N)


@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (4, 2, 384), (6, 3, 256), (16, 1, 640), (9, 7, 128)])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
def test_very_narrow_weights(M, N, K, fmt, group, zeros):
    test_gemv_matches_the_64_bit_form(M, N, K, fmt, group, zeros)
    test_gated_gemv_matches_the_64_bit_form(M, N, K, fmt, group, zeros)


@pytest.mark.parametrize("M,N,K", [(1, 4, 128), (3, 9, 384), (16, 100, 1152), (2, 2112, 256), (7, 3000, 128),
                                   (16, 7168, 128), (1, 12285, 128)])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
def test_gated_gemv_matches_the_64_bit_form(M, N, K, fmt, group, zeros):
    act = "silu" if group == 64 else "gelu"
    say(f"gated gemv {fmt} group={group} zeros={zeros} M={M} N={N} K={K} {act}")
    rng = np.random.default_rng(M + N + K + group)
    x = ref.to_bf16(rng.standard_normal((M, K)) * 0.05)
    (gq, gs, gz), wg, gm = _weight(rng, N, K, fmt, group, zeros)
    (uq, us, uz), wu, um = _weight(rng, N, K, fmt, group, zeros)
    full, out = guarded((M, N))
    fp8.gated_gemv_w4(_bf16(ref.bf16_bits_of(x)), gq, gs, uq, us, zeros_g=gz, zeros_u=uz, act=act, out=out)
    g, u = x @ wg.T, x @ wu.T
    eg, eu = _sum_error(K, x, gm), _sum_error(K, x, um)
    t, a = ref.act_parts(act, g)[0], ref.act_value(act, g)
    eh = 1.13 * np.abs(u) * eg + np.abs(a) * eu + 1.13 * eg * eu + (8 + 4 * np.abs(t)) * ref.U_F32 * np.abs(a * u)
    # where the gate vanishes the exponential's argument carries the gate's own error too
    ref.assert_bf16(bf16_to_f64(bf16_bits(out)), a * u, eh, "y")
    check_guards(full, M * N)


def test_quantizers_feed_the_products():
    """Weights through the framework's quantizers, against their decoded values."""
    M, N, K = 5, 200, 512
    rng = np.random.default_rng(3)
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    x = ref.to_bf16(rng.standard_normal((M, K)))
    xd = _bf16(ref.bf16_bits_of(x))
    say("gemv on quantized weights")
    q, e = fp8.quant_mxfp4(dev(w))
    wd = ref.decode_mxfp4(host(q), host(e).view(np.uint32))
    assert np.abs(wd - w).max() < 0.02
    ref.assert_bf16(bf16_to_f64(bf16_bits(fp8.gemv_w4(xd, q, e))), x @ wd.T, _sum_error(K, x, np.abs(wd)), "mxfp4")
    for group in (32, 64, 128):
        for symmetric in (False, True):
            q, s, z = fp8.quant_int4(dev(w), group, symmetric)
            wd, mag = ref.decode_int4(host(q), bf16_to_f64(bf16_bits(s)), None if z is None else host(z), group)
            assert np.abs(wd - w).max() < 0.02
            ref.assert_bf16(bf16_to_f64(bf16_bits(fp8.gemv_w4(xd, q, s, zeros=z))), x @ wd.T,
                            _sum_error(K, x, mag), "int4")


@pytest.mark.parametrize("N,K", [(1, 128), (4, 128), (33, 640), (200, 1152)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [False, True])
def test_quant_int4_is_exact(N, K, group, symmetric):
    say(f"quant_int4 N={N} K={K} group={group} symmetric={symmetric}")
    rng = np.random.default_rng(N + K + group)
    w = (rng.standard_normal((N, K)) * np.exp(rng.uniform(-8, 4, (N, 1)))).astype(np.float32)
    w[0, :group] = 0                                 # a group of zeros
    w[-1, -group:] = np.abs(w[-1, -group:])          # one sign only
    if N > 2:
        w[1, :group] = -np.abs(w[1, :group])
        w[2, :group] = 3.25                          # one value
    q, s, z = fp8.quant_int4(dev(w), group, symmetric)
    rq, rs, rz = ref.quant_int4(w, group, symmetric)
    assert np.array_equal(bf16_bits(s), rs)
    assert np.array_equal(host(q), rq)
    assert (z is None) == symmetric and (symmetric or np.array_equal(host(z), rz))


def test_refusals():
    rng = np.random.default_rng(0)
    N, K = 64, 256
    (q, s, z), _, _ = _weight(rng, N, K, "int4", 64, True)
    (mq, me, _), _, _ = _weight(rng, N, K, "mxfp4", 32, False)
    x = torch.ones((2, K), dtype=torch.bfloat16, device="cuda")
    say("gemv refusals")
    with pytest.raises(TypeError):
        fp8.gemv_w4(x.float(), q, s, zeros=z)
    with pytest.raises(ValueError):
        fp8.gemv_w4(x, q[:, :64].contiguous(), s, zeros=z)
    with pytest.raises(ValueError):
        fp8.gemv_w4(x, q, s[:3].contiguous(), zeros=z)
    with pytest.raises(ValueError):
        fp8.gemv_w4(x, q, s, zeros=z[:2].contiguous())
    with pytest.raises(ValueError):
        fp8.gemv_w4(x, mq, me, zeros=z)
    with pytest.raises(ValueError):
        fp8.gated_gemv_w4(x, q, s, mq, me)
    with pytest.raises(ValueError):
        fp8.gated_gemv_w4(x, q, s, q, s, zeros_g=z)
    with pytest.raises(ValueError):
        fp8.quant_int4(torch.zeros((4, 128), device="cuda"), group=16)
    with pytest.raises(fp8.Fp8GemmError) as e:
        fp8.gemv_w4(torch.ones((17, K), dtype=torch.bfloat16, device="cuda"), q, s, zeros=z)
    assert e.value.status == 2
    assert fp8.gemv_w4(x[:0], q, s, zeros=z).shape == (0, N)


def test_graph_and_side_stream():
    rng = np.random.default_rng(8)
    (q, s, z), _, _ = _weight(rng, 300, 640, "int4", 32, True)
    x = _bf16(ref.bf16_bits_of(ref.to_bf16(rng.standard_normal((3, 640)))))
    want = fp8.gemv_w4(x, q, s, zeros=z).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("gemv on a side stream")
    with torch.cuda.stream(side):
        got = fp8.gemv_w4(x, q, s, zeros=z)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    say("gemv graph")
    with torch.cuda.graph(graph):
        fp8.gemv_w4(x, q, s, zeros=z, out=out)
    for _ in range(4):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        fp8.gemv_w4(x, q, s, zeros=z)
        torch.cuda.synchronize()
