"""The gradient of the gated block against the formula's 64-bit form and
against differences of the forward pass."""
import numpy as np
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import bf16_bits, bf16_to_f64, check_guards, guarded, say

pytestmark = pytest.mark.gpu


def _bf16(a):
    bits = ref.bf16_bits_of(ref.to_bf16(a)).view(np.int16)
    return torch.from_numpy(np.ascontiguousarray(bits)).cuda().view(torch.bfloat16)


def _values(t):
    return bf16_to_f64(bf16_bits(t))


def _case(M, N, K, seed):
    rng = np.random.default_rng(seed)
    shapes = [(M, N)] * 3 + [(M, K), (N, K), (N, K)]
    scale = [0.1, 1.5, 1.5, 1.0, 0.05, 0.05]
    return [ref.to_bf16(rng.standard_normal(s) * c) for s, c in zip(shapes, scale)]


def _check(got, want, err, dims):
    for t, w, e, name in zip(got, want, err, ("dx", "dwg", "dwu")):
        v = _values(t)
        ref.assert_bf16(v, w, e, name)
        if min(dims) >= 64:
            # two independent roundings, in the 2-norm each below 2^-9 of the values
            assert np.linalg.norm(v - w) <= 2.0 ** -8 * np.linalg.norm(w), name


@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 200, 128), (31, 7, 128), (33, 64, 256), (64, 65, 384),
                                   (129, 500, 640), (300, 8, 128), (257, 130, 1152), (500, 333, 512)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_matches_the_formula(M, N, K, act):
    say(f"grad M={M} N={N} K={K} act={act}")
    data = _case(M, N, K, M + N + K)
    bufs = [guarded(s) for s in ((M, K), (N, K), (N, K))]
    got = fp8.gated_nt_grad(*[_bf16(a) for a in data], act=act, out=[b[1] for b in bufs])
    want, err = ref.gated_grad(*data, act)
    _check(got, want, err, (M, N, K))
    for full, out in bufs:
        check_guards(full, out.numel())


@pytest.mark.parametrize("M,N,K,split", [(64, 2048, 7168, True), (4096, 128, 256, True), (1024, 512, 28672, False)])
def test_gradient_split_and_large(M, N, K, split):
    """Few long contractions (split), and enough work for the large tiles; the
    reference in 64 bits on the GPU."""
    say(f"grad large M={M} N={N} K={K}")
    plain = 2 * 2 * M * ((N + 63) // 64 * 64)
    assert (fp8.load_library().fp8_gated_grad_workspace_size(M, N, K) > plain) == split
    g = torch.Generator(device="cuda").manual_seed(M)

    def rand(r, c, s):
        return (torch.randn((r, c), generator=g, device="cuda") * s).to(torch.bfloat16)

    ops = [rand(M, N, 0.1), rand(M, N, 1.5), rand(M, N, 1.5), rand(M, K, 1.0), rand(N, K, 0.05), rand(N, K, 0.05)]
    got = fp8.gated_nt_grad(*ops)
    dh, gg, u, x, wg, wu = (t.double() for t in ops)
    p = torch.sigmoid(gg)
    dg, du = dh * u * p * (1 + gg * (1 - p)), dh * gg * p
    pairs = [(got[0], torch.matmul(dg, wg) + torch.matmul(du, wu),
              torch.matmul(dg.abs(), wg.abs()) + torch.matmul(du.abs(), wu.abs())),
             (got[1], torch.matmul(dg.t().contiguous(), x), torch.matmul(dg.abs().t().contiguous(), x.abs())),
             (got[2], torch.matmul(du.t().contiguous(), x), torch.matmul(du.abs().t().contiguous(), x.abs()))]
    for t, want, mag in pairs:
        diff = (t.double() - want).abs()
        # dg and du off by one rounding each, sums of at most 2^-24 (n / 16 + 64), one rounding
        n = max(2 * N, M)
        assert bool((diff <= (1.02 * ref.U_BF16 + (n / 16 + 64) * ref.U_F32 + 2 ** -18) * mag
                     + 1.01 * ref.U_BF16 * want.abs()).all())
        assert float(torch.linalg.norm(diff)) <= 2.0 ** -8 * float(torch.linalg.norm(want))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_matches_differences(act):
    """Directional derivatives of sum(dh * h).  x and w are small integers over
    16, so that g and u are BF16 values and the saved projections exact."""
    M, N, K = 24, 40, 128
    rng = np.random.default_rng(11)
    x = rng.integers(-1, 2, (M, K)).astype(np.float64)
    wg, wu = (rng.integers(-2, 3, (N, K)) / 16.0 for _ in range(2))
    g, u = x @ wg.T, x @ wu.T
    assert np.array_equal(g, ref.to_bf16(g)) and np.array_equal(u, ref.to_bf16(u))
    dh = ref.to_bf16(rng.standard_normal((M, N)))
    say(f"grad differences {act}")
    got = [_values(t) for t in fp8.gated_nt_grad(*[_bf16(a) for a in (dh, g, u, x, wg, wu)], act=act)]
    _, err = ref.gated_grad(dh, g, u, x, wg, wu, act)

    def loss(x, wg, wu):
        return float(np.sum(dh * (ref.act_value(act, x @ wg.T) * (x @ wu.T))))

    eps = 1e-5
    at = [x, wg, wu]
    for i in range(3):
        v = rng.standard_normal(at[i].shape)
        plus, minus = ([a + s * eps * v if j == i else a for j, a in enumerate(at)] for s in (1, -1))
        want = (loss(*plus) - loss(*minus)) / (2 * eps)
        tol = np.sum(np.abs(v) * (1.02 * err[i] + 1.01 * ref.U_BF16 * np.abs(got[i])))
        # the difference's own error: third derivatives (order eps^2) and 64-bit rounding over eps
        tol += 1e-4 * np.linalg.norm(v)
        assert abs(np.sum(got[i] * v) - want) <= tol, (i, np.sum(got[i] * v), want, tol)


def test_parts_and_empty():
    M, N, K = 70, 96, 256
    data = _case(M, N, K, 2)
    ops = [_bf16(a) for a in data]
    say("grad parts")
    dx, dwg, dwu = fp8.gated_nt_grad(*ops)
    only = fp8.gated_nt_grad(*ops, need_dw=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
    only = fp8.gated_nt_grad(*ops, need_dx=False)
    assert only[0] is None and torch.equal(only[1], dwg) and torch.equal(only[2], dwu)
    say("grad of no tokens")
    e = [ops[0][:0], ops[1][:0], ops[2][:0], ops[3][:0], ops[4], ops[5]]
    dx0, dg0, du0 = fp8.gated_nt_grad(*e, out=(torch.empty((0, K), dtype=torch.bfloat16, device="cuda"),
                                               torch.full_like(dwg, 7), torch.full_like(dwu, 7)))
    torch.cuda.synchronize()
    assert dx0.shape == (0, K) and not dg0.any() and not du0.any()
    say("grad of no columns")
    e = [t[:, :0].contiguous() for t in ops[:3]] + [ops[3], ops[4][:0], ops[5][:0]]
    dx0, dg0, _ = fp8.gated_nt_grad(*e)
    torch.cuda.synchronize()
    assert not dx0.any() and dg0.shape == (0, K)


def test_extreme_gates_and_rows_of_zeros():
    M, N, K = 16, 64, 128
    data = _case(M, N, K, 4)
    data[1][:] = np.where(np.arange(N) % 2, 1e30, -1e30)
    data[1][:, :8] = [0, 88, -88, 100, -100, 3e38, -3e38, 1e-30]
    data[1] = ref.to_bf16(data[1])
    data[0][3] = 0
    for act in ("silu", "gelu"):
        say(f"grad extreme {act}")
        ops = [_bf16(a) for a in data]
        dx, dwg, dwu = (_values(t) for t in fp8.gated_nt_grad(*ops, act=act))
        keep = np.abs(data[1][0]) < 1e20
        with np.errstate(over="ignore", invalid="ignore"):
            # act'(g) is 0 or 1 there; u's gradient takes act(g) = g or 0
            d = np.where(np.abs(data[1]) < 1e20, ref.act_grad(act, np.where(np.abs(data[1]) < 1e20, data[1], 0.0)),
                         (data[1] > 0) * 1.0)
        dg = data[0] * data[2] * d
        want = dg.T @ data[3]
        mag = np.abs(dg).T @ np.abs(data[3])
        assert np.all(np.isfinite(dwg))
        assert np.all(np.abs(dwg - want) <= 3 * ref.U_BF16 * mag + 1e-12)
        assert np.all(dx[3] == 0) and keep.any()


def test_refusals():
    data = _case(16, 64, 128, 1)
    ops = [_bf16(a) for a in data]
    say("grad refusals")
    with pytest.raises(ValueError, match="act"):
        fp8.gated_nt_grad(*ops, act="tanh")
    with pytest.raises(TypeError):
        fp8.gated_nt_grad(ops[0].float(), *ops[1:])
    with pytest.raises(ValueError):
        fp8.gated_nt_grad(ops[0][:15], *ops[1:])
    with pytest.raises(ValueError):
        fp8.gated_nt_grad(ops[0].t().contiguous().t(), *ops[1:])
    with pytest.raises(fp8.Fp8GemmError) as e:
        fp8.gated_nt_grad(*ops, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 7
    bad = [ops[0], ops[1], ops[2]] + [t[:, :100].contiguous() for t in ops[3:]]
    with pytest.raises(fp8.Fp8GemmError) as e:
        fp8.gated_nt_grad(*bad)
    assert e.value.status == 2


def test_side_stream_and_graph():
    data = _case(200, 130, 384, 9)
    ops = [_bf16(a) for a in data]
    want = [t.clone() for t in fp8.gated_nt_grad(*ops)]
    outs = [torch.empty_like(t) for t in want]
    ws = torch.empty(fp8.load_library().fp8_gated_grad_workspace_size(200, 130, 384), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("grad on a side stream")
    with torch.cuda.stream(side):
        got = fp8.gated_nt_grad(*ops)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    say("grad graph")
    with torch.cuda.graph(graph):
        fp8.gated_nt_grad(*ops, out=outs, workspace=ws)
    for _ in range(4):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        fp8.gated_nt_grad(*ops)
        torch.cuda.synchronize()


@pytest.mark.parametrize("M,N,K", [(777, 500, 640), (2000, 130, 256), (256, 1024, 1024), (20, 600, 1024),
                                   (256, 4096, 7168)])
def test_split_contractions_are_repeatable(M, N, K):
    """Tiles whose splits are joined by whichever comes last: the same bits in
    every call, in a workspace that holds other values each time, eagerly and
    replayed, and for each result alone."""
    g = torch.Generator(device="cuda").manual_seed(M + N)

    def rand(r, c, s):
        return torch.randn((r, c), generator=g, device="cuda").mul_(s).bfloat16()

    ops = [rand(M, N, 0.1), rand(M, N, 1.5), rand(M, N, 1.5), rand(M, K, 1.0), rand(N, K, 0.05), rand(N, K, 0.05)]
    size = fp8.load_library().fp8_gated_grad_workspace_size(M, N, K)
    say(f"grad splits M={M} N={N} K={K} workspace={size}")
    assert size > 2 * 2 * M * ((N + 63) // 64 * 64)
    full, ws = guarded((size // 2,))
    ws = ws.view(torch.uint8)
    want = [t.clone() for t in fp8.gated_nt_grad(*ops)]
    dg, du = (t.bfloat16().float() for t in _act_grads(*(t.float() for t in ops[:3])))
    for got, ref32 in ((want[0], dg @ ops[4].float() + du @ ops[5].float()), (want[1], dg.t() @ ops[3].float()),
                       (want[2], du.t() @ ops[3].float())):
        # one rounding of each result, one of dg and du, in the 2-norm
        assert float((got.float() - ref32).norm()) <= 2.0 ** -8 * float(ref32.norm())
    for i in range(12):
        ws.fill_(17 * i)
        assert all(torch.equal(a, b) for a, b in zip(fp8.gated_nt_grad(*ops, workspace=ws), want))
    check_guards(full, size // 2)
    outs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.gated_nt_grad(*ops, out=outs, workspace=ws)
    for _ in range(4):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        fp8.gated_nt_grad(*ops)


def _act_grads(dh, g, u):
    p = torch.sigmoid(g)
    return dh * u * p * (1 + g * (1 - p)), dh * g * p
