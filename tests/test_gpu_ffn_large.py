"""The feed-forward operators where byte and element offsets pass 32 bits:
operands and results of over 4 GiB, checked on slices at both ends and across
the 4 GiB line against 64-bit products."""
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _codes(shape, seed):
    """Finite E4M3 bytes below 2 in magnitude."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 0x40, shape, generator=g, device="cuda", dtype=torch.uint8)
    c[..., 1::2] |= 0x80
    return c


def _close(got, want, mag, steps):
    """BF16 results of FP32 sums of at most `steps` roundings of sums of `mag`."""
    diff = (got.double() - want).abs()
    assert bool(torch.isfinite(diff).all())
    assert bool((diff <= 1.02 * ref.U_BF16 * want.abs() + (steps * ref.U_F32 + 2.0 ** -30) * mag + 2.0 ** -133).all())


@pytest.mark.parametrize("save", [False, True])
def test_gated_over_4_gib_of_activations(save):
    M, N, K = 70016, 160, 65536
    xq = _codes((M, K), 1)
    gq, uq = _codes((N, K), 2), _codes((N, K), 3)
    sa = torch.full((K // 128, M), 2.0 ** -6, device="cuda")
    sg, su = (torch.full(((N + 127) // 128, K // 128), 2.0 ** -4, device="cuda") for _ in range(2))
    say(f"gated M={M} N={N} K={K} save={save}")
    out = fp8.gated_nt(xq, sa, gq, sg, uq, su, save=save)
    if not save:
        out = (out,)
    w = [q.view(torch.float8_e4m3fn).double() * 2.0 ** -10 for q in (gq, uq)]
    for rows in (slice(0, 64), slice(65500, 65600), slice(M - 64, M)):
        x = xq[rows].view(torch.float8_e4m3fn).double()
        g, u = (torch.matmul(x, a.t()) for a in w)
        mg, mu = (torch.matmul(x.abs(), a.abs().t()) for a in w)
        p = torch.sigmoid(g)
        steps = K / 16 + 2 * K / 128 + 32
        _close(out[0][rows], g * p * u, 1.13 * (u.abs() * mg + (g * p).abs() * mu) + 1e-3 * mg * mu
               + (12 + 4 * g.abs()) / steps * (g * p * u).abs(), steps)
        if save:
            _close(out[1][rows], g, mg, steps)
            _close(out[2][rows], u, mu, steps)


def test_gradient_over_4_gib():
    """K of 4 Mi columns: X and dX hold over 4 GiB, and every run of loads along
    the contraction is cut to a few blocks."""
    M, N, K = 600, 8, 1 << 22
    g0 = torch.Generator(device="cuda").manual_seed(4)

    def rand(r, c, s):
        return torch.randn((r, c), generator=g0, device="cuda", dtype=torch.bfloat16) * s

    dh, g, u = rand(M, N, 0.1), rand(M, N, 1.0), rand(M, N, 1.0)
    x, wg, wu = rand(M, K, 1.0), rand(N, K, 0.5), rand(N, K, 0.5)
    say(f"grad M={M} N={N} K={K}")
    dx, dwg, dwu = fp8.gated_nt_grad(dh, g, u, x, wg, wu)
    gd = g.double()
    p = torch.sigmoid(gd)
    dg, du = dh.double() * u.double() * p * (1 + gd * (1 - p)), dh.double() * gd * p
    for cols in (slice(0, 300), slice((1 << 21) - 100, (1 << 21) + 100), slice(K - 300, K)):
        xs, gs, us = (t[:, cols].double() for t in (x, wg, wu))
        for got, a, b in ((dwg, dg.t(), xs), (dwu, du.t(), xs)):
            a = a.contiguous()
            mag = torch.matmul(a.abs(), b.abs())
            _close(got[:, cols], torch.matmul(a, b), mag * (1 + 1.02 * ref.U_BF16 / (102 * ref.U_F32)), 102)
        mag = torch.matmul(dg.abs(), gs.abs()) + torch.matmul(du.abs(), us.abs())
        _close(dx[:, cols], torch.matmul(dg, gs) + torch.matmul(du, us),
               mag * (1 + 1.02 * ref.U_BF16 / (72 * ref.U_F32)), 72)


def test_gemv_over_4_gib_of_weights():
    M, N, K = 2, 300000, 32768
    g0 = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((M, K), generator=g0, device="cuda", dtype=torch.bfloat16)
    q = torch.randint(0, 256, (N, K // 2), generator=g0, device="cuda", dtype=torch.uint8)
    s = (0.01 + torch.rand((K // 128, N), generator=g0, device="cuda") * 0.01).to(torch.bfloat16)
    z = torch.randint(0, 16, (K // 128, N), generator=g0, device="cuda", dtype=torch.uint8)
    say(f"gemv M={M} N={N} K={K}")
    y = fp8.gemv_w4(x, q, s, zeros=z)
    for rows in (slice(0, 100), slice(262100, 262200), slice(N - 100, N)):
        c = torch.stack((q[rows] & 15, q[rows] >> 4), 2).view(-1, K).double()
        sc, zp = (t[:, rows].t().double().repeat_interleave(128, 1) for t in (s, z))
        w, mag = (c - zp) * sc, (c + zp) * sc
        _close(y[:, rows], torch.matmul(x.double(), w.t()), torch.matmul(x.double().abs(), mag.t()), 3 * K / 32 + 64)


def test_clip_over_4_gib_in_one_tensor():
    n = (1 << 31) + 12345
    g = torch.empty(n + 1, dtype=torch.bfloat16, device="cuda")[1:]
    g.fill_(2.0 ** -10)
    g[-1] = 3.0
    out = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    say(f"clip one tensor of {n}")
    norm = float(fp8.clip_grad_norm([g], 1.0, out=[out]))
    want = float(((n - 1) * 2.0 ** -20 + 9.0) ** 0.5)
    assert abs(norm - want) <= 2.0 ** -23 * want
    coef = 1.0 / (want + 1e-6)
    small, last = float(out[0]), float(out[-1])
    assert abs(small - 2.0 ** -10 * coef) <= ref.U_BF16 * 2.0 ** -10 * coef * 1.01
    assert abs(last - 3.0 * coef) <= ref.U_BF16 * 3.0 * coef * 1.01
    assert bool((out[:-1] == out[0]).all())
