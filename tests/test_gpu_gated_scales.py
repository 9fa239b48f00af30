"""The quantized gated block at the size of a long prefill, against 64 bits on
the GPU: a scale differs from the 64-bit one only where the FP32 error of the
group's maximum reaches a threshold, and code times scale stands for h."""
import numpy as np
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
import oracle
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _decoded(q, s_rows):
    """E4M3 codes (R, K) times their scales (R, K/128), in 64 bits."""
    values = torch.from_numpy(oracle.e4m3_decode(np.arange(256)).astype(np.float64)).cuda()
    R, K = q.shape
    return (values[q.long()].view(R, K // 128, 128) * s_rows.double()[..., None]).view(R, K)


@pytest.mark.parametrize("M,N,K", [(8192, 4096, 7168)])
@pytest.mark.parametrize("pow2", [True, False])
def test_scales_of_a_long_prefill(M, N, K, pow2):
    say(f"gated quantized prefill M={M} N={N} K={K} pow2={pow2}")
    gen = torch.Generator(device="cuda").manual_seed(M + pow2)
    x = torch.randn((M, K), generator=gen, device="cuda")
    x *= 1.0 + 30.0 * (torch.rand((M, K), generator=gen, device="cuda") < 0.001)
    xq, sa = fp8.quant_1x128(x, ue8m0=pow2)
    wq = [fp8.quant_128x128(torch.randn((N, K), generator=gen, device="cuda") * 0.02, ue8m0=pow2) for _ in range(2)]
    hq, sh = fp8.gated_nt_qout(xq, sa, *wq[0], *wq[1], ue8m0=pow2)

    xd = _decoded(xq, sa.t())
    rows = torch.arange(N, device="cuda") // 128
    wd = [_decoded(q, s[rows]) for q, s in wq]
    g, u = (torch.matmul(xd, w.t()) for w in wd)
    steps = K / 16 + 2 * K / 128 + 32           # FP32 roundings of a sum, as in ffn_reference.gated
    eg, eu = (steps * ref.U_F32 * torch.matmul(xd.abs(), w.t().abs()) for w in wd)
    a = g * torch.sigmoid(g)
    h = (a * u).view(M, N // 128, 128)
    e = 1.13 * u.abs() * eg + a.abs() * eu + 1.13 * eg * eu + (8 + 4 * g.abs()) * ref.U_F32 * (a * u).abs()
    e = e.view(M, N // 128, 128)
    del g, u, a, eg, eu

    s, amax = sh.t().double(), h.abs().amax(2)
    lo, hi = ((m.clamp_min(1e-4) / 448) for m in (amax - e.amax(2), amax + e.amax(2)))
    if pow2:
        up = torch.exp2(torch.ceil(torch.log2(amax.clamp_min(1e-4) / 448)))
        lo, hi = (torch.exp2(torch.ceil(torch.log2(v))) for v in (lo, hi))
        assert len(up.unique()) > 1
        # Roundings of a sum add like a random walk: sqrt(steps) * 2^-24 < 2^-19 of
        # the maximum, and maxima spread over factors of two come within that of a
        # threshold for about 2 * 2^-19 / ln 2 of the groups, 1.4 of 262144
        assert int((s != up).sum()) <= 16
    assert bool(((s >= lo * (1 - 2 ** -22)) & (s <= hi * (1 + 2 ** -22))).all())
    pair = _decoded(hq, s).view(h.shape)
    # nearest E4M3: half a unit of 3 fraction bits, or of the subnormals
    bound = 1.01 * e + 2.0 ** -4 * (h.abs() + e) * (1 + 2 ** -20) + 2.0 ** -10 * s[..., None] * (1 + 2 ** -20)
    assert bool(((pair - h).abs() <= bound).all())
