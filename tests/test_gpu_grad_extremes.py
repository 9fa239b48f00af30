"""The gradient of the gated block at gates far beyond where the exponential
overflows or vanishes: all three results, every row."""
import numpy as np
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import bf16_bits, bf16_to_f64, say

pytestmark = pytest.mark.gpu

GATES = {"closed": [-1e30, -3e37, -1000.0, -88.0, -100.0, -89.5, -1e20, 0.0],
         "open": [1e30, 1e20, 1000.0, 88.0, 100.0, 89.5, 1e25, 1e-30],
         "around the range": [87.0, -87.0, 88.0, -88.0, 89.0, -89.0, 100.0, -100.0],
         "both": [1e37, -1e37, 1e30, -1e30, 88.0, -88.0, 0.0, 1e-30]}


def _bf16(a):
    bits = ref.bf16_bits_of(ref.to_bf16(a)).view(np.int16)
    return torch.from_numpy(np.ascontiguousarray(bits)).cuda().view(torch.bfloat16)


@pytest.mark.parametrize("gates", sorted(GATES))
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_extreme_gates(gates, act):
    M, N, K = 19, 72, 128
    say(f"grad extreme gates {gates} {act}")
    rng = np.random.default_rng(len(gates))
    dh, u = (ref.to_bf16(rng.standard_normal((M, N)) * c) for c in (0.1, 1.5))
    g = ref.to_bf16(np.tile(np.resize(GATES[gates], N), (M, 1)))
    dh[3], dh[:, 5] = 0, 0
    x, wg, wu = (ref.to_bf16(rng.standard_normal(s) * c) for s, c in (((M, K), 1.0), ((N, K), 0.05), ((N, K), 0.05)))
    dx, dwg, dwu = (bf16_to_f64(bf16_bits(t)) for t in
                    fp8.gated_nt_grad(*[_bf16(a) for a in (dh, g, u, x, wg, wu)], act=act))
    # beyond +-1000 the gate is 0 or 1 to all of 64 bits' digits
    inner = np.clip(g, -1000, 1000)
    with np.errstate(over="ignore"):
        a = np.where(g > 1000, g, np.where(g < -1000, 0.0, ref.act_value(act, inner)))
        d = np.where(g > 1000, 1.0, np.where(g < -1000, 0.0, ref.act_grad(act, inner)))
    dg, du = dh * u * d, dh * a
    # dg and du off by one rounding each and by FP32's evaluation of the gate
    # (exponent arguments up to 90: 90 * 2^-24 of it, twice), one rounding of the
    # result; gates below 2^-126 may vanish: 1e-30
    for name, got, want, mag in (("dx", dx, dg @ wg + du @ wu, np.abs(dg) @ np.abs(wg) + np.abs(du) @ np.abs(wu)),
                                 ("dwg", dwg, dg.T @ x, np.abs(dg).T @ np.abs(x)),
                                 ("dwu", dwu, du.T @ x, np.abs(du).T @ np.abs(x))):
        assert np.all(np.isfinite(got)), name
        bad = np.abs(got - want) > 3 * ref.U_BF16 * mag + 1e-30
        assert not bad.any(), (name, np.argwhere(bad)[0], got[bad][0], want[bad][0])
    assert np.all(dx[3] == 0) and np.all(dwg[5] == 0) and np.all(dwu[5] == 0)
