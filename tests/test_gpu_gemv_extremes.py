"""MXFP4 weights over the whole range of their scale bytes, and the smallest
activations."""
import numpy as np
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import dev, host, say

pytestmark = pytest.mark.gpu


def _codes():
    """16 rows whose first element is each E2M1 code, the others zero."""
    q = np.zeros((16, 64), np.uint8)
    q[:, 0] = np.arange(16)
    return q


@pytest.mark.parametrize("M", [1, 16])
def test_every_scale_byte(M):
    say(f"MXFP4 scale bytes M={M}")
    q, want = _codes(), np.array([*ref.E2M1, *-ref.E2M1])
    for e in range(256):
        k = 120 if e < 100 else -120 if e > 150 else 0
        x = torch.zeros((M, 128), device="cuda")
        x[:, 0] = 2.0 ** k
        scales = np.full((1, 16, 4), e, np.uint8).view(np.int32).reshape(1, 16)
        y = host(fp8.gemv_w4(x.bfloat16(), dev(q), dev(scales)).float())
        if e == 255:
            assert np.all(np.isnan(y))
            continue
        w = np.ldexp(want, e - 127)
        w = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)
        assert np.array_equal(y, np.tile(np.ldexp(w, k).astype(np.float32), (M, 1))), e


@pytest.mark.parametrize("k", [-133, -127, -126, -120])
def test_smallest_activations(k):
    """Subnormal BF16 activations count."""
    say(f"activations of 2^{k}")
    x = torch.zeros((2, 128), dtype=torch.float32)
    x[0, 0], x[1, 0] = 2.0 ** k, -2.0 ** k
    x = x.bfloat16().cuda()
    scales = np.full((1, 16, 4), 227, np.uint8).view(np.int32).reshape(1, 16)
    want = np.ldexp(np.array([*ref.E2M1, *-ref.E2M1]), k + 100)
    assert np.array_equal(host(fp8.gemv_w4(x, dev(_codes()), dev(scales)).float()), [want, -want])
    s = torch.full((1, 16), 2.0 ** 100, dtype=torch.bfloat16, device="cuda")
    for zeros in (None, torch.full((1, 16), 8, dtype=torch.uint8, device="cuda")):
        q = np.full((16, 64), 0x88, np.uint8)
        q[:, 0] = 0x80 | np.arange(16)
        want = np.ldexp(np.arange(16.0) - 8, k + 100)
        assert np.array_equal(host(fp8.gemv_w4(x, dev(q), s, zeros=zeros).float()), [want, -want])
