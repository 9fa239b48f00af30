"""The gradient of the gated block with operands that are the leading part of
larger buffers: what lies behind them is never read, or a NaN there would show
in the sums."""
import numpy as np
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import bf16_bits, bf16_to_f64, say

pytestmark = pytest.mark.gpu


def _leading(a, tail):
    """BF16 values in the first rows of a buffer whose last `tail` rows are NaN."""
    full = torch.full((a.shape[0] + tail, a.shape[1]), float("nan"), dtype=torch.bfloat16, device="cuda")
    bits = ref.bf16_bits_of(a).view(np.int16)
    full[:a.shape[0]] = torch.from_numpy(np.ascontiguousarray(bits)).cuda().view(torch.bfloat16)
    return full[:a.shape[0]]


# N % 64 in 1..32 (the last 32 columns of the padded dg and du hold none of W's
# rows) and in 33..63; one block, several, and split contractions
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (33, 31, 128), (5, 65, 128), (77, 95, 256), (129, 130, 384),
                                   (201, 600, 640), (31, 607, 128), (19, 1000, 1024), (95, 2113, 384)])
def test_nothing_behind_the_operands_is_read(M, N, K):
    say(f"grad ends M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K)
    shapes, scale = [(M, N)] * 3 + [(M, K), (N, K), (N, K)], [0.1, 1.5, 1.5, 1.0, 0.05, 0.05]
    data = [ref.to_bf16(rng.standard_normal(s) * c) for s, c in zip(shapes, scale)]
    got = fp8.gated_nt_grad(*[_leading(a, 160) for a in data])
    want, err = ref.gated_grad(*data, "silu")
    for t, w, e, name in zip(got, want, err, ("dx", "dwg", "dwu")):
        ref.assert_bf16(bf16_to_f64(bf16_bits(t)), w, e, name)


def test_nothing_behind_a_part_is_read():
    """Each gradient by itself."""
    M, N, K = 131, 321, 256
    say("grad ends, parts")
    rng = np.random.default_rng(7)
    shapes, scale = [(M, N)] * 3 + [(M, K), (N, K), (N, K)], [0.1, 1.5, 1.5, 1.0, 0.05, 0.05]
    data = [ref.to_bf16(rng.standard_normal(s) * c) for s, c in zip(shapes, scale)]
    want, err = ref.gated_grad(*data, "gelu")
    for part in ({"need_dw": False}, {"need_dx": False}):
        got = fp8.gated_nt_grad(*[_leading(a, 160) for a in data], act="gelu", **part)
        for t, w, e, name in zip(got, want, err, ("dx", "dwg", "dwu")):
            if t is not None:
                ref.assert_bf16(bf16_to_f64(bf16_bits(t)), w, e, name)
