"""Adapters of more than 4 GB of tokens, projections and weights, exactly: all
operands are whole numbers small enough that FP32 holds every product, sum and
half, so each output is one rounding of a known value."""
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import say

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


def _whole(gen, shape, most):
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda", dtype=torch.int8).bfloat16()


def _beside(T, *rows):
    """Tokens at both ends and on either side of 2 and 4 GB for rows of these widths (BF16)."""
    at = {0, 1, 2, T - 1, T - 2, T - 3, T // 2}
    for width in rows:
        for bound in (2 ** 31, 2 ** 32):
            t = bound // (2 * width)
            at |= {t - 1, t, t + 1, t + 2}
    return sorted(t for t in at if 0 <= t < T)


def _check(x, a, b, y, idx, out, tokens):
    for t in tokens:
        i, want = int(idx[t]), y[t].double()
        if 0 <= i < a.shape[0]:
            want = want + 0.5 * torch.mv(b[i].double(), torch.mv(a[i].double(), x[t].double()))
        assert float(want.abs().max()) < 2 ** 23
        assert torch.equal(out[t], want.bfloat16()), t


@pytest.mark.parametrize("L,N,group", [(4, 7000, 4), (20000, 64, 1), (20000, 7000, 1)])
def test_many_tokens(L, N, group):
    """In groups of tiles, and in single tiles (many adapters, of which some occur)."""
    say("far adapters", L, N)
    T, K, R = 330000, 7168, 8
    assert fp8.adapters_plan(T, L, N, K, R)["group"] == group
    gen = torch.Generator(device="cuda").manual_seed(12)
    x, a, b, y = _whole(gen, (T, K), 1), _whole(gen, (L, R, K), 1), _whole(gen, (L, N, R), 1), _whole(gen, (T, N), 3)
    ids = min(L, 1000)
    idx = torch.randint(-1, ids, (T,), generator=gen, device="cuda", dtype=torch.int32)
    tokens = _beside(T, K, N)
    none, idx[T - 3] = tokens[1], ids - 1
    idx[none] = -1
    out = fp8.add_adapters(x, a, b, torch.full((L,), 0.5, device="cuda"), fp8.adapter_rows(idx, ids), y)
    extra = torch.randint(0, T, (60,), generator=gen, device="cuda").tolist()
    _check(x, a, b, y, idx, out, tokens + extra)


def test_few_tokens():
    """The one kernel, at both ends and beside 4 GB of a and of b."""
    say("far adapters, few tokens")
    L, K, N, R = 1000, 43008, 40000, 64
    gen = torch.Generator(device="cuda").manual_seed(13)
    a, b = _whole(gen, (L, R, K), 1), _whole(gen, (L, N, R), 1)
    far = [2 ** 32 // (2 * R * width) for width in (K, N)]
    for first in range(2):
        idx = torch.tensor([[L - 1, 0, -1, 499], [far[0], far[0] + 1, far[1], far[1] + 1]][first], device="cuda", dtype=torch.int32)
        T = idx.numel()
        assert fp8.adapters_plan(T, L, N, K, R)["whole"] > 0
        x, y = _whole(gen, (T, K), 1), _whole(gen, (T, N), 3)
        out = fp8.add_adapters(x, a, b, torch.full((L,), 0.5, device="cuda"), fp8.adapter_rows(idx, L), y)
        _check(x, a, b, y, idx, out, range(T))
