"""Rows whose offsets pass 32 bits: more than 4 GB of tokens, experts' rows and
projections."""
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import say

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


def test_rows_behind_four_gigabytes():
    say("large rows")
    T, K, E = 330000, 7168, 3           # 4.7 GB in BF16
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-3, 4, (T, K), generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    ids = torch.randint(0, E, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    pos, src, m_indices, counts = fp8.expert_sort(ids, E)
    rows = src.shape[0]
    assert int(counts.sum()) == T and int(pos.min()) >= 0
    xs = fp8.expert_dispatch(x, pos, src)
    at = torch.cat((torch.arange(200, device="cuda"), torch.arange(T - 200, T, device="cuda")))
    assert torch.equal(xs[pos[at, 0].long()], x[at])
    assert bool((xs[src < 0] == 0).all())
    w = torch.full((T, 1), 0.5, device="cuda")
    back = fp8.expert_combine(xs, pos, w)
    assert torch.equal(back, x * 0.5)
    dy, dw = fp8.expert_combine_grad(x, xs, pos, w, src)
    assert torch.equal(dy, xs * 0.5)
    assert torch.equal(dw[at, 0], x[at].float().square().sum(1))        # whole numbers below 2^24
    del back, dy, xs
    xq, sa = fp8.expert_dispatch_quant(x, pos, rows)
    q, s = fp8.quant_1x128(x[at].float())
    assert torch.equal(xq[pos[at, 0].long()], q) and torch.equal(sa[:, pos[at, 0].long()], s)


@pytest.mark.parametrize("L,N,group", [(4, 7000, 4), (20000, 64, 1)])
def test_adapters_behind_four_gigabytes(L, N, group):
    """In groups of tiles, and in single tiles (many adapters, of which some occur)."""
    say("large adapters", L)
    T, K, R = 330000, 7168, 8
    assert fp8.adapters_plan(T, L, N, K, R)["group"] == group
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randint(-1, 2, (T, K), generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    a = torch.randint(-1, 2, (L, R, K), generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    b = torch.randint(-1, 2, (L, N, R), generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    y = torch.randint(-3, 4, (T, N), generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    idx = torch.randint(-1, min(L, 1000), (T,), generator=gen, device="cuda", dtype=torch.int32)
    scale = torch.full((L,), 0.5, device="cuda")
    rows = fp8.adapter_rows(idx, min(L, 1000))
    out = fp8.add_adapters(x, a, b, scale, rows, y)
    for t in (0, 1, 1999, T // 2, T - 2, T - 1):
        i = int(idx[t])
        want = y[t].double()
        if i >= 0:
            want = want + 0.5 * (b[i].double() @ (a[i].double() @ x[t].double()))
        # whole and half numbers that both products hold exactly: one rounding
        assert float((out[t].double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max())


def test_adapters_of_few_tokens_behind_four_gigabytes():
    """The one kernel, at both ends of a and b of more than 5 GB each."""
    say("large adapters, few tokens")
    T, L, K, N, R = 4, 1000, 43008, 40000, 64
    assert fp8.adapters_plan(T, L, N, K, R)["whole"] > 0
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-1, 2, (T, K), generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    a = torch.randint(-1, 2, (L, R, K), generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    b = torch.randint(-1, 2, (L, N, R), generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    y = torch.randint(-3, 4, (T, N), generator=gen, device="cuda", dtype=torch.int8).bfloat16()
    idx = torch.tensor([L - 1, 0, -1, 499], device="cuda", dtype=torch.int32)
    out = fp8.add_adapters(x, a, b, torch.full((L,), 0.5, device="cuda"), fp8.adapter_rows(idx, L), y)
    for t in range(T):
        i, want = int(idx[t]), y[t].double()
        if i >= 0:
            want = want + 0.5 * (b[i].double() @ (a[i].double() @ x[t].double()))
        # whole and half numbers that both products hold exactly: one rounding
        assert float((out[t].double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max())
