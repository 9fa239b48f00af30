"""The largest grids that the moving of rows and the router launch: just under
2^32 threads, every row checked; and the sizes above them refused."""
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import say

pytestmark = pytest.mark.gpu

GRID = (2 ** 32 - 1) // 256          # workgroups of 256 threads


def _refused(call):
    with pytest.raises(fp8.Fp8GemmError, match="UNSUPPORTED"):
        call()


def test_router():
    T = 4 * GRID
    say("largest router", T)
    logits = torch.zeros((T + 1, 2), dtype=torch.bfloat16, device="cuda")
    second = torch.arange(T, device="cuda") % 3 == 0
    logits[:T, 1] = second.to(torch.bfloat16)
    w, ids = fp8.route_topk(logits[:T], 1)
    assert torch.equal(ids[:, 0] == 1, second) and bool((w == 1).all())
    d = fp8.route_topk_grad(w, logits[:T], ids, renormalize=False)
    # p (1 - p) for the chosen of two, its negative for the other; one half each where they are equal
    p = torch.sigmoid(torch.ones((), dtype=torch.float64))
    want = torch.where(second, float(p * (1 - p)), 0.25)
    at = torch.cat((torch.arange(1000, device="cuda"), torch.arange(T - 1000, T, device="cuda")))
    got = d[at].double().gather(1, ids[at].long())[:, 0]
    assert bool(((got - want[at]).abs() <= 2.0 ** -8 * want[at]).all())
    assert bool(((d.abs().sum(1) > 0.3) & (d.sum(1).abs() < 1e-2)).all())
    _refused(lambda: fp8.route_topk(logits, 1))


def test_rows():
    T = 4 * GRID * 8 // 9            # and a wave per 8 rows to clear
    say("largest dispatch and combine", T)
    x = (torch.arange(T, device="cuda") % 251).to(torch.bfloat16)[:, None]
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")[:, None]
    src = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    src[5] = -1
    pos[T - 6] = -1
    xs = fp8.expert_dispatch(x, pos, src)
    want = x.flip(0)
    want[5] = 0
    assert torch.equal(xs, want)
    back = fp8.expert_combine(xs, pos)
    x[T - 6] = 0
    assert torch.equal(back, x)
    longer = torch.zeros((4 * GRID + 1, 1), dtype=torch.int32, device="cuda")
    _refused(lambda: fp8.expert_combine(xs, longer))


def test_combine_gradient():
    T = GRID
    say("largest combine gradient", T)
    dout = (torch.arange(T, device="cuda") % 13).float()[:, None].repeat(1, 2)
    y = (torch.arange(T, device="cuda") % 7).float()[:, None].repeat(1, 2)
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")[:, None]
    w = torch.full((T, 1), 0.5, device="cuda")
    dy, dw = fp8.expert_combine_grad(dout, y, pos, w)
    assert torch.equal(dy, 0.5 * dout.flip(0)) and torch.equal(dw[:, 0], 2 * dout[:, 0] * y[:, 0].flip(0))
    one = pos.new_zeros((T + 1, 1))
    _refused(lambda: fp8.expert_combine_grad(torch.zeros((T + 1, 2), device="cuda"), y, one, None))
