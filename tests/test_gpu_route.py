"""The router's choice and its gradient against their 64-bit forms: every
width of a lane's share, ties, masked experts, rows without any, NaN and
infinities, odd sizes and alignments."""
import numpy as np
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
import routing_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _check(logits, k, renorm, scale, what):
    w, ids = fp8.route_topk(logits, k, renormalize=renorm, scale=scale)
    l = logits.double().cpu().numpy()
    rw, rids = ref.route(l, k, renorm, scale)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), rids), what
    ref.assert_near(w.double().cpu().numpy(), rw, ref.route_error(l, rw), what)
    return w, ids


@pytest.mark.parametrize("E,k", [(1, 1), (3, 3), (63, 5), (64, 64), (65, 2), (128, 8), (162, 6), (256, 8), (257, 9),
                                 (500, 16), (512, 1), (1000, 33), (1024, 64)])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_choice_and_gradient(E, k, kind):
    g = torch.Generator(device="cuda").manual_seed(E * 100 + k)
    for T, renorm, scale in ((1, True, 1.0), (37, True, 2.5), (130, False, 1.0), (5, False, 0.3)):
        say("route", E, k, kind, T, renorm)
        logits = (3.0 * torch.randn((T, E), generator=g, device="cuda")).to(TYPES[kind])
        if E > 8:
            logits[T // 2, : E - k + 1] = -float("inf")          # fewer than k are left
        if T > 3:
            logits[1] = -float("inf")                              # and none
        w, ids = _check(logits, k, renorm, scale, f"{E} {k} {kind} {T}")
        dw = torch.randn((T, k), generator=g, device="cuda")
        d = fp8.route_topk_grad(dw, logits, ids, renormalize=renorm, scale=scale)
        assert d.dtype == logits.dtype
        l, i = logits.double().cpu().numpy(), ids.cpu().numpy()
        rd, mag = ref.route_grad(dw.double().cpu().numpy(), l, i, renorm, scale)
        # probabilities as in the choice (one factor of route_error), a sum of k terms in six steps, three products
        bound = ref.route_error(l, np.ones((1, 1))) * mag * 2 + (6 + k + 8) * ref.U * mag
        ref.assert_near(d.double().cpu().numpy(), rd, ref.rounded(bound, rd, kind == "bf16"), f"grad {E} {k} {kind}")


def test_ties_take_the_lowest_index():
    say("route ties")
    g = torch.Generator(device="cuda").manual_seed(1)
    for E in (7, 100, 256, 700):
        logits = torch.randint(-2, 3, (64, E), generator=g, device="cuda").float()
        logits[0] = 0.0
        logits[1, ::2] = -0.0                   # equal to the zeros beside it
        logits[1, 1::2] = 0.0
        for dtype in (torch.float32, torch.bfloat16):
            _, ids = _check(logits.to(dtype), min(E, 12), True, 1.0, f"ties {E}")
            assert ids[0].tolist() == ids[1].tolist() == list(range(min(E, 12)))


def test_extremes():
    say("route extremes")
    big = torch.finfo(torch.float32).max
    rows = torch.tensor([[big, -big, 0.0, 1.0], [-big, -big, -big, -big], [1e-45, 0.0, -1e-45, 1.0],
                         [-100.0, -200.0, -300.0, 60.0]], device="cuda")
    for renorm in (True, False):
        _check(rows, 3, renorm, 1.0, "extremes")
    nan, inf = float("nan"), float("inf")
    bad = torch.tensor([[0.0, nan, 1.0, inf], [nan, 5.0, nan, -inf], [inf, 0.0, inf, 1.0], [0.0, 1.0, 2.0, 3.0]], device="cuda")
    w, ids = fp8.route_topk(bad, 2)
    assert ids.tolist() == [[1, 3], [0, 2], [0, 2], [3, 2]]
    assert torch.isnan(w[:3]).all() and torch.isfinite(w[3]).all()
    # a NaN that is not chosen: only weights over all experts see it
    assert torch.isnan(fp8.route_topk(bad, 2, renormalize=False)[0][:3]).all()


def test_alignments_and_outputs():
    """Rows that begin off any vector, and outputs that end in sentinels."""
    g = torch.Generator(device="cuda").manual_seed(2)
    for dtype in (torch.float32, torch.bfloat16):
        for E in (256, 160, 512):
            say("route alignment", dtype, E)
            flat = torch.randn(9 * E + 1, generator=g, device="cuda").to(dtype)
            view = flat[1:].view(9, E)
            w, ids = _check(view, 8, False, 1.0, f"misaligned {E}")
            keep = torch.full((9 * 8 + 2,), -77, dtype=torch.int32, device="cuda")
            out = (torch.full((9 * 8 + 2,), 7.0, device="cuda")[1:-1].view(9, 8), keep[1:-1].view(9, 8))
            got = fp8.route_topk(view, 8, renormalize=False, out=out)
            assert got[0] is out[0] and torch.equal(got[0], w) and torch.equal(got[1], ids)
            assert keep[0] == -77 and keep[-1] == -77
            dw = torch.randn((9, 8), generator=g, device="cuda")
            d = fp8.route_topk_grad(dw, view, ids, renormalize=False)
            edge = torch.full((9 * E + 2,), 7.0, dtype=dtype, device="cuda")
            fp8.route_topk_grad(dw, view, ids, renormalize=False, out=edge[1:-1].view(9, E))
            assert torch.equal(edge[1:-1].view(9, E), d) and edge[0] == 7 and edge[-1] == 7


def test_gradient_of_given_choices():
    """Indices outside the experts add nothing, one that stands twice counts twice."""
    say("route given choices")
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn((6, 20), generator=g, device="cuda")
    ids = torch.randint(-3, 24, (6, 5), generator=g, device="cuda", dtype=torch.int32)
    ids[0] = torch.tensor([3, 3, 7, -1, 3], device="cuda")
    ids[1] = -1
    dw = torch.randn((6, 5), generator=g, device="cuda")
    dw[0, 3] = float("nan")                      # of no expert
    for renorm in (True, False):
        d = fp8.route_topk_grad(dw, logits, ids, renormalize=renorm)
        rd, mag = ref.route_grad(dw.double().cpu().numpy(), logits.double().cpu().numpy(), ids.cpu().numpy(), renorm, 1.0)
        ref.assert_near(d.double().cpu().numpy(), rd, 200 * ref.U * mag, "given")


def test_empty_and_large():
    say("route empty and large")
    w, ids = fp8.route_topk(torch.empty((0, 16), device="cuda"), 4)
    assert w.shape == ids.shape == (0, 4)
    assert fp8.route_topk_grad(w, torch.empty((0, 16), device="cuda"), ids).shape == (0, 16)
    logits = torch.randn((70001, 64), device="cuda").bfloat16()
    _check(logits, 4, True, 1.0, "large")


def test_refusals():
    say("route refusals")
    l = torch.randn((4, 16), device="cuda")
    with pytest.raises(fp8.Fp8GemmError):
        fp8.route_topk(l, 17)
    with pytest.raises(fp8.Fp8GemmError):
        fp8.route_topk(l, 0)
    with pytest.raises(ValueError):
        fp8.route_topk(l.t(), 2)
    with pytest.raises(TypeError):
        fp8.route_topk(l.double(), 2)
    w, ids = fp8.route_topk(l, 2)
    with pytest.raises(ValueError):
        fp8.route_topk(l, 2, out=(w[:3], ids))
    with pytest.raises(TypeError):
        fp8.route_topk_grad(w, l, ids.long())
    with pytest.raises(ValueError):
        fp8.route_topk_grad(w[:, :1].contiguous(), l, ids)
