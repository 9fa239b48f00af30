"""Gradient norm and clipping against the 64-bit form: mixed types, sizes from
zero on, views at any alignment, more tensors than one launch takes, values
whose squares leave FP32's range, NaN and infinities."""
import numpy as np
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import say

pytestmark = pytest.mark.gpu

# relative error of one product after the factor's rounding, and the least step
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def _norm(grads):
    return float(np.sqrt(sum(float((g.double() ** 2).sum()) for g in grads)))


def _grads(sizes, types, seed, scale=1.0, odd=True):
    """Views of one flat buffer per type, an odd number of elements apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n, t in zip(sizes, types):
        pad = 1 + 2 * (len(out) % 3) if odd else 0
        out.append((torch.randn(n + pad, generator=g, device="cuda") * scale).to(t)[pad:])
    return out


def _check(grads, outs, norm, max_norm):
    want = _norm(grads)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    coef = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(grads, outs):
        exact = g.double() * coef
        bound = (1.01 * HALF_ULP[g.dtype] + 2.0 ** -23) * exact.abs() + TINY[g.dtype]
        assert bool(((o.double() - exact).abs() <= bound).all())


SETS = {
    "one": ([1], [torch.float32]),
    "odd": ([1, 2, 3, 7, 255, 256, 257, 8191, 8192, 8193, 0, 50001],
            [torch.float32, torch.bfloat16, torch.float16] * 4),
    "many": ([1 + 37 * (i % 29) for i in range(500)], [torch.float32, torch.bfloat16] * 250),
    "large": ([9000000, 5, 33000000, 1], [torch.bfloat16, torch.float32, torch.float32, torch.float16]),
}


@pytest.mark.parametrize("name", sorted(SETS))
@pytest.mark.parametrize("ratio", [0.3, 3.0])
def test_out_of_place(name, ratio):
    sizes, types = SETS[name]
    grads = _grads(sizes, types, 1, 1e-2)
    keep = [g.clone() for g in grads]
    max_norm = ratio * _norm(grads)
    outs = [torch.full((n + 5,), 3.0, dtype=t, device="cuda") for n, t in zip(sizes, types)]
    views = [o[3:3 + n] for o, n in zip(outs, sizes)]
    say(f"clip {name} ratio={ratio}")
    norm = fp8.clip_grad_norm(grads, max_norm, out=views)
    torch.cuda.synchronize()
    _check(keep, views, norm, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    for o, n in zip(outs, sizes):
        assert bool((o[:3] == 3).all()) and bool((o[3 + n:] == 3).all()), "write outside an output"
    if ratio > 1:
        assert all(torch.equal(a, b) for a, b in zip(views, keep))


@pytest.mark.parametrize("name", sorted(SETS))
def test_in_place(name):
    sizes, types = SETS[name]
    grads = _grads(sizes, types, 2)
    keep = [g.clone() for g in grads]
    max_norm = 0.25 * _norm(grads)
    say(f"clip in place {name}")
    norm = fp8.clip_grad_norm(grads, max_norm)
    torch.cuda.synchronize()
    _check(keep, grads, norm, max_norm)
    say(f"clip in place, nothing to clip {name}")
    again = [g.clone() for g in grads]
    fp8.clip_grad_norm(grads, 1e30)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("scale", [1e30, 1e-30])
def test_squares_outside_fp32(scale):
    grads = _grads([1000, 4097], [torch.float32, torch.bfloat16], 3, scale)
    outs = [torch.empty_like(g) for g in grads]
    max_norm = 0.5 * _norm(grads)
    say(f"clip scale {scale}")
    norm = fp8.clip_grad_norm(grads, max_norm, out=outs)
    torch.cuda.synchronize()
    _check(grads, outs, norm, max_norm)


def test_special_values():
    say("clip zeros")
    z = [torch.zeros(100, device="cuda"), torch.zeros(7, dtype=torch.bfloat16, device="cuda")]
    assert float(fp8.clip_grad_norm(z, 1.0)) == 0.0 and not z[0].any()
    say("clip empty tensors only")
    assert float(fp8.clip_grad_norm([torch.zeros(0, device="cuda")], 1.0)) == 0.0
    say("clip to zero")
    g = _grads([1000], [torch.float32], 4)
    fp8.clip_grad_norm(g, 0.0)
    assert not g[0].any()
    say("clip NaN")
    g = _grads([1000, 50], [torch.float32, torch.bfloat16], 5)
    g[0][17] = float("nan")
    assert np.isnan(float(fp8.clip_grad_norm(g, 1.0)))
    assert bool(torch.isnan(g[0]).all()) and bool(torch.isnan(g[1]).all())
    say("clip infinity")
    g = _grads([1000, 50], [torch.float32, torch.bfloat16], 6)
    g[1][3] = float("-inf")
    assert float(fp8.clip_grad_norm(g, 1.0)) == float("inf")
    assert not g[0].any() and bool(torch.isnan(g[1][3])) and not g[1][4:].any()


def test_repeatable_and_captured():
    sizes, types = SETS["odd"]
    grads = _grads(sizes, types, 7)
    outs = [torch.empty_like(g) for g in grads]
    say("clip repeated")
    norms = [float(fp8.clip_grad_norm(grads, 0.5, out=outs)) for _ in range(3)]
    assert len(set(norms)) == 1
    want = [o.clone() for o in outs]
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    say("clip graph")
    with torch.cuda.graph(graph):
        norm = fp8.clip_grad_norm(grads, 0.5, out=outs, workspace=ws)
    for _ in range(4):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert float(norm) == norms[0] and all(torch.equal(a, b) for a, b in zip(outs, want))
        fp8.clip_grad_norm(grads, 0.7, out=[torch.empty_like(g) for g in grads])
        torch.cuda.synchronize()


def test_refusals():
    g = torch.ones(64, device="cuda")
    say("clip refusals")
    with pytest.raises(ValueError):
        fp8.clip_grad_norm([], 1.0)
    with pytest.raises(TypeError):
        fp8.clip_grad_norm([g.double()], 1.0)
    with pytest.raises(ValueError):
        fp8.clip_grad_norm([g, torch.ones(3)], 1.0)
    with pytest.raises(ValueError):
        fp8.clip_grad_norm([torch.ones((8, 8), device="cuda").t()[:4]], 1.0)
    with pytest.raises(ValueError):
        fp8.clip_grad_norm([g], 1.0, out=[torch.ones(63, device="cuda")])
    with pytest.raises(ValueError):
        fp8.clip_grad_norm([g], 1.0, out=[])
    for bad in (-1.0, float("nan")):
        with pytest.raises(fp8.Fp8GemmError) as e:
            fp8.clip_grad_norm([g], bad)
        assert e.value.status == 1
    with pytest.raises(fp8.Fp8GemmError) as e:
        fp8.clip_grad_norm([torch.ones(100000, device="cuda")], 1.0,
                           workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 7
    assert bool((g == 1).all())
