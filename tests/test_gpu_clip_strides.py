"""Clipping of dense gradients whose dimensions lie in another order of memory
(a transposed or channels-last weight's)."""
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _grads(dtype):
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)
    return [rand(33, 70).t(), rand(2, 5, 7, 3).to(memory_format=torch.channels_last), rand(4, 9, 6).permute(2, 0, 1),
            rand(17, 1, 130).permute(2, 1, 0), rand(1, 50).t(), rand(65), rand(300, 41)]


def _expected(grads, max_norm):
    norm = sum(float(g.double().square().sum()) for g in grads) ** 0.5
    factor = torch.tensor(min(1.0, max_norm / (norm + 1e-6)), dtype=torch.float64).float()
    return norm, [(g.float() * factor.cuda()).to(g.dtype) for g in grads]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("in_place", [True, False])
def test_any_order_of_the_dimensions(dtype, in_place):
    say(f"clip strides {dtype} in_place={in_place}")
    grads = _grads(dtype)
    norm, want = _expected(grads, 3.0)
    strides = [g.stride() for g in grads]
    outs = grads if in_place else [torch.empty_like(g) for g in grads]
    assert all(a.stride() == b.stride() for a, b in zip(grads, outs))
    got = fp8.clip_grad_norm(grads, 3.0, out=None if in_place else outs)
    assert abs(float(got) - norm) <= 2.0 ** -23 * norm
    assert [g.stride() for g in outs] == strides
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refused_strides():
    say("clip refused strides")
    a = torch.ones((8, 12), device="cuda")
    for bad in (a[:, :6], a[::2], a.t()[:4], torch.ones(4, device="cuda").expand(3, 4), a.t()[:, ::2]):
        with pytest.raises(ValueError):
            fp8.clip_grad_norm([bad], 1.0)
    for g, out in ((a, torch.ones((12, 8), device="cuda").t()), (a.t(), torch.ones((12, 8), device="cuda")),
                   (a.t(), torch.ones((12, 8), device="cuda")[:, :8].t())):
        with pytest.raises(ValueError):
            fp8.clip_grad_norm([g], 1.0, out=[out])
    torch.cuda.synchronize()
    assert bool((a == 1).all())
