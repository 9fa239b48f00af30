"""The binding's checks of the feed-forward operators: each operand in turn of
another type, shape, layout or device is refused before a launch, and so are
operands that are not on the current device."""
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import say

pytestmark = pytest.mark.gpu

M, N, K = 3, 130, 256


def _gated():
    u8, f32 = torch.uint8, torch.float32
    shapes = [((M, K), u8), ((2, M), f32), ((N, K), u8), ((2, 2), f32), ((N, K), u8), ((2, 2), f32)]
    return [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes]


def _int4(gated):
    w = [torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda"),
         torch.zeros((K // 64, N), dtype=torch.bfloat16, device="cuda"),
         torch.zeros((K // 64, N), dtype=torch.uint8, device="cuda")]
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    return [x] + w + ([t.clone() for t in w] if gated else [])


def _mxfp4():
    return [torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"),
            torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda"),
            torch.zeros((K // 128, N), dtype=torch.int32, device="cuda")]


def _gated_int4(x, wg, sg, zg, wu, su, zu):
    return fp8.gated_gemv_w4(x, wg, sg, wu, su, zeros_g=zg, zeros_u=zu)


def _grad():
    bf16 = torch.bfloat16
    return [torch.zeros(s, dtype=bf16, device="cuda") for s in ((M, N), (M, N), (M, N), (M, K), (N, K), (N, K))]


CALLS = {"gated": (fp8.gated_nt, _gated), "gated saved": (lambda *a: fp8.gated_nt(*a, save=True), _gated),
         "gated grad": (fp8.gated_nt_grad, _grad),
         "gemv int4": (fp8.gemv_w4, lambda: _int4(False)), "gemv mxfp4": (fp8.gemv_w4, _mxfp4),
         "gated gemv int4": (_gated_int4, lambda: _int4(True)),
         "quant int4": (fp8.quant_int4, lambda: [torch.zeros((N, K), device="cuda")]),
         "clip": (lambda *g: fp8.clip_grad_norm(g, 1.0), _grad)}


def _wrong(t):
    """Copies of t, each wrong in one way."""
    yield "type", t.to(torch.int16)
    yield "one row more", torch.cat((t, t[:1]))
    yield "one column less", t[:, :-1].contiguous()
    yield "transposed strides", t.t().contiguous().t()
    yield "three dims", t[None]
    yield "one dim", t.reshape(-1)
    yield "host memory", t.cpu()
    yield "no tensor", t.cpu().numpy() if t.dtype != torch.bfloat16 else t.tolist()


@pytest.mark.parametrize("name", [n for n in CALLS if n not in ("quant int4", "clip")])
def test_each_operand_is_checked(name):
    call, make = CALLS[name]
    good = make()
    say(f"operands of {name}")
    call(*good)
    for i, t in enumerate(good):
        for what, bad in _wrong(t):
            if isinstance(bad, torch.Tensor) and bad.shape == t.shape and bad.is_contiguous() and bad.dtype == t.dtype \
                    and bad.is_cuda:
                continue                            # (a single row has no other strides)
            if "gemv" in name and i == 0 and what == "one row more":
                continue                            # (a token more is a call as good)
            args = list(good)
            args[i] = bad
            with pytest.raises((TypeError, ValueError, AttributeError)):
                call(*args)
                pytest.fail(f"{name}: operand {i}, {what}, was accepted")
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", list(CALLS))
def test_operands_away_from_the_current_device_are_refused(name, monkeypatch):
    call, make = CALLS[name]
    args = make()
    say(f"current device of {name}")
    call(*args)
    monkeypatch.setattr(fp8, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        call(*args)
    torch.cuda.synchronize()
