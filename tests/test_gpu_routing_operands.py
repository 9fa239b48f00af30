"""The binding's checks of the routing operators and the adapters: each operand
in turn of another type, shape, layout or device is refused before a launch,
and so are operands that are not on the current device."""
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import say

pytestmark = pytest.mark.gpu

T, E, k, K, rows = 6, 5, 2, 256, 24


def _f32(*shape):
    return torch.zeros(shape, device="cuda")


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def _i32(*shape):
    return torch.full(shape, -1, dtype=torch.int32, device="cuda")


CALLS = {
    "route": (lambda l: fp8.route_topk(l, k), lambda: [_f32(T, E)]),
    "route grad": (fp8.route_topk_grad, lambda: [_f32(T, k), _bf16(T, E), _i32(T, k)]),
    "dispatch": (fp8.expert_dispatch, lambda: [_bf16(T, K), _i32(T, k), _i32(rows)]),
    "dispatch quant": (lambda x, pos: fp8.expert_dispatch_quant(x, pos, rows), lambda: [_f32(T, K), _i32(T, k)]),
    "combine": (fp8.expert_combine, lambda: [_bf16(rows, K), _i32(T, k), _f32(T, k)]),
    "combine grad": (fp8.expert_combine_grad, lambda: [_bf16(T, K), _bf16(rows, K), _i32(T, k), _f32(T, k), _i32(rows)]),
    "adapters": (fp8.add_adapters, lambda: [_bf16(T, K), _bf16(3, 16, K), _bf16(3, 70, 16), _f32(3), _i32(2, 32), _bf16(T, 70)]),
}
# calls as good as the first: other tokens, experts, widths, pairs, rows or types
FINE = {("route", 0, "one row more"), ("route", 0, "one column less"), ("dispatch", 2, "one row more"),
        ("dispatch", 1, "one column less"), ("dispatch", 0, "one column less"), ("dispatch quant", 1, "one column less"),
        ("combine", 0, "one row more"), ("combine", 0, "one column less"), ("combine", 0, "three dims"),
        ("combine grad", 1, "three dims"), ("route grad", 1, "one column less")}


def _wrong(t):
    """Copies of t, each wrong in one way."""
    yield "type", t.to(torch.float16)
    yield "one row more", torch.cat((t, t[:1]))
    if t.dim() == 2:
        yield "one column less", t[:, :-1].contiguous()
        yield "transposed strides", t.t().contiguous().t()
    yield "three dims", t[None] if t.dim() == 2 else t[None, None]
    yield "one dim", t.reshape(-1) if t.dim() > 1 else t.reshape(1, -1)
    yield "host memory", t.cpu()
    yield "no tensor", t.tolist()


@pytest.mark.parametrize("name", list(CALLS))
def test_each_operand_is_checked(name):
    call, make = CALLS[name]
    good = make()
    say(f"operands of {name}")
    call(*good)
    for i, t in enumerate(good):
        for what, bad in _wrong(t):
            if (name, i, what) in FINE:
                continue
            if isinstance(bad, torch.Tensor) and bad.shape == t.shape and bad.is_contiguous() and bad.dtype == t.dtype \
                    and bad.is_cuda:
                continue
            args = list(good)
            args[i] = bad
            with pytest.raises((TypeError, ValueError, AttributeError, fp8.Fp8GemmError)):
                call(*args)
                pytest.fail(f"{name}: operand {i}, {what}, was accepted")
    torch.cuda.synchronize()


ALL = {**CALLS, "sort": (lambda i: fp8.expert_sort(i, E), lambda: [_i32(T, k)]),
       "sort masked": (lambda i: fp8.expert_sort_masked(i, E, 4), lambda: [_i32(T, k)]),
       "adapter rows": (lambda i: fp8.adapter_rows(i, 3), lambda: [_i32(T)])}


@pytest.mark.parametrize("name", list(ALL))
def test_operands_away_from_the_current_device_are_refused(name, monkeypatch):
    call, make = ALL[name]
    args = make()
    say(f"current device of {name}")
    call(*args)
    monkeypatch.setattr(fp8, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        call(*args)
    torch.cuda.synchronize()


def test_outputs_are_checked():
    say("outputs of the routing operators")
    x, pos, src, w = _bf16(T, K), _i32(T, k), _i32(rows), _f32(T, k)
    i32 = torch.int32
    bad = [
        lambda: fp8.route_topk(_f32(T, E), k, out=(w, pos.long())),
        lambda: fp8.route_topk_grad(w, _f32(T, E), pos, out=_bf16(T, E)),
        lambda: fp8.expert_sort(pos, E, rows=rows, out=(pos, src, src, torch.empty(E + 1, dtype=i32, device="cuda"))),
        lambda: fp8.expert_sort_masked(pos, E, 4, out=(pos, _i32(19), _i32(E))),
        lambda: fp8.expert_dispatch(x, pos, src, out=_f32(rows, K)),
        lambda: fp8.expert_dispatch_quant(x, pos, rows, out=(torch.empty((rows, K), dtype=torch.uint8, device="cuda"), _f32(rows, K // 128))),
        lambda: fp8.expert_dispatch_quant(x, pos, (4, 6), out=(torch.empty((rows, K), dtype=torch.uint8, device="cuda"), _f32(K // 128, rows))),
        lambda: fp8.expert_combine(_bf16(rows, K), pos, w, out=_bf16(T + 1, K)),
        lambda: fp8.expert_combine_grad(x, _bf16(rows, K), pos, w, src, out=(_bf16(rows, K), _f32(k, T))),
        lambda: fp8.add_adapters(x, _bf16(3, 16, K), _bf16(3, 70, 16), _f32(3), _i32(2, 32), _bf16(T, 70), out=_bf16(T, 71)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            call()
            pytest.fail(f"call {i} was accepted")
    torch.cuda.synchronize()
