"""The routing operators, the grouped products and the adapters together: the
example's layer with its gradients, the chain against the oracle, in graphs, on
two streams at once, with whatever the unused rows hold."""
import os
import sys

import numpy as np
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
import oracle
import routing_reference as ref
from gpu_helpers import REL, ABS_RMS, say

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_runs():
    import expert_layer
    say("expert layer example")
    got = expert_layer.main(tokens=200, width=256, hidden=384, experts=6, steps=3, log=say)
    assert all(np.isfinite(got["losses"])) and bool(torch.isfinite(got["out"].float()).all())
    # root mean square roundings: E4M3 operands 2.6% each, so g and u 3.7%, h
    # about 6%, and with the quantized h and Wd 7%
    assert got["error"] < 0.12


def test_example_gradients():
    """Against autograd through the plain layer in 64 bits.  Quantization is
    taken as the identity: g and u are 3.7% off, h 6% and y 7% (above), so
    gradients formed from them are up to 10% off; the bound is twice that."""
    import expert_layer
    say("expert layer gradients")
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, K, F, E, k = 300, 256, 128, 5, 2

    def rand(*shape, std):
        return torch.randn(shape, generator=gen, device="cuda") * std

    x, wr = rand(T, K, std=1.0), rand(E, K, std=K ** -0.5)
    wg, wu, wd = rand(E, F, K, std=K ** -0.5), rand(E, F, K, std=K ** -0.5), rand(E, K, F, std=F ** -0.5)
    dy = rand(T, K, std=1.0)
    y, saved = expert_layer.forward(x, wr, expert_layer.quantized(torch.cat((wg, wu), 1)), expert_layer.quantized(wd), k)
    got = expert_layer.gradients(x, dy, wr, wg, wu, wd, saved)
    leaves = [t.double().cpu().requires_grad_() for t in (x, wr, wg, wu, wd)]
    out = expert_layer.plain_layer(*leaves, k)
    want = torch.autograd.grad((out * dy.double().cpu()).sum(), leaves)
    assert float((y.double().cpu() - out.detach()).norm() / out.detach().norm()) < 0.2
    for name, a, b in zip(("dx", "dwr", "dwg", "dwu", "dwd"), got, want):
        off = float((a.double().cpu() - b).norm() / b.norm())
        say("  ", name, off)
        assert off < 0.2, (name, off)


def _chain(x, logits, wq, sb, k, layout, max_m, out=None, poison=True):
    """Tokens to experts, one grouped product and back: (out, ids, weights)."""
    E, K = wq.shape[0], x.shape[1]
    w, ids = fp8.route_topk(logits, k)
    if layout == "masked":
        pos, src, m = fp8.expert_sort_masked(ids, E, max_m)
        shape = (E, max_m)
    else:
        pos, src, m, _ = fp8.expert_sort(ids, E)
        shape = src.shape[0]
    n = src.shape[0]
    xq = torch.empty((E, max_m, K) if layout == "masked" else (n, K), dtype=torch.uint8, device="cuda")
    sa = torch.empty((K // 128, n), device="cuda")
    if poison:                      # rows without a token may hold anything
        xq.fill_(0x7F)
        sa.fill_(float("nan"))
    fp8.expert_dispatch_quant(x, pos, shape, out=(xq, sa))
    y = (fp8.grouped_gemm_masked if layout == "masked" else fp8.grouped_gemm_contiguous)(xq, sa, wq, sb, m)
    return fp8.expert_combine(y, pos, w, out=out), ids, w, pos


@pytest.mark.parametrize("layout,max_m", [("contiguous", 0), ("masked", 128), ("masked", 16)])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (37, 5, 3), (300, 16, 4)])
def test_chain_against_the_oracle(layout, max_m, T, E, k):
    say("chain", layout, max_m, T, E, k)
    rng = np.random.default_rng(T)
    K, N = 256, 384
    x = torch.from_numpy(rng.normal(size=(T, K)).astype(np.float32)).bfloat16().cuda()
    logits = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).cuda()
    wq, sb = oracle.quant_128x128(rng.normal(size=(E * N, K)).astype(np.float32) * 0.05)
    out, ids, w, pos = _chain(x, logits, torch.from_numpy(wq).view(E, N, K).cuda(),
                              torch.from_numpy(sb).view(E, N // 128, K // 128).cuda(), k, layout, max_m)
    xq, sa = oracle.quant_1x128(x.float().cpu().numpy())
    ids, w, pos = ids.cpu().numpy(), w.double().cpu().numpy(), pos.cpu().numpy()
    want, mag = np.zeros((T, N)), np.zeros((T, N))
    products = [oracle.gemm_nt(xq, sa, wq[e * N:(e + 1) * N], sb[e * N // 128:(e + 1) * N // 128]) for e in range(E)]
    rms = np.sqrt(np.mean(np.square(products)))
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                y = products[ids[t, j]][t]
                want[t] += w[t, j] * y
                # the product's tolerance (with its BF16 rounding) and the sum's roundings
                mag[t] += w[t, j] * (REL * np.abs(y) + ABS_RMS * rms + (k + 1) * ref.U * np.abs(y))
    if max_m == 16 and T == 300:
        assert (pos < 0).any()
    ref.assert_near(out.double().cpu().numpy(), want, ref.rounded(mag, want, True), "chain")


@pytest.mark.parametrize("layout", ["contiguous", "masked"])
@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("pow2", [False, True])
def test_unused_rows_may_hold_anything(layout, fast, pow2):
    """Every grouped path: rows without a token as NaN codes and scales, or as zeros."""
    say("unused rows", layout, fast, pow2)
    gen = torch.Generator(device="cuda").manual_seed(7)
    T, E, k, K, N, max_m = 333, 7, 3, 512, 384, 256
    wq, sb = fp8.quant_128x128(torch.randn((E * N, K), generator=gen, device="cuda") * 0.05, ue8m0=pow2)
    wq, sb = wq.view(E, N, K), sb.view(E, N // 128, K // 128)
    x = torch.randn((T, K), generator=gen, device="cuda").bfloat16()
    w, ids = fp8.route_topk(torch.randn((T, E), generator=gen, device="cuda"), k)
    got = []
    for code, scale in ((0, 0.0), (0x7F, float("nan"))):
        if layout == "masked":
            pos, src, m = fp8.expert_sort_masked(ids, E, max_m)
        else:
            pos, src, m, _ = fp8.expert_sort(ids, E)
        shape = (E, max_m) if layout == "masked" else src.shape[0]
        xq = torch.full((E, max_m, K) if layout == "masked" else (shape, K), code, dtype=torch.uint8, device="cuda")
        sa = torch.full((K // 128, src.shape[0]), scale, device="cuda")
        fp8.expert_dispatch_quant(x, pos, shape, ue8m0=pow2, out=(xq, sa))
        product = fp8.grouped_gemm_masked if layout == "masked" else fp8.grouped_gemm_contiguous
        got.append(fp8.expert_combine(product(xq, sa, wq, sb, m, ue8m0=pow2, fast_accum=fast), pos, w))
    assert bool(torch.isfinite(got[0].float()).all()) and torch.equal(got[0], got[1])


@pytest.mark.parametrize("layout,max_m", [("contiguous", 0), ("masked", 64)])
def test_chain_in_a_graph(layout, max_m):
    """Captured once, replayed on changing tokens and choices, against eager."""
    say("chain in a graph", layout)
    gen = torch.Generator(device="cuda").manual_seed(5)
    T, E, k, K, N = 96, 6, 2, 256, 256
    wq, sb = fp8.quant_128x128(torch.randn((E * N, K), generator=gen, device="cuda") * 0.05)
    wq, sb = wq.view(E, N, K), sb.view(E, N // 128, K // 128)
    a = torch.randn((4, 16, N), generator=gen, device="cuda").bfloat16()
    b = torch.randn((4, 80, 16), generator=gen, device="cuda").bfloat16()
    scale = torch.ones(4, device="cuda")
    x, logits = torch.zeros((T, K), device="cuda").bfloat16(), torch.zeros((T, E), device="cuda")
    idx = torch.zeros(T, dtype=torch.int32, device="cuda")
    base, dout = torch.zeros((T, 80), device="cuda").bfloat16(), torch.zeros((T, N), device="cuda").bfloat16()

    def step():
        out, ids, w, pos = _chain(x, logits, wq, sb, k, layout, max_m, poison=False)
        dy, dw = fp8.expert_combine_grad(dout, out, pos.clamp_max(T - 1).contiguous(), w)
        return (out, ids, fp8.add_adapters(out, a, b, scale, fp8.adapter_rows(idx, 4), base), dw,
                fp8.route_topk_grad(dw, logits, ids))

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn((T, K), generator=g, device="cuda"))
        logits.copy_(torch.randn((T, E), generator=g, device="cuda"))
        idx.copy_(torch.randint(-1, 5, (T,), generator=g, device="cuda"))
        base.copy_(torch.randn((T, 80), generator=g, device="cuda"))
        dout.copy_(torch.randn((T, N), generator=g, device="cuda"))

    fill(0)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
    for seed in range(1, 5):
        fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for g, e in zip(got, step()):
            assert torch.equal(g, e)


def test_two_streams_at_once():
    """Calls on two streams, each with its own tensors, give what they give alone."""
    say("two streams")
    gen = torch.Generator(device="cuda").manual_seed(6)
    T, E, k, K = 3000, 64, 4, 512
    x = [torch.randn((T, K), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    logits = [torch.randn((T, E), generator=gen, device="cuda") for _ in range(2)]
    a = torch.randn((8, 16, K), generator=gen, device="cuda").bfloat16()
    b = torch.randn((8, 200, 16), generator=gen, device="cuda").bfloat16()
    y = [torch.randn((T, 200), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    scale = torch.rand(8, generator=gen, device="cuda")

    def work(i):
        w, ids = fp8.route_topk(logits[i], k)
        pos, src, m, counts = fp8.expert_sort(ids, E)
        xs = fp8.expert_dispatch(x[i], pos, src)
        out = fp8.expert_combine(xs, pos, w)
        return w, ids, pos, src, m, counts, xs, out, fp8.add_adapters(x[i], a, b, scale, fp8.adapter_rows(ids[:, 0].contiguous(), 8), y[i])

    alone = [work(0), work(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work(i))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for g, e in zip(run, alone[i]):
                assert torch.equal(g, e)
