"""Host-side checks of the routing and adapter entry points, and of their
references (no GPU needed): bad arguments are refused before any device call,
plans cover their problems, and the references' gradients are those of their
own forward passes by differences."""
import ctypes
import os

import numpy as np
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
import routing_reference as ref

OK, INVALID, SHAPE, ALIGN, UNSUP, NODEV, LAUNCH, SCRATCH = range(8)
P = ctypes.c_void_p
A = P(4096)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fp8.LIB_PATH):
        from fine_grained_block_e4m3_amd import build
        build.build()
    return fp8.load_library()


def test_route_validation(L):
    def call(l=A, w=A, ids=A, T=3, E=8, k=2, kind=0):
        return L.fp8_route_topk(l, T, E, k, kind, 1, 1.0, w, ids, None)
    assert call(l=None) == INVALID and call(w=None) == INVALID and call(ids=None) == INVALID
    assert call(T=-1) == INVALID and call(E=0) == INVALID and call(k=0) == INVALID
    assert call(kind=2) == INVALID and call(kind=-1) == INVALID
    assert call(k=9) == SHAPE
    assert call(E=1025) == UNSUP and call(E=100, k=65) == UNSUP
    assert call(l=P(4098)) == ALIGN and call(w=P(4098)) == ALIGN and call(ids=P(4097)) == ALIGN
    assert call(l=P(4097), kind=1) == ALIGN
    assert call(T=0, l=None) == OK

    def grad(dw=A, l=A, ids=A, d=A, T=3, E=8, k=2, kind=0):
        return L.fp8_route_topk_grad(dw, l, ids, T, E, k, kind, 0, 1.0, d, None)
    assert grad(dw=None) == INVALID and grad(l=None) == INVALID and grad(ids=None) == INVALID and grad(d=None) == INVALID
    assert grad(d=P(4098)) == ALIGN and grad(k=9) == SHAPE and grad(T=0, d=None) == OK


def test_sort_validation(L):
    def call(ids=A, size=4, n=10, E=4, align=128, rows=640, pos=A, src=A, idx=A, counts=A, ws=None, ws_bytes=0):
        return L.fp8_expert_sort_contiguous(ids, size, n, E, align, rows, 0, pos, src, idx, counts, ws, ws_bytes, None)
    assert call(ids=None) == INVALID and call(src=None) == INVALID and call(idx=None) == INVALID
    assert call(size=2) == INVALID and call(n=-1) == INVALID and call(E=0) == INVALID and call(rows=-1) == INVALID
    assert call(align=0) == INVALID and call(align=48) == INVALID and call(align=2048) == INVALID
    assert call(ws_bytes=4) == INVALID
    assert call(E=1025) == UNSUP and call(n=(1 << 30) + 1) == UNSUP
    assert call(ids=P(4100), size=8) == ALIGN and call(pos=P(4098)) == ALIGN and call(ws=P(4104), ws_bytes=400) == ALIGN
    assert call(n=2049) == SCRATCH and call(n=100000, ws=A, ws_bytes=16) == SCRATCH

    def masked(ids=A, E=4, max_m=16, src=A, m=A):
        return L.fp8_expert_sort_masked(ids, 4, 10, E, max_m, A, src, m, None, 0, None)
    assert masked(ids=None) == INVALID and masked(src=None) == INVALID and masked(m=None) == INVALID
    assert masked(max_m=-1) == INVALID and masked(E=1024, max_m=1 << 21) == UNSUP
    assert L.fp8_expert_sort_workspace_size(2048, 256) == 0
    assert L.fp8_expert_sort_workspace_size(2049, 256) == 4 * 257 * 4       # three chunks, a multiple of 4
    assert L.fp8_expert_sort_workspace_size(-1, 256) == 0 and L.fp8_expert_sort_workspace_size(10, 2000) == 0
    for n in (8193, 1 << 20, 1 << 30):       # at most 256 chunks
        assert L.fp8_expert_sort_workspace_size(n, 1024) <= 256 * 1025 * 4


def test_rows_are_what_the_worst_choice_needs():
    for n, E, align in ((0, 8, 128), (1, 8, 128), (5, 8, 16), (64, 4, 16), (1000, 16, 128), (37, 3, 8), (9, 9, 1)):
        worst = 0
        if E <= 4 and n <= 64:               # every split of n over E experts
            def splits(left, e):
                if e == 1:
                    yield (left,)
                    return
                for c in range(left + 1):
                    for rest in splits(left - c, e - 1):
                        yield (c,) + rest
            worst = max(sum(-(-c // align) for c in s) for s in splits(n, E)) * align
        else:
            # one row in all experts but one, the rest in it, as far as they go round
            for full in range(0, min(E, n) + 1):
                for extra in range(0, align + 1):
                    c = [1] * full
                    left = n - full
                    if not c and left:
                        c, left = [0], left
                    if c:
                        c[0] += max(0, left - extra * max(0, len(c) - 1))
                        for i in range(1, len(c)):
                            c[i] += extra
                    if c and sum(c) == n and min(c) >= 0:
                        worst = max(worst, sum(-(-v // align) for v in c) * align)
        rows = fp8.expert_rows(n, E, align)
        assert rows >= worst and rows % align == 0
        assert rows <= n + min(E, n) * (align - 1)
        if E <= 4 and n <= 64:
            assert rows == worst
    with pytest.raises(ValueError):
        fp8.expert_rows(-1, 4)


def test_rows_validation(L):
    def dispatch(x=A, pos=A, src=A, xs=A, T=3, k=2, rows=8, K=16, kind=1):
        return L.fp8_expert_dispatch(x, pos, src, xs, T, k, rows, K, kind, None)
    assert dispatch(x=None) == INVALID and dispatch(pos=None) == INVALID and dispatch(xs=None) == INVALID
    assert dispatch(k=0) == INVALID and dispatch(kind=2) == INVALID and dispatch(rows=-1) == INVALID
    assert dispatch(T=1 << 30, k=2) == UNSUP
    assert dispatch(x=P(4097)) == ALIGN and dispatch(xs=P(4098), kind=0) == ALIGN and dispatch(src=P(4098)) == ALIGN
    assert dispatch(rows=0, x=None) == OK and dispatch(K=0) == OK and dispatch(T=0, src=None, x=None) == OK

    def quant(x=A, pos=A, xq=A, sa=A, T=3, k=2, rows=8, K=256, kind=1, flags=0):
        return L.fp8_expert_dispatch_quant(x, pos, xq, sa, T, k, rows, K, kind, flags, None)
    assert quant(x=None) == INVALID and quant(sa=None) == INVALID and quant(flags=2) == INVALID
    assert quant(K=100) == SHAPE
    assert quant(x=P(4104)) == ALIGN and quant(xq=P(4104)) == ALIGN and quant(sa=P(4100)) == ALIGN
    assert quant(T=0, x=None) == OK

    def combine(y=A, pos=A, w=None, out=A, T=3, k=2, rows=8, N=16, kind=0):
        return L.fp8_expert_combine(y, pos, w, out, T, k, rows, N, kind, None)
    assert combine(y=None) == INVALID and combine(pos=None) == INVALID and combine(out=None) == INVALID
    assert combine(w=P(4098)) == ALIGN and combine(T=0, y=None) == OK and combine(k=-1) == INVALID

    def grad(dout=A, y=A, pos=A, w=A, src=A, dy=A, dw=A, T=3, k=2, rows=8, N=16, kind=1):
        return L.fp8_expert_combine_grad(dout, y, pos, w, src, dy, dw, T, k, rows, N, kind, None)
    assert grad(dout=None) == INVALID and grad(y=None) == INVALID and grad(pos=None) == INVALID
    assert grad(dy=P(4097)) == ALIGN and grad(dw=P(4098)) == ALIGN
    assert grad(dy=None, dw=None, pos=None) == OK and grad(T=0, dy=None) == OK


def test_adapter_validation(L):
    def call(x=A, a=A, b=A, scale=A, src=A, index=A, y=A, out=A, T=3, N=20, K=256, n=2, R=16, rows=48, ws=A, ws_bytes=1 << 40):
        return L.fp8_add_adapters(x, a, b, scale, src, index, y, out, T, N, K, n, R, rows, ws, ws_bytes, None)
    for name in ("x", "a", "b", "scale", "src", "index", "y", "out"):
        assert call(**{name: None}) == INVALID, name
    assert call(ws=None, ws_bytes=8) == INVALID and call(n=0) == INVALID and call(R=0) == INVALID
    assert call(K=100) == SHAPE and call(K=0) == SHAPE and call(R=12) == SHAPE and call(rows=40) == SHAPE
    assert call(R=136) == UNSUP and call(K=(1 << 22) + 128) == UNSUP
    for name in ("x", "a", "b", "ws"):
        assert call(**{name: P(4104)}) == ALIGN, name
    assert call(scale=P(4098)) == ALIGN and call(y=P(4097)) == ALIGN
    assert call(T=0, x=None) == OK and call(N=0) == OK and call(rows=0) == OK
    assert L.fp8_adapters_workspace_size(3, 2, 48, 20, 100, 16) == 0


@pytest.mark.parametrize("T,adapters", [(1, 1), (1, 1000), (100, 64), (320, 9), (8192, 8), (8192, 300), (1 << 20, 16)])
@pytest.mark.parametrize("N,K", [(1, 128), (300, 1536), (7168, 7168), (24576, 128), (2112, 28672)])
def test_adapter_plan_covers_the_problem(T, adapters, N, K):
    for cus in (256, 64):
        p = fp8.adapters_plan(T, adapters, N, K, 16, compute_units=cus)
        rows = fp8.expert_rows(T, adapters + 1, 16)
        assert p["tiles"] * 16 == rows
        assert p["group"] == (4 if T >= 24 * (adapters + 1) and T * 16 >= 48 << 10 else 1)
        assert p["k_range"] % 128 == 0 and (p["k_splits"] - 1) * p["k_range"] < K <= p["k_splits"] * p["k_range"]
        assert p["n_range"] % 256 == 0 and p["n_range"] > 0
        if p["whole"]:          # a power of two of workgroups per tile, about one per compute unit in all
            assert p["whole"] in (1, 2, 4, 8, 16) and 3 * p["tiles"] * p["whole"] <= 4 * cus and p["workspace_bytes"] == 0
            assert 16 * T <= 64 * p["tiles"]
        else:
            assert p["workspace_bytes"] == p["k_splits"] * rows * 16 * 4


def test_binding_refuses_cpu_tensors():
    f, i = torch.zeros((2, 128)), torch.zeros((2, 2), dtype=torch.int32)
    for call in (lambda: fp8.route_topk(f, 2), lambda: fp8.route_topk_grad(f, f, i), lambda: fp8.expert_sort(i, 4),
                 lambda: fp8.expert_sort_masked(i, 4, 4), lambda: fp8.expert_dispatch(f, i, i[0]),
                 lambda: fp8.expert_dispatch_quant(f, i, 8), lambda: fp8.expert_combine(f, i),
                 lambda: fp8.expert_combine_grad(f, f, i), lambda: fp8.adapter_rows(i[0], 4)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        fp8.route_topk(f.half(), 2)
    with pytest.raises(TypeError):
        fp8.expert_sort(f, 4)


@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_by_differences(renorm):
    rng = np.random.default_rng(5)
    l, dw = rng.normal(size=(4, 9)), rng.normal(size=(4, 3))
    l[1, 2] = -np.inf
    ids = ref.order(l, 3)
    d = ref.route_grad(dw, l, ids, renorm, 1.7)[0]
    h = 1e-6
    for e in range(9):
        if e == 2:
            continue
        step = np.zeros_like(l)
        step[:, e] = h
        # (the choice is fixed)
        diff = 1.7 * (ref._parts(l + step, ids, renorm)[0] - ref._parts(l - step, ids, renorm)[0]) / (2 * h)
        assert np.allclose((diff * dw).sum(1), d[:, e], atol=1e-8)


def test_reference_combine_gradient_by_differences():
    rng = np.random.default_rng(6)
    y, w, dout = rng.normal(size=(6, 5)), rng.normal(size=(3, 2)), rng.normal(size=(3, 5))
    pos = np.array([[0, 4], [-1, 2], [5, 9]])
    dy, dw, _ = ref.combine_grad(dout, y, pos, w, np.zeros_like(y))

    def loss(y, w):
        return (ref.combine(y, pos, w)[0] * dout).sum()
    h = 1e-6
    for i in np.ndindex(y.shape):
        s = np.zeros_like(y)
        s[i] = h
        assert abs((loss(y + s, w) - loss(y - s, w)) / (2 * h) - dy[i]) < 1e-8
    for i in np.ndindex(w.shape):
        s = np.zeros_like(w)
        s[i] = h
        assert abs((loss(y, w + s) - loss(y, w - s)) / (2 * h) - dw[i]) < 1e-8
