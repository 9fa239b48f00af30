"""Tokens sorted by expert and back, with the gradients, against plain forms:
the tables exactly, moved rows bit for bit, sums against 64 bits."""
import numpy as np
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
import oracle
import routing_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _buffers(shapes, fill=-77):
    """int32 outputs, each between sentinels."""
    full = [torch.full((int(np.prod(s)) + 64,), fill, dtype=torch.int32, device="cuda") for s in shapes]
    return full, [f[32:32 + int(np.prod(s))].view(s) for f, s in zip(full, shapes)]


def _edges(full, fill=-77):
    for f in full:
        assert bool((f[:32] == fill).all()) and bool((f[-32:] == fill).all())


def _ids(rng, shape, E, kind):
    if kind == "one":
        return np.full(shape, E - 1)
    if kind == "outside":
        return rng.integers(-3, E + 3, shape)
    if kind == "far":
        return rng.choice([-2 ** 31, 2 ** 31 - 1, 0, E - 1, E], shape)
    if kind == "skewed":
        return np.minimum(rng.geometric(0.2, shape) - 1, E - 1)
    return rng.integers(0, E, shape)


@pytest.mark.parametrize("E", [1, 3, 16, 64, 255, 256, 1000, 1024])
@pytest.mark.parametrize("shape", [(0, 2), (1, 1), (1, 8), (63, 1), (65, 1), (300, 5), (1024, 2), (1025, 2), (2731, 3), (5000, 4)])
def test_sort_contiguous(E, shape):
    rng = np.random.default_rng(E + shape[0])
    for kind, dtype, align, keep in (("even", torch.int32, 128, False), ("outside", torch.int64, 16, True),
                                     ("skewed", torch.int32, 1, False), ("one", torch.int64, 1024, False),
                                     ("far", torch.int32, 64, True)):
        say("sort", E, shape, kind, align)
        a = _ids(rng, shape, E, kind)
        ids = torch.from_numpy(a).to(dtype).cuda()
        most = fp8.expert_rows(a.size, E + 1 if keep else E, align)
        for rows in (most, most // 2, 0):
            full, out = _buffers([shape, (rows,), (rows,), (E,)])
            got = fp8.expert_sort(ids, E, align=align, rows=rows, keep=keep, out=out)
            for g, r, name in zip(got, ref.sort_contiguous(a, E, align, rows, keep), ("pos", "src", "m_indices", "counts")):
                assert np.array_equal(g.cpu().numpy(), r), (name, E, shape, kind, align, rows)
            _edges(full)


@pytest.mark.parametrize("E,max_m", [(1, 5), (16, 256), (7, 0), (300, 33), (1024, 16)])
def test_sort_masked(E, max_m):
    rng = np.random.default_rng(E)
    for shape in ((0, 2), (1, 2), (200, 2), (3000, 4)):
        for kind in ("even", "outside", "one"):
            say("sort masked", E, max_m, shape, kind)
            a = _ids(rng, shape, E, kind)
            full, out = _buffers([shape, (E * max_m,), (E,)])
            got = fp8.expert_sort_masked(torch.from_numpy(a).cuda(), E, max_m, out=out)
            for g, r, name in zip(got, ref.sort_masked(a, E, max_m), ("pos", "src", "masked_m")):
                assert np.array_equal(g.cpu().numpy(), r), (name, E, max_m, shape, kind)
            _edges(full)


def test_sort_of_many_pairs():
    """As many chunks as there can be, of each kernel's size."""
    rng = np.random.default_rng(9)
    for n, E in ((262145, 256), (700000, 40), (530000, 1024), (1200001, 17)):
        say("sort", n, E)
        a = _ids(rng, (n,), E, "outside")
        most = fp8.expert_rows(n, E)
        got = fp8.expert_sort(torch.from_numpy(a).int().cuda(), E)
        for g, r in zip(got, ref.sort_contiguous(a, E, 128, most, False)):
            assert np.array_equal(g.cpu().numpy(), r)


def _places(rng, T, k, rows, dropped=0.2):
    """Distinct rows for some of the pairs; the others -1 or outside."""
    pos = np.full(T * k, -1, np.int64)
    n = min(T * k, rows)
    held = rng.permutation(T * k)[: int(n * (1 - dropped)) if n > 1 else n]
    pos[held] = rng.permutation(rows)[: held.size]
    pos[(pos < 0) & (rng.random(T * k) < 0.5)] = rows + 3
    src = np.full(rows, -1, np.int64)
    src[pos[held]] = held
    return pos.reshape(T, k).astype(np.int32), src.astype(np.int32)


WIDTHS = [1, 2, 3, 7, 8, 130, 511, 1024, 1530, 2049, 7168]


@pytest.mark.parametrize("W", WIDTHS)
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_rows_there_and_back(W, kind):
    rng = np.random.default_rng(W)
    dtype = TYPES[kind]
    for T, k, rows in ((1, 1, 1), (5, 3, 9), (33, 2, 128), (40, 9, 300)):
        say("rows", W, kind, T, k, rows)
        pos, src = _places(rng, T, k, rows)
        dpos, dsrc = torch.from_numpy(pos).cuda(), torch.from_numpy(src).cuda()
        x = torch.from_numpy(rng.normal(size=(T, W)).astype(np.float32)).to(dtype).cuda()
        # there: bit for bit, zeros where no token goes, nothing outside
        full = torch.full((rows * W + 32,), 9.0, dtype=dtype, device="cuda")
        xs = fp8.expert_dispatch(x, dpos, dsrc, out=full[16:16 + rows * W].view(rows, W))
        want = torch.zeros((rows, W), dtype=dtype, device="cuda")
        held = torch.from_numpy(np.flatnonzero(src >= 0)).cuda()
        want[held] = x[dsrc[held].long() // k]
        assert torch.equal(xs, want)
        assert bool((full[:16] == 9).all()) and bool((full[-16:] == 9).all())
        # back
        y = torch.from_numpy(rng.normal(size=(rows, W)).astype(np.float32)).to(dtype).cuda()
        y[torch.from_numpy(src < 0).cuda()] = float("nan")         # rows of no pair are not read
        yn = y.double().cpu().numpy()
        w = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).cuda()
        for weights in (w, None):
            full = torch.full((T * W + 32,), 9.0, dtype=dtype, device="cuda")
            got = fp8.expert_combine(y, dpos, weights, out=full[16:16 + T * W].view(T, W))
            r, mag = ref.combine(yn, pos, None if weights is None else w.double().cpu().numpy())
            ref.assert_near(got.double().cpu().numpy(), r, ref.rounded((k + 1) * ref.U * mag, r, kind == "bf16"), "combine")
            assert bool((full[:16] == 9).all()) and bool((full[-16:] == 9).all())
        # the gradient
        dout = torch.from_numpy(rng.normal(size=(T, W)).astype(np.float32)).to(dtype).cuda()
        for weights, with_src in ((w, True), (None, False)):
            full = torch.full((rows * W + 32,), 9.0, dtype=dtype, device="cuda")
            buf = full[16:16 + rows * W].view(rows, W)
            dw_full = torch.full((T * k + 2,), 9.0, device="cuda")
            dy, dw = fp8.expert_combine_grad(dout, y, dpos, weights, dsrc if with_src else None,
                                             out=(buf, dw_full[1:-1].view(T, k)))
            rdy, rdw, mag = ref.combine_grad(dout.double().cpu().numpy(), yn, pos, None if weights is None else w.double().cpu().numpy(),
                                             np.full((rows, W), 0.0 if with_src else 9.0))
            ref.assert_near(dy.double().cpu().numpy(), rdy, ref.rounded(ref.U * np.abs(rdy), rdy, kind == "bf16"), "dy")
            # a thread sums every 256th vector, then 64 lanes and 4 waves
            ref.assert_near(dw.double().cpu().numpy(), rdw, (W / 64 + 24) * ref.U * mag + 1e-300, "dw")
            assert bool((full[:16] == 9).all()) and bool((full[-16:] == 9).all())
            assert dw_full[0] == 9 and dw_full[-1] == 9


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("k", [1, 4, 5, 8, 9, 17])
def test_rows_of_whole_lines(kind, k):
    """Buffers at line boundaries and beside them take different loads and
    stores: one result, the 64-bit form's."""
    rng = np.random.default_rng(k)
    dtype = TYPES[kind]
    for T, rows, W in ((3, 20, 64), (30, 300, 1024), (9, 64, 7168)):
        say("whole lines", kind, k, T, W)
        pos, src = _places(rng, T, k, rows)
        dpos, dsrc = torch.from_numpy(pos).cuda(), torch.from_numpy(src).cuda()
        y = torch.from_numpy(rng.normal(size=(rows, W)).astype(np.float32)).to(dtype).cuda()
        dout = torch.from_numpy(rng.normal(size=(T, W)).astype(np.float32)).to(dtype).cuda()
        w = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).cuda()
        beside = torch.empty(rows * W + 8, dtype=dtype, device="cuda")[8:].view(rows, W)
        beside.copy_(y)
        assert y.data_ptr() % 128 == 0 and beside.data_ptr() % 128 != 0
        out = fp8.expert_combine(y, dpos, w)
        assert torch.equal(out, fp8.expert_combine(beside, dpos, w))
        r, mag = ref.combine(y.double().cpu().numpy(), pos, w.double().cpu().numpy())
        ref.assert_near(out.double().cpu().numpy(), r, ref.rounded((k + 1) * ref.U * mag, r, kind == "bf16"), "combine")
        dy, dw = fp8.expert_combine_grad(dout, y, dpos, w, dsrc)
        dy2, dw2 = fp8.expert_combine_grad(dout, beside, dpos, w, dsrc)
        assert torch.equal(dy, dy2) and torch.equal(dw, dw2)
        rdy, rdw, mag = ref.combine_grad(dout.double().cpu().numpy(), y.double().cpu().numpy(), pos, w.double().cpu().numpy(),
                                         np.zeros((rows, W)))
        ref.assert_near(dy.double().cpu().numpy(), rdy, ref.rounded(ref.U * np.abs(rdy), rdy, kind == "bf16"), "dy")
        ref.assert_near(dw.double().cpu().numpy(), rdw, (W / 64 + 24) * ref.U * mag + 1e-300, "dw")


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("pow2", [False, True])
def test_codes_larger_than_the_caches(kind, pow2):
    """Over 256 MB of codes, against the quantizer's."""
    say("large codes", kind, pow2)
    T, K = 40000, 7168
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((T, K), generator=gen, device="cuda").to(TYPES[kind])
    ids = torch.randint(0, 7, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    pos, src, _, _ = fp8.expert_sort(ids, 7)
    xq, sa = fp8.expert_dispatch_quant(x, pos, src.shape[0], ue8m0=pow2)
    q, s = fp8.quant_1x128(x.float(), ue8m0=pow2)
    at = pos[:, 0].long()
    assert torch.equal(xq[at], q) and torch.equal(sa[:, at], s)


def test_gradients_alone():
    """Each of the two gradients without the other; y is not read for dy."""
    say("gradients alone")
    rng = np.random.default_rng(4)
    T, k, rows, W = 20, 3, 70, 300
    pos, src = _places(rng, T, k, rows)
    pos, src = torch.from_numpy(pos).cuda(), torch.from_numpy(src).cuda()
    y, dout = torch.randn((rows, W), device="cuda").bfloat16(), torch.randn((T, W), device="cuda").bfloat16()
    w = torch.rand((T, k), device="cuda")
    both = fp8.expert_combine_grad(dout, y, pos, w, src)
    dy, none = fp8.expert_combine_grad(dout, torch.full_like(y, float("nan")), pos, w, src, need_dw=False)
    assert none is None and torch.equal(dy, both[0])
    none, dw = fp8.expert_combine_grad(dout, y, pos, w, src, need_dy=False)
    assert none is None and torch.equal(dw, both[1])
    assert fp8.expert_combine_grad(dout, y, pos, w, src, need_dy=False, need_dw=False) == (None, None)


def test_infinities_stay_with_their_pairs():
    """An infinite dout or weight shows in its own pairs, not in those without a row."""
    say("infinities")
    pos = torch.tensor([[0, -1], [1, 2]], dtype=torch.int32, device="cuda")
    src = torch.tensor([0, 2, 3, -1], dtype=torch.int32, device="cuda")
    y = torch.ones((4, 40), device="cuda")
    dout = torch.ones((2, 40), device="cuda")
    dout[0, 3] = float("inf")
    w = torch.ones((2, 2), device="cuda")
    dy, dw = fp8.expert_combine_grad(dout, y, pos, w, src)
    assert dw.tolist() == [[float("inf"), 0.0], [40.0, 40.0]]
    assert torch.isfinite(dy[1:]).all() and torch.isinf(dy[0, 3]) and bool((dy[3] == 0).all())
    w[0, 1] = float("nan")                       # of a pair without a row
    assert bool((fp8.expert_combine(y, pos, w) == torch.tensor([[1.0], [2.0]], device="cuda")).all())


@pytest.mark.parametrize("K", [128, 256, 1024, 1152, 7168])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantizing_dispatch(K, kind, pow2):
    """Codes and scales as the quantizer's, in the tokens' rows only."""
    rng = np.random.default_rng(K)
    for T, k, rows in ((1, 1, 1), (7, 3, 20), (200, 2, 640)):
        say("quantizing dispatch", K, kind, pow2, T)
        pos, src = _places(rng, T, k, rows)
        a = rng.normal(size=(T, K)).astype(np.float32) * np.exp(rng.normal(size=(T, 1)) * 4).astype(np.float32)
        a[0, :128] = 0.0
        x = torch.from_numpy(a).to(TYPES[kind]).cuda()
        q, s = oracle.quant_1x128(x.float().cpu().numpy(), oracle.FLAG_UE8M0 if pow2 else 0)
        xq = torch.full((rows * K + 32,), 0x55, dtype=torch.uint8, device="cuda")
        sa = torch.full((K // 128 * rows + 32,), -3.0, device="cuda")
        buf = (xq[16:16 + rows * K].view(rows, K), sa[16:16 + K // 128 * rows].view(K // 128, rows))
        got = fp8.expert_dispatch_quant(x, torch.from_numpy(pos).cuda(), rows, ue8m0=pow2, out=buf)
        wq, ws = np.full((rows, K), 0x55, np.uint8), np.full((K // 128, rows), -3.0, np.float32)
        held = np.flatnonzero(src >= 0)
        wq[held], ws[:, held] = q[src[held] // k], s[:, src[held] // k]
        assert np.array_equal(got[0].cpu().numpy(), wq) and np.array_equal(got[1].cpu().numpy(), ws)
        assert bool((xq[:16] == 0x55).all()) and bool((xq[-16:] == 0x55).all())
        assert bool((sa[:16] == -3).all()) and bool((sa[-16:] == -3).all())


def test_empty_calls():
    say("empty calls")
    i32 = torch.int32
    pos0, src = torch.empty((0, 2), dtype=i32, device="cuda"), torch.full((8,), -1, dtype=i32, device="cuda")
    x0 = torch.empty((0, 40), device="cuda")
    assert bool((fp8.expert_dispatch(x0, pos0, src) == 0).all())
    assert fp8.expert_combine(torch.empty((8, 40), device="cuda"), pos0).shape == (0, 40)
    dy, dw = fp8.expert_combine_grad(x0, torch.ones((8, 40), device="cuda"), pos0, None, src)
    assert bool((dy == 0).all()) and dw.shape == (0, 2)
    # no rows at all: every token's sum is empty
    pos = torch.full((3, 2), -1, dtype=i32, device="cuda")
    pos[0, 0] = 5
    none = torch.empty((0, 40), device="cuda")
    assert bool((fp8.expert_combine(none, pos) == 0).all())
    dy, dw = fp8.expert_combine_grad(torch.ones((3, 40), device="cuda"), none, pos)
    assert dy.shape == (0, 40) and bool((dw == 0).all())
    assert fp8.expert_dispatch(torch.ones((3, 40), device="cuda"), pos, pos0.view(-1)).shape == (0, 40)
    # no columns: empty sums
    y = torch.empty((8, 0), device="cuda")
    dy, dw = fp8.expert_combine_grad(torch.empty((3, 0), device="cuda"), y, pos)
    assert bool((dw == 0).all())


def test_refusals():
    say("expert refusals")
    i32 = torch.int32
    ids = torch.zeros((4, 2), dtype=i32, device="cuda")
    x, pos = torch.ones((4, 256), device="cuda"), torch.zeros((4, 2), dtype=i32, device="cuda")
    src = torch.full((8,), -1, dtype=i32, device="cuda")
    for call, err in (
            (lambda: fp8.expert_sort(ids.float(), 4), TypeError),
            (lambda: fp8.expert_sort(ids.t(), 4), ValueError),
            (lambda: fp8.expert_sort(ids, 4, align=48), fp8.Fp8GemmError),
            (lambda: fp8.expert_sort(ids, 4, out=(pos, src)), ValueError),
            (lambda: fp8.expert_sort(ids, 4, rows=8, out=(pos, src, src, src)), ValueError),
            (lambda: fp8.expert_sort(torch.zeros(9000, dtype=i32, device="cuda"), 4,
                                     workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), fp8.Fp8GemmError),
            (lambda: fp8.expert_dispatch(x, pos[:3], src), ValueError),
            (lambda: fp8.expert_dispatch(x, pos, src, out=torch.empty((7, 256), device="cuda")), ValueError),
            (lambda: fp8.expert_dispatch(x.half(), pos, src), TypeError),
            (lambda: fp8.expert_dispatch_quant(x[:, :100].contiguous(), pos, 8), (ValueError, fp8.Fp8GemmError)),
            (lambda: fp8.expert_combine(x, pos, torch.ones((4, 3), device="cuda")), ValueError),
            (lambda: fp8.expert_combine(x, pos.long()), TypeError),
            (lambda: fp8.expert_combine(x, pos, out=torch.empty((4, 255), device="cuda")), ValueError),
            (lambda: fp8.expert_combine_grad(x.bfloat16(), x, pos), TypeError),
            (lambda: fp8.expert_combine_grad(x, x, pos, None, src), ValueError),
            (lambda: fp8.expert_combine(x, pos.cpu()), ValueError)):
        with pytest.raises(err):
            call()
