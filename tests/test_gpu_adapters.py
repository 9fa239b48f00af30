"""Low-rank adapters of many requests against their 64-bit form: every rank's
kernel, one token to long prompts, tokens without an adapter, in place and
out of place, shared and split tiles."""
import ctypes

import numpy as np
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
import routing_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _operands(rng, T, L, R, K, N):
    def bf16(a):
        return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().cuda()
    return (bf16(rng.normal(size=(T, K))), bf16(rng.normal(size=(L, R, K)) / K ** 0.5), bf16(rng.normal(size=(L, N, R)) * 0.3),
            torch.from_numpy(rng.uniform(0.5, 2, L).astype(np.float32)).cuda(), bf16(rng.normal(size=(T, N))))


def _f64(t):
    return t.double().cpu().numpy()


def _check(rng, T, L, R, K, N, idx, what):
    x, a, b, s, y = _operands(rng, T, L, R, K, N)
    rows = fp8.adapter_rows(torch.from_numpy(np.asarray(idx)).cuda(), L)
    full = torch.full((T * N + 32,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = fp8.add_adapters(x, a, b, s, rows, y, out=full[16:16 + T * N].view(T, N))
    r, err = ref.adapters(_f64(x), _f64(a), _f64(b), _f64(s), idx, _f64(y))
    ref.assert_near(_f64(out), r, ref.rounded(err, r, True), what)
    assert bool((full[:16] == 9).all()) and bool((full[-16:] == 9).all())
    none = torch.from_numpy((np.asarray(idx) < 0) | (np.asarray(idx) >= L)).cuda()
    assert torch.equal(out[none].view(torch.int16), y[none].view(torch.int16))
    again = fp8.add_adapters(x, a, b, s, rows, y)
    assert torch.equal(again, out)
    here = y.clone()
    assert fp8.add_adapters(x, a, b, s, rows, here, out=here) is here
    assert torch.equal(here, out)


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128])
def test_ranks(R):
    rng = np.random.default_rng(R)
    for T, L, K, N in ((1, 1, 128, 1), (1, 3, 7168, 2048), (5, 2, 640, 77), (40, 6, 256, 300), (100, 64, 1536, 130)):
        say("adapters", R, T, L, K, N)
        _check(rng, T, L, R, K, N, rng.integers(-1, L + 1, T), f"{R} {T} {L} {K} {N}")


@pytest.mark.parametrize("N", [1, 3, 8, 63, 64, 65, 255, 257, 1000])
def test_widths(N):
    rng = np.random.default_rng(N)
    say("adapters width", N)
    _check(rng, 33, 3, 16, 384, N, rng.integers(-1, 3, 33), f"width {N}")


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
def test_orders(dtype):
    """One adapter for all, runs, none at all, every token its own."""
    rng = np.random.default_rng(1)
    T, L = 150, 200
    for name, idx in (("one", np.full(T, 7)), ("runs", np.arange(T) // 40), ("none", np.full(T, -1)),
                      ("own", rng.permutation(L)[:T]), ("far", rng.choice([-2 ** 31, 2 ** 31 - 1, 5], T))):
        say("adapters order", name)
        _check(rng, T, L, 16, 256, 200, idx.astype(dtype), name)


def test_many_tiles():
    """So many tokens per adapter that a workgroup takes four tiles, of one adapter, of two, of one and none."""
    rng = np.random.default_rng(2)
    for T, L, R, K, N, group in ((8301, 5, 16, 128, 72, 4), (4000, 300, 24, 256, 130, 1), (2700, 40, 64, 384, 65, 4),
                                 (3080, 12, 32, 2048, 600, 4), (3080, 12, 32, 512, 640, 4), (2000, 3, 64, 256, 192, 4),
                                 (1000, 3, 128, 1152, 340, 4), (1400, 5, 72, 640, 128, 4), (2100, 60, 24, 1152, 333, 4),
                                 (1500, 60, 40, 896, 520, 4), (500, 19, 104, 640, 1030, 4), (6200, 250, 8, 128, 64, 4)):
        idx = rng.integers(-1, L, T)
        assert fp8.adapters_plan(T, L, N, K, R)["group"] == group
        say("adapters many tiles", T, L, R)
        _check(rng, T, L, R, K, N, idx, "many tiles")


@pytest.mark.parametrize("R", [8, 16, 24, 40, 56, 64])
def test_one_kernel(R):
    """Few tokens per adapter, of which each workgroup of a tile takes a share or
    a part of N: from one token to a full tile, K and N long and short."""
    rng = np.random.default_rng(100 + R)
    for T, L, K, N in ((1, 4, 128, 1), (1, 1, 640, 4099), (2, 40, 7168, 2100), (16, 200, 1152, 2048), (16, 40, 128, 9000),
                       (30, 60, 512, 600), (40, 70, 8192, 130)):
        plan = fp8.adapters_plan(T, L, N, K, R)
        assert plan["whole"] > 0 and plan["workspace_bytes"] == 0
        for name, idx in (("any", rng.integers(-1, L + 1, T)), ("one", np.full(T, L - 1)), ("pairs", np.arange(T) // 2 % L),
                          ("sevens", np.arange(T) // 7 % L), ("none", np.full(T, -1))):
            say("adapters one kernel", R, T, L, K, N, name)
            _check(rng, T, L, R, K, N, idx, f"{name} {R} {T} {L} {K} {N}")


def test_either_side_of_one_kernel():
    """The sizes beside each bound of the rule, and both forms on the same tokens."""
    rng = np.random.default_rng(9)
    for T, L, R, whole in ((84, 200, 16, True), (86, 200, 16, False), (8, 8, 64, True), (8, 8, 72, False), (21, 4, 64, False),
                           (9, 0, 64, True)):
        L = L or 9
        assert (fp8.adapters_plan(T, L, 300, 256, R)["whole"] > 0) == whole, (T, L, R)
        say("adapters beside a bound", T, L, R)
        _check(rng, T, L, R, 256, 300, rng.integers(-1, L, T), f"{T} {L} {R}")
    # the same rows in a table with more tiles: two kernels
    T, L, R, K, N = 20, 30, 16, 2048, 1000
    x, a, b, s, y = _operands(rng, T, L, R, K, N)
    idx = rng.integers(-1, 5, T)
    rows = fp8.adapter_rows(torch.from_numpy(idx).cuda(), L)
    more = torch.full((2, 16 * 90), -1, dtype=torch.int32, device="cuda")
    more[:, :rows.shape[1]] = rows
    r, err = ref.adapters(_f64(x), _f64(a), _f64(b), _f64(s), idx, _f64(y))
    for table in (rows, more):
        ref.assert_near(_f64(fp8.add_adapters(x, a, b, s, table, y)), r, ref.rounded(err, r, True), "both forms")


def test_infinities_stay_with_their_token():
    """What one token, adapter or column holds does not reach another's."""
    say("adapters infinities")
    rng = np.random.default_rng(10)
    T, L, R, K, N = 20, 40, 24, 640, 200
    x, a, b, s, y = _operands(rng, T, L, R, K, N)
    idx = np.array([3] * 7 + [4] * 6 + [-1] * 3 + [5] * 4)
    r, err = ref.adapters(_f64(x), _f64(a), _f64(b), _f64(s), idx, _f64(y))
    x[2, 639], a[4, 23, 600], b[5, 199, 23], y[14, 3] = float("inf"), float("nan"), float("-inf"), float("nan")
    rows = fp8.adapter_rows(torch.from_numpy(idx).cuda(), L)
    assert fp8.adapters_plan(T, L, N, K, R)["whole"] > 0
    out = fp8.add_adapters(x, a, b, s, rows, y)
    bad = torch.zeros((T, N), dtype=torch.bool)
    bad[2], bad[7:13], bad[16:20, 199], bad[14, 3] = True, True, True, True
    assert not bool(torch.isfinite(out.cpu()[bad]).any())
    good = ~bad.numpy()
    ref.assert_near(_f64(out)[good], r[good], ref.rounded(err, r, True)[good], "infinities")


@pytest.mark.parametrize("R,whole", [(16, False), (8, True)])
def test_given_tables(R, whole):
    """Rows outside the tokens, tiles of mixed indices, tiles without a row."""
    say("adapters given tables", R)
    rng = np.random.default_rng(3)
    T, L, K, N = 20, 3, 256, 100
    plan = fp8.AdaptersPlan()
    assert fp8.load_library().fp8_adapters_plan(T, L, 64, N, K, R, 256, ctypes.byref(plan)) == 0
    assert (plan.whole > 0) == whole
    x, a, b, s, y = _operands(rng, T, L, R, K, N)
    src = torch.full((64,), -1, dtype=torch.int32, device="cuda")
    index = torch.full((64,), 1, dtype=torch.int32, device="cuda")
    src[3], src[5], src[7] = 4, T, 9            # T: no token
    index[3], index[7] = 2, 0                   # token 9 is not computed: the tile is token 4's
    src[33], src[34], index[33], index[34] = 0, 19, 1, 1
    out = fp8.add_adapters(x, a, b, s, torch.stack((src, index)), y, out=torch.full_like(y, 5.0))
    idx = np.full(T, -1)
    idx[[4, 0, 19]] = 2, 1, 1
    r, err = ref.adapters(_f64(x), _f64(a), _f64(b), _f64(s), idx, _f64(y))
    done = [0, 4, 19]
    ref.assert_near(_f64(out)[done], r[done], ref.rounded(err, r, True)[done], "given")
    assert bool((out[[i for i in range(T) if i not in done]] == 5).all())


def test_workspace_and_refusals():
    say("adapters refusals")
    rng = np.random.default_rng(4)
    x, a, b, s, y = _operands(rng, 10, 3, 128, 2048, 1200)
    rows = fp8.adapter_rows(torch.zeros(10, dtype=torch.int32, device="cuda"), 3)
    plan = fp8.adapters_plan(10, 3, 1200, 2048, 128)
    assert plan["group"] == 1 and plan["k_splits"] > 1
    size = plan["workspace_bytes"]
    want = fp8.add_adapters(x, a, b, s, rows, y)
    ws = torch.full((size + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(fp8.add_adapters(x, a, b, s, rows, y, workspace=ws[:size]), want)
    assert bool((ws[size:] == 0xFF).all())
    with pytest.raises(fp8.Fp8GemmError):
        fp8.add_adapters(x, a, b, s, rows, y, workspace=ws[:size - 16])
    for bad in ((x[:9], a, b, s, rows, y), (x, a[:2], b, s, rows, y), (x, a, b[:, :1199].contiguous(), s, rows, y),
                (x, a, b, s[:2], rows, y), (x, a, b, s, rows[:1], y), (x.t(), a, b, s, rows, y),
                (x, a, b, s, rows, y.cpu())):
        with pytest.raises(ValueError):
            fp8.add_adapters(*bad)
    with pytest.raises(TypeError):
        fp8.add_adapters(x.float(), a, b, s, rows, y)
    with pytest.raises(fp8.Fp8GemmError):          # a rank that is no multiple of 8
        fp8.add_adapters(x, a[:, :12].contiguous(), b[:, :, :12].contiguous(), s, rows, y)
    assert fp8.add_adapters(x[:0], a, b, s, fp8.adapter_rows(torch.zeros(0, dtype=torch.int32, device="cuda"), 3),
                            y[:0]).shape == (0, 1200)


@pytest.mark.parametrize("T,L,R,whole,group", [(6, 40, 16, True, 1), (70, 3, 16, False, 1), (1600, 5, 32, False, 4)])
def test_graph_replays(T, L, R, whole, group):
    """Two captured projections of one table, replayed with other tokens and
    other adapters, eager calls on another stream in between."""
    say("adapters graph", T, L)
    rng = np.random.default_rng(11)
    K, N = 768, 200
    plan = fp8.adapters_plan(T, L, N, K, R)
    assert (plan["whole"] > 0) == whole and plan["group"] == group
    x, a, b, s, y = _operands(rng, T, L, R, K, N)
    a2, b2 = b.new_empty(a.shape).copy_(a.flip(1)), b.flip(1).contiguous()
    idx = torch.zeros(T, dtype=torch.int32, device="cuda")

    def step():
        rows = fp8.adapter_rows(idx, L)
        return fp8.add_adapters(x, a, b, s, rows, y), fp8.add_adapters(x, a2, b2, s, rows, y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(4):
        new = np.random.default_rng(20 + seed)
        x.copy_(torch.from_numpy(new.normal(size=(T, K)).astype(np.float32)))
        idx.copy_(torch.from_numpy(new.integers(-1, L if seed else 1, T).astype(np.int32)))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w), seed
        r, err = ref.adapters(_f64(x), _f64(a), _f64(b), _f64(s), idx.cpu().numpy(), _f64(y))
        ref.assert_near(_f64(got[0]), r, ref.rounded(err, r, True), f"replay {seed}")
