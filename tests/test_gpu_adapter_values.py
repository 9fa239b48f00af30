"""Values of the adapters' first product that are not ordinary: infinities,
NaN and magnitudes at the types' ends, in each of the three forms."""
import numpy as np
import pytest
import torch

import fine_grained_block_e4m3_amd as fp8
import routing_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu

# (T, adapters, K, N) of one kernel, of two with a tile each, and of groups of four tiles
FORMS = {"whole": (20, 40, 640, 200), "tiles": (150, 3, 640, 200), "groups": (6200, 5, 256, 72)}
RANKS = {"whole": (8, 24, 40, 64), "tiles": (8, 24, 40, 104), "groups": (8, 24, 40, 104)}
CASES = [(form, R) for form in FORMS for R in RANKS[form]]


def _sizes(form, R):
    T, L, K, N = FORMS[form]
    plan = fp8.adapters_plan(T, L, N, K, R)
    assert (plan["whole"] > 0) == (form == "whole") and plan["group"] == (4 if form == "groups" else 1)
    return T, L, K, N


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().cuda()


def _f64(t):
    return t.double().cpu().numpy()


def _signs(rng, shape):
    """Magnitudes between 0.5 and 2 of either sign: no zero, which times an infinity is no number."""
    return rng.uniform(0.5, 2, shape) * rng.choice([-1.0, 1.0], shape)


def _same(got, want, err):
    """NaN where `want` is, its infinities with their signs, and its finite values within err and the last rounding."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf])
    ok = np.isfinite(want)
    ref.assert_near(got[ok], want[ok], ref.rounded(err[ok], want[ok], True), "finite values")


@pytest.mark.parametrize("form,R", CASES)
def test_infinities_keep_their_sign(form, R):
    """An infinite element of a, x or y makes what the definition makes of it."""
    say("adapters infinite", form, R)
    rng = np.random.default_rng(R)
    T, L, K, N = _sizes(form, R)
    x, a, b, y = _bf16(_signs(rng, (T, K))), _bf16(_signs(rng, (L, R, K)) / K), _bf16(_signs(rng, (L, N, R))), _bf16(_signs(rng, (T, N)))
    s = torch.from_numpy(_signs(rng, L).astype(np.float32)).cuda()
    idx = rng.integers(0, L, T)
    idx[:8] = [0, 1, 2, 0, 1, 2, 0, 1]
    err = ref.adapters(_f64(x), _f64(a), _f64(b), _f64(s), idx, _f64(y))[1]
    inf = float("inf")
    a[0, R - 1, K - 1] = inf                            # +-inf by the signs of its token's x, its column's b and the scale
    a[1, 0, 3], b[1, 5, 0] = -inf, 0.0                  # and no number in column 5
    a[2, :, 7] = a[2, :, 7].abs()                       # one token's x: all of its z are infinities of one sign ...
    b[2, :20] = b[2, :20].abs()                         # ... and so are the first columns' terms; others differ in sign
    x[2, 7], y[5, 9] = -inf, inf
    with np.errstate(invalid="ignore"):
        want = _f64(y)
        xa, aa, ba = _f64(x), _f64(a), _f64(b)
        for t in range(T):
            want[t] += float(s[idx[t]]) * (ba[idx[t]] @ (aa[idx[t]] @ xa[t]))
    assert np.isnan(want[1, 5]) and np.isinf(want[0]).all() and np.isinf(want[2, :20]).all() and np.isnan(want[2]).any()
    out = fp8.add_adapters(x, a, b, s, fp8.adapter_rows(torch.from_numpy(idx).cuda(), L), y)
    _same(_f64(out), want, err)


@pytest.mark.parametrize("form,R", CASES)
def test_magnitudes_at_the_end_of_the_type(form, R):
    """A scaled z between BF16's largest value (3.39e38) and FP32's (3.40e38)
    is a number like others: times a small b it is in the middle of the range."""
    say("adapters at the end of the type", form, R)
    rng = np.random.default_rng(100 + R)
    T, L, K, N = _sizes(form, R)
    x, a, b, y = np.zeros((T, K)), np.zeros((L, R, K)), _signs(rng, (L, N, R)) * 2.0 ** -120, _signs(rng, (T, N))
    x[:, 0], a[:, :, 0] = 1.0, rng.choice([-1.0, 1.0], (L, R))
    x, a, b, y = _bf16(x), _bf16(a), _bf16(b), _bf16(y)
    s = torch.full((L,), 3.4e38, device="cuda")
    idx = rng.integers(-1, L, T)
    want, err = ref.adapters(_f64(x), _f64(a), _f64(b), _f64(s), idx, _f64(y))
    assert np.abs(want).max() > 100
    out = fp8.add_adapters(x, a, b, s, fp8.adapter_rows(torch.from_numpy(idx).cuda(), L), y)
    _same(_f64(out), want, err)


@pytest.mark.parametrize("form,R", CASES)
def test_infinite_scales(form, R):
    """An infinite scale of terms of one sign gives infinities of that sign,
    whatever the rank is rounded up to; other adapters' tokens see nothing of it."""
    say("adapters infinite scale", form, R)
    rng = np.random.default_rng(200 + R)
    T, L, K, N = _sizes(form, R)
    x, a = _bf16(rng.uniform(0.5, 2, (T, K))), _bf16(rng.uniform(0.5, 2, (L, R, K)) / K)
    b = rng.uniform(0.5, 2, (L, N, R)) * rng.choice([-1.0, 1.0], (L, N, 1))
    b, y = _bf16(b), _bf16(_signs(rng, (T, N)))
    s = torch.ones(L, device="cuda")
    s[0], s[1] = float("inf"), float("-inf")
    idx = rng.integers(-1, L, T)
    idx[:4] = [0, 1, 0, 1]
    finite = torch.ones(L, device="cuda")
    want, err = ref.adapters(_f64(x), _f64(a), _f64(b), _f64(finite), idx, _f64(y))
    for i, sign in ((0, 1.0), (1, -1.0)):
        want[idx == i] = sign * np.sign(_f64(b)[i, :, 0]) * np.inf
    out = fp8.add_adapters(x, a, b, s, fp8.adapter_rows(torch.from_numpy(idx).cuda(), L), y)
    _same(_f64(out), want, err)


@pytest.mark.parametrize("form,R", CASES)
@pytest.mark.parametrize("scale", [1.0, -0.125])
def test_every_bit_of_the_first_product(form, R, scale):
    """What is left where y takes away the leading bits of the added term.

    x and a are whole numbers up to 255 and x has 128 places that are not zero:
    every z and every sum on the way to it is a whole number below 2^23, which
    FP32 holds.  b has one 1 per column and y is the term rounded to BF16: the
    last sum is exact in FP32 too, and out is its one rounding."""
    say("adapters every bit", form, R, scale)
    rng = np.random.default_rng(300 + R)
    T, L, K, N = _sizes(form, R)
    x, a = rng.integers(100, 256, (T, K)), rng.integers(100, 256, (L, R, K))
    x[:, rng.permutation(K)[128:]] = 0
    b = np.zeros((L, N, R))
    b[:, np.arange(N), np.arange(N) % R] = 1.0
    idx = rng.integers(0, L, T)
    z = np.stack([a[i] @ x[t] for t, i in enumerate(idx)])
    assert z.max() < 2 ** 23 and (z & 0xFF).any()
    term = torch.from_numpy(np.ascontiguousarray(scale * z[:, np.arange(N) % R], np.float32))
    y = -term.bfloat16()
    want = (y.float() + term).bfloat16()                    # both operands and the sum exact
    x, a, b, s = _bf16(x), _bf16(a), _bf16(b), torch.full((L,), scale, device="cuda")
    out = fp8.add_adapters(x, a, b, s, fp8.adapter_rows(torch.from_numpy(idx).cuda(), L), y.cuda())
    assert torch.equal(out.cpu(), want)
