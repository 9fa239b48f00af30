"""Integer zero points of the 4-bit products: q - z enters the product, so that
weights of zero add nothing, infinities follow the definition, and the error is
that of a sum of x (q - z)."""
import numpy as np
import pytest
import torch

import ffn_reference as ref
import fine_grained_block_e4m3_amd as fp8
from gpu_helpers import bf16_bits, bf16_to_f64, dev, say

pytestmark = pytest.mark.gpu

GROUPS = [32, 64, 128]


def _bf16(a):
    bits = ref.bf16_bits_of(ref.to_bf16(a)).view(np.int16)
    return torch.from_numpy(np.ascontiguousarray(bits)).cuda().view(torch.bfloat16)


def _pack(c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def _gemv(x, c, s, z):
    return bf16_to_f64(bf16_bits(fp8.gemv_w4(x, dev(_pack(c)), _bf16(s), zeros=None if z is None else dev(z))))


def _zeros_of(rng, K, N, group, zeros):
    return rng.integers(0, 16, (K // group, N), dtype=np.uint8) if zeros else None


def _spread(z, K, N, group):
    """Zero point of every weight, (N, K)."""
    return np.full((N, K), 8, np.int64) if z is None else np.repeat(z.T.astype(np.int64), group, axis=1)


@pytest.mark.parametrize("M", [1, 4, 5, 16])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
def test_weights_of_zero_add_nothing(M, group, zeros):
    """Rows of zeros give zeros, and a row with one other weight gives its
    product alone, whatever x is."""
    N, K = 67, 640
    say(f"zero weights M={M} group={group} zeros={zeros}")
    rng = np.random.default_rng(M + group)
    z = _zeros_of(rng, K, N, group, zeros)
    c = _spread(z, K, N, group).copy()
    row, at = np.arange(0, N, 2), rng.integers(0, K, (N + 1) // 2)
    off = np.where(c[row, at] == 15, -1, 1)
    c[row, at] += off
    s = ref.to_bf16(np.exp(rng.uniform(-6, 1, (K // group, N))))
    x = ref.to_bf16(rng.standard_normal((M, K)) + 300.0)
    got = _gemv(_bf16(x), c, s, z)
    want = np.zeros((M, N))
    want[:, row] = x[:, at] * off * s[at // group, row]     # a product of two BF16 values
    assert np.array_equal(got, ref.to_bf16(want.astype(np.float32)))
    one = dev(_pack(c)), _bf16(s)
    zd = None if z is None else dev(z)
    y = fp8.gated_gemv_w4(_bf16(x * 1e-3), *one, *one, zeros_g=zd, zeros_u=zd)
    assert not y[:, 1::2].any()


@pytest.mark.parametrize("M,N,K", [(1, 33, 384), (3, 130, 1152), (16, 500, 640), (9, 24570, 128)])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
def test_error_is_that_of_the_difference(M, N, K, group, zeros):
    """Bounded by |x| |q - z| s, not by the larger |x| (q + z) s."""
    say(f"zero points M={M} N={N} K={K} group={group} zeros={zeros}")
    rng = np.random.default_rng(N + group)
    z = _zeros_of(rng, K, N, group, zeros)
    full = _spread(z, K, N, group)
    c = np.clip(full + rng.integers(-1, 2, (N, K)), 0, 15)
    s = ref.to_bf16(np.exp(rng.uniform(-6, 1, (K // group, N))))
    x = ref.to_bf16(rng.standard_normal((M, K)) + 8.0)
    w = (c - full) * np.repeat(s.T, group, axis=1)
    got = _gemv(_bf16(x), c, s, z)
    # sums of 32 products at a time, within a group first, 8 waves joined
    ref.assert_bf16(got, x @ w.T, (K / 32 * 3 + 64) * ref.U_F32 * (np.abs(x) @ np.abs(w).T), "y")


@pytest.mark.parametrize("M", [1, 4, 7, 16])
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
def test_infinities_and_nan_follow_the_definition(M, group, zeros):
    N, K = 45, 384
    say(f"infinite x M={M} group={group} zeros={zeros}")
    rng = np.random.default_rng(3 * M + group)
    z = _zeros_of(rng, K, N, group, zeros)
    c = rng.integers(0, 16, (N, K))
    s = ref.to_bf16(np.exp(rng.uniform(-6, 1, (K // group, N))))
    w = (c - _spread(z, K, N, group)) * np.repeat(s.T, group, axis=1)
    x = ref.to_bf16(rng.standard_normal((M, K)))
    at = int(rng.integers(0, K))
    for token, value in enumerate((np.inf, -np.inf, np.nan)[:M]):
        x[token, at] = value
    with np.errstate(invalid="ignore"):
        want = x @ w.T                  # infinity times a weight of zero is NaN
    bits = torch.from_numpy(x.astype(np.float32)).cuda().bfloat16()
    got = _gemv(bits, c, s, z)
    k = min(M, 3)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[:k][np.isinf(want[:k])], want[:k][np.isinf(want[:k])])
    assert np.all(np.isfinite(got[k:])) and np.any(np.isinf(want[0]))


@pytest.mark.parametrize("group", GROUPS)
def test_products_below_the_largest_value_stay_finite(group):
    """x times the code alone would overflow FP32; x (q - z) s does not."""
    N, K = 32, 128
    say(f"large x group={group}")
    c = np.full((N, K), 13)
    z = np.full((K // group, N), 12, np.uint8)
    x = np.zeros((2, K))
    x[0, 5], x[1, 70] = 2.0 ** 127, -2.0 ** 127
    got = _gemv(_bf16(x), c, np.full((K // group, N), 2.0 ** -3), z)
    assert np.array_equal(got, np.repeat([[2.0 ** 124], [-2.0 ** 124]], N, axis=1))


def test_zero_points_of_every_value():
    """All 256 pairs of a code and a zero point."""
    say("codes and zero points")
    c = np.zeros((16, 128), np.int64)
    c[:, 0] = np.arange(16)
    x = np.zeros((1, 128))
    x[0, 0] = 1.0
    for z in range(16):
        c[:, 1:] = z
        got = _gemv(_bf16(x), c, np.ones((1, 16)), np.full((1, 16), z, np.uint8))
        assert np.array_equal(got[0], np.arange(16.0) - z)


def test_high_bits_of_a_zero_point_do_not_count():
    say("zero points with high bits")
    rng = np.random.default_rng(9)
    N, K = 40, 256
    c, z = rng.integers(0, 16, (N, K)), rng.integers(0, 16, (K // 64, N), dtype=np.uint8)
    s = ref.to_bf16(np.exp(rng.uniform(-6, 1, (K // 64, N))))
    x = _bf16(rng.standard_normal((3, K)))
    assert np.array_equal(_gemv(x, c, s, z), _gemv(x, c, s, z | 0xA0))
