"""Plain 64-bit forms of the feed-forward operators and the bounds of their
rounding errors (not a test module).  NumPy only; shares no code with the
kernels.

Error model used throughout: a BF16 rounding (8 significant bits) is off by at
most half a unit in the last place, 2^-8 of the value; an FP32 sum of n rounded steps by at most n * 2^-24 of the sum of the
magnitudes; one FP32 evaluation of an activation by a few units of 2^-24, the
exponential's argument t entering relatively (|t| * 2^-24)."""
from __future__ import annotations

import numpy as np

import oracle

U_BF16 = 2.0 ** -8
U_F32 = 2.0 ** -24


def to_bf16(a: np.ndarray) -> np.ndarray:
    """Nearest-even BF16 values of finite numbers, as float64 (one rounding)."""
    a = np.asarray(a, np.float64)
    m, e = np.frexp(a)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def bf16_bits_of(a: np.ndarray) -> np.ndarray:
    """Bit patterns of values that BF16 holds exactly."""
    f = np.asarray(a, np.float64).astype(np.float32)
    bits = f.view(np.uint32)
    assert np.all(bits & 0xFFFF == 0)
    return (bits >> 16).astype(np.uint16)


def act_parts(act: str, g: np.ndarray):
    """(t, p, dt/dg): act(g) = g * p, p = 1 / (1 + e^-t)."""
    if act == "silu":
        t, dt = g, np.ones_like(g)
    else:
        c = 2.0 * np.sqrt(2.0 / np.pi)
        t, dt = c * (g + 0.044715 * g ** 3), c * (1.0 + 3 * 0.044715 * g * g)
    with np.errstate(over="ignore"):
        p = 1.0 / (1.0 + np.exp(-t))
    return t, p, dt


def act_value(act: str, g: np.ndarray) -> np.ndarray:
    return g * act_parts(act, g)[1]


def act_grad(act: str, g: np.ndarray) -> np.ndarray:
    _, p, dt = act_parts(act, g)
    return p + g * dt * p * (1.0 - p)


def decode_x(q: np.ndarray, sa: np.ndarray) -> np.ndarray:
    return oracle.e4m3_decode(np.arange(256))[q] * np.repeat(sa.astype(np.float64).T, 128, axis=1)


def decode_w(q: np.ndarray, sb: np.ndarray) -> np.ndarray:
    s = np.repeat(np.repeat(sb.astype(np.float64), 128, axis=0)[:q.shape[0]], 128, axis=1)
    return oracle.e4m3_decode(np.arange(256))[q] * s


def gated(x: np.ndarray, wg: np.ndarray, wu: np.ndarray, act: str):
    """h, g, u and the bounds of their FP32 errors before the last rounding."""
    K = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    # sums of 16 products at a time, rescaled once per 128, joined over splits
    steps = K / 16 + 2 * K / 128 + 32
    eg, eu = (steps * U_F32 * (np.abs(x) @ np.abs(w).T) for w in (wg, wu))
    t = act_parts(act, g)[0]
    a = act_value(act, g)
    # |act'| <= 1.13; the activation itself: 8 roundings and the exponential's argument
    eh = 1.13 * np.abs(u) * eg + np.abs(a) * eu + 1.13 * eg * eu + (8 + 4 * np.abs(t)) * U_F32 * np.abs(a * u)
    return (a * u, g, u), (eh, eg, eu)


def assert_bf16(got: np.ndarray, ref: np.ndarray, err: np.ndarray, what: str = "") -> None:
    """got: BF16 values; ref exact, computed with an error of at most err and
    then rounded."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    # half a unit in the last place of the largest value in reach
    _, e = np.frexp(np.abs(ref) + 1.01 * err)
    bound = 1.01 * err + np.ldexp(1.0, np.maximum(e, -125) - 9)
    bad = np.abs(got - ref) > bound
    if np.any(bad):
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.size} outside the bound; first {i}: "
                             f"{got[i]} against {ref[i]}, bound {np.broadcast_to(bound, got.shape)[i]}")


def gated_grad(dh, g, u, x, wg, wu, act: str):
    """(dx, dwg, dwu) and their error bounds before the last rounding: dg and
    du are rounded once to BF16."""
    M, N = dh.shape
    a, d = act_value(act, g), act_grad(act, g)
    t, p, dt = act_parts(act, g)
    dg, du = dh * u * d, dh * a
    # the derivative's terms, p and g dt p (1 - p), are evaluated with a few
    # roundings of each and of 1 - p
    ed = (16 + 8 * np.abs(t)) * U_F32 * (p + np.abs(g * dt) * p)
    eg = np.abs(dh * u) * ed + U_BF16 * 1.01 * np.abs(dg)
    eu = (16 + 8 * np.abs(t)) * U_F32 * np.abs(du) + U_BF16 * 1.01 * np.abs(du)
    sx, sw = (2 * N / 16 + 64) * U_F32, (M / 16 + 64) * U_F32
    out = (dg @ wg + du @ wu, dg.T @ x, du.T @ x)
    err = (eg @ np.abs(wg) + eu @ np.abs(wu) + 1.02 * sx * (np.abs(dg) @ np.abs(wg) + np.abs(du) @ np.abs(wu)),
           eg.T @ np.abs(x) + 1.02 * sw * (np.abs(dg).T @ np.abs(x)),
           eu.T @ np.abs(x) + 1.02 * sw * (np.abs(du).T @ np.abs(x)))
    return out, err


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nibbles(q: np.ndarray) -> np.ndarray:
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.int64)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def decode_mxfp4(q: np.ndarray, e: np.ndarray) -> np.ndarray:
    """q (N, K/2), e uint32 (K/128, N): group 4 kb + t of row n in byte t."""
    c = nibbles(q)
    v = np.where(c >= 8, -E2M1[c & 7], E2M1[c & 7])
    b = np.stack([(e >> (8 * t)) & 255 for t in range(4)], axis=2)          # (K/128, N, 4)
    b = b.transpose(1, 0, 2).reshape(q.shape[0], -1).astype(np.int64)
    return v * np.repeat(np.ldexp(1.0, b - 127), 32, axis=1)


def decode_int4(q: np.ndarray, s: np.ndarray, z, group: int):
    """(w, magnitudes of the two terms s q and s z that it is formed from)."""
    c = nibbles(q).astype(np.float64)
    sc = np.repeat(np.asarray(s, np.float64).T, group, axis=1)
    zp = 8.0 if z is None else np.repeat(z.astype(np.float64).T, group, axis=1)
    return (c - zp) * sc, (c + zp) * sc


def quant_int4(w: np.ndarray, group: int, symmetric: bool):
    """Codes (N, K/2), BF16 scale bits (K/group, N), zero points (K/group, N)."""
    f = np.float32
    N, K = w.shape
    g = w.astype(f).reshape(N, K // group, group)
    lo, hi = np.minimum(g.min(2), f(0)), np.maximum(g.max(2), f(0))
    wide = np.maximum(hi, -lo) / f(7) if symmetric else (hi - lo) / f(15)
    bits = bf16_bits_of(to_bf16(np.maximum(wide, f(1e-8))))
    s = (bits.astype(np.uint32) << 16).view(f)
    z = np.full(s.shape, f(8)) if symmetric else np.clip(np.rint(-lo / s), f(0), f(15))
    c = np.clip(np.rint(g / s[..., None]) + z[..., None], 0, 15).astype(np.uint8).reshape(N, K)
    return c[:, 0::2] | (c[:, 1::2] << 4), np.ascontiguousarray(bits.T), np.ascontiguousarray(z.T.astype(np.uint8))
