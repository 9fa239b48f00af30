"""Plain 64-bit forms of the operators around the experts' products and the
shared projection, and the bounds of their rounding errors (not a test
module).  NumPy only; shares no code with the kernels.

Error model: an FP32 operation is off by at most 2^-24 of its value, an
exponential by two units of 2^-23 and the rounding of its argument's
difference, a rounding to BF16 by 2^-8 of the value at most (half a step)."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def order(logits: np.ndarray, k: int) -> np.ndarray:
    """ids (T, k): by falling logit, ties by rising index; NaN first, -inf never (-1)."""
    l = np.asarray(logits, np.float64)
    rank = np.where(np.isnan(l), np.inf, l)
    first = np.where(np.isnan(l), 0, 1)                 # NaN before +inf
    index = np.broadcast_to(np.arange(l.shape[1]), l.shape)
    ids = np.lexsort((index, -rank, first), axis=1)[:, :k]
    return np.where(np.take_along_axis(rank, ids, 1) == -np.inf, -1, ids)


def _parts(logits, ids, renorm):
    """(p of the chosen (T, k), p of all (T, E)) before the scale, zeros where there is no expert."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    on = (ids >= 0) & (ids < E)
    lc = np.where(on, np.take_along_axis(l, np.clip(ids, 0, E - 1), 1), -np.inf)
    top = (lc if renorm else l).max(1, keepdims=True)
    if renorm is False:
        top = np.maximum(top, lc.max(1, keepdims=True))
    top = np.where(np.isfinite(top), top, 0.0)
    ec, ea = np.exp(lc - top), np.exp(l - top)
    s = (ec if renorm else ea).sum(1, keepdims=True)
    s = np.where(s == 0, 1.0, s)
    return ec / s, ea / s


def route(logits, k: int, renorm: bool, scale: float):
    ids = order(logits, k)
    return scale * _parts(logits, ids, renorm)[0], ids


def route_error(logits, weights) -> np.ndarray:
    """Bound of |computed - weights|: the largest exponent's difference that
    still counts (an exponential below e^-30 changes no sum), two exponentials,
    a sum of up to 16 + 6 steps, a quotient and a product."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isfinite(l), l, 0.0)
    d = np.minimum(l.max(1, keepdims=True) - l.min(1, keepdims=True), 110.0)
    return (2 * d + 8 + 22 + 4) * U * np.abs(weights) + 2.0 ** -140


def route_grad(dw, logits, ids, renorm: bool, scale: float):
    """(dlogits, sum of its terms' magnitudes)."""
    T, E = logits.shape
    pc, pa = _parts(logits, ids, renorm)
    on = (ids >= 0) & (ids < E)
    terms = np.where(on, pc * np.where(on, dw, 0.0), 0.0)
    total = terms.sum(1, keepdims=True)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    if not renorm:
        d -= pa * total
        mag += pa * np.abs(terms).sum(1, keepdims=True)
    rows = np.arange(T)
    for j in range(ids.shape[1]):
        t = rows[on[:, j]]
        e = ids[t, j]
        d[t, e] += terms[t, j] - (pc[t, j] * total[t, 0] if renorm else 0.0)
        mag[t, e] += np.abs(terms[t, j]) + (pc[t, j] * np.abs(terms[t]).sum(1) if renorm else 0.0)
    return scale * d, abs(scale) * mag


def sort_contiguous(ids, E: int, align: int, rows: int, keep: bool):
    """(pos, src, m_indices, counts), expert by expert."""
    flat = np.asarray(ids).reshape(-1)
    pos, src = np.full(flat.size, -1, np.int32), np.full(rows, -1, np.int32)
    m_indices, counts, at = np.full(rows, -1, np.int32), np.zeros(E, np.int32), 0
    for e in range(E + (1 if keep else 0)):
        pairs = np.flatnonzero(flat == e) if e < E else np.flatnonzero((flat < 0) | (flat >= E))
        if e < E:
            counts[e] = pairs.size
        fit = max(0, min(pairs.size, rows - at))
        pos[pairs[:fit]] = at + np.arange(fit)
        src[at:at + fit] = pairs[:fit]
        m_indices[at:at + fit] = e if e < E else -1
        at += -(-pairs.size // align) * align
    return pos.reshape(np.shape(ids)), src, m_indices, counts


def sort_masked(ids, E: int, max_m: int):
    flat = np.asarray(ids).reshape(-1)
    pos, src, masked_m = np.full(flat.size, -1, np.int32), np.full(E * max_m, -1, np.int32), np.zeros(E, np.int32)
    for e in range(E):
        pairs = np.flatnonzero(flat == e)[:max_m]
        pos[pairs] = e * max_m + np.arange(pairs.size)
        src[e * max_m:e * max_m + pairs.size] = pairs
        masked_m[e] = pairs.size
    return pos.reshape(np.shape(ids)), src, masked_m


def combine(y, pos, w):
    """(out, sum of its terms' magnitudes); a place outside y's rows adds nothing."""
    T, k = pos.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < y.shape[0]:
                term = (1.0 if w is None else float(w[t, j])) * y[pos[t, j]]
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def combine_grad(dout, y, pos, w, dy):
    """(dy filled where a pair has a row, dw, sum of dw's terms' magnitudes)."""
    T, k = pos.shape
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = pos[t, j]
            if 0 <= r < y.shape[0]:
                dy[r] = (1.0 if w is None else float(w[t, j])) * dout[t]
                dw[t, j] = dout[t] @ y[r]
                mag[t, j] = np.abs(dout[t]) @ np.abs(y[r])
    return dy, dw, mag


def adapters(x, a, b, scale, idx, y):
    """(out, the bound of its error before the last rounding).  The first
    product sums K terms in FP32; its result is kept as two BF16 values, off by
    2^-8 of the rest after a rounding by 2^-8 (2^-16 in all); the second sums 2 R."""
    T, K = x.shape
    R = a.shape[1]
    out, err = np.array(y, np.float64), np.zeros(y.shape)
    for t in range(T):
        i = int(idx[t])
        if 0 <= i < a.shape[0]:
            z, zm = a[i] @ x[t], np.abs(a[i]) @ np.abs(x[t])
            s = abs(float(scale[i]))
            out[t] += float(scale[i]) * (b[i] @ z)
            mag = np.abs(b[i])
            err[t] = s * (mag @ ((K / 8 + 64) * U * zm + (2.0 ** -16 + 2 * U) * np.abs(z))) \
                + (2 * R + 8) * U * (s * (mag @ np.abs(z)) + np.abs(y[t]))
    return out, err


def assert_near(got, ref, bound, what: str = "") -> None:
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bound = np.broadcast_to(bound, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)
    if np.any(bad):
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.size} outside the bound; first {i}: {got[i]} against "
                             f"{ref[i]}, bound {bound[i]}")


def rounded(bound, ref, bf16: bool):
    """`bound` with the last rounding's error: half a step of the type at the
    largest value in reach."""
    _, e = np.frexp(np.abs(ref) + 1.01 * bound)
    return 1.01 * bound + (np.ldexp(1.0, np.maximum(e, -125) - 9) if bf16 else np.ldexp(1.0, np.maximum(e, -125) - 25))
