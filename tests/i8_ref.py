"""Plain 64-bit implementations of the 8-bit integer operators for the tests,
from the definitions in include/hocf.h."""

import numpy as np

TINY = np.float32(2.0 ** -126)


def to_bf16(v):
    """float64 -> the nearest bfloat16 (halves to even) as float64; infinities and NaN stay."""
    v = np.asarray(v, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        m, e = np.frexp(v)                        # v = m 2^e, 0.5 <= |m| < 1
        step = np.ldexp(1.0, np.where(np.isfinite(v), np.maximum(e, -125), 0) - 8)
        r = np.round(v / step) * step             # (v / step is exact: a power of two)
        r = np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, v), r)
    return np.where(np.isfinite(v), r, v)


def silu(x):
    with np.errstate(over="ignore", invalid="ignore"):
        return x / (1.0 + np.exp(-x))


def silu_slope(h):
    with np.errstate(over="ignore", invalid="ignore"):
        p = 1.0 / (1.0 + np.exp(-h))
    return p * (1.0 + h * (1.0 - p))


def scale_of(a):
    """Scales (fp32) of the rows of a: largest magnitude / 127 in fp32, at least 2^-126; NaN where a row is not finite."""
    top = np.abs(a).max(axis=-1).astype(np.float32)
    with np.errstate(invalid="ignore"):
        s = np.maximum(top / np.float32(127), TINY)
    return np.where(np.isfinite(a).all(axis=-1), s, np.float32(np.nan)).astype(np.float32)


def quant(a):
    """(codes int8, scales fp32) of rows of float64 numbers that fp32 holds."""
    s = scale_of(a)
    with np.errstate(invalid="ignore"):
        q = np.round(a / s.astype(np.float64)[..., None])   # (numpy rounds halves to even)
    return np.where(np.isnan(s)[..., None], 0, q).astype(np.int8), s


def held(q, s):
    """What codes stand for where bf16 numbers are wanted (fp32 product, rounded)."""
    v = q.astype(np.float64) * s.astype(np.float64)[..., None]
    return to_bf16(v.astype(np.float32).astype(np.float64))


def groups(offsets, E, T):
    return [(0, T)] if offsets is None else [(int(offsets[e]), int(offsets[e + 1])) for e in range(E)]


def gemm(xq, xs, wq, ws, offsets=None):
    """out, NaN where no group has the row."""
    out = np.full((xq.shape[0], wq.shape[1]), np.nan)
    for e, (a, b) in enumerate(groups(offsets, wq.shape[0], xq.shape[0])):
        sums = xq[a:b].astype(np.float64) @ wq[e].astype(np.float64).T     # (whole numbers below 2^53: exact)
        out[a:b] = sums * xs[a:b].astype(np.float64)[:, None] * ws[e].astype(np.float64)
    return out


def dx(dy, wq, ws, offsets=None, pre=None):
    """(dx, sums of the terms' magnitudes), NaN where no group has the row; pre: (codes, scales)."""
    T, K = dy.shape[0], wq.shape[2]
    out, size = np.full((T, K), np.nan), np.full((T, K), np.nan)
    for e, (a, b) in enumerate(groups(offsets, wq.shape[0], T)):
        w = held(wq[e], ws[e])
        out[a:b], size[a:b] = dy[a:b] @ w, np.abs(dy[a:b]) @ np.abs(w)
    if pre is not None:
        slope = silu_slope(held(*pre))
        out, size = out * slope, size * np.abs(slope)
    return out, size


def dw(xq, xs, dy, E, offsets=None):
    """(dw, sums of the terms' magnitudes)."""
    out = np.zeros((E, xq.shape[1], dy.shape[1]))
    size = np.zeros_like(out)
    for e, (a, b) in enumerate(groups(offsets, E, xq.shape[0])):
        x = held(xq[a:b], xs[a:b])
        out[e], size[e] = x.T @ dy[a:b], np.abs(x).T @ np.abs(dy[a:b])
    return out, size
