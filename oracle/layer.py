"""Oracle of the operators around the einsums, in NumPy float64, from their
definitions: the root-mean-square norm and its gradients, quantisation into
e4m3 blocks with power-of-two scales, the product of two such matrices and the
products of rows grouped by expert.  Shares no code with the device path."""

from __future__ import annotations

import numpy as np

TOP = 448.0           # largest finite e4m3 value
COLS = 128            # columns that share a scale


def rmsnorm(r, weight, eps):
    r = np.asarray(r, np.float64)
    return r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps) * weight


def rmsnorm_backward(x, weight, dout, eps, d_residual=None):
    """(dx, dweight) of sum(rmsnorm(x, weight) * dout) [+ sum(x * d_residual)]."""
    x, weight, dout = (np.asarray(t, np.float64) for t in (x, weight, dout))
    root = np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps)
    n, g = x / root, weight * dout
    dx = (g - n * np.mean(g * n, axis=1, keepdims=True)) / root
    if d_residual is not None:
        dx = dx + d_residual
    return dx, np.sum(dout * n, axis=0)


def e4m3_round(v):
    """v (|v| <= 464) to the nearest e4m3 value, ties to the even one; NaN stays."""
    v = np.asarray(v, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(v == 0, 1.0, np.abs(v))))
        e = np.where(np.abs(v) >= 2.0 ** (e + 1), e + 1, np.where(np.abs(v) < 2.0 ** e, e - 1, e))
    step = 2.0 ** (np.maximum(np.nan_to_num(e), -6.0) - 3.0)
    return np.clip(np.rint(v / step) * step, -TOP, TOP)


def expand(scales, shape, block_rows):
    """One factor per element from one per block."""
    s = np.repeat(np.repeat(scales, block_rows, axis=0), COLS, axis=1)
    return s[:shape[0], :shape[1]]


def block_scales(x, block_rows):
    """The factors of x's blocks: the smallest 2^e, e >= -126, with max|x| <= 448 * 2^e; NaN for
    a block with a NaN or an infinity."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    out = np.empty((-(-rows // block_rows), -(-cols // COLS)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            b = np.abs(x[i * block_rows:(i + 1) * block_rows, j * COLS:(j + 1) * COLS])
            top = b.max()
            if not np.isfinite(top):
                out[i, j] = np.nan
                continue
            e = -126
            if top > TOP * 2.0 ** -126:
                e = max(-126, int(np.floor(np.log2(top / TOP))) - 1)
                while top > TOP * 2.0 ** e:
                    e += 1
            out[i, j] = 2.0 ** e
    return out


def quantize(x, block_rows):
    """(e4m3 values, factors)."""
    s = block_scales(x, block_rows)
    with np.errstate(invalid="ignore"):
        return e4m3_round(np.asarray(x, np.float64) / expand(s, np.shape(x), block_rows)), s


def block_scaled_product(a, sa, b, sb):
    """(a in 1 x 128 blocks) @ (b in 128 x 128 blocks)^T, and the sum of the products' magnitudes."""
    a = a * expand(sa, a.shape, 1)
    b = b * expand(sb, b.shape, 128)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def segments(offsets):
    return [(int(lo), int(hi)) for lo, hi in zip(offsets[:-1], offsets[1:])]


def ragged(a, b, offsets, before):
    """c[r] = a[r] @ b[e]^T over each expert's rows; other rows as `before`."""
    c = np.array(before, np.float64)
    for e, (lo, hi) in enumerate(segments(offsets)):
        c[lo:hi] = a[lo:hi] @ b[e].T
    return c


def ragged_dgrad(dc, b, offsets, before):
    da = np.array(before, np.float64)
    for e, (lo, hi) in enumerate(segments(offsets)):
        da[lo:hi] = dc[lo:hi] @ b[e]
    return da


def ragged_wgrad(dc, a, offsets):
    return np.stack([dc[lo:hi].T @ a[lo:hi] for lo, hi in segments(offsets)])
