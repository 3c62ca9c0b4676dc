"""The products of grouped rows, their gradients, and the norm in front of an
expert layer, in float64 (CPU oracle; test only).

P2, review comments: one routing serves every step, so the grouped rows are the
plan's: expert e's from offsets[e] on, counts[e] of them.  The 4-bit operands are
R22's and the 8-bit ones R11's.  Nothing is rounded here but where a function
says so: callers compare with the bounds of the arithmetic they check.
"""

import numpy as np

from . import formats as F
from . import mxfp8


def spans(counts, offsets):
    return [(e, slice(int(offsets[e]), int(offsets[e]) + int(counts[e]))) for e in range(len(counts))]


def gemm(rows, weight, counts, offsets):
    """out[g] = weight[e] rows[g] (zeros elsewhere) and the sums of the terms' magnitudes."""
    out = np.zeros((rows.shape[0], weight.shape[1]))
    mag = np.zeros_like(out)
    for e, at in spans(counts, offsets):
        out[at] = rows[at] @ weight[e].T
        mag[at] = np.abs(rows[at]) @ np.abs(weight[e]).T
    return out, mag


def dgrad(dout, weight, counts, offsets):
    return gemm(dout, np.swapaxes(weight, 1, 2), counts, offsets)


def wgrad(dout, rows, counts, offsets):
    out = np.zeros((len(counts), dout.shape[1], rows.shape[1]))
    mag = np.zeros_like(out)
    for e, at in spans(counts, offsets):
        out[e] = dout[at].T @ rows[at]
        mag[e] = np.abs(dout[at]).T @ np.abs(rows[at])
    return out, mag


def rmsnorm(h, weight, eps):
    """rstd and y of h [T, H]."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return rstd, h * rstd[:, None] * weight


def drmsnorm(dy, h, weight, rstd, dh=None):
    """dx, dweight (rstd as given, not taken again from h)."""
    r = rstd[:, None]
    g = dy * weight
    dx = r * (g - h * (r * r * (g * h).mean(axis=1, keepdims=True)))
    return dx if dh is None else dx + dh, (dy * h * r).sum(axis=0)


def mxfp8_f32(y):
    """R11 of FP32 rows: (data, scale bytes); 255 for a block that is not finite, whose data is not fixed."""
    y = np.asarray(y, dtype=np.float32)
    n, h = y.shape
    blocks = y.reshape(n, h // 32, 32).astype(np.float64)
    fine = np.isfinite(blocks).all(axis=2)
    blocks = np.where(fine[:, :, None], blocks, 0.0)
    e = mxfp8.scale_exponent(np.abs(blocks).max(axis=2))
    q = F.e4m3_encode(np.abs(blocks) / np.ldexp(1.0, e)[:, :, None])
    data = (np.signbit(blocks).astype(np.uint8) << 7) | q.astype(np.uint8)
    return data.reshape(n, h), np.where(fine, e + 127, 255).astype(np.uint8)
