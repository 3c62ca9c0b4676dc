"""The expert layer's unquantized steps, in float64 (CPU oracle; test only).

P2, review comments: one routing serves the dispatch and the combine.  The
products take the packed NVFP4 rows of P1 (R7) as weights; the 8-bit checkpoint
is MXFP8 (R11).  Nothing is rounded here: callers compare with the bounds of the
arithmetic they check.
"""

import numpy as np

from . import formats as F
from . import mxfp8, nvfp4


def f64(bits):
    return F.bf16_to_f32(bits).astype(np.float64)


def dispatch(x, src_row):
    """out[g] = x[src_row[g]], zeros where src_row[g] is no token."""
    out = np.zeros((len(src_row), x.shape[1]), dtype=x.dtype)
    for g, s in enumerate(src_row):
        if 0 <= s < x.shape[0]:
            out[g] = x[s]
    return out


def combine(rows, dst_row, weights=None):
    """out[t] = sum_j weights[t, j] rows[dst_row[t, j]] over the used slots, and the
    sum of the terms' magnitudes (for error bounds)."""
    t, k = dst_row.shape
    out, mag = np.zeros((t, rows.shape[1])), np.zeros((t, rows.shape[1]))
    for i in range(t):
        for j in range(k):
            g = dst_row[i, j]
            if 0 <= g < rows.shape[0]:
                term = rows[g] * (1.0 if weights is None else float(weights[i, j]))
                out[i] += term
                mag[i] += np.abs(term)
    return out, mag


def combine_bwd(dout, rows, dst_row, weights):
    """drows, dweights and, for bounds, the sums of the magnitudes behind dweights."""
    t, k = dst_row.shape
    drows = np.zeros_like(rows)
    dw, mag = np.zeros((t, k)), np.zeros((t, k))
    for i in range(t):
        for j in range(k):
            g = dst_row[i, j]
            if 0 <= g < rows.shape[0]:
                drows[g] = float(weights[i, j]) * dout[i]
                p = dout[i] * rows[g]
                dw[i, j], mag[i, j] = p.sum(), np.abs(p).sum()
    return drows, dw, mag


def matvec(x, weight, topk_idx=None):
    """y[t, j] = W[topk_idx[t, j]] x[t] (x [T, K]) or x[t, j] (x [T, k, K]) for packed
    NVFP4 weights [E, N, 9K/16 + 4]; the sums of the terms' magnitudes beside it.
    Ids outside [0, E) give zero rows.  Without topk_idx: weight [N, .], y [T, N]."""
    K = x.shape[-1]
    if topk_idx is None:
        w = nvfp4.decode_exact(weight, K)
        return x @ w.T, np.abs(x) @ np.abs(w).T
    t, k = topk_idx.shape
    y, mag = np.zeros((t, k, weight.shape[1])), np.zeros((t, k, weight.shape[1]))
    cache = {}
    for i in range(t):
        for j in range(k):
            e = int(topk_idx[i, j])
            if 0 <= e < weight.shape[0]:
                if e not in cache:
                    cache[e] = nvfp4.decode_exact(weight[e], K)
                v = x[i, j] if x.ndim == 3 else x[i]
                y[i, j], mag[i, j] = cache[e] @ v, np.abs(cache[e]) @ np.abs(v)
    return y, mag


def sigmoid(a):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-a))


def swiglu(p):
    """silu(a) * b of [.., 2F] = [a | b]."""
    a, b = np.split(p, 2, axis=-1)
    return a * sigmoid(a) * b


def swiglu_grad(p, dy):
    """Gradient of sum(dy * swiglu(p)) by p."""
    a, b = np.split(p, 2, axis=-1)
    s = sigmoid(a)
    return np.concatenate([dy * b * s * (1.0 + a * (1.0 - s)), dy * a * s], axis=-1)


def checkpoint_values(preact_bits):
    """What the 8-bit checkpoint of preact stands for."""
    return mxfp8.decode(*mxfp8.pack_rows(preact_bits))
