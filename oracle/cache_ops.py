"""Plain numpy fp64 statements of the operators over key/value caches: the
E4M3 cache and attention with lengths and masks.  Shares no code with the GPU
path."""

from __future__ import annotations

import numpy as np


def quantize_rows(x):
    """(values of the E4M3 codes, scales) of the rows x [..., D].

    scale = the least power of two, 2^-126 or more, with max|x| <= 448 *
    scale; the code is x / scale on the E4M3 grid (four significand bits,
    exponents -6..8, subnormal step 2^-9), ties to even.  A row with a NaN or
    an infinity has scale NaN and codes 0."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        top = np.max(np.abs(x), axis=-1)
        finite = np.isfinite(top)
        m, e = np.frexp(np.where(finite, top, 1.0))      # top = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
        e = np.where(top == 0, -126, np.maximum(np.where(m <= 0.875, e - 9, e - 8), -126))
        scale = np.ldexp(1.0, e)
        y = np.where(finite[..., None], x, 0.0) / scale[..., None]
    _, ey = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))   # |y| in [2^(ey-1), 2^ey): step 2^(ey-4)
    step = np.ldexp(1.0, ey - 4)
    return np.round(y / step) * step, np.where(finite, scale, np.nan)


def attention(q, parts, scale):
    """One head: q [T][D] against the visible keys of parts, a list of (k
    [N][D], v [N][D], visible [N] bool).  Returns (out [T][D], lse [T]) and
    weights' sum of |v| [T][D] (for error bounds); a query that sees nothing
    gives 0 and -inf."""
    k = np.concatenate([np.asarray(k, np.float64)[w] for k, _, w in parts])
    v = np.concatenate([np.asarray(v, np.float64)[w] for _, v, w in parts])
    q = np.asarray(q, np.float64)
    if k.shape[0] == 0:
        z = np.zeros((q.shape[0], q.shape[1]))
        return z, np.full(q.shape[0], -np.inf), z
    s = scale * (q @ k.T)
    top = s.max(axis=1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(axis=1, keepdims=True)
    return p @ v / total, (top + np.log(total))[:, 0], p @ np.abs(v) / total
