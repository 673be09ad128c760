"""Plain fp64 definitions of the 8-bit format and the operators that use it.

TEST INFRASTRUCTURE ONLY, as ``dora_oracle``: it shares no code with the CUDA
library.  A stretch of values v is kept as the integers nearest to
127 v / max|v| (ties to even) and the scale max|v| / 127; a stretch is a whole
row, or ``width`` columns of one.  Stretches below 2^-100 keep zeros, stretches
with an infinity or a NaN keep the scale NaN.
"""

from __future__ import annotations

import numpy as np

TINY = 2.0 ** -100


def encode(v, width=None):
    """(codes int64 [rows, cols], scale fp64 [rows, stretches]) of the rows of v."""
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    width = cols if width is None else width
    codes = np.zeros((rows, cols), dtype=np.int64)
    scale = np.zeros((rows, -(-cols // width)))
    for j in range(scale.shape[1]):
        part = v[:, j * width:(j + 1) * width]
        top = np.max(np.abs(part), axis=1)
        ok = np.isfinite(top) & (top >= TINY)
        scale[:, j] = np.where(ok, top / 127.0, np.where(np.isfinite(top), 0.0, np.nan))
        codes[ok, j * width:(j + 1) * width] = np.rint(127.0 * part[ok] / top[ok, None]).astype(np.int64)
    return codes, scale


def decode(codes, scale, width=None):
    """codes * scale, fp64."""
    codes, scale = np.asarray(codes, dtype=np.float64), np.asarray(scale, dtype=np.float64)
    cols = codes.shape[1]
    width = cols if width is None else width
    return codes * scale.reshape(codes.shape[0], -1)[:, np.arange(cols) // width]


def rms_factor(h, eps):
    """1 / sqrt(mean(h^2) + eps) of each row, [rows, 1]."""
    h = np.asarray(h, dtype=np.float64)
    return 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)


def linear_i8(x_q, x_scale, W_q, w_scale, x, A, B, m, n, s, bias):
    """b + (m / n) * (x_scale w_scale (x_q W_q^T) + s (x A^T) B^T); x, A, B or m, n or bias may be None."""
    f = lambda t: np.asarray(t, dtype=np.float64)  # noqa: E731
    z = (f(x_q) @ f(W_q).T) * f(x_scale)[:, None] * f(w_scale)[None, :]
    if A is not None:
        z = z + s * ((f(x) @ f(A).T) @ f(B).T)
    if m is not None:
        z = z * (f(m) / f(n))[None, :]
    return z if bias is None else z + f(bias)[None, :]


def compose_backward_kept(dy, z, m, n, s):
    """(d_base, d_lora, d_m) from the kept z (the bias already out of it), n constant."""
    dy, z, m, n = (np.asarray(t, dtype=np.float64) for t in (dy, z, m, n))
    g = m / n
    return g * dy, s * g * dy, np.sum(dy * z, axis=0) / n
