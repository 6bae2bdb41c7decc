"""int8 codes with a scale per row and their products in plain numpy.

The formulas are those of include/gptq.h (gptq_int8_quantize, gptq_int8_matmul,
gptq_int8_matmul_grouped), one row at a time; sums are 64-bit whole numbers.
"""
from __future__ import annotations

import numpy as np

FLOOR = 2.0 ** -100


def quantize(X):
    """(codes int8 [m x k], scales fp32 [m])."""
    X = np.asarray(X).astype(np.float64)
    m, k = X.shape
    codes, scales = np.zeros((m, k), np.int8), np.full(m, np.nan, np.float32)
    for i in range(m):
        if not np.isfinite(X[i]).all():
            continue
        a = max(np.max(np.abs(X[i])), FLOOR)
        r = np.float64(np.float32(1.0 / a))                   # fp32 quotients and products: the
        inv = np.float64(np.float32(127.0 * r))               # 64-bit ones, rounded
        t = np.float32(X[i] * inv)
        codes[i] = np.rint(t.astype(np.float64))
        scales[i] = a / 127.0
    return codes, scales


def matmul(x_codes, x_scales, w_codes, w_scales, bias=None):
    """(Y in fp64, sum of the magnitudes of its two terms)."""
    acc = np.asarray(x_codes, np.float64) @ np.asarray(w_codes, np.float64).T        # below 2^53: exact
    y = acc * (np.asarray(x_scales, np.float64)[:, None] * np.asarray(w_scales, np.float64))
    mag = np.abs(y)
    if bias is not None:
        b = np.asarray(bias, np.float64)
        y, mag = y + b, mag + np.abs(b)
    return y, mag


def grouped(x_codes, x_scales, w_codes, w_scales, offsets, rows=None, bias=None):
    """(Y, magnitudes, mask of the rows that belong to an expert)."""
    m = len(x_codes) if rows is None else len(rows)
    n = np.shape(w_codes)[1]
    y, mag, has = np.zeros((m, n)), np.zeros((m, n)), np.zeros(m, bool)
    for e in range(len(w_codes)):
        for i in range(int(offsets[e]), int(offsets[e + 1])):
            r = i if rows is None else int(rows[i])
            has[i] = True
            if not 0 <= r < len(x_codes):
                y[i] = np.nan
                continue
            a, b = matmul(x_codes[r:r + 1], x_scales[r:r + 1], w_codes[e], w_scales[e], None if bias is None else bias[e])
            y[i], mag[i] = a[0], b[0]
    return y, mag, has
