"""e4m3 block codes, their product and token log probabilities in plain fp64 numpy.

The formulas are those of include/gptq.h (gptq_fp8_quantize, gptq_fp8_matmul,
gptq_token_logprobs), written for reading, one block or row at a time.
"""
from __future__ import annotations

import numpy as np

BLK = 128
E4M3_NAN = 0x7F


def e4m3_value(codes):
    """The number an e4m3 bit pattern stands for (NaN for 0x7F and 0xFF)."""
    table = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        mag = (8 + f) * 2.0 ** (e - 10) if e else f * 2.0 ** -9
        if (b & 0x7F) == 0x7F:
            mag = np.nan
        table[b] = -mag if b > 127 else mag
    return table[np.asarray(codes, dtype=np.uint8)]


_MAGS = e4m3_value(np.arange(127))                       # 0 .. 448, ascending


def e4m3_code(u):
    """Nearest e4m3 pattern of |u| <= 448 (half to even code), 0x7F where u is not finite."""
    u = np.asarray(u, dtype=np.float64)
    a = np.where(np.isfinite(u), np.abs(u), 0.0)
    lo = np.clip(np.searchsorted(_MAGS, a, side="right") - 1, 0, 125)
    mid = (_MAGS[lo] + _MAGS[lo + 1]) / 2
    code = lo + ((a > mid) | ((a == mid) & (lo % 2 == 1)))
    code = np.where(np.signbit(u), code + 128, code)
    return np.where(np.isfinite(u), code, E4M3_NAN).astype(np.uint8)


def block_scale(x) -> float:
    """2^e, e the smallest integer >= -126 with max|finite x| <= 448 2^e; 1 without a maximum."""
    x = np.asarray(x, dtype=np.float64)
    a = np.max(np.abs(x[np.isfinite(x)]), initial=0.0)
    if a == 0.0:
        return 1.0
    e = -126
    while a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def quantize(X, block_rows):
    """(codes uint8 [m x k], scales in the layout of gptq_fp8_quantize)."""
    X = np.asarray(X).astype(np.float64)
    m, k = X.shape
    mb, kb = -(-m // block_rows), -(-k // BLK)
    codes, scales = np.empty((m, k), np.uint8), np.empty((mb, kb), np.float32)
    for i in range(mb):
        for b in range(kb):
            at = np.s_[i * block_rows:(i + 1) * block_rows, b * BLK:(b + 1) * BLK]
            s = block_scale(X[at])
            codes[at] = e4m3_code(X[at] / s)
            scales[i, b] = s
    return codes, (np.ascontiguousarray(scales.T) if block_rows == 1 else scales)


def dequantize(codes, scales, block_rows):
    codes = np.asarray(codes, dtype=np.uint8)
    m, k = codes.shape
    s = np.asarray(scales, dtype=np.float64)
    s = s.T if block_rows == 1 else s
    return e4m3_value(codes) * s[np.arange(m) // block_rows][:, np.arange(k) // BLK]


def matmul(x_codes, x_scales, w_codes, w_scales, bias=None):
    """(Y in fp64, sum of the magnitudes that Y is the sum of)."""
    x, w = dequantize(x_codes, x_scales, 1), dequantize(w_codes, w_scales, 128)
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        y, mag = y + b, mag + np.abs(b)
    return y, mag


def token_logprobs(logits, tokens, top_k):
    """(logprobs, entropy, top_ids, top_logprobs) of the rows of logits."""
    logits = np.asarray(logits).astype(np.float64)
    n, v = logits.shape
    lp, ent = np.empty(n), np.empty(n)
    ids, tops = np.empty((n, top_k), np.int64), np.empty((n, top_k))
    for r in range(n):
        x = logits[r]
        order = sorted(range(v), key=lambda i: (0 if np.isnan(x[i]) else 1, -x[i] if not np.isnan(x[i]) else 0.0, i))
        ids[r] = order[:top_k]
        M = np.max(x) if not np.isnan(x).any() else np.nan
        if np.isfinite(M):
            d = x - M
            p = np.exp(d)
            S = np.sum(p)
            logp = d - np.log(S)
            ent[r] = np.log(S) - np.sum(p[p > 0] * d[p > 0]) / S
        else:
            logp = np.full(v, np.nan)
            ent[r] = np.nan
        tops[r] = logp[ids[r]]
        t = int(tokens[r])
        lp[r] = 0.0 if t < 0 else np.nan if t >= v else logp[t]
    return lp, ent, ids, tops
