"""The divergence from a teacher's top tokens and its gradient in plain fp64 numpy, one row
at a time (gptq_distill_loss of include/gptq.h)."""
from __future__ import annotations

import math

import numpy as np


def teacher(ids, logprobs, v, temperature, tail):
    """(q over all v tokens without the rest's, q_r) of a row."""
    q = np.zeros(v)
    j = [i for i in range(len(ids)) if ids[i] >= 0]
    t = np.array([float(logprobs[i]) for i in j])
    rest = 0.0
    if tail:
        e = np.exp(t)
        rest = max(0.0, 1.0 - math.fsum(e))
    else:
        e = np.exp((t - np.max(t)) / temperature)
        e = e / math.fsum(e)
    for i, w in zip(j, e):
        q[ids[i]] += w
    return q, rest


def row(z, ids, logprobs, temperature=1.0, tail=False, weight=1.0):
    """(loss, gradient [v], spread): spread is the mean of |z - max| / temperature under p and
    under p given the tokens that are not listed, which bounds what rounding can do."""
    z, ids = np.asarray(z, np.float64), [int(i) for i in ids]
    v = len(z)
    if any(i >= v for i in ids):
        return math.nan, np.full(v, math.nan if weight else 0.0), (0.0, 0.0)
    if all(i < 0 for i in ids):
        return 0.0, np.zeros(v), (0.0, 0.0)
    with np.errstate(all="ignore"):
        q, rest = teacher(ids, logprobs, v, temperature, tail)
        M = np.max(z)
        if not np.isfinite(M) or np.isnan(z).any() or not np.isfinite(q).all():
            return math.nan, np.full(v, math.nan if weight else 0.0), (0.0, 0.0)
        d = (z - M) / temperature
        e = np.exp(d)
        p = e / math.fsum(e)
        log_p = d - math.log(math.fsum(e))
        listed = np.zeros(v, bool)
        listed[[i for i in ids if i >= 0]] = True
        # every entry has its own term: a token listed twice is no token of the summed q
        loss = 0.0
        t = {}
        for i, j in enumerate(ids):
            if j >= 0:
                t.setdefault(j, []).append(float(logprobs[i]))
        flat = [x for xs in t.values() for x in xs]
        for j, xs in t.items():
            for x in xs:
                if tail:
                    lq = x
                else:
                    top = max(flat)
                    lq = (x - top) / temperature - math.log(math.fsum(math.exp((y - top) / temperature) for y in flat))
                if math.exp(lq) > 0.0:
                    loss += math.exp(lq) * (lq - log_p[j])
        grad = p * (q.sum() + rest) - q
        dr = d[~listed]
        er = np.exp(dr - np.max(dr)) if dr.size else dr
        share = er / math.fsum(er) if dr.size else er
        if rest > 0.0:
            Sr = math.fsum(np.exp(dr))
            top = np.max(dr)
            log_pr = top + math.log(math.fsum(er)) - math.log(math.fsum(e)) if np.isfinite(top) else -math.inf
            loss += rest * (math.log(rest) - log_pr)
            grad[~listed] -= rest * share
        spread = (float(np.sum(np.where(p > 0, p * -np.where(p > 0, d, 0.0), 0.0))),
                  float(np.sum(np.where(share > 0, share * (np.max(dr) - np.where(share > 0, dr, 0.0)), 0.0))) if dr.size else 0.0)
        return loss, (grad * (weight / temperature) if weight else np.zeros(v)), spread
