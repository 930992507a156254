"""Oracle of the operators at the vocabulary end of a step: embedding lookup and log probabilities.

Plain numpy in float64, one row at a time.  The pages name neither operator's details (the draft
tree's score is the sum of log probabilities along a path: summary page, best-first tree); the
conventions for masked rows, ties and NaN are this build's own:
  * equal logits (-0 equals +0) go by the lower column, NaN sorts above every number;
  * a -Inf logit has probability 0; a row of -Inf alone gives log probabilities -Inf, entropy 0;
  * a row with a NaN or +Inf logit gives NaN; a token outside the columns gives -Inf always.
"""
from __future__ import annotations

import numpy as np


def embed_bits(w_bits, ids) -> np.ndarray:
    """Rows ids of W (bfloat16 bits); zeros for an id outside 0 .. n-1."""
    w = np.asarray(w_bits, dtype=np.uint16)
    out = np.zeros((len(ids), w.shape[1]), dtype=np.uint16)
    for j, t in enumerate(ids):
        if 0 <= t < w.shape[0]:
            out[j] = w[t]
    return out


def logprobs64(y, tokens, top):
    """(logp [m, t], entropy [m], top_index [m, top], top_logp [m, top]) of float64 logits y [m, n]."""
    y = np.asarray(y, dtype=np.float64) + 0.0
    m, n = y.shape
    tokens = np.asarray(tokens, dtype=np.int64).reshape(m, -1)
    logp = np.full(tokens.shape, -np.inf)
    ent = np.zeros(m)
    idx = np.zeros((m, top), dtype=np.int32)
    tlp = np.full((m, top), -np.inf)
    for r in range(m):
        x = y[r]
        # descending by value, ascending by column; NaN first
        order = np.lexsort((np.arange(n), -np.where(np.isnan(x), 0.0, x), ~np.isnan(x)))[:top]
        idx[r] = order
        valid = (tokens[r] >= 0) & (tokens[r] < n)
        if np.isnan(x).any() or np.isposinf(x).any():
            logp[r, valid] = np.nan
            ent[r] = np.nan
            tlp[r] = np.nan
            continue
        if np.isneginf(x).all():
            continue
        big = x.max()
        p = np.exp(x - big)
        z = np.log1p(p.sum() - 1.0) if p.sum() > 1.5 else np.log1p(np.delete(p, np.argmax(x)).sum())
        lp = x - big - z
        logp[r, valid] = lp[tokens[r][valid]]
        live = p > 0
        ent[r] = -(np.exp(lp[live]) * lp[live]).sum()
        tlp[r] = lp[order]
    return logp, ent, idx, tlp


def logprobs_tol(y):
    """Error bounds of a float32 evaluation, per row of y: (absolute error of log1p(s) from the error
    of s, the sum of the exponentials without one maximum; absolute error of the entropy).

    With u = 2^-24: an exponential carries its argument's roundings (the difference, and the
    product with log2 e rounded in both factors: 3 u |d|) and its own (4 u); a sum of c terms added
    in any order carries at most c u, where a lane adds n / 64 terms at most before the 64 lanes and
    the parts (80 more).  So s is off by at most u sum e^d (c + 4 + 4 |d|), and log1p(s) by that
    over 1 + s.  The entropy's other half sum p |d| is off by u sum p |d| (c + 5 + 4 |d|) and by its
    denominator's error; the logarithm, the quotient and the sum round once or twice each."""
    y = np.asarray(y, dtype=np.float64)
    m, n = y.shape
    u = 2.0 ** -24
    ls, ent = np.zeros(m), np.zeros(m)
    adds = n / 64 + 80
    for r in range(m):
        x = y[r][np.isfinite(y[r])]
        if x.size == 0:
            continue
        d = np.maximum(x - x.max(), -1000.0)
        e = np.exp(d)
        one = e.sum()
        s = np.delete(e, np.argmax(d)).sum()
        md, md2 = -(e * d).sum() / one, (e * d * d).sum() / one
        ls[r] = u * ((adds + 4) * s / one + 4 * md)
        ent[r] = ls[r] * (1 + md) + u * ((adds + 5) * md + 4 * md2 + 4 * md + 4 * np.log1p(s))
    return ls, ent
