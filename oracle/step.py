"""Oracle of the operators between the products of a decoding step: cache append with rotation,
attention over the paged cache, sampling.

Plain numpy in float64, one row at a time.  The pages name a verification attention over a split cache
(summary page) and a best-first tree of drafts, but no details; the conventions are this build's own:
  * a place outside the table, or on a page outside the cache, does not exist: nothing is appended there
    and nobody sees it;
  * a row that sees nothing gives zeros; what a row does not see never reaches it;
  * equal logits (-0 equals +0) go by the lower column; a row of -Inf alone gives token -1, log
    probability -Inf and 0 kept; one with a NaN or +Inf logit, or a NaN temperature, token -1, NaN and 0.
"""
from __future__ import annotations

import numpy as np


def new_tokens(lens, q_start, rows):
    """[(row, sequence, j, T, length)] of the rows that belong to a sequence."""
    out = []
    for s, n in enumerate(lens):
        a, b = (s, s + 1) if q_start is None else (int(q_start[s]), int(q_start[s + 1]))
        out += [(a + j, s, j, b - a, int(n)) for j in range(b - a) if a + j < rows]
    return out


def page_of(table, s, c, page, pages):
    """The page of place c of sequence s, or None."""
    if c < 0 or c // page >= table.shape[1]:
        return None
    p = int(table[s, c // page])
    return p if 0 <= p < pages else None


def rotate64(x, cos, sin, pairs):
    """x [..., dim] with its first 2 len(cos) columns rotated."""
    h = len(cos)
    a = np.arange(0, 2 * h, 2) if pairs else np.arange(h)
    b = a + 1 if pairs else a + h
    r = np.array(x, dtype=np.float64)
    r[..., a] = x[..., a] * cos - x[..., b] * sin
    r[..., b] = x[..., b] * cos + x[..., a] * sin
    return r


def append64(q, k, v, rope, pairs, table, lens, q_start, positions, page, pages):
    """(q rotated [m, hq, dim] with NaN in rows that stay, and {(page, place): (k, v)} as [heads, dim]).
    q, k, v: float64 [m, heads, dim] (q may be None)."""
    m = k.shape[0]
    out = None if q is None else np.full(q.shape, np.nan)
    put = {}
    for i, s, j, t, n in new_tokens(lens, q_start, m):
        c = n - t + j
        kk = k[i]
        pos = c if positions is None else int(positions[i])
        if rope is not None:
            if not 0 <= pos < rope.shape[0]:
                if out is not None:
                    out[i] = 0.0
                continue
            h = rope.shape[1] // 2
            cos, sin = rope[pos, :h].astype(np.float64), rope[pos, h:].astype(np.float64)
            kk = rotate64(kk, cos, sin, pairs)
            if out is not None:
                out[i] = rotate64(q[i], cos, sin, pairs)
        elif out is not None:
            out[i] = q[i]
        p = page_of(table, s, c, page, pages)
        if p is not None:
            put[p, c % page] = (kk, v[i])
    return out, put


def attention64(q, k, v, table, lens, q_start, tree, scale):
    """(y, sum p |v|, largest sum |q k| scale) with q [m, hq, dim], k and v [pages, heads, page, dim]
    float64; rows of no sequence are NaN."""
    m, hq, dim = q.shape
    pages, heads, page, _ = k.shape
    g = hq // heads
    y, mag, big = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros((m, hq))
    for i, s, j, t, n in new_tokens(lens, q_start, m):
        y[i] = 0.0
        base = n - t
        at = []
        for c in range(max(n, 0)):
            b = c - base
            if b >= 0 and not (b <= j if tree is None else b < 64 and int(tree[i]) >> b & 1):
                continue
            p = page_of(table, s, c, page, pages)
            if p is not None:
                at.append((p, c % page))
        if not at:
            continue
        pg, off = (np.array(z) for z in zip(*at))
        for h in range(hq):
            kk, vv = k[pg, h // g, off], v[pg, h // g, off]
            x = (kk @ q[i, h]) * scale
            big[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
            if np.isneginf(x).all():
                continue
            e = np.exp(x - x.max())
            p = e / e.sum()
            y[i, h] = p @ vv
            mag[i, h] = p @ np.abs(vv)
    return y, mag, big


def sample64(y, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(token, logp, kept) per row of y [m, n]."""
    y = np.asarray(y, dtype=np.float64) + 0.0
    m, n = y.shape
    tok, logp, kept = np.full(m, -1, np.int32), np.full(m, -np.inf), np.zeros(m, np.int32)
    for r in range(m):
        x = y[r]
        temp = 1.0 if temperature is None else float(temperature[r])
        if np.isnan(x).any() or np.isposinf(x).any() or np.isnan(temp):
            logp[r] = np.nan
            continue
        if np.isneginf(x).all():
            continue
        order = np.lexsort((np.arange(n), -x))
        order = order[x[order] > -np.inf]
        if temp <= 0:
            tok[r], logp[r], kept[r] = order[0], 0.0, 1
            continue
        d = np.where(x == x.max(), 0.0, (x - x.max()) / temp)
        w = np.exp(d)
        if top_k is not None and top_k[r] > 0:
            order = order[:top_k[r]]
        p = 1.0 if top_p is None else float(top_p[r])
        if p < 1.0:
            cum = np.cumsum(w[order])
            before = np.concatenate([[0.0], cum[:-1]])
            order = order[:max(1, int((before < p * cum[-1]).sum()))]
        mp = 0.0 if min_p is None else float(min_p[r])
        if mp > 0.0:
            order = order[:max(1, int((w[order] >= mp).sum()))]
        cols = np.sort(order)
        cum = np.cumsum(w[cols])
        want = float(u[r]) if u[r] > 0 else 0.0
        live = np.nonzero(w[cols] > 0)[0]
        at = live[-1] if want >= 1 else min(int((cum <= want * cum[-1]).sum()), live[-1])
        tok[r], kept[r] = cols[at], len(cols)
        logp[r] = d[cols[at]] - np.log(cum[-1])
    return tok, logp, kept
