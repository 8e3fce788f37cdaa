"""Verification of drafted tokens in 64 bits, one sequence after another, from the
definition (numpy)."""
from __future__ import annotations

import numpy as np


LEAST = 2.0 ** -126  # of the row's largest probability: below this tokens are not drawn


def _row(z):
    """Log probabilities of one row of logits; -inf everywhere in a row without any
    token, NaN where a NaN or +inf spoils it."""
    z = np.asarray(z, np.float64)
    if np.isnan(z).any() or np.isposinf(z).any():
        return np.full(z.shape, np.nan)
    if np.isneginf(z).all():
        return z.copy()
    m = z.max()
    return z - m - np.log(np.exp(z - m).sum())


def _draw(residual, noise):
    """The token with the largest residual / noise among those with a positive one
    and a noise of 0 or more (0 wins, -0 is less); the lowest index of equal ones; or -1."""
    ok = (residual > 0) & (noise >= 0) & ~np.signbit(noise) & (noise < np.inf)
    if not ok.any():
        return -1
    with np.errstate(divide="ignore", invalid="ignore"):
        score = np.where(ok, residual / noise, -1.0)
    return int(np.argmax(score))


def verify(logits, draft_logits, ids, uniform, noise, scale=1.0, draft_scale=1.0):
    """logits [n, k + 1, V], draft_logits [n, k, V] or None, ids and uniform [n, k],
    noise [n, V] -> accepted [n], tokens [n, k + 1], logprobs [n, k + 1]."""
    n, k1, V = logits.shape
    k = k1 - 1
    accepted = np.zeros(n, np.int32)
    tokens = np.full((n, k1), -1, np.int32)
    lps = np.zeros((n, k1))
    for s in range(n):
        j, refused, q = 0, False, None
        lp = _row(np.asarray(logits[s, 0], np.float64) * scale)
        broken = False
        while True:
            if np.isnan(lp).any():
                broken = True
                break
            d = int(ids[s, j]) if j < k else -1
            if not 0 <= d < V:
                break
            if draft_logits is None:
                q = np.where(np.arange(V) == d, 0.0, -np.inf)
            else:
                q = _row(np.asarray(draft_logits[s, j], np.float64) * draft_scale)
                if np.isnan(q).any():
                    broken = True
                    break
            with np.errstate(divide="ignore"):
                lu = np.log(np.float64(uniform[s, j]))
            if not lu + q[d] < lp[d]:
                refused = True
                break
            tokens[s, j], lps[s, j] = d, lp[d]
            j += 1
            lp = _row(np.asarray(logits[s, j], np.float64) * scale)
        accepted[s] = j
        if broken:
            lps[s, j] = np.nan
            continue
        p = np.exp(lp)
        p[p < p.max() * LEAST] = 0  # too unlikely to be drawn
        e = np.asarray(noise[s], np.float64)
        t = _draw(p - np.exp(q), e) if refused else -1
        if t < 0:
            t = _draw(p, e)
        tokens[s, j] = t
        lps[s, j] = lp[t] if t >= 0 else -np.inf
    return accepted, tokens, lps
