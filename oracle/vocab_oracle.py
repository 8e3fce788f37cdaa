"""Vocabulary operators from their definitions, in 64 bits (numpy).

Inputs are arrays of any float type, taken to float64 first; nothing is
rounded.  Ignored ids are those outside [0, vocab).
"""
from __future__ import annotations

import numpy as np

NEG = -np.inf


def embedding_forward(table, ids, scale):
    t = np.asarray(table, np.float64)
    out = np.zeros((len(ids), t.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < t.shape[0]:
            out[i] = t[v] * scale
    return out


def embedding_backward(dout, ids, scale, vocab, base=None):
    """The table's gradient, and per row the sum of absolute contributions
    and their number (for error bounds)."""
    d = np.asarray(dout, np.float64)
    g = np.zeros((vocab, d.shape[1]))
    mag = np.zeros_like(g)
    count = np.zeros(vocab, np.int64)
    for i, v in enumerate(ids):
        if 0 <= v < vocab:
            g[v] += d[i] * scale
            mag[v] += np.abs(d[i] * scale)
            count[v] += 1
    if base is not None:
        g = g + np.asarray(base, np.float64)
    return g, mag, count


def scaled(x, scale):
    """x * scale; what overflows binary32 is infinite."""
    z = np.asarray(x, np.float64) * scale
    return np.where(np.abs(z) >= 2.0 ** 128 - 2.0 ** 103, np.copysign(np.inf, z), z)


def _log_softmax(z):
    """(log softmax, lse); rows of -inf alone give -inf everywhere.  The
    maximum is taken off before the logarithm of the sum: at 1e38 the sum of
    the two would lose it."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = z.max(axis=-1, keepdims=True)
        m = np.where(m == NEG, 0.0, m)
        logs = np.log(np.exp(z - m).sum(axis=-1, keepdims=True))
        logp = np.where(logs == NEG, NEG, z - m - logs)
    return logp, (m + logs)[..., 0]


def token_logprobs(logits, targets, scale, k=0):
    x = np.asarray(logits, np.float64)
    logp, lse = _log_softmax(scaled(x, scale))
    n, V = x.shape
    lp = np.array([logp[i, t] if 0 <= t < V else 0.0 for i, t in enumerate(targets)])
    with np.errstate(invalid="ignore"):
        p = np.exp(logp)
        ent = -np.where(p == 0, 0.0, p * np.where(p == 0, 0.0, logp)).sum(axis=1)
    top = np.zeros((n, k), np.int64)
    for i in range(n):
        top[i] = np.argsort(-x[i], kind="stable")[:k]  # ties to the lowest index
    return dict(logprob=lp, lse=lse, entropy=ent, top_ids=top,
                top_logprobs=np.take_along_axis(logp, top, 1))


def token_logprobs_backward(logits, targets, scale, dlogprob=None, dentropy=None):
    x = np.asarray(logits, np.float64)
    n, V = x.shape
    out = token_logprobs(x, targets, scale)
    logp, lse = _log_softmax(scaled(x, scale))
    p = np.exp(logp)
    dx = np.zeros_like(x)
    for i, t in enumerate(targets):
        if lse[i] == NEG:
            continue
        on = p[i] > 0
        if dlogprob is not None and 0 <= t < V:
            dx[i] -= dlogprob[i] * p[i]
            dx[i, t] += dlogprob[i]
        if dentropy is not None:
            dx[i, on] -= dentropy[i] * p[i, on] * (logp[i, on] + out["entropy"][i])
    return dx * scale


def teacher_probabilities(teacher, teacher_ids, scale, vocab):
    """[n, k] probabilities; 0 for entries that do not count."""
    t = scaled(teacher, scale)
    ids = np.asarray(teacher_ids)
    t = np.where((ids >= 0) & (ids < vocab), t, NEG)
    logq, lse = _log_softmax(t)
    return np.exp(logq), logq, lse > NEG


def distill(logits, teacher, teacher_ids, scale, weight=None):
    """(loss [n], gradient of sum weight * loss [n, vocab], lse [n], and per
    row the sum of the loss terms' magnitudes)."""
    x = np.asarray(logits, np.float64)
    n, V = x.shape
    logp, lse = _log_softmax(scaled(x, scale))
    q, logq, some = teacher_probabilities(teacher, teacher_ids, scale, V)
    w = np.ones(n) if weight is None else np.asarray(weight, np.float64)
    loss, mag, dx = np.zeros(n), np.zeros(n), np.zeros_like(x)
    for i in range(n):
        if not some[i] or lse[i] == NEG:
            continue
        dx[i] = np.exp(logp[i])
        for k in range(q.shape[1]):
            if q[i, k] > 0:
                j = teacher_ids[i][k]
                loss[i] += q[i, k] * (logq[i, k] - logp[i, j])
                mag[i] += q[i, k] * (abs(logq[i, k]) + abs(logp[i, j]))
                dx[i, j] -= q[i, k]
    return loss / scale ** 2, dx * (w / scale)[:, None], lse, mag / scale ** 2
