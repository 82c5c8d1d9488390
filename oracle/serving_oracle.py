"""Float64 NumPy definitions of the operators around a decode step -- verification of drafted tokens,
the attention weight that cached keys receive, eviction -- written apart from the GPU code.  Slow and plain.
"""
from __future__ import annotations

import math

import numpy as np


def verify(target, draft, tokens, draft_len, u_accept, u_sample):
    """One sequence: target [n + 1, V], draft [n, V] or None, tokens [n], u_accept [n] -> (tokens [n + 1] with
    -1 behind the drawn one, drafts taken).  A token outside the vocabulary is not taken."""
    n, V = target.shape[0] - 1, target.shape[1]
    out = np.full(n + 1, -1, dtype=np.int32)
    p = np.asarray(target, dtype=np.float64)
    q = None if draft is None else np.asarray(draft, dtype=np.float64)
    length = n if draft_len is None else min(max(int(draft_len), 0), n)
    a = 0
    while a < length:
        x = int(tokens[a])
        if not 0 <= x < V:
            break
        if not float(u_accept[a]) * (1.0 if q is None else q[a, x]) < p[a, x]:
            break
        out[a] = x
        a += 1
    r = np.where(p[a] > 0.0, p[a], 0.0)
    if a < length:
        if q is not None:
            with np.errstate(invalid="ignore"):
                diff = p[a] - q[a]
            r = np.where(diff > 0.0, diff, 0.0)
        elif 0 <= int(tokens[a]) < V:
            r = r.copy()
            r[int(tokens[a])] = 0.0
        if not np.any(r > 0.0):
            r = np.where(p[a] > 0.0, p[a], 0.0)
    total = math.fsum(r) if np.all(np.isfinite(r)) else math.inf
    if total > 0.0 and total < math.inf:
        u = float(u_sample)
        at = u * total if u > 0.0 else 0.0
        over = np.nonzero((np.cumsum(r) > at) & (r > 0.0))[0]
        out[a] = over[0] if over.size else np.nonzero(r > 0.0)[0][-1]
    return out, a


def key_weights(q, kv, lse, tau):
    """One row: q [H, 576], kv [L, 576], lse [H] -> (sum over heads of exp(tau q . kv_j - lse) [L], a bound of
    |tau q . kv_j|'s terms per head and key [H, L])."""
    s = tau * (q @ kv.T)
    with np.errstate(invalid="ignore"):
        w = np.exp(s - lse[:, None])
    w[np.isneginf(lse)] = 0.0
    return w.sum(axis=0), w, tau * (np.abs(q) @ np.abs(kv).T)


def evict(weight, length, n_keep, n_first, n_last):
    """Positions that stay, ascending: everything of a sequence of at most n_keep keys, else the first n_first,
    the last n_last and the heaviest of the others (ties: the lower position; NaN weighs least)."""
    if length <= n_keep:
        return np.arange(length)
    a, b = n_first, length - n_last
    w = np.asarray(weight[a:b], dtype=np.float64)
    order = sorted(range(b - a), key=lambda i: (math.isnan(w[i]), 0.0 if math.isnan(w[i]) else -w[i], i))
    middle = sorted(order[:n_keep - n_first - n_last])
    return np.concatenate([np.arange(a), np.asarray(middle, dtype=np.int64) + a, np.arange(b, length)]).astype(np.int64)
