"""CPU oracle of the paged-cache calls (dartree_paged_*): append, attention, accumulated
weights, eviction, commit. Float64, from the definitions; a cache is a plain array of
rows per request and head, read through the block table.

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import numpy as np

from .tree_attention import ROPE_THETA, rope


def place(table, c, j, page):
    """(page id, row in it) of cached rows j of request c."""
    j = np.asarray(j, np.int64)
    return np.asarray(table)[c, j // page], j % page


def rows_of(pages, table, c, n):
    """The first n cached rows of request c, [Hkv, n, D] (float64)."""
    p, r = place(table, c, np.arange(n), pages.shape[2])
    return np.moveaxis(np.asarray(pages[p, :, r], np.float64), 0, 1)


def head_norm(x, gain, eps):
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)


def append(x, gain, positions, eps=1e-6, theta=ROPE_THETA):
    """Normed (gain may be None) and rotated heads of x [n, heads, D] at positions [n]."""
    y = np.asarray(x, np.float64) if gain is None else head_norm(x, gain, eps)
    return np.moveaxis(rope(np.moveaxis(y, 0, 1), positions, theta), 0, 1)


def sees(n_old, n_new, mask=None):
    """[n_new, n_old + n_new]: which rows each new token sees (mask [n_new, n_new], None: causal)."""
    new = np.tril(np.ones((n_new, n_new), bool)) if mask is None else np.asarray(mask)[:n_new, :n_new] != 0
    return np.concatenate([np.ones((n_new, n_old), bool), new], axis=1)


def attention(q, k, v, seen, scale):
    """q [n, Hq, D], k and v [Hkv, m, D], seen [n, m] -> (out [n, Hq, D], lse [n, Hq], mean |v| under the
    same weights [n, Hq, D], largest scale * sum |q_d k_d| of each row [n, Hq])."""
    n, Hq, D = q.shape
    grp = Hq // k.shape[0]
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    mag, most = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    q = np.asarray(q, np.float64)
    for h in range(Hq):
        g = h // grp
        for i in range(n):
            j = np.flatnonzero(seen[i])
            if not len(j):
                continue
            s = k[g, j] @ q[i, h] * scale
            w = np.exp(s - s.max())
            lse[i, h] = s.max() + np.log(w.sum())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ v[g, j], w @ np.abs(v[g, j])
            most[i, h] = (np.abs(k[g, j]) @ np.abs(q[i, h])).max() * scale
    return out, lse, mag, most


def weights(q, k, seen, lse, scale, before, n_old, decay):
    """Weights [Hkv, m] of the cached rows after the step; before [Hkv, >= n_old]."""
    Hkv, m, _ = k.shape
    n, Hq, _ = q.shape
    w = np.zeros((Hkv, m))
    w[:, :n_old] = decay * np.asarray(before, np.float64)[:, :n_old]
    for h in range(Hq):
        g = h // (Hq // Hkv)
        for i in range(n):
            j = np.flatnonzero(seen[i])
            w[g, j] += np.exp(k[g, j] @ np.asarray(q[i, h], np.float64) * scale - lse[i, h])
    return w


def kept_rows(w, n, budget, sink, recent):
    """Rows of one head kept of n, ascending: the first `sink`, the last `recent`, and the largest of w
    (NaN lowest, ties to the lowest row) up to `budget`."""
    if n <= budget:
        return list(range(n))
    mid = list(range(sink, n - recent))
    key = {j: -np.inf if np.isnan(w[j]) else float(w[j]) for j in mid}
    # NaN counts below every number, -inf included
    mid.sort(key=lambda j: (np.isnan(w[j]), -key[j], j))
    return sorted(list(range(sink)) + mid[:budget - sink - recent] + list(range(n - recent, n)))


def commit_moves(path, accepted, n_ctx):
    """(source rows, destination rows, rows cached afterwards) of one request."""
    src = [n_ctx + int(s) for s in path[:accepted]]
    return src, [n_ctx + 1 + i for i in range(accepted)], n_ctx + 1 + accepted
