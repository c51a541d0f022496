"""CPU oracle of a serving step's calls: pages and rows from lengths (dartree_paged_reserve,
dartree_paged_release), draws under temperature, top-k, top-p and min-p (dartree_sample) and the walk
of a tree on them (dartree_verify_filtered). Integers and float64, from the definitions.

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import numpy as np


def reserve(table, n_ctx, n_new, stack, page, S, T, fixed):
    """table [C, max_pages], stack: the free pages (last one first) -> dict(table, granted, q_start, slot, pos,
    request, n_free). fixed: S rows of q to a request; else rows follow one another, T in all. A request that
    does not fit gets nothing."""
    table, stack = np.array(table), list(stack)
    C = len(n_ctx)
    granted, q = [], [0]
    slot, pos, req = (np.full(T, -1, np.int64) for _ in range(3))
    for c in range(C):
        o, m = int(n_ctx[c]), int(n_new[c])
        have, want = -(-o // page), -(-(o + m) // page)
        fits = want <= table.shape[1] and want - have <= len(stack) and (fixed or q[-1] + m <= T)
        granted.append(m if fits else 0)
        if fits:
            for i in range(have, want):
                table[c, i] = stack.pop()
            for i in range(m):
                r = (c * S if fixed else q[-1]) + i
                slot[r] = int(table[c, (o + i) // page]) * page + (o + i) % page
                pos[r], req[r] = o + i, c
        q.append(q[-1] + granted[-1])
    return dict(table=table, granted=np.array(granted), q_start=np.array(q), slot=slot, pos=pos, request=req,
                n_free=len(stack))


def release(table, n_held, n_keep, n_shared, stack, page):
    """The stack once the pages behind the kept and the shared rows are on it."""
    stack = list(stack)
    for c in range(len(n_held)):
        first = -(-max(int(n_keep[c]), int(n_shared[c])) // page)
        for i in range(first, -(-int(n_held[c]) // page)):
            stack.append(int(table[c, i]))
    return stack


def kept(x, temperature, top_k, top_p, min_p):
    """(tokens kept, ascending, their weights) of one row of logits."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max()
    if m == -np.inf:
        return np.zeros(0, np.int64), np.zeros(0)
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == m, 1.0, np.exp((x - m) / temperature) if temperature > 0 else 0.0)
    if m == np.inf:
        w = (x == m).astype(np.float64)
    order = np.flatnonzero(x > -np.inf)
    order = order[np.argsort(-x[order], kind="stable")]
    if temperature == 0:
        order = order[:1]
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        run = np.cumsum(w[order])
        order = order[(np.arange(len(order)) == 0) | (run - w[order] < top_p * run[-1])]
    order = np.sort(order[(w[order] >= min_p) | (order == order[0])])
    return order, w[order]


def draw(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, how near the decision was: the least distance of u from a border, -1 for an empty row)."""
    tok, w = kept(x, temperature, top_k, top_p, min_p)
    if not len(tok):
        return -1, 1.0
    c = np.cumsum(w) / w.sum()
    i = min(int(np.searchsorted(c, u, side="right")), len(tok) - 1)
    return int(tok[i]), float(np.min(np.abs(c[:-1] - u))) if len(tok) > 1 else 1.0


def verify(tree, target, rows, L, u, settings):
    """The walk of each request's tree on draws: settings(c) gives a request's keywords of draw()."""
    C = len(tree["n_nodes"])
    acc, path, bonus = np.zeros(C, np.int64), np.full((C, L), -1, np.int64), np.full(C, -1, np.int64)
    for c in range(C):
        cur = 0
        while True:
            r = cur if rows == "node" else int(tree["depth"][c, cur])
            if r >= target.shape[1]:
                break
            t, _ = draw(target[c, r], float(u[c, r]), **settings(c))
            kid = [j for j in range(1, int(tree["n_nodes"][c])) if tree["par"][c, j] == cur and tree["tok"][c, j] == t]
            if not kid:
                bonus[c] = t
                break
            cur = kid[0]
            path[c, acc[c]] = cur
            acc[c] += 1
    return dict(accepted_len=acc, path=path, bonus=bonus)
