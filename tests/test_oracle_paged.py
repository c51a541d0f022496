"""Pins of the oracle's paged-cache calls against facts that do not come from it: a chain
tree equals causal attention, one page equals a plain cache, weights of a softmax sum to
one per row, closed-form norms, and hand-made evictions and commits."""
import math

import numpy as np
import pytest
import scipy.special

from oracle import paged as op
from oracle import tree_attention as ota


def _cache(rng, C=2, Hkv=2, D=8, page=4, rows=10):
    per = -(-rows // page)
    table = rng.permutation(C * per).reshape(C, per)
    return rng.standard_normal((C * per, Hkv, page, D)), table


def test_rows_of_reads_through_the_table():
    rng = np.random.default_rng(0)
    pages, table = _cache(rng)
    got = op.rows_of(pages, table, 1, 10)
    for j in range(10):
        np.testing.assert_array_equal(got[:, j], pages[table[1, j // 4], :, j % 4])


def test_head_norm_closed_form():
    x = np.array([[[3.0, 4.0]]])
    np.testing.assert_allclose(op.head_norm(x, [2.0, 1.0], 0.5), [[[6 / math.sqrt(13), 4 / math.sqrt(13)]]])
    y = op.append(x, [1.0, 1.0], [0], eps=1e-12)
    assert abs((y ** 2).mean() - 1) < 1e-9                 # position 0 turns nothing
    assert abs((op.append(x, None, [5]) ** 2).sum() - 25) < 1e-12


def test_causal_attention_and_a_chain_tree_agree_with_scipy():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((2, 9, 8)), rng.standard_normal((2, 9, 8))
    out, lse, mag, _ = op.attention(q, k, v, op.sees(4, 5), 0.3)
    chain, _, _, _ = op.attention(q, k, v, op.sees(4, 5, np.tril(np.ones((7, 7)))), 0.3)
    np.testing.assert_array_equal(out, chain)
    for h in range(4):
        s = q[:, h] @ k[h // 2].T * 0.3
        s[np.triu_indices(5, 5, 9)] = -np.inf
        np.testing.assert_allclose(out[:, h], scipy.special.softmax(s, 1) @ v[h // 2], atol=1e-13)
        np.testing.assert_allclose(lse[:, h], scipy.special.logsumexp(s, 1), atol=1e-13)
    assert (mag >= np.abs(out) - 1e-15).all()


def test_attention_agrees_with_the_contiguous_tree_attention():
    rng = np.random.default_rng(2)
    Hq, Hkv, D, N, S = 4, 2, 8, 6, 3
    q, kt, vt = (rng.standard_normal((1, S, h, D)) for h in (Hq, Hkv, Hkv))
    kc, vc = rng.standard_normal((2, 1, Hkv, N, D))
    mask = np.array([[[1, 0, 0], [1, 1, 0], [1, 0, 1]]], np.uint8)
    pos = np.array([[0, 1, 1]])
    want = ota.tree_attention(q, kt, vt, kc, vc, np.array([N]), mask, pos, np.array([S]), "f32")
    p = N + pos[0]
    k = np.concatenate([kc[0], np.moveaxis(op.append(kt[0], None, p), 0, 1)], 1)
    v = np.concatenate([vc[0], np.moveaxis(vt[0], 0, 1)], 1)
    got = op.attention(op.append(q[0], None, p), k, v, op.sees(N, S, mask[0]), 1 / math.sqrt(D))[0]
    np.testing.assert_allclose(got, want[0], atol=1e-5)


def test_a_row_that_sees_nothing_is_zero():
    q, k = np.ones((1, 1, 4)), np.ones((1, 1, 4))
    out, lse, _, _ = op.attention(q, k, k, np.zeros((1, 1), bool), 1.0)
    assert (out == 0).all() and lse[0, 0] == -np.inf


def test_weights_of_a_step_sum_to_one_per_token_and_head():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((3, 4, 8)), rng.standard_normal((2, 8, 8))
    seen = op.sees(5, 3)
    lse = op.attention(q, k, k, seen, 0.5)[1]
    before = rng.random((2, 16))
    w = op.weights(q, k, seen, lse, 0.5, before, 5, 0.25)
    np.testing.assert_allclose((w - np.pad(0.25 * before[:, :5], ((0, 0), (0, 3)))).sum(1), 3 * 2)


@pytest.mark.parametrize("w,n,budget,sink,recent,want", [
    ([5, 1, 4, 2, 3, 0], 6, 3, 1, 1, [0, 2, 5]),
    ([0, 1, 1, 1, 0, 9], 6, 4, 1, 1, [0, 1, 2, 5]),          # ties: the lowest rows
    ([0, math.nan, -math.inf, 2, 0, 9], 6, 4, 0, 0, [0, 3, 4, 5]),
    ([math.nan, -math.inf, 1], 3, 2, 0, 0, [1, 2]),          # NaN below -inf
    ([1, 2, 3], 3, 5, 1, 1, [0, 1, 2]),                      # all fit
    ([1, 2, 3, 4], 4, 2, 1, 1, [0, 3]),                      # no room but for the fixed rows
    ([], 0, 2, 0, 0, []),
])
def test_kept_rows_by_hand(w, n, budget, sink, recent, want):
    assert op.kept_rows(np.asarray(w, float), n, budget, sink, recent) == want


def test_commit_moves_by_hand():
    assert op.commit_moves([2, 5, -1], 2, 100) == ([102, 105], [101, 102], 103)
    assert op.commit_moves([-1], 0, 7) == ([], [], 8)
