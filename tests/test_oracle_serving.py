"""Pins of the serving step's oracle: hand-made tables and draws, the law of the draws."""
import numpy as np

from oracle import serving as sv


def test_reserve_by_hand():
    # pages of 4: request 0 fills its page, 1 needs two pages of three free, 2 needs two (one is left: refused),
    # 3 needs one (served from what is left), 4 wants nothing
    table = np.full((5, 3), -1)
    table[0, 0], table[2, 0] = 9, 8
    r = sv.reserve(table, [3, 0, 4, 0, 0], [1, 5, 5, 2, 0], [20, 21, 22], 4, 5, 9, False)
    assert r["granted"].tolist() == [1, 5, 0, 2, 0] and r["n_free"] == 0
    assert r["table"].tolist() == [[9, -1, -1], [22, 21, -1], [8, -1, -1], [20, -1, -1], [-1, -1, -1]]
    assert r["q_start"].tolist() == [0, 1, 6, 6, 8, 8]
    assert r["slot"].tolist() == [39, 88, 89, 90, 91, 84, 80, 81, -1]
    assert r["pos"].tolist() == [3, 0, 1, 2, 3, 4, 0, 1, -1]
    assert r["request"].tolist() == [0, 1, 1, 1, 1, 1, 3, 3, -1]
    f = sv.reserve(table, [3, 0, 4, 0, 0], [1, 5, 5, 2, 0], [20, 21, 22], 4, 5, 25, True)
    assert f["slot"][:11].tolist() == [39, -1, -1, -1, -1, 88, 89, 90, 91, 84, -1]
    assert sv.release(r["table"], [4, 5, 4, 2, 0], [4, 1, 0, 0, 0], [0, 0, 0, 2, 0], [], 4) == [21, 8]


def test_kept_by_hand():
    x = np.log([0.5, 0.25, 0.125, 0.125])
    k = lambda **kw: sv.kept(x, **{**dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0), **kw})[0].tolist()  # noqa: E731
    assert k() == [0, 1, 2, 3] and k(top_k=3) == [0, 1, 2] and k(top_p=0.75) == [0, 1] and k(top_p=0.8) == [0, 1, 2]
    assert k(min_p=0.3) == [0, 1] and k(temperature=0.0) == [0] and k(top_p=0.0) == [0]
    assert k(top_k=2, top_p=0.6) == [0]            # top-p of what top-k left: 1/2 of 3/4 is two thirds
    assert sv.kept([0.0, -np.inf, np.nan, 0.0], 1.0, 0, 1.0, 0.0)[0].tolist() == [0, 3]
    assert sv.draw([-np.inf, np.nan], 0.5)[0] == -1
    assert [sv.draw(x, u)[0] for u in (0.0, 0.49, 0.5, 0.74, 0.76, 0.99)] == [0, 0, 1, 1, 2, 3]


def test_law_of_the_draws():
    rng = np.random.default_rng(0)
    x, T = rng.standard_normal(7), 0.7
    p = np.exp(x / T) / np.exp(x / T).sum()
    n = 20000
    got = np.bincount([sv.draw(x, u, T)[0] for u in rng.random(n)], minlength=7)
    assert (((got - n * p) ** 2 / (n * p)).sum()) < 27.9      # chi-square, 6 degrees of freedom, 1e-4
