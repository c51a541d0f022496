"""Draws and walks of shapes that take the kernel's other ways: clusters of eight CTAs that walk several rows, fewer
tokens than top-k asks for in rows that start anywhere, values whose difference is no float. Compared as in
test_gpu_filtered."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_filtered as tf  # noqa: E402
from oracle import serving as sv  # noqa: E402

pytestmark = pytest.mark.gpu
dd = tf.dd
DT = tf.DT


def _single(kw, c):
    """Settings of request c as the oracle takes them."""
    return {k: v[c].item() if isinstance(v, np.ndarray) else float(np.float32(v)) if k != "top_k" else v
            for k, v in kw.items()}


def _walk(dd, t, x, rows, L, u, **kw):
    """A walk through the binding, equal to the oracle's -> accepted lengths."""
    dev = {k: torch.from_numpy(v).cuda() for k, v in t.items()}
    mode = dd.ROWS_PER_NODE if rows == "node" else dd.ROWS_PER_POSITION
    ws = dd.new_workspace(256)
    got = dd.verify_filtered(dev, x, mode, L, torch.from_numpy(u).cuda(), ws=ws, **{
        k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in kw.items()})
    assert dd.read_status(ws) == 0
    want = sv.verify(t, x.double().cpu().numpy(), rows, L, u, lambda c: _single(kw, c))
    for k in want:
        np.testing.assert_array_equal(got[k].cpu().numpy(), want[k], err_msg=f"{k} {kw}")
    return want["accepted_len"]


def _liked(rng, t, rows, n, V, boost):
    """Rows of logits in which the tree's tokens are far above the others."""
    C = len(t["n_nodes"])
    x = torch.from_numpy(rng.standard_normal((C, n, V)))
    for c in range(C):
        for j in range(1, int(t["n_nodes"][c])):
            r = int(t["par"][c, j]) if rows == "node" else int(t["depth"][c, t["par"][c, j]])
            if r < n:
                x[c, r, int(t["tok"][c, j])] += boost
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ["node", "position"])
@pytest.mark.parametrize("C,S,L,V", [(2, 17, 8, 20001), (9, 9, 5, 8200), (1, 12, 6, 151937)])
def test_clusters_of_eight_walk_several_rows(dd, C, S, L, V, rows, dtype):
    """Every CTA of a cluster reaches the first exchange in its own time: the call again and again, the kernel behind
    itself in the stream."""
    rng = np.random.default_rng(V + C)
    t = tf._tree(rng, C, S, L, V)
    n = S if rows == "node" else L
    x = _liked(rng, t, rows, n, V, 12.0).to(DT[dtype]).cuda()
    deepest = 0
    for kw in tf.SETTINGS[:4]:
        u = rng.random((C, n), dtype=np.float32).clip(0, 1 - 2.0 ** -24)
        deepest = max(deepest, int(_walk(dd, t, x, rows, L, u, **kw).max()))
    assert deepest >= 2                                        # (the oracle's: more rows than one)
    dev, un = {k: torch.from_numpy(v).cuda() for k, v in t.items()}, torch.from_numpy(u).cuda()
    mode = dd.ROWS_PER_NODE if rows == "node" else dd.ROWS_PER_POSITION
    first = dd.verify_filtered(dev, x, mode, L, un, **kw)
    for got in [dd.verify_filtered(dev, x, mode, L, un, **kw) for _ in range(50)]:
        for k in first:
            assert torch.equal(got[k], first[k]), k


def _leave_narrow_borders(dd, V, dtype):
    """Rows on every SM of which one token far above any other is kept: what a later call must not take for its own
    border."""
    x = torch.zeros(1200, V, dtype=DT[dtype], device="cuda")
    x[:, 0] = 1000.0
    assert (dd.sample(x, torch.full((1200,), 0.5, device="cuda"), top_p=0.01) == 0).all()
    assert (dd.sample(x, torch.full((1200,), 0.5, device="cuda"), top_k=V - 1, top_p=0.01) == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first", range(8))
def test_fewer_tokens_than_top_k(dd, first, dtype):
    """Masked rows at every offset from 16 bytes: with k of more than the finite logits all of these are kept, and
    nothing else."""
    rng = np.random.default_rng(20 + first)
    V, R = 3001, 16                                            # (an odd pitch: each row has its own offset)
    for finite in (1, 60, 296, 1100, 2400):
        x = np.full((R, V), -np.inf)
        for r in range(R):
            x[r, rng.choice(V, finite, replace=False)] = rng.standard_normal(finite) * 2.5
            if r % 4 == 3:                                     # NaN counts as -inf
                x[r, np.isinf(x[r]) & (rng.random(V) < 0.5)] = np.nan
        big = torch.full((R * V + first,), float("inf"), dtype=DT[dtype], device="cuda")
        rows = big[first:].view(R, V)
        rows.copy_(torch.from_numpy(x))
        for kw in (dict(top_k=2500), dict(top_k=2999, temperature=0.7, top_p=0.9), dict(top_k=3000, min_p=0.02),
                   dict(top_k=np.where(np.arange(R) % 2, 2400, 1025).astype(np.int32))):
            for _ in range(3):
                _leave_narrow_borders(dd, V, dtype)
                tf._check(dd, rows, rng.random(R, dtype=np.float32).clip(0, 1 - 2.0 ** -24), dtype, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_under_a_large_top_k(dd, dtype):
    """The tokens that reach +inf share the weight, whatever k asks for."""
    rng = np.random.default_rng(30)
    V, R = 3001, 16
    x = rng.standard_normal((R, V)) * 2.5
    at = [rng.choice(V, n, replace=False) for n in np.resize([1, 2, 3, 1200], R)]
    for r in range(R):
        x[r, at[r]] = np.inf
    for kw in (dict(top_k=2500), dict(top_k=2500, top_p=0.5), dict(top_k=1100)):
        _leave_narrow_borders(dd, V, dtype)
        got = tf._check(dd, x, rng.random(R, dtype=np.float32).clip(0, 1 - 2.0 ** -24), dtype, **kw)
        assert all(got[r] in at[r] for r in range(R))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [3001, 20001])
def test_a_walk_from_a_full_row_into_masked_ones(dd, V, dtype):
    """The rows of one walk share their CTAs: a border far above the next rows' logits stays with its row."""
    rng = np.random.default_rng(V)
    C, S, L = 6, 9, 8
    t = tf._tree(rng, C, S, L, V, width=1)                     # chains
    x = np.full((C, S, V), -np.inf)
    for c in range(C):
        x[c, 0] = 100.0 + rng.standard_normal(V)
        for j in range(1, S):
            x[c, j, rng.choice(V, 40, replace=False)] = rng.standard_normal(40)
        for j in range(1, int(t["n_nodes"][c])):
            p = int(t["par"][c, j])
            x[c, p, t["tok"][c, j]] = 115.0 if p == 0 else 5.0
    x = torch.from_numpy(x).to(DT[dtype]).cuda()
    deepest = 0
    for i in range(8):
        u = rng.random((C, S), dtype=np.float32).clip(0, 1 - 2.0 ** -24)
        deepest = max(deepest, int(_walk(dd, t, x, "node", L, u, top_k=2500, top_p=[1.0, 0.95][i % 2]).max()))
    assert deepest >= 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,lo,hi,T", [(20.0, -9.1e-7, 9.1e-7, 10.0), (100.0, -3e-6, 3e-6, 50.0), (-1e-5, -6.0, -9.0, 4.0),
                                       (-3e-6, -3.5, -1.75, 1.0)])
def test_differences_that_are_no_floats(dd, m, lo, hi, T, dtype):
    """A maximum and values so far apart in magnitude that fp32 rounds their difference: numbers u between the border of
    two runs of such values and where weights of rounded differences would put it."""
    V = 512
    x = torch.full((V,), lo, dtype=torch.float64)
    tried = 0
    for n in (3, 4, 6, 8, 11, 16, 23, 32, 45, 64, 100, 200):
        x[:n], x[n:], x[V // 2] = hi, lo, m
        h = x.to(DT[dtype]).double().numpy()
        top = h.max()
        exact, rounded = (np.cumsum(np.exp(-d / T)) for d in (top - h, (top - h).astype(np.float32).astype(np.float64)))
        a, b = exact[n - 1] / exact[-1], rounded[n - 1] / rounded[-1]
        margin = 2 * V * 2.0 ** -42
        u = np.float32(0.5 * (a + b))
        if min(abs(u - a), abs(u - b)) < 2 * margin or not min(a, b) < u < max(a, b):
            continue                                           # (no float lies between)
        tried += 1
        tf._check(dd, x[None].to(DT[dtype]).cuda(), np.array([u]), dtype, temperature=T)
        tf._check(dd, x[None].to(DT[dtype]).cuda(), np.array([u]), dtype, temperature=T, top_p=float(np.float32(0.9999999)))
    assert tried >= 3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_minus_zero_is_zero(dd, dtype):
    """u and settings of -0, as numbers and as tensors, are settings: they draw what 0 draws."""
    rng = np.random.default_rng(40)
    R = 6
    x = rng.standard_normal((R, 3001))
    z, f = np.full(R, -0.0, np.float32), rng.random(R, dtype=np.float32).clip(0, 1 - 2.0 ** -24)
    for kw in (dict(), dict(top_p=0.9), dict(top_k=50), dict(top_k=2000), dict(min_p=0.05)):
        assert (tf._check(dd, x, z, dtype, **kw) == tf._check(dd, x, -z, dtype, **kw)).all()
    for key in ("temperature", "top_p", "min_p"):
        for value in (-0.0, z):
            tf._check(dd, x, f, dtype, **{key: value})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1.4e-45, 3e-42, 1e-39, 2e-36, 1e-30, 5e-20, 6e-20, 1e-10, 1e18, 2e19, 1e30, 2e37])
def test_logits_of_the_temperatures_size(dd, T, dtype):
    """Temperatures from the smallest float to the largest ones, logits a few of them apart."""
    T = float(np.float32(T))
    rng = np.random.default_rng(50)
    quantum = max(T, 2.0 ** -133) if dtype == "bf16" else T    # (the smallest bf16)
    x = np.stack([rng.integers(0, 8, 3001) * quantum, -rng.integers(0, 60, 3001) * quantum * 0.5,
                  np.where(rng.random(3001) < 0.01, 9 * quantum, 0.0), rng.standard_normal(3001) * 3 * quantum])
    for kw in (dict(), dict(top_p=0.9), dict(top_k=40), dict(top_k=2000, top_p=0.97), dict(min_p=0.3), dict(top_p=0.8, min_p=0.01)):
        for _ in range(4):
            tf._check(dd, x, rng.random(4, dtype=np.float32).clip(0, 1 - 2.0 ** -24), dtype, temperature=T, **kw)
