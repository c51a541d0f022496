"""Batches of more rows than run at once in shared memory: every pass reads them again, by clusters of one to four CTAs.
(Rows that take more than one CTA's 76 KB, and more CTAs than two to an SM: fp32 beyond 19 thousand tokens, bf16 beyond 38
thousand, from 153 rows on, fewer where a row takes more CTAs.) Compared as in test_gpu_filtered."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_filtered as tf  # noqa: E402

pytestmark = pytest.mark.gpu
dd = tf.dd
DT = tf.DT


def _rows(rng, R, V, dtype):
    """Peaked rows, and of every kind that can go wrong some."""
    x = rng.standard_normal((R, V)) * 2.5
    low = float(torch.finfo(DT[dtype]).min)
    for r in range(R):
        x[r, rng.integers(0, V, 6)] += 12 * rng.random(6)
    x[0] = -np.inf
    x[1] = -np.inf
    x[1, V - 1] = -3.0
    x[2, [0, V // 2, V - 1]] = np.inf
    x[3, rng.random(V) < 0.95] = -np.inf
    x[4, rng.random(V) < 0.5] = np.nan
    x[5, rng.random(V) < 0.9] = low
    x[6] = np.round(x[6])
    x[7] = 1.5
    x[8] = 40.0 + np.round(x[8] * 0.5) * 0.5
    x[9] = -np.inf
    x[9, rng.choice(V, 900, replace=False)] = rng.standard_normal(900)
    return x


SHAPES = [("f32", 160, 20001, 20003, 1), ("f32", 160, 20001, 20001, 3), ("bf16", 160, 40003, 40005, 1),
          ("bf16", 160, 40003, 40003, 5), ("f32", 40, 151937, 151939, 2), ("bf16", 80, 151937, 151937, 7)]


@pytest.mark.parametrize("dtype,R,V,ld,first", SHAPES)
def test_settings(dd, dtype, R, V, ld, first):
    rng = np.random.default_rng(R + V + first)
    big = torch.full((R * ld + first,), float("inf"), dtype=DT[dtype], device="cuda")   # (around the rows: not theirs)
    x = big[first:].view(R, ld)[:, :V]
    x.copy_(torch.from_numpy(_rows(rng, R, V, dtype)))
    pick = lambda a, t: rng.choice(np.array(a, t), R)  # noqa: E731
    mixed = dict(temperature=pick([0, 0.3, 1, 1.5], np.float32), top_k=pick([0, 0, 1, 20, 400, 3000], np.int32),
                 top_p=pick([1, 0.95, 0.3, 0], np.float32), min_p=pick([0, 0, 0.1, 1], np.float32))
    for kw in tf.SETTINGS[:5] + [dict(top_k=2500, top_p=0.9), dict(top_k=V - 1), dict(temperature=0.05, top_p=0.999), mixed]:
        tf._check(dd, x, tf._u(rng, R), dtype, **kw)


@pytest.mark.parametrize("dtype,R,V", [("f32", 300, 30001), ("bf16", 200, 50000)])
def test_a_row_does_not_depend_on_its_batch(dd, dtype, R, V):
    """Held in shared memory or read again: the same tokens."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(R, V, generator=gen, device="cuda") * 2).to(DT[dtype])
    u = torch.rand(R, generator=gen, device="cuda")
    for kw in tf.SETTINGS[:4] + [dict(top_k=5000, top_p=0.8), dict(top_k=700)]:
        whole = dd.sample(x, u, **kw)
        for n in (1, 7, 60, 150):
            assert torch.equal(dd.sample(x[:n], u[:n], **kw), whole[:n]), (kw, n)


def test_a_captured_batch(dd):
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, u = torch.randn(170, 24001, generator=gen, device="cuda") * 2, torch.rand(170, generator=gen, device="cuda")
    out, ws = torch.zeros(170, dtype=torch.int32, device="cuda"), dd.new_workspace(256)
    kw = dict(temperature=0.8, top_p=0.9)
    dd.sample(x, u, out=out, ws=ws, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dd.sample(x, u, out=out, ws=ws, **kw)
    for _ in range(3):
        x.copy_(torch.randn(170, 24001, generator=gen, device="cuda") * 2)
        u.copy_(torch.rand(170, generator=gen, device="cuda"))
        g.replay()
        got = out.clone()
        assert torch.equal(dd.sample(x, u, **kw), got)
