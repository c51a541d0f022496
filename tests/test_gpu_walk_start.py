"""Walks by nodes whose slices are nearly or wholly empty: their CTAs come to the first exchange of the cluster at once,
behind one that loads a long slice. Greedy and sampled walks against the oracles, again and again."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import sampling as osm  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from diffusion_drafter_draft_gb300 import _build
    _build.build()
    import diffusion_drafter_draft_gb300 as m
    m.lib()
    return m


def _tree(rng, C, S, V):
    """Chains with a side branch now and then; slots' tokens differ."""
    t = {k: np.full((C, S), -1, np.int64) for k in ("tok", "par", "depth")}
    for c in range(C):
        t["tok"][c] = rng.permutation(max(V, S))[:S] % V
        t["depth"][c, 0] = 0
        for j in range(1, S):
            p = j - 1 if rng.random() < 0.7 else int(rng.integers(0, j))
            t["par"][c, j], t["depth"][c, j] = p, t["depth"][c, p] + 1
    return dict(t, n_nodes=np.full(C, S, np.int64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,S,V", [(1, 5, 9), (40, 6, 17), (3, 9, 57), (200, 8, 100)])
def test_short_slices(dd, C, S, V, dtype):
    rng = np.random.default_rng(C + V)
    t = _tree(rng, C, S, V)
    L = int(t["depth"].max())
    x = rng.standard_normal((C, S, V)).astype(np.float32)
    for c in range(C):
        for j in range(1, S):
            x[c, t["par"][c, j], t["tok"][c, j]] += 6.0
    d = torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    dev = {k: torch.from_numpy(v.astype(np.int32)).cuda() for k, v in t.items()}
    h = d.float().cpu().numpy()
    greedy = dd.verify(dev, d, dd.ROWS_PER_NODE, L)
    for c in range(C):
        cur, path = 0, []
        while True:
            tok = int(np.argmax(h[c, cur]))
            kid = [j for j in range(1, S) if t["par"][c, j] == cur and t["tok"][c, j] == tok]
            if not kid:
                break
            cur = kid[0]
            path.append(cur)
        assert greedy["path"][c].tolist() == path + [-1] * (L - len(path)) and greedy["bonus"][c].item() == tok
    assert int(greedy["accepted_len"].max()) >= 2
    drawn = dd.verify_sample(dev, d, dd.ROWS_PER_NODE, L, 0.7, 99)
    target = d.view(torch.int16).cpu().numpy().view(np.uint16) if dtype == "bf16" else h
    want = osm.verify_sample(t, target, dtype, "node", L, 0.7, 99)
    for k in ("accepted_len", "path", "bonus"):
        np.testing.assert_array_equal(drawn[k].cpu().numpy(), want[k], err_msg=k)
    for _ in range(100):
        a, b = dd.verify(dev, d, dd.ROWS_PER_NODE, L), dd.verify_sample(dev, d, dd.ROWS_PER_NODE, L, 0.7, 99)
        for k in greedy:
            assert torch.equal(a[k], greedy[k]) and torch.equal(b[k], drawn[k]), k
