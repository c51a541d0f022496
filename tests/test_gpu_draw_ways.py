"""Draws and walks of shapes that take the kernel's other ways: clusters of eight CTAs that walk several rows.
Compared as in test_gpu_filtered."""
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
