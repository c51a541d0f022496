"""Lengths without a tree (tree=dict(n_nodes=...) in the fixed layout): append, attention and weights of batches whose
requests have fewer tokens than S, by the tests of the paged calls over their own cases, each laid out with S rows to a
request; shared prefixes; a captured step whose lengths change in place."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_paged as tp  # noqa: E402
import test_gpu_shared as ts  # noqa: E402

pytestmark = pytest.mark.gpu
dd = tp.dd


class Lengths(tp.Case):
    """A batch in the fixed layout with 0 to 2 rows more than its longest request has tokens."""

    def __init__(self, dd, new, old, S=None, tree=False, ragged=False, pad=(0, 0), seed=0, **kw):
        super().__init__(dd, new, old, S=(S or max(1, max(new))) + seed % 3, ragged=False, seed=seed, **kw)
        self.tree = dict(n_nodes=torch.tensor(self.new, dtype=torch.int32, device="cuda"))
        self.depth = [np.arange(self.S) for _ in new]


@pytest.fixture
def lengths(monkeypatch):
    monkeypatch.setattr(tp, "Case", Lengths)


RUNS = lambda cases: [i for i, kw in enumerate(cases) if not kw.get("tree")]  # noqa: E731


@pytest.mark.parametrize("i", RUNS(tp.ATTN))
def test_attention(dd, lengths, i):
    tp.test_attention_matches_oracle(dd, i)


@pytest.mark.parametrize("i", RUNS(tp.WEIGHTS))
def test_weights(dd, lengths, i):
    tp.test_weights_match_oracle(dd, i)


@pytest.mark.parametrize("i", RUNS(tp.APPEND))
def test_append(dd, lengths, i):
    tp.test_append_matches_oracle(dd, i, bool(i % 2), "bf16" if i % 3 else "f32")


@pytest.mark.parametrize("i,kw,start,rows", [
    (0, dict(new=[1, 0, 1, 2, 0, 1], old=[300, 301, 317, 428, 300, 300], spare=6000), [0, 6], [300]),
    (1, dict(new=[3, 0, 1, 2], old=[200, 130, 300, 64], page=32, D=64, Hq=8, Hkv=4, spare=6000), [0, 2, 4], [130, 50]),
    (2, dict(new=[40, 0, 17, 64, 1], old=[700, 650, 640, 900, 641], Hq=8, Hkv=2, page=64, spare=6000), [0, 5], [640]),
    (3, dict(new=[0] * 3, old=[90] * 3, spare=3000), [0, 3], [90]),
])
def test_shared(dd, i, kw, start, rows):
    x = Lengths(dd, seed=i, **kw).fill()
    ts._check(x, ts._groups(x, start, rows))


def test_lengths_that_do_not_fit_and_a_tree_after_them(dd):
    """More tokens than S and fewer than none are reported; a tree's call behind one with lengths is a tree's."""
    x = Lengths(dd, [2, 3], [40, 50], S=4, seed=0).fill()
    for n in ([5, 3], [2, -1]):
        x.cache.attention(x.q, tree=dict(n_nodes=torch.tensor(n, dtype=torch.int32, device="cuda")))
        torch.cuda.synchronize()
        assert dd.read_status(x.cache.ws) == dd.EINTERNAL
        dd.clear_status(x.cache.ws)
    y = tp.Case(dd, [4, 4], [40, 50], S=4, tree=True, seed=1).fill()
    lse = torch.empty(y.T, y.Hq, device="cuda")
    want = y.cache.attention(y.q, tree=y.tree)
    y.cache.attention(y.q, tree=dict(n_nodes=y.tree["n_nodes"]))
    got = y.cache.attention(y.q, tree=y.tree, lse=lse)
    y.ok()
    assert torch.equal(got, want)
    tp._check_attention(y, got, lse)
    for half in (dict(n_nodes=y.tree["n_nodes"], pos=y.tree["pos"]),):
        with pytest.raises(KeyError):
            y.cache.attention(y.q, tree=half)
    with pytest.raises(dd.DartreeError):                        # q_start has the lengths
        z = tp.Case(dd, [2, 3], [40, 50], seed=2).fill()
        z.cache.attention(z.q, tree=dict(n_nodes=y.tree["n_nodes"]))


def test_a_captured_step(dd):
    x = Lengths(dd, [3] * 5, [100, 33, 64, 0, 17], S=3, seed=3, Hq=8, Hkv=2).fill()
    out, lse = torch.zeros_like(x.q), torch.zeros(x.T, x.Hq, device="cuda")
    step = lambda s=None: x.cache.attention(x.q, tree=x.tree, out=out, lse=lse, stream=s)  # noqa: E731
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for new in ([0, 1, 2, 3, 0], [3, 0, 0, 1, 2], [0] * 5):
        x.new = new
        x.tree["n_nodes"].copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(7.0), lse.fill_(7.0)
        g.replay()
        x.ok()
        tp._check_attention(x, out, lse)
        for c in range(x.C):
            dead = slice(x.first[c] + new[c], x.first[c] + x.S)
            assert (out[dead] == 0).all() and (lse[dead] == 0).all()
        got, side = out.clone(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        side.synchronize()
        assert torch.equal(out, got)
