"""Groups whose shared rows pass a request's cached ones are reported, by a row as by a page, wherever the request lies
in its group and by both ways of own rows (at most 16 rows of q to a request, and more)."""
import pytest

torch = pytest.importorskip("torch")

import test_gpu_paged as tp  # noqa: E402

pytestmark = pytest.mark.gpu
dd = tp.dd


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,tree", [(1, False), (9, False), (12, True)])
def test_rows_past_the_cached_ones(dd, new, tree, D):
    C, page = 40, 32
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for start, rows, short, n in (([0, 40], [300], 0, 299), ([0, 40], [300], 39, 299), ([0, 40], [300], 17, 288),
                                  ([0, 40], [300], 17, 287), ([3, 9, 9, 33], [64, 10, 70], 32, 69),
                                  (list(range(41)), [64] * 39 + [65], 39, 64)):
        old = [300] * C
        x = tp.Case(dd, new=[new] * C, old=old, Hq=8, Hkv=2, D=D, page=page, tree=tree, ragged=not tree, seed=D, spare=3000).fill()
        s = x.cache.shared(i(start), i(rows), always=True)
        x.cache.attention(x.q, tree=x.tree, shared=s)
        torch.cuda.synchronize()
        assert dd.read_status(s.ws) == 0
        x.n_ctx[short] = n
        x.cache.attention(x.q, tree=x.tree, shared=s)
        torch.cuda.synchronize()
        assert dd.read_status(s.ws) == dd.EINTERNAL, (start, rows, short, n)
        dd.clear_status(s.ws)
        x.n_ctx[short] = n + 1                                 # (287: still a row short of the page)
        x.cache.attention(x.q, tree=x.tree, shared=s)
        torch.cuda.synchronize()
        g = sum(b <= short for b in start) - 1
        assert dd.read_status(s.ws) == (0 if n + 1 >= rows[g] else dd.EINTERNAL), (start, rows, short, n + 1)
