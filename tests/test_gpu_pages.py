"""Pages and rows from lengths (PagedCache.reserve and release) against the oracle: every entry equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import serving as sv  # noqa: E402

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


def _dev(a, dt=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dt))).cuda()


class Batch:
    def __init__(self, dd, C, S, ctx, page, fixed, seed=0, spare=5, T=None, width=None, old=None, new=None):
        rng = self.rng = np.random.default_rng(seed)
        self.C, self.S, self.page, self.fixed = C, S, page, fixed
        self.old = rng.integers(0, ctx + 1, C) if old is None else np.array(old)
        self.new = rng.integers(0, S + 1, C) if new is None else np.array(new)
        held = -(-self.old // page)
        self.width = width or max(1, -(-(ctx + S) // page))
        self.n_pages = int(held.sum()) + max(spare, 0) + 3
        ids = rng.permutation(self.n_pages)
        self.table = np.full((C, self.width), -7, np.int64)
        at = 0
        for c in range(C):
            self.table[c, :held[c]] = ids[at:at + held[c]]
            at += held[c]
        self.stack = ids[at:at + spare].tolist()
        self.T = C * S if fixed else int(self.new.sum()) if T is None else T
        self.q_start = None if fixed else torch.full((C + 1,), -3, dtype=torch.int32, device="cuda")
        self.d_table, self.free = _dev(self.table), torch.full((self.n_pages,), -9, dtype=torch.int32, device="cuda")
        self.free[:spare] = _dev(self.stack)
        self.n_free = _dev([spare])
        pages = torch.zeros(self.n_pages, 1, page, 64, dtype=torch.bfloat16, device="cuda")
        self.cache = dd.PagedCache(pages, pages.clone(), self.d_table, _dev(self.old), 1, max(S, 1), T=self.T,
                                   q_start=self.q_start)
        self.dd = dd

    def check(self, **kw):
        want = sv.reserve(self.table, self.old, self.new, self.stack, self.page, self.S, self.T, self.fixed)
        got = self.cache.reserve(_dev(self.new), self.free, self.n_free, **kw)
        torch.cuda.synchronize()
        assert self.dd.read_status(self.cache.ws) == 0
        for k in ("granted", "slot", "pos", "request"):
            if got.get(k) is not None:
                np.testing.assert_array_equal(got[k].cpu().numpy(), want[k], err_msg=k)
        np.testing.assert_array_equal(self.d_table.cpu().numpy(), want["table"])
        assert got["n_free"].item() == want["n_free"]
        if not self.fixed:
            np.testing.assert_array_equal(self.q_start.cpu().numpy(), want["q_start"])
        return want


@pytest.mark.parametrize("fixed", [True, False])
@pytest.mark.parametrize("C,S,ctx,page", [(1, 1, 100, 16), (1, 1, 0, 64), (3, 65, 500, 64), (64, 65, 2048, 64), (64, 1, 300, 16),
                                          (512, 33, 900, 16), (513, 7, 64, 256), (1500, 3, 40, 32), (2, 9000, 100, 128)])
def test_reserve(dd, C, S, ctx, page, fixed):
    n = C * (-(-S // page) + 1)
    for seed, spare in enumerate((n, n // 3, n // 20, 0)):     # enough, and ever more requests refused
        Batch(dd, C, S, ctx, page, fixed, seed, spare).check()


def test_reserve_short_of_rows_and_of_table(dd):
    Batch(dd, 200, 40, 300, 16, False, 1, 900, T=1500).check()
    Batch(dd, 200, 40, 300, 16, False, 2, 900, T=0).check()
    # request 1 would pass its row of the table, 3 fills it to the last row
    w = Batch(dd, 4, 40, 60, 16, True, 3, 30, width=4, old=[10, 50, 0, 60], new=[40, 20, 40, 4]).check()
    assert w["granted"].tolist() == [40, 0, 40, 4]
    # the largest first, then small ones that still fit, one that wants nothing among them
    w = Batch(dd, 5, 64, 0, 16, False, 4, 5, old=[0] * 5, new=[64, 33, 16, 0, 1]).check()
    assert w["granted"].tolist() == [64, 0, 16, 0, 0]


def test_reserve_in_place_and_without_slots(dd):
    b = Batch(dd, 40, 30, 200, 16, False, 5, 100)
    out = dict(granted=torch.zeros(40, dtype=torch.int32, device="cuda"), slot=None, pos=None, request=None, n_free=b.n_free)
    b.check(out=out)


def test_release(dd):
    for C, ctx, page in ((1, 50, 16), (64, 2000, 64), (700, 300, 16), (1100, 64, 32)):
        b = Batch(dd, C, 1, ctx, page, True, C, 4)
        rng = b.rng
        keep = np.minimum(b.old, rng.integers(0, ctx + 1, C) * rng.integers(0, 2, C))
        for shared in (None, rng.integers(0, ctx + 1, C)):
            stack = sv.release(b.table, b.old, keep, np.zeros(C) if shared is None else shared, b.stack, page)
            n = b.cache.release(_dev(b.old), _dev(keep), b.free, b.n_free, n_shared=None if shared is None else _dev(shared))
            torch.cuda.synchronize()
            assert dd.read_status(b.cache.ws) == 0 and n.item() == len(stack)
            assert b.free[:len(stack)].tolist() == stack
            np.testing.assert_array_equal(b.d_table.cpu().numpy(), b.table)


def test_pages_come_back(dd):
    """Reserve, give back, reserve: in place, the same pages again."""
    b = Batch(dd, 30, 50, 100, 16, True, 9, 150)
    first = b.cache.reserve(_dev(b.new), b.free, b.n_free)
    b.cache.release(_dev(b.old + first["granted"].cpu().numpy()), _dev(b.old), b.free, first["n_free"], n_out=first["n_free"])
    assert first["n_free"].item() == 150 and sorted(b.free[:150].tolist()) == sorted(b.stack)
    again = b.cache.reserve(_dev(b.new), b.free, first["n_free"])
    slots = [s for s in again["slot"].tolist() if s >= 0]
    assert len(slots) == int(b.new.sum()) == len(set(slots))       # no row is given twice
    assert dd.read_status(b.cache.ws) == 0


def test_bad_lengths_and_pages(dd):
    def status(change, **kw):
        b = Batch(dd, 6, 20, 100, 16, False, 11, 40, T=120, old=[5, 90, 20, 33, 0, 7], **kw)
        n_new = _dev([3, 20, 0, 9, 4, 1])
        change(b, n_new)
        got = b.cache.reserve(n_new, b.free, b.n_free)
        torch.cuda.synchronize()
        return b, got, dd.read_status(b.cache.ws)

    def put(name, i, v):
        def f(b, n_new):
            t = n_new if name == "new" else b.cache.n_ctx if name == "ctx" else getattr(b, name)
            t.view(-1)[i] = v
        return f

    for name, i, v in (("new", 1, 21), ("new", 1, -1), ("ctx", 3, -1), ("ctx", 3, 10 ** 6), ("ctx", 3, 2 ** 31 - 1)):
        b, got, st = status(put(name, i, v))
        assert st == dd.EINTERNAL and got["granted"][i].item() == 0
        assert got["granted"][0].item() == 3
    for v, left in ((-1, 0), (10 ** 6, None)):
        b, got, st = status(put("n_free", 0, v))
        assert st == dd.EINTERNAL and 0 <= got["n_free"].item() <= b.n_pages
    b, got, st = status(put("free", 39, 10 ** 6))              # the first page taken is none
    assert st == dd.EINTERNAL and (got["slot"] >= -1).all() and (got["slot"] < b.n_pages * 16).all()
    b, got, st = status(put("d_table", 0, -1))                 # nor is the one that request 0 goes on in
    assert st == dd.EINTERNAL and got["slot"][0].item() == -1
    b = Batch(dd, 2, 1, 100, 16, True, 12, 4)
    b.cache.release(_dev([10 ** 6, 5]), _dev([-1, 0]), b.free, b.n_free)
    assert dd.read_status(b.cache.ws) == dd.EINTERNAL
    dd.clear_status(b.cache.ws)
    b.n_free.fill_(b.n_pages)
    n = b.cache.release(_dev([48, 48]), _dev([0, 0]), b.free, b.n_free)
    assert dd.read_status(b.cache.ws) == dd.EINTERNAL and n.item() == b.n_pages


def test_refusals_and_empty_batches(dd):
    b = Batch(dd, 3, 4, 50, 16, True, 13, 9)
    n = _dev([1, 2, 3])
    for a in ((n[:2], b.free, b.n_free), (n.long(), b.free, b.n_free), (n, b.free[:3], b.n_free), (n, b.free, n)):
        with pytest.raises(ValueError):
            b.cache.reserve(*a)
    with pytest.raises(dd.DartreeError):
        b.cache.reserve(n, b.free, b.n_free, out=dict(granted=n, n_free=b.n_free))
    with pytest.raises(ValueError):
        b.cache.release(n, n[:1], b.free, b.n_free)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    pages = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    cache = dd.PagedCache(pages, pages.clone(), e.view(0, 2), e, 1, 1, T=3, q_start=q)
    free, nf = _dev([0, 1, 2, 3]), _dev([4])
    r = cache.reserve(e, free, nf)
    assert r["n_free"].item() == 4 and q.item() == 0 and r["slot"].tolist() == [-1, -1, -1]
    assert cache.release(e, e, free, nf).item() == 4


def test_graph(dd):
    b = Batch(dd, 20, 30, 200, 16, False, 14, 60, T=700)
    new, nf = _dev(b.new), _dev([60])
    out = b.cache.reserve(new, b.free, nf)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.cache.reserve(new, b.free, nf, out=out)
    for seed in range(3):
        b.new = np.random.default_rng(seed).integers(0, 31, 20)
        new.copy_(_dev(b.new))
        b.d_table.copy_(_dev(b.table))
        g.replay()
        want = sv.reserve(b.table, b.old, b.new, b.stack, 16, 30, 700, False)
        for k in ("granted", "slot", "pos", "request"):
            np.testing.assert_array_equal(out[k].cpu().numpy(), want[k], err_msg=k)
        np.testing.assert_array_equal(b.d_table.cpu().numpy(), want["table"])
