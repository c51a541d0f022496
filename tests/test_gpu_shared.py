"""Attention of requests that share prefixes (PagedCache.attention with groups) against the float64 oracle of the
plain call, with its tolerances: the same sums in another order. Page rows that hold nothing are NaN."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_paged as tp  # noqa: E402

pytestmark = pytest.mark.gpu
dd = tp.dd


def _groups(x, start, rows, **kw):
    """The groups' requests get the pages of their first ones; the copies that they had are NaN."""
    for g in range(len(rows)):
        whole = rows[g] // x.page
        first = x.np_table[start[g]:start[g] + 1, :whole].copy()
        for c in range(start[g] + 1, start[g + 1]):
            assert rows[g] <= x.old[c]
            old = torch.from_numpy(x.np_table[c, :whole].astype(np.int64)).cuda()
            x.k[old], x.v[old] = float("nan"), float("nan")
            x.np_table[c, :whole] = first
    x.table.copy_(torch.from_numpy(x.np_table))
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return x.cache.shared(dev(start), dev(rows), **{**dict(always=True), **kw})


def _run(x, s, scale=None):
    lse = torch.full((x.T, x.Hq), 7.0, device="cuda")
    out = torch.full((x.T, x.Hq, x.D), 7.0, device="cuda", dtype=torch.bfloat16)
    got = x.cache.attention(x.q, tree=x.tree, shared=s, scale=scale, out=out, lse=lse)
    torch.cuda.synchronize()
    assert got is out and x.dd.read_status(s.ws) == 0
    return out, lse


def _check(x, s, scale=None):
    out, lse = _run(x, s, scale)
    tp._check_attention(x, out, lse, scale)
    first = np.array(x.first)
    live = np.zeros(x.T, bool)
    for c in range(x.C):
        live[first[c]:first[c] + x.new[c]] = True
    rest = torch.from_numpy(~live).cuda()
    want = 7.0 if x.q_start is not None else 0.0               # rows of no token; slots without a node
    assert (out[rest] == want).all() and (lse[rest] == want).all()


BIG = dict(spare=6000)   # the chunks are planned for longer rows
CASES = [
    # single tokens: own rows from none to several blocks, lengths around pages and blocks
    (dict(new=[1] * 6, old=[300, 301, 317, 428, 813, 300], ragged=False, **BIG), [0, 6], [300]),
    (dict(new=[1] * 5, old=[128, 129, 255, 256, 400], Hq=8, Hkv=1, page=64, ragged=False, **BIG), [0, 5], [128]),
    (dict(new=[1] * 9, old=[130 + 40 * c for c in range(9)], Hq=6, Hkv=6, D=64, page=32, **BIG), [0, 9], [130]),
    # several groups, one of one request, one empty, one with less than a page, requests of no group
    (dict(new=[1, 2, 1, 3, 1, 1, 2], old=[200, 130, 300, 64, 70, 9, 33], page=32, **BIG), [0, 2, 3, 3, 5], [130, 300, 50, 64]),
    (dict(new=[2] * 6, old=[500, 90, 100, 90, 20, 7], page=16, ragged=False, **BIG), [1, 4], [90]),
    (dict(new=[1] * 4, old=[40, 40, 15, 20], page=16, **BIG), [0, 2, 4], [0, 15]),
    # chunks of tokens, ragged, with rows of q before and behind
    (dict(new=[40, 0, 17, 64, 1], old=[700, 650, 640, 900, 641], Hq=8, Hkv=2, page=64, pad=(3, 5), **BIG), [0, 5], [640]),
    (dict(new=[30, 31], old=[256, 300], Hq=10, Hkv=2, D=64, page=256, **BIG), [0, 2], [256]),
    (dict(new=[3] * 12, old=[2000] * 12, Hq=28, Hkv=4, page=128, **BIG), [0, 12], [2000]),
    (dict(new=[9, 2], old=[140, 150], Hq=128, Hkv=1, page=16, D=64, **BIG), [0, 2], [140]),
    # trees, some without nodes
    (dict(new=[12, 1, 0, 7], old=[260, 300, 255, 256], S=12, tree=True, **BIG), [0, 4], [250]),
    (dict(new=[65] * 5, old=[1000, 1024, 1100, 1023, 1500], tree=True, Hq=8, Hkv=2, page=64, **BIG), [0, 5], [1000]),
    (dict(new=[33, 20, 33], old=[400, 400, 500], S=33, tree=True, Hq=16, Hkv=8, D=64, page=32, **BIG), [0, 1, 3], [300, 400]),
    (dict(new=[2, 4, 3], old=[90, 80, 100], S=4, tree=True, page=16, **BIG), [0, 3], [80]),
    # a batch of many; more groups than a warp
    (dict(new=[1] * 64, old=[4000 + 11 * c for c in range(64)], Hq=16, Hkv=4, page=64, ragged=False), [0, 64], [3990]),
    (dict(new=[1, 2] * 35, old=[150 + c for c in range(70)], Hq=8, Hkv=2, D=64, page=16, spare=2500),
     list(range(0, 70, 2)) + [69, 70], [150 + 2 * g for g in range(34)] + [218, 219]),
    # long prefixes: many chunks
    (dict(new=[1] * 3, old=[20000, 20100, 20001], Hq=4, Hkv=1, page=256, ragged=False), [0, 3], [20000]),
    (dict(new=[16, 5, 9, 16], old=[9000, 9100, 9000, 9500], Hq=16, Hkv=1, D=64, page=64, pad=(0, 2)), [0, 4], [9000]),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_oracle(dd, i):
    kw, start, rows = CASES[i]
    x = tp.Case(dd, seed=i, **kw).fill()
    _check(x, _groups(x, start, rows))
    # planned for what there is: other chunks
    _check(x, x.cache.shared(*(torch.tensor(a, dtype=torch.int32, device="cuda") for a in (start, rows)), always=True,
                             most_rows=max(rows), most_rest=64))


def test_large_scores_and_far_keys(dd):
    """Rising maxima: the shared rows' weights vanish beside the own ones, and the other way round."""
    for k, (lo, hi) in enumerate(((0.05, 6.0), (6.0, 0.05))):
        x = tp.Case(dd, new=[1, 3, 2], old=[600, 700, 650], Hq=8, Hkv=2, page=64, seed=40 + k, spare=6000, scaleq=3.0).fill()
        s = _groups(x, [0, 3], [600])
        for c in range(3):
            n = x.old[c] + x.new[c]
            p, r = tp.op.place(x.np_table, c, np.arange(n), x.page)
            f = torch.from_numpy(np.where(np.arange(n) < 576, lo, hi)).to(torch.bfloat16).cuda()
            p, r = torch.from_numpy(p.astype(np.int64)).cuda(), torch.from_numpy(r).cuda()
            if c == 0:
                x.k[p, :, r] *= f[:, None, None]
            else:
                x.k[p[576:], :, r[576:]] *= f[576:, None, None]
        _check(x, s, scale=0.3)


def test_equal_inputs_give_equal_outputs_and_fallback(dd):
    x = tp.Case(dd, new=[1] * 8, old=[900 + c for c in range(8)], Hq=8, Hkv=2, page=64, seed=50, spare=6000).fill()
    s = _groups(x, [0, 8], [900])
    a = _run(x, s)
    for _ in range(3):
        b = _run(x, s)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # too little to share by what is expected: the plain call, bit for bit
    t = x.cache.shared(s.start, s.rows, most_rows=64, most_rest=6000)
    assert not t.plan().use
    c = _run(x, t)
    lse = torch.empty_like(c[1])
    assert torch.equal(c[0], x.cache.attention(x.q, lse=lse)) and torch.equal(c[1], lse)
    # expectations that do not hold change nothing but the time
    tight = x.cache.shared(s.start, s.rows, most_rows=6500, most_rest=1, always=True)
    _check(x, tight)
    # no groups: every request for itself
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    z = x.cache.shared(torch.zeros(1, dtype=torch.int32, device="cuda"), e)
    assert torch.equal(_run(x, z)[0], c[0])


def test_bad_groups_are_reported(dd):
    def status(start, rows, old=(300, 300, 300, 300)):
        x = tp.Case(dd, new=[1] * 4, old=list(old), Hq=4, Hkv=2, page=16, seed=60, spare=6000).fill()
        dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        s = x.cache.shared(dev(start), dev(rows), always=True)
        x.cache.attention(x.q, shared=s)
        torch.cuda.synchronize()
        return dd.read_status(s.ws)

    assert status([0, 4], [300]) == 0
    for start, rows in (([0, 5], [300]), ([-1, 4], [300]), ([3, 1], [300]), ([0, 3, 2], [16, 16]), ([0, 4], [-1]),
                        ([0, 4], [10 ** 6]), ([0, 4], [2 ** 31 - 1]), ([0, 4], [320])):
        assert status(start, rows) == dd.EINTERNAL, (start, rows)
    assert status([0, 4], [256], old=(300, 300, 255, 300)) == dd.EINTERNAL


def test_bad_pages_are_reported(dd):
    x = tp.Case(dd, new=[1] * 4, old=[300] * 4, Hq=4, Hkv=2, page=16, seed=61, spare=6000).fill()
    s = _groups(x, [0, 4], [256])
    for c, j, v in ((0, 3, -1), (0, 5, 10 ** 6), (2, 17, -5)):
        t = x.table.clone()
        x.table[c, j] = v
        out = x.cache.attention(x.q, shared=s)
        torch.cuda.synchronize()
        assert dd.read_status(s.ws) == dd.EINTERNAL and torch.isfinite(out).all()
        dd.clear_status(s.ws)
        x.table.copy_(t)
    _check(x, s)


def test_refusals(dd):
    x = tp.Case(dd, new=[1] * 3, old=[50] * 3, seed=62).fill()
    y = tp.Case(dd, new=[1] * 3, old=[50] * 3, seed=62).fill()
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for a in ((i([0, 3]), i([1, 2])), (i([0, 3]).long(), i([1])), (i([0, 3]), i([[1]])), (i([0, 3]).cpu(), i([1]))):
        with pytest.raises(ValueError):
            x.cache.shared(*a)
    with pytest.raises(dd.DartreeError):
        x.cache.shared(i([0, 1, 2, 3, 3]), i([1] * 4))         # more groups than requests
    with pytest.raises(dd.DartreeError):
        x.cache.shared(i([0, 3]), i([1]), most_rows=-1)
    s = x.cache.shared(i([0, 3]), i([16]))
    with pytest.raises(ValueError):
        y.cache.attention(y.q, shared=s)
    with pytest.raises(dd.DartreeError) as e:
        x.cache.attention(x.q, shared=x.cache.shared(i([0, 3]), i([16]), ws=dd.new_workspace(256)))
    assert e.value.code == dd.EWORKSPACE


def test_lengths_change_in_place_graph_and_streams(dd):
    """One captured step, replayed as groups, lengths and contents change; the same on a side stream."""
    x = tp.Case(dd, new=[2] * 6, old=[500] * 6, Hq=8, Hkv=2, page=16, ragged=False, seed=63, spare=4000).fill()
    s = _groups(x, [0, 6], [480])
    out, lse = torch.zeros_like(x.q), torch.zeros(x.T, x.Hq, device="cuda")
    step = lambda: x.cache.attention(x.q, shared=s, out=out, lse=lse)  # noqa: E731
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for start, rows, old in (([0, 6], [480], [500, 490, 480, 700, 481, 500]), ([0, 4], [300], [300, 310, 600, 300, 5, 0]),
                             ([2, 6], [16], [9, 3, 20, 30, 16, 100])):
        x.old = old
        x.n_ctx.copy_(torch.tensor(old, dtype=torch.int32))
        s.start.copy_(torch.tensor(start, dtype=torch.int32)), s.rows.copy_(torch.tensor(rows, dtype=torch.int32))
        x.fill()                                               # (tables still share pages: the same contents)
        g.replay()
        torch.cuda.synchronize()
        assert dd.read_status(s.ws) == 0
        tp._check_attention(x, out, lse)
        got = out.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out2 = x.cache.attention(x.q, shared=s, stream=side)
        side.synchronize()
        assert torch.equal(out2, got)


@pytest.mark.parametrize("D", [64, 128])
def test_many_requests_to_a_cta_again_and_again(dd, D):
    """Several (request, head) pairs follow one another in a CTA, with rings that are refilled across them: every wait
    ends, call after call, and outputs are the same."""
    rng = np.random.default_rng(D)
    rows = 320
    x = tp.Case(dd, new=[1] * 128, old=[rows + int(n) for n in rng.integers(0, 700, 128)], Hq=8, Hkv=8, D=D, page=16,
                seed=70 + D).fill()
    s = _groups(x, [0, 128], [rows])
    first = _run(x, s)
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(8):
            x.cache.attention(x.q, shared=s, out=out, lse=lse)
    for _ in range(25):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert dd.read_status(s.ws) == 0
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    _check(x, s)


def test_two_caches_on_two_streams_at_once(dd):
    xs, ss = [], []
    for i in range(2):
        x = tp.Case(dd, new=[1] * 48, old=[700 + 11 * c for c in range(48)], Hq=8, Hkv=8, page=32, seed=80 + i, spare=3000).fill()
        xs.append(x), ss.append(_groups(x, [0, 48], [700]))
    alone = [x.cache.attention(x.q, shared=s) for x, s in zip(xs, ss)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got += [(i, xs[i].cache.attention(xs[i].q, shared=ss[i], stream=streams[i])) for i in range(2)]
    torch.cuda.synchronize()
    for i, out in got:
        assert torch.equal(out, alone[i])
    for s in ss:
        assert dd.read_status(s.ws) == 0
