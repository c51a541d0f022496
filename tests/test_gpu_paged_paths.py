"""The paged-cache calls on the paths that large and wide shapes take, in the states that only errors
reach, and captured: two query tiles to a CTA (also with chunks that meet in memory), tables much
wider than the contexts, tables, lengths and paths that are wrong, eviction and commit on a side
stream and in a graph. Cases, oracle and tolerances are those of test_gpu_paged."""
import copy
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import paged as op  # noqa: E402
from test_gpu_paged import E32, Case, _check_attention, _check_evict, _evict_case, _status, dd  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def _plan(dd, x):  # noqa: F811
    plan = dd.PagedPlan()
    assert dd.lib().dartree_paged_attention_plan(dd.ctypes.byref(x.cache.p), dd.ctypes.byref(plan)) == 0
    return plan


def _one(x, c):
    """Request c of Case x alone, for the checks."""
    y = copy.copy(x)
    y.C, y.new, y.old, y.first, y.masks = 1, [x.new[c]], [x.old[c]], [x.first[c]], [x.masks[c]]
    y.np_table = x.np_table[c:c + 1]
    return y


def _check_weights(x, q, lse, w, before, decay, which=None):
    """Weights of Case x's requests against the oracle, rows behind the new ones against what they were."""
    scale = 1 / math.sqrt(x.D)
    hw, hq, z = w.cpu().numpy().astype(np.float64), x.host(q).astype(np.float64), lse.cpu().numpy().astype(np.float64)
    k, hb = x.host(x.k), before.cpu().numpy()
    for c in range(x.C) if which is None else which:
        n, r = x.old[c] + x.new[c], slice(x.first[c], x.first[c] + x.new[c])
        kc, seen = op.rows_of(k, x.np_table, c, n), op.sees(x.old[c], x.new[c], x.masks[c])
        want = op.weights(hq[r], kc, seen, z[r], scale, hb[c], x.old[c], decay)
        ab = np.abs(hq[r]).max(initial=0) * np.abs(kc).sum(-1).max(initial=0) * scale
        arg = 2 * (ab + np.abs(np.where(np.isfinite(z[r]), z[r], 0)).max(initial=0))
        rel = x.D * 2 * E32 * ab + arg * 2.0 ** -22 + 2.0 ** -20 + x.new[c] * (x.Hq // x.Hkv) * E32
        assert (np.abs(hw[c, :, :n] - want) <= rel * want + 1e-30).all(), c
        np.testing.assert_array_equal(hw[c, :, n:], hb[c, :, n:])


# ------------------------------------------------------------------------------ two tiles to a CTA

PAIRS = [
    dict(new=[2050], old=[300], Hq=32, Hkv=8, page=64, ragged=False),                    # an odd number of tiles
    # last pairs of one tile, a request of one row, one without a token
    dict(new=[700, 33, 0, 300, 65], old=[900, 0, 50, 129, 1000], Hq=32, Hkv=8, page=64, pad=(2, 3)),
    dict(new=[33] * 8, old=[4063 - 500 * c for c in range(8)], Hq=32, Hkv=8, page=64),  # chunks through memory
    dict(new=[65 - c for c in range(16)], old=[1435 - 80 * c for c in range(16)], S=65, tree=True, Hq=32, Hkv=8,
         page=64),
    dict(new=[530, 1], old=[370, 800], Hq=40, Hkv=8, page=16),                           # 25 tokens of 5 heads: 125 rows
    dict(new=[1000], old=[300], Hq=128, Hkv=8, page=32, ragged=False),
]


def _pairs(dd, i, seed):  # noqa: F811
    x = Case(dd, seed=seed + i, **PAIRS[i]).fill()
    plan = _plan(dd, x)
    assert plan.tiles_per_cta == 2 and (plan.part_bytes > 0) == (i == 2)
    return x


def _attend(x, scale=None):
    lse = torch.full((x.T, x.Hq), 5.0, device="cuda")
    out = torch.full((x.T, x.Hq, x.D), 5.0, device="cuda", dtype=torch.bfloat16)
    x.cache.attention(x.q, tree=x.tree, scale=scale, out=out, lse=lse)
    x.ok()
    _check_attention(x, out, lse, scale=scale, most=8)
    return out, lse


def _keys(x, c, rows, values):
    p, r = op.place(x.np_table, c, np.asarray(rows), x.page)
    x.k[torch.from_numpy(p.astype(np.int64)).cuda(), :, torch.from_numpy(r).cuda()] = values


@pytest.mark.parametrize("i", range(len(PAIRS)))
def test_two_tiles_a_cta(dd, i):  # noqa: F811
    x = _pairs(dd, i, 200)
    out, lse = _attend(x)
    used = np.zeros(x.T, bool)
    for c in range(x.C):
        used[x.first[c]:x.first[c] + x.new[c]] = True
    rest = torch.from_numpy(~used).cuda()
    fill = 5 if x.q_start is not None else 0               # rows outside a ragged batch stay, slots without a node are 0
    assert (out[rest] == fill).all() and (lse[rest] == fill).all()
    for _ in range(5):
        z = torch.empty_like(lse)
        assert torch.equal(x.cache.attention(x.q, tree=x.tree, lse=z)[~rest], out[~rest])
        assert torch.equal(z[~rest], lse[~rest])


@pytest.mark.parametrize("i", range(len(PAIRS)))
@pytest.mark.parametrize("fall", [False, True])
def test_two_tiles_maximum_that_keeps_growing(dd, i, fall):  # noqa: F811
    x = _pairs(dd, i, 220)
    for c in range(x.C):
        n = x.old[c] + x.new[c]
        ramp = torch.linspace(-1, 1, n, device="cuda")[:, None, None] * (-6 if fall else 6)
        _keys(x, c, range(n), (x.rand(n, x.Hkv, x.D).float() * 0.2 + ramp).to(torch.bfloat16))
    x.q.copy_((x.q.float() * 0.2 + 1).to(torch.bfloat16))
    _attend(x)


@pytest.mark.parametrize("i", [1, 2, 4])
@pytest.mark.parametrize("at", [0, 63, 64, 127, 200])
def test_two_tiles_a_key_far_above_the_others(dd, i, at):  # noqa: F811
    """Both halves of a block of keys; a second key as far above the first."""
    x = _pairs(dd, i, 230 + at)
    x.q.copy_((x.q.float() * 0.1 + 1).to(torch.bfloat16))
    for c in range(x.C):
        n = x.old[c] + x.new[c]
        for j, v in ((at, 7.0), (at + 97, 14.0)):
            if j < n:
                _keys(x, c, [j], v)
    _attend(x)


@pytest.mark.parametrize("scale,scaleq", [(1.0, 8.0), (0.02, 1.0)])
def test_two_tiles_scales(dd, scale, scaleq):  # noqa: F811
    for i in (1, 2, 3):
        x = Case(dd, seed=260 + i, scaleq=scaleq, **PAIRS[i]).fill()
        assert _plan(dd, x).tiles_per_cta == 2
        _attend(x, scale)


def test_two_tiles_of_bad_tables_and_lengths(dd):  # noqa: F811
    x = _pairs(dd, 1, 270)
    good = int(x.table[0, 1])
    lse, out = torch.zeros(x.T, x.Hq, device="cuda"), torch.zeros_like(x.q)
    for bad in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        x.table[0, 1] = bad
        x.cache.attention(x.q, out=out, lse=lse)
        assert _status(dd, x) == dd.EINTERNAL
        assert torch.isfinite(out.float()).all()
        for c in (1, 3, 4):
            _check_attention(_one(x, c), out, lse, most=4)
    x.table[0, 1] = good
    for ctx in (x.cache.rows - 1, x.cache.rows + 5, -1, 2 ** 31 - 1, -2 ** 31):
        x.n_ctx[0] = ctx
        x.cache.attention(x.q, out=out, lse=lse)
        assert _status(dd, x) == dd.EINTERNAL
        for c in (1, 3, 4):
            _check_attention(_one(x, c), out, lse, most=4)
    x.n_ctx[0] = 900
    was = x.q_start.clone()
    for j, v in ((0, -3), (1, 10 ** 6), (5, x.T + 9), (3, 0), (0, 2 ** 31 - 1), (5, -2 ** 31)):
        x.q_start[j] = v
        x.cache.attention(x.q)
        assert _status(dd, x) == dd.EINTERNAL
        x.q_start.copy_(was)
    _attend(x)


# ------------------------------------------------------------------------------ tables wider than the contexts

WIDE = [
    dict(new=[1, 1], old=[130, 700], Hq=4, Hkv=1, D=64, page=256, spare=60000),
    dict(new=[1], old=[2047], Hq=32, Hkv=8, page=256, spare=30000),
    dict(new=[1] * 3, old=[500, 0, 127], Hq=8, Hkv=2, page=256, ragged=False, spare=16000),
    dict(new=[65], old=[700], S=65, tree=True, Hq=32, Hkv=8, page=256, spare=16000),
    dict(new=[20, 9], old=[300, 128], S=20, tree=True, Hq=8, Hkv=2, D=64, page=128, spare=16000),
    dict(new=[300, 2], old=[0, 600], Hq=8, Hkv=2, page=256, spare=16000),
    dict(new=[600], old=[100], Hq=32, Hkv=8, page=256, ragged=False, spare=8000),
]


@pytest.mark.parametrize("i", range(len(WIDE)))
def test_tables_much_wider_than_the_contexts(dd, i):  # noqa: F811
    """Chunks without a key, entries behind the last row that are no page."""
    x = Case(dd, seed=280 + i, **WIDE[i]).fill()
    for c in range(x.C):
        x.table[c, -(-(x.old[c] + x.new[c]) // x.page):] = -7
    out, lse = _attend(x)
    before = torch.rand(x.C, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    w = before.clone()
    x.cache.weights(x.q, lse, w, tree=x.tree, decay=0.5)
    x.ok()
    _check_weights(x, x.q, lse, w, before, 0.5)


# ------------------------------------------------------------------------------ what the device checks

def test_the_other_requests_of_a_bad_table_entry_are_right(dd):  # noqa: F811
    x = Case(dd, [3, 4], [40, 300], seed=290).fill()
    before = torch.rand(x.C, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    for bad in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        x.table[0, 1] = bad
        lse = torch.empty(x.T, x.Hq, device="cuda")
        out = x.cache.attention(x.q, lse=lse)
        assert _status(dd, x) == dd.EINTERNAL
        _check_attention(_one(x, 1), out, lse)
        w = before.clone()
        x.cache.weights(x.q, lse, w, decay=0.5)
        assert _status(dd, x) == dd.EINTERNAL
        _check_weights(x, x.q, lse, w, before, 0.5, [1])
        # append: every row of the batch's queries, and the other request's rows, as with a good table
        k, v = x.rand(x.T, x.Hkv, x.D), x.rand(x.T, x.Hkv, x.D)
        keep = x.table.clone()
        x.table[0, 2] = bad                                  # the new tokens' page
        pools = x.k.clone(), x.v.clone()
        got = x.cache.append(x.q, k, v)
        assert _status(dd, x) == dd.EINTERNAL
        mine = x.k.clone(), x.v.clone()
        x.k.copy_(pools[0]), x.v.copy_(pools[1]), x.table.copy_(torch.from_numpy(x.np_table))
        want = x.cache.append(x.q, k, v)
        assert _status(dd, x) == 0 and torch.equal(got, want)
        pg = int(x.np_table[0, 2])
        for a, b, was in ((mine[0], x.k, pools[0]), (mine[1], x.v, pools[1])):
            rest = [p for p in range(x.n_pages) if p != pg]
            np.testing.assert_array_equal(x.host(a[rest]), x.host(b[rest]))
            np.testing.assert_array_equal(x.host(a[pg]), x.host(was[pg]))
        x.table.copy_(keep)


CTX = [lambda x: x.cache.rows - 1, lambda x: x.cache.rows + 5, lambda x: -1, lambda x: 2 ** 31 - 1, lambda x: -2 ** 31]


@pytest.mark.parametrize("b", range(len(CTX)))
def test_weights_of_lengths_that_do_not_fit(dd, b):  # noqa: F811
    x = Case(dd, [5, 3], [20, 40], seed=300 + b).fill()
    lse = torch.empty(x.T, x.Hq, device="cuda")
    x.cache.attention(x.q, lse=lse)
    before = torch.rand(x.C, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    w = before.clone()
    x.n_ctx[0] = CTX[b](x)
    x.cache.weights(x.q, lse, w, decay=0.5)
    assert _status(dd, x) == dd.EINTERNAL
    _check_weights(x, x.q, lse, w, before, 0.5, [1])
    if CTX[b](x) < 0:                                        # taken for 0: the rows behind the new ones stay
        assert torch.equal(w[0, :, 5:], before[0, :, 5:])


def test_weights_of_a_bad_q_start(dd):  # noqa: F811
    x = Case(dd, [5, 3], [20, 40], seed=310).fill()
    lse = torch.empty(x.T, x.Hq, device="cuda")
    x.cache.attention(x.q, lse=lse)
    before = torch.rand(x.C, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    for st in ([0, 9, 8], [-3, 5, 8], [0, 5, 50], [5, 2, 8], [2 ** 31 - 1, -2 ** 31, 8]):
        x.q_start.copy_(torch.tensor(st, dtype=torch.int32))
        w = before.clone()
        x.cache.weights(x.q, lse, w, decay=0.5)
        assert _status(dd, x) == dd.EINTERNAL, st
        for c in range(2):                                   # at most S new rows
            assert torch.equal(w[c, :, x.old[c] + x.S:], before[c, :, x.old[c] + x.S:])
            assert not torch.isnan(w[c, :, :x.old[c]]).any()


@pytest.mark.parametrize("b", range(1, len(CTX)))
def test_eviction_of_lengths_that_do_not_fit(dd, b):  # noqa: F811
    """A length is taken for 0 or the capacity and reported; the other request as ever."""
    x, w, dst = _evict_case(dd, [64, 50], 32, 3, 4, seed=320 + b)
    bk, bv = x.host(x.k), x.host(x.v)
    n = CTX[b](x)
    x.n_ctx[0] = n
    r = x.cache.evict(torch.from_numpy(w).cuda(), 32, dst, 3, 4)
    assert _status(dd, x) == dd.EINTERNAL
    x.old[0] = min(max(n, 0), x.cache.rows)
    _check_evict(x, w, r, 32, 3, 4, bk, bv)


@pytest.mark.parametrize("b", range(len(CTX)))
def test_commit_of_lengths_that_do_not_fit(dd, b):  # noqa: F811
    x = Case(dd, [9, 9], [20, 35], S=9, seed=330 + b, ragged=False).fill()
    path = torch.tensor([[2, 5], [3, 8]], dtype=torch.int32).cuda()
    w = torch.rand(x.C, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    want, bk, bv = w.cpu().numpy().copy(), x.host(x.k), x.host(x.v)
    n, rows = CTX[b](x), x.cache.rows
    x.n_ctx[0] = n
    got = x.cache.commit(path, torch.tensor([2, 2], dtype=torch.int32).cuda(), weights=w)
    assert _status(dd, x) == dd.EINTERNAL
    x.old[0] = min(max(n, 0), rows)
    assert got.tolist() == [min(x.old[0] + 3, rows), 38]
    for c in range(2):
        moves = [(x.old[c] + int(s), x.old[c] + 1 + i) for i, s in enumerate(path[c].tolist())]
        moves = [m for m in moves if max(m) < rows]          # rows past the capacity are not moved
        if moves:
            src, dst = [m[0] for m in moves], [m[1] for m in moves]
            want[c][:, dst] = want[c][:, src].copy()
            (sp, sr), (dp, dr) = op.place(x.np_table, c, src, x.page), op.place(x.np_table, c, dst, x.page)
            for pool in (bk, bv):
                pool[dp, :, dr] = pool[sp, :, sr].copy()
    np.testing.assert_array_equal(x.host(x.k), bk)
    np.testing.assert_array_equal(x.host(x.v), bv)
    np.testing.assert_array_equal(w.cpu().numpy(), want)


@pytest.mark.parametrize("path,acc,moves,n", [
    ([0, 4], 2, {12: 14}, 13), ([3, 9], 2, {11: 13}, 13), ([-1, 5], 2, {12: 15}, 13), ([-1, 2], 1, {}, 12),
    ([4, 7], -1, {}, 11), ([4, 7], 3, {11: 14, 12: 17}, 13), ([2 ** 31 - 1, 8], 2, {12: 18}, 13),
    ([-2 ** 31, -2 ** 31], 2 ** 31 - 1, {}, 13)])
def test_only_the_slots_a_path_names_move(dd, path, acc, moves, n):  # noqa: F811
    """Nine slots behind ten rows: entries that are no slot leave their rows, the others move exactly."""
    x = Case(dd, [9], [10], S=9, seed=340, ragged=False).fill()
    w = torch.rand(1, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    want, bk, bv = w.cpu().numpy().copy(), x.host(x.k), x.host(x.v)
    got = x.cache.commit(torch.tensor([path], dtype=torch.int32).cuda(), torch.tensor([acc], dtype=torch.int32).cuda(),
                         weights=w)
    assert _status(dd, x) == dd.EINTERNAL
    assert int(got[0]) == n
    src, dst = list(moves.values()), list(moves)
    if moves:
        want[0][:, dst] = want[0][:, src].copy()
        (sp, sr), (dp, dr) = op.place(x.np_table, 0, src, x.page), op.place(x.np_table, 0, dst, x.page)
        for pool in (bk, bv):
            pool[dp, :, dr] = pool[sp, :, sr].copy()
    np.testing.assert_array_equal(x.host(x.k), bk)
    np.testing.assert_array_equal(x.host(x.v), bv)
    np.testing.assert_array_equal(w.cpu().numpy(), want)


@pytest.mark.parametrize("old,budget,sink,recent,page", [([1500, 90], 77, 3, 9, 32), ([60000], 700, 3, 5, 256)])
def test_eviction_by_weights_off_a_16_byte_boundary(dd, old, budget, sink, recent, page):  # noqa: F811
    x, w, dst = _evict_case(dd, old, budget, sink, recent, seed=350, page=page, Hkv=1)
    bk, bv = x.host(x.k), x.host(x.v)
    room = torch.empty(w.size + 1, device="cuda")
    view = room[1:].view(w.shape)
    view.copy_(torch.from_numpy(w))
    assert view.data_ptr() % 16 == 4
    r = x.cache.evict(view, budget, dst, sink, recent)
    x.ok()
    _check_evict(x, w, r, budget, sink, recent, bk, bv)


# ------------------------------------------------------------------------------ no tokens, no requests

def test_a_step_without_tokens_decays_the_weights(dd):  # noqa: F811
    x = Case(dd, [0, 0], [40, 300], S=3, seed=355).fill()
    w = torch.rand(x.C, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    before, lse = w.clone(), torch.empty(0, x.Hq, device="cuda")
    assert x.T == 0
    x.cache.append(x.q, x.rand(0, x.Hkv, x.D), x.rand(0, x.Hkv, x.D))
    x.cache.attention(x.q, lse=lse)
    x.cache.weights(x.q, lse, w, decay=0.25)
    x.ok()
    for c, n in enumerate(x.old):
        assert torch.equal(w[c, :, :n], before[c, :, :n] * 0.25) and torch.equal(w[c, :, n:], before[c, :, n:])


def test_a_batch_without_requests(dd):  # noqa: F811
    x = Case(dd, [3], [20], seed=356).fill()
    none = lambda *s, t=torch.int32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    cache = dd.PagedCache(x.k, x.v, none(0, 4), none(0), x.Hq, 1)
    q, k, w = x.rand(0, x.Hq, x.D), x.rand(0, x.Hkv, x.D), none(0, x.Hkv, cache.rows, t=torch.float32)
    pools = x.host(x.k), x.host(x.v)
    cache.append(q, k, k)
    assert cache.attention(q).shape == q.shape
    cache.weights(q, none(0, x.Hq, t=torch.float32), w)
    assert cache.commit(none(0, 2), none(0), weights=w).shape == (0,)
    assert cache.evict(w, 5, none(0, 1))["keep"].shape == (0, x.Hkv, 5)
    torch.cuda.synchronize()
    assert dd.read_status(cache.ws) == 0
    np.testing.assert_array_equal(x.host(x.k), pools[0])
    np.testing.assert_array_equal(x.host(x.v), pools[1])


# ------------------------------------------------------------------------------ streams and graphs

def test_eviction_and_commit_on_a_side_stream(dd):  # noqa: F811
    side = torch.cuda.Stream()
    x, w, dst = _evict_case(dd, [900, 40, 333], 100, 4, 16, seed=360)
    bk, bv = x.host(x.k), x.host(x.v)
    dw = torch.from_numpy(w).cuda()
    torch.cuda.synchronize()
    r = x.cache.evict(dw, 100, dst, 4, 16, stream=side)
    side.synchronize()
    x.ok()
    _check_evict(x, w, r, 100, 4, 16, bk, bv)
    y = Case(dd, [9, 9], [20, 35], S=9, seed=361, ragged=False).fill()
    bk, bv = y.host(y.k), y.host(y.v)
    path, acc = torch.tensor([[2, 5], [3, -1]], dtype=torch.int32).cuda(), torch.tensor([2, 1], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    n = y.cache.commit(path, acc, stream=side)
    side.synchronize()
    y.ok()
    assert n.tolist() == [23, 37]
    for c, a in ((0, 2), (1, 1)):
        src, to, _ = op.commit_moves(path[c].tolist(), a, y.old[c])
        (sp, sr), (dp, dr) = op.place(y.np_table, c, src, y.page), op.place(y.np_table, c, to, y.page)
        for pool in (bk, bv):
            pool[dp, :, dr] = pool[sp, :, sr].copy()
    np.testing.assert_array_equal(y.host(y.k), bk)
    np.testing.assert_array_equal(y.host(y.v), bv)


def test_caches_on_streams_at_once(dd):  # noqa: F811
    """Trees in clusters, single tokens, a prompt's weights shared by clusters and a chunk through memory, each
    with a workspace of its own on a stream of its own, give what they give alone."""
    cases = [dict(new=[65] * 4, old=[1900, 1500, 1000, 700], S=65, tree=True, Hq=32, Hkv=8, page=64),
             dict(new=[1] * 3, old=[2000, 900, 50], Hq=32, Hkv=8, page=64, ragged=False),
             dict(new=[500], old=[1], Hq=32, Hkv=8, page=64, ragged=False),
             dict(new=[33] * 8, old=[4063] * 8, Hq=32, Hkv=8, page=64)]
    xs = [Case(dd, seed=380 + i, **kw).fill() for i, kw in enumerate(cases)]
    ways = [_plan(dd, x) for x in xs]
    assert ways[0].cluster and ways[1].few and ways[3].part_bytes > 0

    def step(x, stream=None):
        lse = torch.empty(x.T, x.Hq, device="cuda") if stream is None else x.lse
        w = torch.zeros(x.C, x.Hkv, x.cache.rows, device="cuda") if stream is None else x.w
        out = x.cache.attention(x.q, tree=x.tree, out=None if stream is None else x.out, lse=lse, stream=stream)
        x.cache.weights(x.q, lse, w, tree=x.tree, decay=0.0 if stream is not None else 1.0, stream=stream)
        return out, lse, w

    alone = [step(x) for x in xs]
    for x, a in zip(xs, alone):
        x.ok()
        _check_attention(x, a[0], a[1], most=4)
        x.out, x.lse, x.w = (torch.zeros_like(t) for t in a)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(40):
        for x, s in zip(xs, streams):
            step(x, s)
    torch.cuda.synchronize()
    for x, a in zip(xs, alone):
        x.ok()
        assert torch.equal(x.out, a[0]) and torch.equal(x.lse, a[1]) and torch.equal(x.w, a[2])


def test_a_captured_commit_and_eviction(dd):  # noqa: F811
    """Captured together, the commit's lengths feeding the eviction; replayed on other paths, weights, lengths
    and rows."""
    budget, sink, recent, S, L = 40, 2, 5, 9, 4
    x, w, dst = _evict_case(dd, [200, 60, 30], budget, sink, recent, seed=370)
    n_ctx = torch.zeros(3, dtype=torch.int32, device="cuda")
    tree = dd.PagedCache(x.k, x.v, x.table, n_ctx, x.Hq, S)
    after = dd.PagedCache(x.k, x.v, x.table, x.n_ctx, x.Hq, 1, ws=tree.ws)
    dw = torch.from_numpy(w).cuda()
    path, acc = torch.full((3, L), -1, dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    keep, n_out = torch.empty(3, x.Hkv, budget, dtype=torch.int32, device="cuda"), torch.empty_like(n_ctx)
    w_out = torch.zeros(3, x.Hkv, dst.shape[1] * x.page, device="cuda")

    def step():
        tree.commit(path, acc, n_out=x.n_ctx, weights=dw)
        return after.evict(dw, budget, dst, sink, recent, keep=keep, n_out=n_out, weights_out=w_out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step()
    for i in range(4):
        old = [int(v) for v in x.rng.integers(1, [180, 50, 20])]
        n_ctx.copy_(torch.tensor(old, dtype=torch.int32))
        hp = np.full((3, L), -1, np.int32)
        ha = [int(a) for a in x.rng.integers(0, L + 1, 3)]
        for c in range(3):
            hp[c, :ha[c]] = np.sort(x.rng.choice(np.arange(1, S), ha[c], replace=False))
        path.copy_(torch.from_numpy(hp)), acc.copy_(torch.tensor(ha, dtype=torch.int32))
        w = x.rng.random(w.shape).astype(np.float32)
        dw.copy_(torch.from_numpy(w))
        x.k.copy_(x.rand(*x.k.shape)), x.v.copy_(x.rand(*x.v.shape))
        w_out.zero_()
        bk, bv = x.host(x.k), x.host(x.v)
        graph.replay()
        torch.cuda.synchronize()
        assert dd.read_status(tree.ws) == 0
        for c in range(3):
            src, to, x.old[c] = op.commit_moves(hp[c], ha[c], old[c])
            w[c][:, to] = w[c][:, src].copy()
            (sp, sr), (dp, dr) = op.place(x.np_table, c, src, x.page), op.place(x.np_table, c, to, x.page)
            for pool in (bk, bv):
                pool[dp, :, dr] = pool[sp, :, sr].copy()
        np.testing.assert_array_equal(dw.cpu().numpy(), w)
        assert x.n_ctx.tolist() == x.old
        _check_evict(x, w, r, budget, sink, recent, bk, bv)
