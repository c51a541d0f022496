"""The entry points of a serving step reject bad arguments on the host, before any CUDA call (no GPU
needed; the fake pointers are never dereferenced)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dd():
    from diffusion_drafter_draft_gb300 import _build
    _build.build()
    import diffusion_drafter_draft_gb300 as m
    m.lib()
    return m


FAKE, WS = ctypes.c_void_p(256), ctypes.c_void_p(1 << 20)
GOOD = dict(C=2, T=6, S=3, Hq=8, Hkv=2, D=128, page=64, n_pages=8, max_pages=4, dtype=1)
NAN, INF = float("nan"), float("inf")


def _p(dd, **kw):
    return dd.PagedParams(**{**GOOD, **kw})


def _filter(dd, **kw):
    return dd.Filter(**{**dict(temperature=0.7, top_k=20, top_p=0.9, min_p=0.0), **kw})


BAD_FILTERS = [dict(temperature=-1.0), dict(temperature=NAN), dict(temperature=INF), dict(top_k=-1), dict(top_p=-0.1),
               dict(top_p=1.5), dict(top_p=NAN), dict(min_p=-0.1), dict(min_p=1.1), dict(min_p=NAN)]


def test_sample_arguments(dd):
    L = dd.lib()

    def call(x=FAKE, rows=2, V=100, ld=100, dtype=1, f=None, u=FAKE, tok=FAKE, ws=WS, n=256):
        return L.dartree_sample(x, rows, V, ld, dtype, ctypes.byref(f or _filter(dd)), u, tok, ws, n, None)

    for kw in BAD_FILTERS:
        assert call(f=_filter(dd, **kw)) == dd.EINVAL, kw
    for kw in (dict(rows=-1), dict(V=0), dict(ld=99), dict(x=None), dict(x=ctypes.c_void_p(257)), dict(u=None),
               dict(tok=None), dict(x=ctypes.c_void_p(258), dtype=0)):
        assert call(**kw) == dd.EINVAL, kw
    assert L.dartree_sample(FAKE, 2, 100, 100, 1, None, FAKE, FAKE, WS, 256, None) == dd.EINVAL
    assert call(dtype=3) == dd.EDTYPE
    assert call(V=(1 << 20) + 1, ld=1 << 21) == dd.EUNSUPPORTED
    assert call(V=400000, ld=400000, dtype=0) == dd.EUNSUPPORTED
    assert call(rows=1 << 24) == dd.EUNSUPPORTED
    assert call(ws=None) == dd.EWORKSPACE
    assert call(ws=ctypes.c_void_p((1 << 20) + 8)) == dd.EWORKSPACE
    assert call(n=255) == dd.EWORKSPACE
    assert call(rows=0) == dd.OK
    # arrays take the place of numbers
    assert call(rows=0, f=_filter(dd, temperature=NAN, temperatures=256, top_p=NAN, top_ps=256, top_k=-1, top_ks=256,
                                  min_p=NAN, min_ps=256)) == dd.OK


def test_verify_filtered_arguments(dd):
    L = dd.lib()
    tree = dict(tok=256, par=256, depth=256, n_nodes=256)

    def call(p=None, tree=tree, x=FAKE, rows=0, V=100, dtype=1, f=None, u=FAKE, out=FAKE, ws=WS, n=256):
        t = dd.Tree(tree["tok"], tree["par"], tree["depth"], None, tree["n_nodes"], None, None)
        return L.dartree_verify_filtered(ctypes.byref(p or dd.Params(2, 4, 1, 1, 8, 0.0)), ctypes.byref(t), x, rows, V,
                                         dtype, ctypes.byref(f or _filter(dd)), u, out, FAKE, FAKE, ws, n, None)

    for kw in BAD_FILTERS:
        assert call(f=_filter(dd, **kw)) == dd.EINVAL, kw
    for kw in (dict(V=0), dict(x=None), dict(u=None), dict(out=None), dict(x=ctypes.c_void_p(257)),
               dict(p=dd.Params(-1, 4, 1, 1, 8, 0.0)), dict(p=dd.Params(2, 0, 1, 1, 8, 0.0)),
               dict(p=dd.Params(2, 4, 1, 1, 0, 0.0))):
        assert call(**kw) == dd.EINVAL, kw
    for k in tree:
        assert call(tree={**tree, k: None}) == dd.EINVAL, k
    assert call(rows=2) == dd.EDTYPE
    assert call(dtype=2) == dd.EDTYPE
    assert call(p=dd.Params(2, 65, 1, 1, 8, 0.0)) == dd.EUNSUPPORTED
    assert call(p=dd.Params(2, 4, 1, 1, 1024, 0.0)) == dd.EUNSUPPORTED
    assert call(V=(1 << 20) + 1) == dd.EUNSUPPORTED
    assert call(n=255) == dd.EWORKSPACE
    assert call(p=dd.Params(0, 4, 1, 1, 8, 0.0)) == dd.OK


def test_reserve_and_release_arguments(dd):
    L = dd.lib()
    need = L.dartree_paged_workspace_bytes(ctypes.byref(_p(dd)))
    names = ("table", "n_ctx", "n_new", "free_pages", "n_free", "n_free_out", "granted", "q_start", "slot", "pos", "request")

    def res(p=None, n=None, **kw):
        x = dd.PagedStep(**{**{k: 4096 * (i + 1) for i, k in enumerate(names)}, **kw})
        return L.dartree_paged_reserve(ctypes.byref(p or _p(dd)), ctypes.byref(x), WS, need if n is None else n, None)

    for k in ("table", "n_ctx", "n_new", "free_pages", "n_free", "n_free_out", "granted"):
        assert res(**{k: None}) == dd.EINVAL, k
    assert res(granted=3 * 4096 + 4) == dd.EINVAL              # in n_new's last entry
    assert res(slot=4100) == dd.EINVAL
    assert res(p=_p(dd, T=7), q_start=None) == dd.EINVAL
    assert res(p=_p(dd, n_pages=0)) == dd.EINVAL
    assert res(p=_p(dd, max_pages=0)) == dd.EINVAL
    assert res(p=_p(dd, page=24)) == dd.EUNSUPPORTED
    assert res(n=511) == dd.EWORKSPACE
    assert L.dartree_paged_reserve(ctypes.byref(_p(dd)), None, WS, need, None) == dd.EINVAL

    def rel(p=None, n=None, **kw):
        a = {**dict(table=1 << 16, held=4096, keep=8192, shared=None, free=1 << 17, nf=12288, out=12288), **kw}
        return L.dartree_paged_release(ctypes.byref(p or _p(dd)), *(ctypes.c_void_p(a[k]) for k in (
            "table", "held", "keep", "shared", "free", "nf", "out")), WS, need if n is None else n, None)

    for k in ("table", "held", "keep", "free", "nf", "out"):
        assert rel(**{k: None}) == dd.EINVAL, k
    assert rel(free=(1 << 16) + 16) == dd.EINVAL               # in the table
    assert rel(p=_p(dd, n_pages=0)) == dd.EINVAL
    assert rel(n=511) == dd.EWORKSPACE


def test_shared_attention_arguments(dd):
    L = dd.lib()
    g = lambda G=1, most_rows=0, most_rest=0, always=1, start=256, rows=256: dd.PagedGroups(  # noqa: E731
        G, most_rows, most_rest, always, start, rows)
    need = L.dartree_paged_shared_workspace_bytes(ctypes.byref(_p(dd)), ctypes.byref(g()))
    assert need > 512
    m = dd.PagedCacheDesc(256, 256, 256, 256, None)
    at = lambda n: ctypes.c_void_p((1 << 24) + n)  # noqa: E731
    n = 6 * 8 * 128 * 2

    def call(p=None, s=None, q=at(0), m=m, tree=None, scale=0.0, out=at(n), lse=None, bytes_=None):
        return L.dartree_paged_shared_attention(ctypes.byref(p or _p(dd)), q, ctypes.byref(m), tree, ctypes.byref(s or g()),
                                                scale, out, lse, WS, need if bytes_ is None else bytes_, None)

    bad = [dict(G=-1), dict(G=3), dict(most_rows=-1), dict(most_rest=-5)]
    for kw in bad:
        assert call(s=g(**kw)) == dd.EINVAL, kw
        assert L.dartree_paged_shared_workspace_bytes(ctypes.byref(_p(dd)), ctypes.byref(g(**kw))) == 0
        assert L.dartree_paged_shared_plan(ctypes.byref(_p(dd)), ctypes.byref(g(**kw)), ctypes.byref(dd.PagedSharedPlan())) \
            == dd.EINVAL
    for kw in (dict(s=g(start=None)), dict(s=g(rows=None)), dict(q=None), dict(q=at(8)), dict(out=None), dict(out=at(16)),
               dict(lse=at(n - 4)), dict(lse=at(2 * n - 4)), dict(lse=at(2 * n + 2)), dict(scale=-1.0), dict(scale=NAN),
               dict(p=_p(dd, T=7)), dict(m=dd.PagedCacheDesc(256, 256, None, 256, None))):
        assert call(**kw) == dd.EINVAL, kw
    assert call(p=_p(dd, dtype=0)) == dd.EUNSUPPORTED
    assert call(p=_p(dd, D=96)) == dd.EUNSUPPORTED
    assert call(bytes_=need - 1) == dd.EWORKSPACE
    assert call(bytes_=255) == dd.EWORKSPACE
    assert call(p=_p(dd, C=0, T=0), s=g(G=0)) == dd.OK
    assert L.dartree_paged_shared_plan(ctypes.byref(_p(dd)), ctypes.byref(g()), None) == dd.EINVAL


def test_every_way_of_sharing_is_taken(dd):
    """(own rows by the transposed kernel, tiles per CTA, alone): what is compiled is what plans choose; the
    workspace holds what the plan stores, and little more of it than half a gigabyte where chunks are a choice."""
    import random
    rng, taken, used = random.Random(5), {64: set(), 128: set()}, set()
    for _ in range(4000):
        C, S = rng.randint(1, 100), rng.choice([1, 1, 2, int(2 ** rng.uniform(0, 9))])
        Hkv, grp = rng.choice([(1, 8), (2, 5), (4, 4), (8, 4), (8, 1), (4, 7), (2, 16), (1, 1)])
        width = int(2 ** rng.uniform(0, 11))
        for D, seen in taken.items():
            p = dd.PagedParams(C, C * S, S, Hkv * grp, Hkv, D, 64, 1 << 20, width, 1)
            s = dd.PagedGroups(rng.randint(1, C), rng.choice([0, rng.randint(1, 10000)]), rng.choice([0, rng.randint(1, 2000)]),
                               rng.choice([0, 1]), None, None)
            o = dd.PagedSharedPlan()
            assert dd.lib().dartree_paged_shared_plan(ctypes.byref(p), ctypes.byref(s), ctypes.byref(o)) == dd.OK
            need = dd.lib().dartree_paged_shared_workspace_bytes(ctypes.byref(p), ctypes.byref(s))
            assert 256 + o.part_bytes <= need <= 256 + 4 * C + 512 + o.part_bytes
            used.add((bool(s.always), bool(o.use)))
            if o.use:
                seen.add((o.few, o.tiles_per_cta, o.alone))
                row = C * S * Hkv * grp * (D * 4 + 8)
                assert o.part_bytes <= max(512 << 20, 2 * row) * 1.1 + 1024
    assert used == {(True, True), (False, True), (False, False)}
    one = {(f, 1, a) for f in (0, 1) for a in (0, 1)}
    assert taken[64] == one and taken[128] == one | {(0, 2, 0), (1, 2, 0)}


def test_kernel_families_are_named(dd):
    names = [dd.lib().dartree_kernel_name(i).decode() for i in range(dd.num_kernel_ids())]
    for n in ("paged_reserve_kernel", "paged_release_kernel", "sample_kernel", "sample_walk_kernel", "paged_own_kernel"):
        assert n in names


def test_reserve_and_release_sums_and_lengths_apart(dd):
    L = dd.lib()
    ptr = lambda n: ctypes.c_void_p(n)  # noqa: E731
    # 512 requests that give back 2^22 pages each pass 31 bits (whatever the pool holds)
    for C, pages, e in ((512, 1 << 22, dd.EUNSUPPORTED), (4096, 1 << 22, dd.EUNSUPPORTED), (511, 1 << 22, dd.EWORKSPACE),
                        (512, (1 << 22) - 1, dd.EWORKSPACE)):
        p = _p(dd, C=C, T=C, S=1, Hq=1, Hkv=1, page=16, max_pages=pages)
        assert L.dartree_paged_release(ctypes.byref(p), ptr(1 << 44), ptr(4096), ptr(8192), None, ptr(1 << 20), ptr(12288),
                                       ptr(12288), WS, 0, None) == e
    x = dd.PagedStep(table=4096, n_ctx=1 << 20, n_new=1 << 21, free_pages=1 << 22, n_free=256, n_free_out=256,
                     granted=(1 << 20) + 4)                     # lengths are read while grants are written
    assert L.dartree_paged_reserve(ctypes.byref(_p(dd)), ctypes.byref(x), WS, 1 << 20, None) == dd.EINVAL
