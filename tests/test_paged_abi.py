"""The paged-cache entry points reject bad arguments on the host, before any CUDA call
(no GPU needed; the fake pointers are never dereferenced)."""
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


def _p(dd, **kw):
    return dd.PagedParams(**{**GOOD, **kw})


def _m(dd, k=256, v=256, table=256, n_ctx=256, q_start=None):
    return dd.PagedCacheDesc(k, v, table, n_ctx, q_start)


def _x(dd, **kw):
    d = dict(q=256, k=256, v=256, ldq=1024, ldk=256, ldv=256, gq=256, gk=256, pos_base=None, eps=1e-6, theta=1e6)
    return dd.PagedTokens(**{**d, **kw})


def _tree(dd, mask=256, pos=256, n_nodes=256):
    return ctypes.byref(dd.Tree(None, None, None, None, n_nodes, mask, pos))


BAD = [(dict(C=-1), "EINVAL"), (dict(S=0), "EINVAL"), (dict(T=-1), "EINVAL"), (dict(Hq=7), "EINVAL"),
       (dict(Hkv=0), "EINVAL"), (dict(dtype=5), "EDTYPE"), (dict(D=96), "EUNSUPPORTED"),
       (dict(D=256), "EUNSUPPORTED"), (dict(page=8), "EUNSUPPORTED"), (dict(page=48), "EUNSUPPORTED"),
       (dict(page=512), "EUNSUPPORTED"), (dict(Hq=258, Hkv=2), "EUNSUPPORTED"),
       (dict(page=256, max_pages=1 << 23), "EUNSUPPORTED"),   # 2^31 rows
       (dict(C=1 << 15, S=1 << 16, T=1 << 30), "EUNSUPPORTED"),
       (dict(T=(1 << 31) // 8, Hq=8, Hkv=2), "EUNSUPPORTED")]  # T * Hq = 2^31


@pytest.mark.parametrize("kw,err", BAD)
def test_sizes(dd, kw, err):
    L, code, p = dd.lib(), getattr(dd, err), _p(dd, **kw)
    b, m, x = ctypes.byref(p), _m(dd), _x(dd)
    assert L.dartree_paged_workspace_bytes(b) == 0
    assert L.dartree_paged_append(b, ctypes.byref(x), ctypes.byref(m), None, FAKE, WS, 1 << 30, None) == code
    assert L.dartree_paged_attention(b, FAKE, ctypes.byref(m), None, 0.0, FAKE, None, WS, 1 << 30, None) == code
    assert L.dartree_paged_weights(b, FAKE, FAKE, ctypes.byref(m), None, 0.0, 1.0, FAKE, WS, 1 << 30, None) == code
    assert L.dartree_paged_evict(b, ctypes.byref(m), FAKE, 4, 0, 0, FAKE, 9, FAKE, FAKE, None, WS, 1 << 30,
                                 None) == code
    assert L.dartree_paged_commit(b, ctypes.byref(m), FAKE, FAKE, 4, FAKE, WS, 1 << 30, None) == code


def test_append_arguments(dd):
    L = dd.lib()
    need = L.dartree_paged_workspace_bytes(ctypes.byref(_p(dd)))
    assert need > 256

    def call(p=None, x=None, m=None, tree=None, out=FAKE, ws=WS, n=None):
        return L.dartree_paged_append(ctypes.byref(p or _p(dd)), ctypes.byref(x or _x(dd)), ctypes.byref(m or _m(dd)),
                                      tree, out, ws, need if n is None else n, None)

    for kw in (dict(q=None), dict(k=260), dict(v=264), dict(gq=258), dict(ldq=1020), dict(ldq=1016), dict(ldk=248),
               dict(ldv=0), dict(theta=0.0), dict(theta=float("inf")), dict(eps=0.0), dict(eps=float("nan"))):
        assert call(x=_x(dd, **kw)) == dd.EINVAL, kw
    assert call(x=_x(dd, ldq=1032), out=FAKE) == dd.EINVAL     # in place needs packed queries
    for kw in (dict(k=None), dict(v=264), dict(table=None), dict(n_ctx=None)):
        assert call(m=_m(dd, **kw)) == dd.EINVAL, kw
    assert call(p=_p(dd, n_pages=0)) == dd.EINVAL
    assert call(p=_p(dd, max_pages=0)) == dd.EINVAL
    assert call(p=_p(dd, T=5)) == dd.EINVAL                    # T = C * S without q_start
    assert call(m=_m(dd, q_start=256), tree=_tree(dd)) == dd.EINVAL
    assert call(tree=_tree(dd, pos=None)) == dd.EINVAL
    assert call(tree=_tree(dd, n_nodes=None)) == dd.EINVAL
    assert call(out=None) == dd.EINVAL
    assert call(ws=None) == dd.EWORKSPACE
    assert call(n=need - 1) == dd.EWORKSPACE
    assert call(p=_p(dd, C=0, T=0)) == dd.OK


def test_attention_and_weights_arguments(dd):
    L = dd.lib()
    need = L.dartree_paged_workspace_bytes(ctypes.byref(_p(dd)))

    def att(p=None, q=FAKE, m=None, tree=None, scale=0.0, out=FAKE, lse=None, n=None):
        return L.dartree_paged_attention(ctypes.byref(p or _p(dd)), q, ctypes.byref(m or _m(dd)), tree, scale, out, lse,
                                         WS, need if n is None else n, None)

    def wts(p=None, q=FAKE, lse=FAKE, m=None, tree=None, scale=0.0, decay=0.5, w=FAKE, n=None):
        return L.dartree_paged_weights(ctypes.byref(p or _p(dd)), q, lse, ctypes.byref(m or _m(dd)), tree, scale, decay,
                                       w, WS, need if n is None else n, None)

    for f in (att, wts):
        assert f(p=_p(dd, dtype=0)) == dd.EUNSUPPORTED         # bf16 only
        assert f(q=ctypes.c_void_p(264)) == dd.EINVAL
        assert f(q=None) == dd.EINVAL
        assert f(scale=-1.0) == dd.EINVAL
        assert f(scale=float("nan")) == dd.EINVAL
        assert f(tree=_tree(dd, mask=None)) == dd.EINVAL
        assert f(m=_m(dd, q_start=256), tree=_tree(dd)) == dd.EINVAL
        assert f(p=_p(dd, T=7)) == dd.EINVAL
        assert f(n=need - 1) == dd.EWORKSPACE
        assert f(p=_p(dd, C=0, T=0)) == dd.OK
    assert att(out=None) == dd.EINVAL
    assert att(lse=ctypes.c_void_p(258)) == dd.EINVAL
    assert att(p=_p(dd, T=0), m=_m(dd, q_start=256)) == dd.OK  # no new token
    for d in (-0.1, 1.5, float("nan")):
        assert wts(decay=d) == dd.EINVAL
    assert wts(lse=None) == dd.EINVAL
    assert wts(w=None) == dd.EINVAL


def test_evict_and_commit_arguments(dd):
    L = dd.lib()
    need = L.dartree_paged_workspace_bytes(ctypes.byref(_p(dd)))

    def ev(p=None, m=None, w=FAKE, budget=64, sink=4, recent=8, dst=FAKE, pages=1, keep=FAKE, n_out=FAKE, n=None):
        return L.dartree_paged_evict(ctypes.byref(p or _p(dd)), ctypes.byref(m or _m(dd)), w, budget, sink, recent,
                                     dst, pages, keep, n_out, None, WS, need if n is None else n, None)

    for kw in (dict(budget=0), dict(budget=65), dict(sink=-1), dict(recent=-1), dict(sink=60, recent=5),
               dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(pages=0), dict(w=None), dict(dst=None),
               dict(keep=None), dict(n_out=None), dict(m=_m(dd, k=None))):
        assert ev(**kw) == dd.EINVAL, kw
    assert ev(p=_p(dd, C=1 << 12, T=3 << 12, Hq=4096, Hkv=4096), budget=128, pages=2) == dd.EUNSUPPORTED
    assert ev(n=need - 1) == dd.EWORKSPACE
    assert ev(p=_p(dd, C=0, T=0)) == dd.OK

    def cm(p=None, m=None, path=FAKE, acc=FAKE, Lp=16, n_out=FAKE, n=None):
        return L.dartree_paged_commit(ctypes.byref(p or _p(dd)), ctypes.byref(m or _m(dd)), path, acc, Lp, n_out, WS,
                                      need if n is None else n, None)

    for kw in (dict(path=None), dict(acc=None), dict(Lp=0), dict(n_out=None), dict(m=_m(dd, table=None))):
        assert cm(**kw) == dd.EINVAL, kw
    assert cm(Lp=65) == dd.EUNSUPPORTED
    assert cm(n=need - 1) == dd.EWORKSPACE
    assert cm(p=_p(dd, C=0, T=0)) == dd.OK


def test_commit_with_weights_arguments(dd):
    L = dd.lib()
    need = L.dartree_paged_workspace_bytes(ctypes.byref(_p(dd)))

    def cm(p=None, m=None, path=FAKE, acc=FAKE, Lp=16, w=FAKE, n_out=FAKE, n=None):
        return L.dartree_paged_commit_weights(ctypes.byref(p or _p(dd)), ctypes.byref(m or _m(dd)), path, acc, Lp, w,
                                              n_out, WS, need if n is None else n, None)

    for kw in (dict(w=None), dict(path=None), dict(acc=None), dict(Lp=0), dict(n_out=None),
               dict(m=_m(dd, table=None))):
        assert cm(**kw) == dd.EINVAL, kw
    assert cm(Lp=65) == dd.EUNSUPPORTED
    assert cm(n=need - 1) == dd.EWORKSPACE
    assert cm(p=_p(dd, C=0, T=0)) == dd.OK
    assert cm(p=_p(dd, C=0, T=0), path=None, acc=None, w=None, n_out=None) == dd.OK    # empty tensors


def test_outputs_inside_inputs_are_refused(dd):
    """Kernels read these inputs while other CTAs write the outputs."""
    L, p, m = dd.lib(), ctypes.byref(_p(dd)), ctypes.byref(_m(dd))
    need = L.dartree_paged_workspace_bytes(p)
    at = lambda n: ctypes.c_void_p((1 << 24) + n)   # one buffer of q rows: T * Hq * D * 2 bytes
    n = 6 * 8 * 128 * 2

    def app(out, **kw):
        x = _x(dd, **{**dict(q=1 << 24, k=1 << 28, v=1 << 29), **kw})
        return L.dartree_paged_append(p, ctypes.byref(x), m, None, out, WS, need, None)

    assert app(at(16)) == dd.EINVAL
    assert app(at(n - 16)) == dd.EINVAL
    assert app(at(16 - n)) == dd.EINVAL
    assert app(at(0), k=(1 << 24) + n - 16) == dd.EINVAL     # in place, keys in its last bytes
    assert app(at(0), v=(1 << 24) - 6 * 2 * 128 * 2 + 16) == dd.EINVAL
    assert app(at(0), q=(1 << 24) - 2048, ldq=3 * 1024) == dd.EINVAL

    def att(out, lse=None):
        return L.dartree_paged_attention(p, at(0), m, None, 0.0, out, lse, WS, need, None)

    for d in (0, 16, n - 16, 16 - n):
        assert att(at(d)) == dd.EINVAL, d
    assert att(at(n), at(n - 4)) == dd.EINVAL                # lse in q's last bytes
    assert att(at(n), at(n + 64)) == dd.EINVAL               # in out

    def ev(dst, w, wo):
        return L.dartree_paged_evict(p, m, w, 64, 4, 8, dst, 1, FAKE, FAKE, wo, WS, need, None)

    w = 2 * 2 * 4 * 64 * 4                                   # bytes of weights: C, Hkv, max_pages * page floats
    assert ev(FAKE, at(0), None) == dd.EINVAL                # the cache's own table
    assert ev(at(-4096), at(0), at(0)) == dd.EINVAL
    assert ev(at(-4096), at(0), at(w - 4)) == dd.EINVAL
    assert ev(at(-4096), at(0), at(4 - w // 4)) == dd.EINVAL


PLAN_SIZES = dict(C=64, T=64, S=1, Hq=32, Hkv=8, D=128, page=64, n_pages=1 << 20, max_pages=128, dtype=1)


def _plan(dd, **kw):
    p, out = dd.PagedParams(**{**PLAN_SIZES, **kw}), dd.PagedPlan()
    assert dd.lib().dartree_paged_attention_plan(ctypes.byref(p), ctypes.byref(out)) == dd.OK
    return out


def _bytes(dd, **kw):
    n = dd.lib().dartree_paged_workspace_bytes(ctypes.byref(dd.PagedParams(**{**PLAN_SIZES, **kw})))
    assert n > 0
    return n


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv,grp", [(8, 4), (1, 8), (2, 16), (8, 1), (4, 7), (1, 128), (32, 1)])
def test_a_workspace_serves_every_smaller_batch(dd, Hkv, grp, D):
    """The bytes grow with C, S and the table's width, and cover what each batch's own plan stores."""
    heads = dict(Hq=Hkv * grp, Hkv=Hkv, D=D)
    Cs, Ss = (0, 1, 2, 3, 5, 8, 16, 31, 48, 64, 200), (1, 2, 3, 4, 16, 17, 33, 65, 128, 500, 2048)
    pages = (1, 7, 8, 9, 16, 64, 128, 500, 1024, 4096)
    need = {}
    for C in Cs:
        for S in Ss:
            for m in pages:
                b = need[C, S, m] = _bytes(dd, C=C, S=S, T=C * S, max_pages=m, **heads)
                plan = _plan(dd, C=C, S=S, T=C * S, max_pages=m, **heads)
                assert 256 + 4 * C + plan.part_bytes <= b <= 256 + 4 * C + 256 + (140 << 20), (C, S, m)
                for C2, S2, m2 in ((Cs[max(Cs.index(C) - 1, 0)], S, m), (C, Ss[max(Ss.index(S) - 1, 0)], m),
                                   (C, S, pages[max(pages.index(m) - 1, 0)])):
                    assert need[C2, S2, m2] <= b, (C, S, m)


def test_plan_arguments(dd):
    L, out = dd.lib(), dd.PagedPlan()
    ok = _p(dd)
    assert L.dartree_paged_attention_plan(ctypes.byref(ok), None) == dd.EINVAL
    assert L.dartree_paged_attention_plan(None, ctypes.byref(out)) == dd.EINVAL
    assert L.dartree_paged_attention_plan(ctypes.byref(_p(dd, dtype=0)), ctypes.byref(out)) == dd.EUNSUPPORTED
    for kw, err in BAD:
        assert L.dartree_paged_attention_plan(ctypes.byref(_p(dd, **kw)), ctypes.byref(out)) == getattr(dd, err)
    assert _plan(dd).few == 1 and _plan(dd, S=2048, C=1, T=2048).few == 0


def test_every_way_of_the_attention_is_taken(dd):
    """(few, tiles per CTA, chunks through memory, cluster, alone): what is compiled for a head size is
    what its plans choose."""
    import random
    rng, taken = random.Random(3), {64: set(), 128: set()}
    for _ in range(6000):
        C, S = int(2 ** rng.uniform(0, 8)), rng.choice([1, int(2 ** rng.uniform(0, 13))])
        Hkv, grp = rng.choice([(1, 8), (2, 5), (4, 4), (8, 4), (8, 1), (4, 7), (2, 16), (1, 1)])
        for D, seen in taken.items():
            p = _plan(dd, C=C, S=S, T=C * S, Hq=Hkv * grp, Hkv=Hkv, D=D, max_pages=int(2 ** rng.uniform(0, 11)))
            seen.add((p.few, p.tiles_per_cta, int(p.part_bytes > 0), p.cluster, p.alone))
            assert (p.part_bytes > 0) == (p.chunks > 1 and not p.cluster)
    few = {(1, 1, m, c, a) for m, c, a in ((0, 0, 0), (0, 0, 1), (1, 0, 0), (1, 0, 1), (0, 1, 1))}
    one = {(0, 1, m, c, a) for m, c in ((0, 0), (1, 0), (0, 1)) for a in (0, 1)}
    assert taken[64] == few | one
    assert taken[128] == few | one | {(0, 2, 0, 0, 0), (0, 2, 1, 0, 0)}


def test_kernel_families_are_named(dd):
    names = [dd.lib().dartree_kernel_name(i).decode() for i in range(dd.num_kernel_ids())]
    for n in ("append", "attn", "weights", "select", "move", "commit"):
        assert f"paged_{n}_kernel" in names
