"""A step in which the pool does not hold all requests' tokens, taken on through the step's other calls with what was
granted: a refused request's tokens are stored nowhere, although its block table still names pages that others have by
now, and it is served once pages come back. With trees, and with runs of tokens in the fixed layout."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import paged as op  # noqa: E402
from oracle import serving as sv  # noqa: E402
from test_gpu_serving_step import _dev, _host, _trees  # noqa: E402

pytestmark = pytest.mark.gpu
E16, E32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def dd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from diffusion_drafter_draft_gb300 import _build
    _build.build()
    import diffusion_drafter_draft_gb300 as m
    m.lib()
    return m


def _bits(t):
    return t.view(torch.int16).clone()


@pytest.mark.parametrize("kind,S,Hq,D", [("tree", 9, 4, 64), ("tree", 20, 8, 128), ("run", 1, 4, 64), ("run", 3, 4, 128),
                                         ("run", 40, 8, 128), ("run", 70, 4, 64)])
def test_refused_requests_touch_nothing(dd, kind, S, Hq, D):
    C, Hkv, page, L, V, steps, width = 6, 2, 16, 6, 300, 6, 24
    prefix, spare = (111, 2) if S == 1 else (110, 3 if S < 40 else 6)
    rng, gen = np.random.default_rng(S), torch.Generator(device="cuda").manual_seed(S)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    whole = prefix // page
    n_pages = whole + C + spare
    k, v = (torch.full((n_pages, Hkv, page, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    order = rng.permutation(n_pages)
    table = np.empty((C, width), np.int64)
    table[:, :whole], table[:, whole] = order[:whole], order[whole:whole + C]
    for c in range(C):                                                  # what release left there: others' pages
        table[c, whole + 1:] = order[whole + (c + 1) % C]
    rows = rand(prefix, Hkv, D), rand(prefix, Hkv, D)
    for c in range(C):
        p, r = op.place(table, c, np.arange(prefix), page)
        p, r = _dev(p, np.int64), _dev(r, np.int64)
        k[p, :, r], v[p, :, r] = rows
    stack = order[whole + C:].tolist()
    free, n_free = _dev(stack + [0] * (n_pages - len(stack))), _dev([len(stack)])
    old = np.full(C, prefix)
    d_table, n_ctx = _dev(table), _dev(old)
    x = dd.PagedCache(k, v, d_table, n_ctx, Hq, S)
    groups = x.shared(_dev([0, C]), _dev([whole * page]), always=True)
    w = torch.rand(C, Hkv, width * page, generator=gen, device="cuda")
    shared_rows = _dev([whole * page] * C)
    refused = np.zeros(C, int)
    later = 0
    for step in range(steps):
        if step == 3:                                                   # request 0 is done: its pages come back
            x.release(n_ctx, _dev([0] + old[1:].tolist()), free, n_free, n_shared=shared_rows, n_out=n_free)
            stack = sv.release(table, old, [0] + old[1:].tolist(), [whole * page] * C, stack, page)
            old[0] = whole * page
            n_ctx[0] = whole * page
        tree = d_tree = None
        if kind == "tree":
            tree, d_tree = _trees(rng, C, S, L, V)
            n_new = tree["n_nodes"]
        else:
            n_new = rng.integers(0, S + 1, C) if S > 1 else np.ones(C, np.int64)
        if step >= 3:
            n_new = n_new.copy()
            n_new[0] = 0
        want = sv.reserve(table, old, n_new, stack, page, S, C * S, True)
        got = x.reserve(_dev(n_new), free, n_free)
        granted = got["granted"]
        n_free.copy_(got["n_free"])
        np.testing.assert_array_equal(granted.cpu().numpy(), want["granted"])
        table, stack = want["table"], stack[:want["n_free"]]
        g = want["granted"]
        later += int(((refused > 0) & (g > 0)).any())
        refused += (n_new > 0) & (g == 0)
        t = dict(n_nodes=granted) if kind == "run" else dict(d_tree, n_nodes=granted)
        # stored: the granted tokens' rows and nothing else
        bk, bv = _bits(k), _bits(v)
        kn, vn = rand(x.T, Hkv, D), rand(x.T, Hkv, D)
        q = x.append(rand(x.T, Hq, D), kn, vn, tree=t)
        ak, av = _bits(k), _bits(v)
        for c in range(C):
            p, r = op.place(table, c, old[c] + np.arange(g[c]), page)
            p, r = _dev(p, np.int64), _dev(r, np.int64)
            assert torch.equal(v[p, :, r], vn[c * S:c * S + int(g[c])])
            ak[p, :, r], av[p, :, r] = bk[p, :, r], bv[p, :, r]
        assert torch.equal(ak, bk) and torch.equal(av, bv)
        # attended: the granted tokens as ever, zeros for the others, with the prefix shared and without
        hk, hv, hq = _host(k), _host(v), _host(q)
        for s in (None, groups):
            out = torch.full((x.T, Hq, D), 7.0, device="cuda", dtype=torch.bfloat16)
            lse = torch.full((x.T, Hq), 7.0, device="cuda")
            x.attention(q, tree=t, shared=s, out=out, lse=lse)
            assert dd.read_status(x.ws) == 0 and dd.read_status(groups.ws) == 0
            ho = _host(out)
            for c in range(C):
                n, mine = int(g[c]), slice(c * S, c * S + int(g[c]))
                rest = slice(c * S + n, c * S + S)
                assert (out[rest] == 0).all() and (lse[rest] == 0).all()
                if n == 0:
                    continue
                kc, vc = op.rows_of(hk, table, c, int(old[c]) + n), op.rows_of(hv, table, c, int(old[c]) + n)
                seen = op.sees(int(old[c]), n, None if tree is None else tree["mask"][c])
                wo, wz, mag, ab = op.attention(hq[mine], kc, vc, seen, D ** -0.5)
                # (weights rounded to bf16, scores off by D sums, one rounding of the output)
                inner = (E16 + 2 * D * 2 * E32 * ab[..., None] + 2.0 ** -18) * mag
                assert (np.abs(ho[mine] - wo) <= inner + E16 * (np.abs(wo) + inner)).all(), (step, c)
                tz = D * 2 * E32 * ab + (old[c] + n) * E32 + 2.0 ** -20 + np.abs(wz) * 2.0 ** -22
                assert (np.abs(lse[mine].cpu().numpy() - wz) <= tz).all(), (step, c)
        # counted: a refused request's rows only decay
        before = w.clone()
        x.weights(q, lse, w, tree=t, decay=0.5)
        assert dd.read_status(x.ws) == 0
        for c in np.flatnonzero(g == 0):
            o = int(old[c])
            assert torch.equal(w[c, :, :o], before[c, :, :o] * 0.5) and torch.equal(w[c, :, o:], before[c, :, o:])
        if kind == "run":
            n_ctx += granted
            old = old + g
            continue
        # verified, committed, the rejected slots' pages given back: a refused request stays where it was
        target = torch.randn(C, S, V, generator=gen, device="cuda")
        r = dd.verify_filtered(t, target, dd.ROWS_PER_NODE, L, torch.rand(C, S, generator=gen, device="cuda"), top_k=40)
        held = n_ctx + granted
        n_ctx.copy_(torch.where(granted > 0, x.commit(r["path"], r["accepted_len"]), n_ctx))
        x.release(held, n_ctx, free, n_free, n_shared=shared_rows, n_out=n_free)
        assert dd.read_status(x.ws) == 0
        new_old = np.where(g > 0, old + 1 + r["accepted_len"].cpu().numpy(), old)
        stack = sv.release(table, old + g, new_old, [whole * page] * C, stack, page)
        old = new_old
        assert n_ctx.tolist() == old.tolist() and free[:len(stack)].tolist() == stack and n_free.item() == len(stack)
        own = [int(p) for c in range(C) for p in table[c, whole:-(-int(old[c]) // page)]]
        assert len(set(own + stack)) == len(own) + len(stack) == C + spare
    assert refused.any() and later
