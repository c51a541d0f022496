"""A batch of requests behind one prefix served step by step with the calls as they are used together: pages
reserved, tokens appended and attended with the prefix read once, tokens drawn, trees verified by draws, their paths
committed, pages given back. Every step is checked against the oracles; every page has one owner."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import paged as op  # noqa: E402
from oracle import serving as sv  # noqa: E402

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


def _dev(a, dt=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dt))).cuda()


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _trees(rng, C, S, L, V):
    t = {k: np.full((C, S), -1, np.int64) for k in ("tok", "par", "depth")}
    mask, n = np.zeros((C, S, S), np.uint8), rng.integers(2, S + 1, C)
    for c in range(C):
        t["tok"][c, 0] = t["depth"][c, 0] = 0
        mask[c, 0, 0] = 1
        toks = rng.choice(V, S, replace=False)
        for j in range(1, n[c]):
            ok = [i for i in range(max(0, j - 4), j) if t["depth"][c, i] < L]
            p = int(rng.choice(ok or [0]))
            t["par"][c, j], t["depth"][c, j], t["tok"][c, j] = p, t["depth"][c, p] + 1, toks[j]
            mask[c, j] = mask[c, p]
            mask[c, j, j] = 1
    d = {k: _dev(v) for k, v in t.items()}
    d.update(n_nodes=_dev(n), pos=_dev(t["depth"]), mask=torch.from_numpy(mask).cuda())
    return dict(t, n_nodes=n, mask=mask), d


@pytest.mark.parametrize("S,Hq,D", [(9, 4, 64), (20, 8, 128)])    # few rows of a head; more than that
def test_steps_of_a_batch_behind_one_prefix(dd, S, Hq, D):
    C, Hkv, page, L, V, prefix, steps = 5, 2, 16, 6, 300, 100, 5
    rng, gen = np.random.default_rng(S), torch.Generator(device="cuda").manual_seed(S)
    width, n_pages = 24, 90
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    k, v = (torch.full((n_pages, Hkv, page, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    # the prefix: whole pages in common, the rest of it in every request's own page
    whole = prefix // page
    order = rng.permutation(n_pages)
    table = np.full((C, width), -1, np.int64)
    table[:, :whole], table[:, whole] = order[:whole], order[whole:whole + C]
    rows = rand(prefix, Hkv, D), rand(prefix, Hkv, D)
    for c in range(C):
        p, r = op.place(table, c, np.arange(prefix), page)
        p, r = _dev(p, np.int64), _dev(r, np.int64)
        k[p, :, r], v[p, :, r] = rows
    stack = order[whole + C:].tolist()
    free, n_free = _dev(stack + [0] * (n_pages - len(stack))), _dev([len(stack)])
    d_table, n_ctx = _dev(table), _dev([prefix] * C)
    old = np.full(C, prefix)
    shared_rows = _dev([whole * page] * C)
    one = dd.PagedCache(k, v, d_table, n_ctx, Hq, 1)                    # single tokens
    many = dd.PagedCache(k, v, d_table, n_ctx, Hq, S)                   # trees
    groups = [x.shared(_dev([0, C]), _dev([prefix]), always=True) for x in (one, many)]
    proj = torch.randn(Hq * D, V, generator=gen, device="cuda") * 0.4
    for step in range(steps):
        tree_step = step % 2 == 1
        x, s, n_new = (many, groups[1], None) if tree_step else (one, groups[0], np.ones(C, np.int64))
        tree = d_tree = None
        if tree_step:
            tree, d_tree = _trees(rng, C, S, L, V)
            n_new = tree["n_nodes"]
        # pages for the step
        want = sv.reserve(table, old, n_new, stack, page, x.S, x.T, True)
        got = x.reserve(_dev(n_new), free, n_free, out=dict(
            granted=torch.zeros(C, dtype=torch.int32, device="cuda"), slot=torch.zeros(x.T, dtype=torch.int64, device="cuda"),
            pos=torch.zeros(x.T, dtype=torch.int32, device="cuda"), request=None, n_free=n_free))
        np.testing.assert_array_equal(d_table.cpu().numpy(), want["table"])
        np.testing.assert_array_equal(got["slot"].cpu().numpy(), want["slot"])
        assert got["granted"].tolist() == list(n_new) and n_free.item() == want["n_free"]
        table, stack = want["table"], stack[:want["n_free"]]
        # tokens into the cache, attention
        q = x.append(rand(x.T, Hq, D), rand(x.T, Hkv, D), rand(x.T, Hkv, D), tree=d_tree)
        lse = torch.zeros(x.T, Hq, device="cuda")
        o = x.attention(q, tree=d_tree, shared=s, lse=lse)
        assert dd.read_status(x.ws) == 0 and dd.read_status(s.ws) == 0
        hk, hv, hq, ho = _host(k), _host(v), _host(q), _host(o)
        for c in range(C):
            n = int(old[c] + n_new[c])
            kc, vc = op.rows_of(hk, table, c, n), op.rows_of(hv, table, c, n)
            mine = slice(c * x.S, c * x.S + int(n_new[c]))
            seen = op.sees(int(old[c]), int(n_new[c]), None if tree is None else tree["mask"][c])
            wo, _, mag, ab = op.attention(hq[mine], kc, vc, seen, D ** -0.5)
            # (as for the plain call: weights rounded to bf16, scores off by D sums, one rounding of the output)
            inner = (E16 + 2 * D * 2 * E32 * ab[..., None] + 2.0 ** -18) * mag
            assert (np.abs(ho[mine] - wo) <= inner + E16 * (np.abs(wo) + inner)).all(), (step, c)
        # what the rows of the tokens say, drawn
        logits = o.float().view(x.T, Hq * D) @ proj
        kw = dict(temperature=0.8, top_k=40, top_p=0.9)
        as64 = dict(temperature=float(np.float32(0.8)), top_k=40, top_p=float(np.float32(0.9)))
        if not tree_step:
            u = torch.rand(C, generator=gen, device="cuda")
            tok = dd.sample(logits, u, **kw).tolist()
            for c in range(C):
                assert tok[c] == sv.draw(logits[c].cpu().numpy(), float(u[c]), **as64)[0]
            n_ctx += 1
            old = old + 1
            continue
        target = logits.view(C, S, V)
        for c in range(C):                                              # the target likes one path of each tree
            for j in range(1, int(n_new[c])):
                target[c, tree["par"][c, j], tree["tok"][c, j]] += 8.0
        u = torch.rand(C, S, generator=gen, device="cuda")
        r = dd.verify_filtered(d_tree, target, dd.ROWS_PER_NODE, L, u, **kw)
        walk = sv.verify(tree, target.cpu().numpy(), "node", L, u.cpu().numpy(), lambda c: as64)
        for key in walk:
            np.testing.assert_array_equal(r[key].cpu().numpy(), walk[key], err_msg=key)
        # the accepted path behind the root, the other slots' pages back
        held = _dev(old + n_new)
        before = _host(k)
        x.commit(r["path"], r["accepted_len"], n_out=n_ctx)
        x.release(held, n_ctx, free, n_free, n_shared=shared_rows, n_out=n_free)
        stack = sv.release(table, old + n_new, old + 1 + walk["accepted_len"], [whole * page] * C, stack, page)
        assert free[:len(stack)].tolist() == stack and n_free.item() == len(stack)
        after = _host(k)
        for c in range(C):
            src, dst, end = op.commit_moves(walk["path"][c], int(walk["accepted_len"][c]), int(old[c]))
            (sp, sr), (dp, dr) = op.place(table, c, src, page), op.place(table, c, dst, page)
            np.testing.assert_array_equal(after[dp, :, dr], before[sp, :, sr])
            old[c] = end
        assert n_ctx.tolist() == old.tolist() and dd.read_status(x.ws) == 0
        # no page has two owners
        own = [int(p) for c in range(C) for p in table[c, whole:-(-int(old[c]) // page)]]
        assert len(set(own + stack + table[0, :whole].tolist())) == len(own) + len(stack) + whole
