"""Parity of the paged-cache calls (dartree_paged_*) with the float64 oracle, through the
C ABI, at the sizes and masks where they can go wrong; every page row that holds nothing
is NaN.

Tolerances (a rounding to bf16 is off by at most 2^-8 relative, to fp32 by 2^-24):
  append     fp32 arithmetic on |y_i| + |y_i+D/2|: mean square (20 additions, halved by the
             root) 10, rsqrt 4, three products 3, the angle's reduction and rounding 2 * 2,
             sine and cosine 2 * 2, the rotation 3 roundings: below 32 * 2^-24 = 2^-19 of
             the pair's magnitudes; then one rounding to the stored type.
  scores     D products summed in fp32, each partial sum off by at most 2^-23 (the tensor
             core may truncate): ds = D * 2^-23 * scale * sum |q_d k_d| (its largest value
             over the row's keys).
  attention  weights rounded to bf16 and formed from scores off by ds: (2^-8 + 2 ds + 2^-18)
             of the mean of |v| under the same weights, then one rounding to bf16.
  lse        ds, the sum of n weights (n * 2^-24) and 2^-20 for the exponentials and the
             logarithm, and 2^-22 of its own value.
  weights    relative: ds, the argument's rounding (|s| + |lse|) * 2^-22 and 2^-20 for the
             exponential; the sum of R terms R * 2^-24.
Copied rows, kept rows and lengths are exact.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import paged as op  # noqa: E402

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


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tree_of(rng, S, n, width=5):
    """One tree of n <= S slots: mask of ancestors, depths (-1 for unused slots)."""
    mask, depth = np.zeros((S, S), np.uint8), np.full(S, -1, np.int32)
    for j in range(n):
        par = -1 if j == 0 else int(rng.integers(max(0, j - width), j))
        depth[j] = 0 if j == 0 else depth[par] + 1
        if par >= 0:
            mask[j] = mask[par]
        mask[j, j] = 1
    return mask, depth


class Case:
    """A batch on the GPU with what the oracle needs of it. new/old: tokens and cached rows per request;
    pad: rows of q before and behind the batch's (ragged batches); spare: capacity rows beyond the last."""

    def __init__(self, dd, new, old, S=None, Hq=4, Hkv=2, D=128, page=16, dtype="bf16", tree=False, ragged=True,
                 seed=0, pad=(0, 0), spare=0, nodes=None, scaleq=1.0):
        self.rng = rng = np.random.default_rng(seed)
        self.new, self.old = list(new), list(old)
        self.C, self.S = len(new), S or max(1, max(new))
        self.Hq, self.Hkv, self.D, self.page, self.dtype = Hq, Hkv, D, page, dtype
        self.tree, self.masks = None, [None] * self.C
        self.q_start = None
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        if tree or not ragged:
            self.first = [c * self.S for c in range(self.C)]
            self.T = self.C * self.S
            if tree:
                t = [_tree_of(rng, self.S, n) for n in new]
                self.masks, self.depth = [m for m, _ in t], [d for _, d in t]
                self.tree = dict(mask=dev(np.stack(self.masks)), pos=dev(np.stack(self.depth)),
                                 n_nodes=dev(np.array(new, np.int32)))
        else:
            st = pad[0] + np.concatenate([[0], np.cumsum(new)])
            self.first, self.T = list(st[:-1]), int(st[-1]) + pad[1]
            self.q_start = dev(st.astype(np.int32))
        width = max(1, -(-(max(o + n for o, n in zip(old, new)) + spare) // page))
        self.n_pages = self.C * width + 3
        self.np_table = rng.permutation(self.n_pages)[:self.C * width].reshape(self.C, width).astype(np.int32)
        self.table, self.n_ctx = dev(self.np_table), dev(np.array(old, np.int32))
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        shape = (self.n_pages, Hkv, page, D)
        self.k, self.v = (torch.full(shape, float("nan"), device="cuda", dtype=DT[dtype]) for _ in range(2))
        self.q = self.rand(self.T, Hq, D, scale=scaleq)
        self.dd = dd
        self.cache = dd.PagedCache(self.k, self.v, self.table, self.n_ctx, Hq, self.S, T=self.T, q_start=self.q_start)

    def rand(self, *s, scale=1.0):
        return (torch.randn(s, generator=self.gen, device="cuda") * scale).to(DT[self.dtype])

    def fill(self, new_too=True):
        """Rows of every request (and of its new tokens) get values."""
        for c in range(self.C):
            n = self.old[c] + (self.new[c] if new_too else 0)
            if n:
                p, r = op.place(self.np_table, c, np.arange(n), self.page)
                p, r = torch.from_numpy(p.astype(np.int64)).cuda(), torch.from_numpy(r).cuda()
                self.k[p, :, r] = self.rand(n, self.Hkv, self.D)
                self.v[p, :, r] = self.rand(n, self.Hkv, self.D)
        return self

    def host(self, t):
        return t.float().cpu().numpy()

    def rows(self, pages, c, n):
        return op.rows_of(self.host(pages), self.np_table, c, n)

    def ok(self):
        torch.cuda.synchronize()
        assert self.dd.read_status(self.cache.ws) == 0


def _check_attention(x, out, lse, scale=None, most=24):
    """out/lse of Case x against the oracle, at up to `most` tokens of each request."""
    scale = scale or 1 / math.sqrt(x.D)
    k, v, q = x.host(x.k), x.host(x.v), x.host(x.q).astype(np.float64)
    o, z = x.host(out).astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for c in range(x.C):
        n = x.old[c] + x.new[c]
        seen = op.sees(x.old[c], x.new[c], x.masks[c])
        pick = np.arange(x.new[c])
        if len(pick) > most:
            pick = np.unique(np.concatenate([[0, 1, x.new[c] - 1], x.rng.choice(x.new[c], most, replace=False)]))
        kc, vc = op.rows_of(k, x.np_table, c, n), op.rows_of(v, x.np_table, c, n)
        rows = x.first[c] + pick
        wo, wz, mag, ab = op.attention(q[rows], kc, vc, seen[pick], scale)
        ds = x.D * 2 * E32 * ab
        inner = (E16 + 2 * ds[..., None] + 2.0 ** -18) * mag
        tol = inner + E16 * (np.abs(wo) + inner) + 1e-30
        err = np.abs(o[rows] - wo)
        assert (err <= tol).all(), (c, float((err / tol).max()), np.argwhere(err > tol)[:3])
        fin = np.isfinite(wz)
        assert (z[rows][~fin] == -np.inf).all() and (o[rows][~fin] == 0).all()
        tz = ds + n * E32 + 2.0 ** -20 + np.abs(np.where(fin, wz, 0)) * 2.0 ** -22
        ez = np.where(fin, np.abs(np.where(fin, z[rows] - np.where(fin, wz, 0), 0)), 0)
        assert (ez <= tz).all(), (c, float((ez / tz).max()))


ATTN = [
    # single tokens: ragged contexts, empty ones, lengths around pages and 128-row blocks
    dict(new=[1, 1, 1, 1, 1], old=[0, 15, 16, 127, 128], ragged=False),
    dict(new=[1] * 4, old=[129, 300, 1023, 2047], Hq=32, Hkv=8, page=64, ragged=False),
    dict(new=[1], old=[5000], Hq=8, Hkv=1, page=256, ragged=False),
    dict(new=[1, 1], old=[700, 33], Hq=6, Hkv=6, D=64, page=32),
    # chunks: one row per request up to many tiles; empty chunks; odd head groups
    dict(new=[1, 0, 130, 37], old=[0, 50, 0, 200], Hq=10, Hkv=2),
    dict(new=[257, 5], old=[3, 511], Hq=14, Hkv=2, D=64, page=64),
    dict(new=[300], old=[1000], Hq=8, Hkv=2, page=128, ragged=False),
    dict(new=[129, 128, 127], old=[128, 1, 0], Hq=2, Hkv=2, page=32),
    dict(new=[40, 3], old=[77, 500], Hq=32, Hkv=2, page=16),          # 16 heads of a group
    dict(new=[9, 2], old=[140, 0], Hq=128, Hkv=1, page=16, D=64),     # a token fills a tile
    dict(new=[5, 2], old=[40, 0], Hq=200, Hkv=2, page=16),            # 100 heads of a group
    dict(new=[1500], old=[900], Hq=4, Hkv=1, page=64, ragged=False),
    # trees
    dict(new=[65, 65], old=[200, 77], tree=True, Hq=8, Hkv=2, page=64),
    dict(new=[7, 1, 0, 12], old=[0, 130, 9, 128], S=12, tree=True),
    dict(new=[128, 100], old=[500, 31], tree=True, S=128, Hq=8, Hkv=8, D=64, page=32),
    dict(new=[300], old=[90], tree=True, S=300, Hq=4, Hkv=2),
    # long contexts of few rows: many chunks, merged through memory
    dict(new=[20, 11], old=[6000, 3000], tree=True, S=20, Hq=4, Hkv=1, page=64),
    dict(new=[2, 0, 1], old=[7000, 10, 130], Hq=8, Hkv=1, D=64, page=256, pad=(1, 2)),
    dict(new=[3], old=[70000], Hq=4, Hkv=1, D=64, page=256),
    # at most 16 rows of a key/value head: causal and tree masks inside them, empty requests, both head sizes
    dict(new=[4, 0, 2, 3], old=[700, 5, 0, 127], Hq=8, Hkv=2, page=32, pad=(3, 2)),
    dict(new=[16, 3, 0], old=[250, 1000, 4], S=16, Hq=2, Hkv=2, D=64, tree=True),
    dict(new=[8, 8], old=[120, 1], Hq=4, Hkv=2, page=16, ragged=False, spare=2000),
    dict(new=[2], old=[9000], Hq=16, Hkv=2, D=64, page=128, ragged=False),
    dict(new=[1], old=[4000], Hq=16, Hkv=1, page=16, ragged=False),
    dict(new=[5], old=[0], Hq=3, Hkv=1, D=64, page=256),
    dict(new=[1] * 40, old=[37 * c for c in range(40)], Hq=16, Hkv=8, D=64, page=32, ragged=False),
    dict(new=[1, 2] * 10, old=[100 * c for c in range(20)], Hq=8, Hkv=8, page=64),
    # several tiles of many heads, more CTAs than run at once; a tile alone on its SM
    dict(new=[65] * 20, old=[45 * c for c in range(20)], tree=True, Hq=16, Hkv=8, page=64),
    dict(new=[130] * 22, old=[600 - 20 * c for c in range(22)], Hq=8, Hkv=8, D=64, page=32, spare=100),
    dict(new=[100], old=[100], Hq=32, Hkv=8, page=16, ragged=False),
    dict(new=[17, 9], old=[500, 333], S=17, tree=True, Hq=16, Hkv=2, D=64, page=16),
    # single tokens of more heads than that
    dict(new=[1, 1], old=[3000, 50], Hq=32, Hkv=1, page=64, ragged=False),
    dict(new=[1] * 20, old=[60 * c for c in range(20)], Hq=68, Hkv=4, D=64, page=16, ragged=False),
]


@pytest.mark.parametrize("i", range(len(ATTN)))
def test_attention_matches_oracle(dd, i):
    x = Case(dd, seed=i, **ATTN[i]).fill()
    lse = torch.full((x.T, x.Hq), 7.0, device="cuda")
    out = torch.full((x.T, x.Hq, x.D), 7.0, device="cuda", dtype=torch.bfloat16)
    got = x.cache.attention(x.q, tree=x.tree, out=out, lse=lse)
    x.ok()
    assert got is out
    _check_attention(x, out, lse)
    if x.tree is not None:
        for c in range(x.C):
            dead = slice(x.first[c] + x.new[c], x.first[c] + x.S)
            assert (out[dead] == 0).all() and (lse[dead] == 0).all()


def test_attention_of_a_full_batch(dd):
    x = Case(dd, [1] * 64, [int(n) for n in np.random.default_rng(5).integers(0, 700, 64)], Hq=32, Hkv=8, page=64,
             ragged=False, seed=64).fill()
    lse = torch.empty(x.T, x.Hq, device="cuda")
    out = x.cache.attention(x.q, lse=lse)
    x.ok()
    _check_attention(x, out, lse)


def test_attention_leaves_rows_outside_the_batch(dd):
    x = Case(dd, [3, 0, 70], [20, 5, 130], pad=(4, 9), seed=3).fill()
    out = torch.full((x.T, x.Hq, x.D), 5.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((x.T, x.Hq), 5.0, device="cuda")
    x.cache.attention(x.q, out=out, lse=lse)
    x.ok()
    _check_attention(x, out, lse)
    for s in (slice(0, 4), slice(x.T - 9, x.T)):
        assert (out[s] == 5).all() and (lse[s] == 5).all()


def test_attention_rows_that_see_nothing(dd):
    """An empty mask row without context; with a context it sees that alone."""
    x = Case(dd, [6, 6], [0, 40], S=6, tree=True, seed=9).fill()
    for m in x.masks:
        m[3] = 0
    x.tree["mask"] = torch.from_numpy(np.stack(x.masks)).cuda()
    lse = torch.empty(x.T, x.Hq, device="cuda")
    out = x.cache.attention(x.q, tree=x.tree, lse=lse)
    x.ok()
    _check_attention(x, out, lse)
    assert (out[3] == 0).all() and torch.isinf(lse[3]).all()


@pytest.mark.parametrize("scale,scaleq", [(1.0, 8.0), (0.02, 1.0), (0.5, 1e-3)])
def test_attention_scales_and_large_scores(dd, scale, scaleq):
    """Scores of several hundred (one key takes all) down to almost equal ones."""
    x = Case(dd, [3, 150], [900, 64], Hq=8, Hkv=2, seed=11, scaleq=scaleq).fill()
    lse = torch.empty(x.T, x.Hq, device="cuda")
    out = x.cache.attention(x.q, scale=scale, lse=lse)
    x.ok()
    _check_attention(x, out, lse, scale=scale)


def test_attention_running_maximum_that_keeps_growing(dd):
    """Keys whose scores rise block by block: every block rescales what came before."""
    x = Case(dd, [1, 140], [1500, 700], Hq=4, Hkv=1, page=32, seed=13).fill()
    for c in range(2):
        n = x.old[c] + x.new[c]
        p, r = op.place(x.np_table, c, np.arange(n), x.page)
        ramp = torch.linspace(-1, 1, n, device="cuda")[:, None, None] * 3
        x.k[torch.from_numpy(p.astype(np.int64)).cuda(), :, torch.from_numpy(r).cuda()] = \
            (x.rand(n, 1, x.D).float() * 0.2 + ramp).to(torch.bfloat16)
    x.q.copy_((x.q.float() * 0.2 + 1).to(torch.bfloat16))
    lse = torch.empty(x.T, x.Hq, device="cuda")
    out = x.cache.attention(x.q, lse=lse)
    x.ok()
    _check_attention(x, out, lse)


@pytest.mark.parametrize("at", [0, 63, 64, 127, 128, 190, 255, 300, 511])
def test_attention_a_key_far_above_the_others(dd, at):
    """One key's score lies a hundred powers of two above what came before it, at the ends of a block's
    halves and inside them; a second one as far above the first."""
    x = Case(dd, [1, 70], [600, 530], Hq=8, Hkv=2, page=64, seed=at).fill()
    x.q.copy_((x.q.float() * 0.1 + 1).to(torch.bfloat16))
    for c in range(2):
        for j, v in ((at, 7.0), (min(at + 97, 599 - 70 * c), 14.0)):
            p, r = op.place(x.np_table, c, [j], x.page)
            x.k[int(p[0]), :, int(r[0])] = v
    lse = torch.empty(x.T, x.Hq, device="cuda")
    out = x.cache.attention(x.q, lse=lse)
    x.ok()
    _check_attention(x, out, lse)


# one request (its blocks spread over a cluster), a batch (a CTA has all of a head's blocks)
FEW = [dict(new=[1], old=[1500], Hq=4, Hkv=1), dict(new=[2] * 22, old=[1400 - 3 * c for c in range(22)], Hq=16, Hkv=8),
       dict(new=[3], old=[1100], Hq=8, Hkv=2, D=64), dict(new=[1] * 40, old=[900] * 40, Hq=8, Hkv=8, D=64)]


@pytest.mark.parametrize("i", range(len(FEW)))
@pytest.mark.parametrize("fall", [False, True])
def test_few_rows_maximum_that_keeps_growing(dd, i, fall):
    """Scores that rise (or fall) block by block, by more than the weights may carry."""
    x = Case(dd, page=32, seed=130 + i, **FEW[i]).fill()
    for c in range(x.C):
        n = x.old[c] + x.new[c]
        p, r = op.place(x.np_table, c, np.arange(n), x.page)
        ramp = torch.linspace(-1, 1, n, device="cuda")[:, None, None] * (-6 if fall else 6)
        x.k[torch.from_numpy(p.astype(np.int64)).cuda(), :, torch.from_numpy(r).cuda()] = \
            (x.rand(n, x.Hkv, x.D).float() * 0.2 + ramp).to(torch.bfloat16)
    x.q.copy_((x.q.float() * 0.2 + 1).to(torch.bfloat16))
    lse = torch.empty(x.T, x.Hq, device="cuda")
    out = x.cache.attention(x.q, lse=lse)
    x.ok()
    _check_attention(x, out, lse)


@pytest.mark.parametrize("i", range(len(FEW)))
@pytest.mark.parametrize("at", [0, 127, 128, 500, 895])
def test_few_rows_a_key_far_above_the_others(dd, i, at):
    x = Case(dd, page=64, seed=140 + at, **FEW[i]).fill()
    x.q.copy_((x.q.float() * 0.1 + 1).to(torch.bfloat16))
    for c in range(x.C):
        p, r = op.place(x.np_table, c, [at], x.page)
        x.k[int(p[0]), :, int(r[0])] = 9.0
    lse = torch.empty(x.T, x.Hq, device="cuda")
    out = x.cache.attention(x.q, lse=lse)
    x.ok()
    _check_attention(x, out, lse)


@pytest.mark.parametrize("scale,scaleq", [(1.0, 8.0), (0.02, 1.0)])
def test_few_rows_scales(dd, scale, scaleq):
    x = Case(dd, [3, 1], [900, 64], Hq=8, Hkv=2, seed=151, scaleq=scaleq).fill()
    lse = torch.empty(x.T, x.Hq, device="cuda")
    out = x.cache.attention(x.q, scale=scale, lse=lse)
    x.ok()
    _check_attention(x, out, lse, scale=scale)


def test_few_rows_that_see_nothing_for_a_block(dd):
    """Tree slots whose mask is empty, without a context and behind one, in batches small and large."""
    for C in (1, 90):
        x = Case(dd, [6] * C, [0, 130][:C] + [0] * (C - 2), S=6, tree=True, seed=153).fill()
        for m in x.masks:
            m[3] = 0
            m[5, :5] = 0
        x.tree["mask"] = torch.from_numpy(np.stack(x.masks)).cuda()
        lse = torch.empty(x.T, x.Hq, device="cuda")
        out = x.cache.attention(x.q, tree=x.tree, lse=lse)
        x.ok()
        _check_attention(x, out, lse)
        assert (out[3] == 0).all() and torch.isinf(lse[3]).all()


def test_equal_inputs_give_equal_outputs(dd):
    """Every way the chunks are merged, called again and again."""
    for kw in (FEW[0], FEW[1], dict(new=[1], old=[9000], Hq=4, Hkv=1), dict(new=[20], old=[2000], Hq=8, Hkv=2),
               dict(new=[300], old=[700], Hq=8, Hkv=2)):
        x = Case(dd, page=64, seed=157, **kw).fill()
        lse = torch.empty(x.T, x.Hq, device="cuda")
        want = x.cache.attention(x.q, lse=lse).clone()
        want_lse = lse.clone()
        for _ in range(20):
            lse.fill_(7.0)
            assert torch.equal(x.cache.attention(x.q, lse=lse), want) and torch.equal(lse, want_lse)
        sums = [x.cache.weights(x.q, lse, torch.zeros(x.C, x.Hkv, x.cache.rows, device="cuda")) for _ in range(20)]
        assert all(torch.equal(w, sums[0]) for w in sums)
        x.ok()


def test_one_workspace_for_batches_of_every_size(dd):
    """Made for the largest batch and the most tokens: smaller ones, some with more partial results than the
    largest, run in it, and the other calls, too."""
    rows, Hq, Hkv, page = 4096, 32, 8, 64
    p = dd.PagedParams(64, 64 * 65, 65, Hq, Hkv, 128, page, 1, rows // page, dd.BF16)
    n = dd.lib().dartree_paged_workspace_bytes(dd.ctypes.byref(p))
    ws = dd.new_workspace(n)
    stored = 0
    for C, S, old in ((8, 33, 500), (8, 65, 300), (1, 1, 4000), (12, 9, 200), (3, 20, 4000), (1, 64, 2000), (20, 2, 60)):
        x = Case(dd, [S] * C, [old - c for c in range(C)], Hq=Hq, Hkv=Hkv, page=page, ragged=False, seed=C + S,
                 spare=rows - old - S).fill()
        x.cache = dd.PagedCache(x.k, x.v, x.table, x.n_ctx, Hq, S, ws=ws)
        plan = dd.PagedPlan()
        assert dd.lib().dartree_paged_attention_plan(dd.ctypes.byref(x.cache.p), dd.ctypes.byref(plan)) == 0
        stored += plan.part_bytes > 0
        lse = torch.empty(x.T, Hq, device="cuda")
        out = x.cache.attention(x.q, lse=lse)
        w = torch.zeros(C, Hkv, x.cache.rows, device="cuda")
        x.cache.weights(x.q, lse, w)
        x.ok()
        _check_attention(x, out, lse, most=4)
        path, acc = torch.full((C, 4), -1, dtype=torch.int32), torch.zeros(C, dtype=torch.int32)
        if S > 2:
            path[:, 0], acc[:] = 2, 1
        n_out = x.cache.commit(path.cuda(), acc.cuda(), weights=w)
        x.ok()
        assert n_out.tolist() == [o + 1 + int(S > 2) for o in x.old]
    assert stored                                        # (eight requests of 33 tokens, on 148 and on 152 SMs)


# ------------------------------------------------------------------------------ append

APPEND = [
    dict(new=[1, 1, 1], old=[0, 15, 16], ragged=False),
    dict(new=[1], old=[100000], ragged=False, page=256, Hkv=1, Hq=1),   # far positions
    dict(new=[5, 0, 70, 1], old=[3, 9, 60, 0], Hq=10, Hkv=2, page=32, pad=(2, 3)),
    dict(new=[65, 20], old=[100, 31], S=65, tree=True, Hq=32, Hkv=8, page=64),
    dict(new=[700], old=[5], ragged=False, Hq=3, Hkv=1, D=64),          # four rows per CTA, an odd tail
    dict(new=[701, 2], old=[5, 9], Hq=3, Hkv=3, D=128),
    # a warp per row, eight rows a CTA and an odd tail (from 16 rows an SM on; those above have a CTA each):
    # more heads than a warp has in hand, requests without tokens, rows outside the batch
    dict(new=[1200, 0, 901, 437], old=[3, 9, 60, 0], Hq=20, Hkv=10, D=128, page=32, pad=(3, 2)),
    dict(new=[1200, 0, 901, 437], old=[3, 9, 60, 0], Hq=40, Hkv=20, D=64, pad=(3, 2)),
    dict(new=[65 - c for c in range(39)], old=[11 * c for c in range(39)], S=65, tree=True, Hq=3, Hkv=1, page=64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("i", range(len(APPEND)))
def test_append_matches_oracle(dd, i, norm, dtype):
    x = Case(dd, seed=i, dtype=dtype, **APPEND[i])
    x.fill(new_too=False)
    before_k, before_v = x.k.clone(), x.v.clone()
    qkv = x.rand(x.T, (x.Hq + 2 * x.Hkv) * x.D + 16)    # one projection's output, with a gap behind each token
    q = qkv[:, :x.Hq * x.D].view(x.T, x.Hq, x.D)
    k = qkv[:, x.Hq * x.D:(x.Hq + x.Hkv) * x.D].view(x.T, x.Hkv, x.D)
    v = qkv[:, (x.Hq + x.Hkv) * x.D:-16].view(x.T, x.Hkv, x.D)
    gains = [(1 + 0.2 * x.rand(x.D).float()).to(DT[dtype]) if norm else None for _ in range(2)]
    base = [int(b) for b in x.rng.integers(0, 3000, x.C)] if i % 2 else None
    out = torch.full((x.T, x.Hq, x.D), 5.0, device="cuda", dtype=DT[dtype])
    x.cache.append(q, k, v, *gains, eps=1e-5, tree=x.tree, out=out,
                   pos_base=None if base is None else torch.tensor(base, dtype=torch.int32, device="cuda"))
    x.ok()
    hq, hk, hv, ho = (x.host(a) for a in (q, k, v, out))
    g = [None if a is None else x.host(a) for a in gains]
    new_k, new_v = x.host(x.k), x.host(x.v)
    wk, wv = x.host(before_k), x.host(before_v)
    step = E16 if dtype == "bf16" else E32
    seen = np.zeros(x.T, bool)
    for c in range(x.C):
        n = x.new[c]
        r = slice(x.first[c], x.first[c] + n)
        seen[r] = True
        p = (x.old[c] if base is None else base[c]) + (x.depth[c][:n] if x.tree else np.arange(n))
        pg, at = op.place(x.np_table, c, x.old[c] + np.arange(n), x.page)
        for got, src, gain in ((ho[r], hq[r], g[0]), (new_k[pg, :, at], hk[r], g[1])):
            if n == 0:
                continue
            want = op.append(src, gain, p, eps=1e-5)
            y = np.abs(src if gain is None else op.head_norm(src, gain, 1e-5))
            pair = np.tile(y[..., :x.D // 2] + y[..., x.D // 2:], 2)
            tol = 2.0 ** -19 * pair + step * (np.abs(want) + 2.0 ** -19 * pair)
            assert (np.abs(got - want) <= tol).all()
        wk[pg, :, at] = new_k[pg, :, at]
        wv[pg, :, at] = hv[r]
    np.testing.assert_array_equal(new_k, wk)       # no other page row changed (NaN equal to NaN)
    np.testing.assert_array_equal(new_v, wv)
    rest = ho[~seen]
    assert (rest == (0 if x.q_start is None else 5)).all()


def test_append_in_place(dd):
    x = Case(dd, [9, 4], [3, 20], seed=2)
    k, v = x.rand(x.T, x.Hkv, x.D), x.rand(x.T, x.Hkv, x.D)
    g = x.rand(x.D)
    want = x.cache.append(x.q, k, v, g, g)
    got = x.cache.append(x.q, k, v, g, g, out=x.q)
    x.ok()
    assert got is x.q and torch.equal(got, want)


# ------------------------------------------------------------------------------ weights

WEIGHTS = [
    dict(new=[1] * 5, old=[0, 15, 128, 129, 700], ragged=False, Hq=8, Hkv=2),
    dict(new=[1, 1], old=[300, 31], Hq=6, Hkv=6, D=64, page=32, spare=300),
    dict(new=[40, 0, 1, 129], old=[100, 50, 0, 64], Hq=10, Hkv=2, page=16),
    dict(new=[33], old=[1000], Hq=32, Hkv=2, page=64),
    dict(new=[3, 2], old=[140, 0], Hq=200, Hkv=2, page=16),
    dict(new=[65, 20], old=[200, 7], S=65, tree=True, Hq=8, Hkv=2, page=64, D=64),
    dict(new=[200], old=[0], Hq=4, Hkv=4, ragged=False),
    # trees: more than 32 slots in a tile, heads that 16 columns do not divide, slots over a block's end
    dict(new=[100, 40], old=[200, 7], S=100, tree=True, Hq=2, Hkv=2, page=32),
    dict(new=[50, 33], old=[100, 127], S=50, tree=True, Hq=6, Hkv=2, page=16, D=64),
    dict(new=[300], old=[90], S=300, tree=True, Hq=1, Hkv=1, page=64),
    # tiles that 16 columns do not divide, whole ones and their last
    dict(new=[150, 18], old=[2100, 300], Hq=28, Hkv=4, page=64),
    dict(new=[60], old=[1500], Hq=10, Hkv=2, D=64, page=32, ragged=False),
    # many query tiles over few key blocks: CTAs share a block's tiles
    dict(new=[300, 3, 0, 130], old=[27, 300, 50, 0], Hq=16, Hkv=1, page=64),
    dict(new=[260], old=[1], Hq=8, Hkv=1, D=64, page=16, ragged=False),
    dict(new=[200, 90], old=[60, 3], S=200, tree=True, Hq=8, Hkv=2, page=32),
]


@pytest.mark.parametrize("i", range(len(WEIGHTS)))
def test_weights_match_oracle(dd, i):
    x = Case(dd, seed=20 + i, **WEIGHTS[i]).fill()
    scale = 1 / math.sqrt(x.D)
    lse = torch.full((x.T, x.Hq), float("nan"), device="cuda")
    x.cache.attention(x.q, tree=x.tree, lse=lse)
    w = torch.rand(x.C, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    w0 = w.clone()
    for c in range(x.C):
        w[c, :, x.old[c]:x.old[c] + x.new[c]] = float("nan")   # a new row has no weight yet
    again = w.clone()
    x.cache.weights(x.q, lse, w, tree=x.tree, decay=0.5)
    x.cache.weights(x.q, lse, again, tree=x.tree, decay=0.5)
    x.ok()
    assert torch.equal(w, again)
    h, q, z = w.cpu().numpy().astype(np.float64), x.host(x.q), lse.cpu().numpy().astype(np.float64)
    for c in range(x.C):
        n, r = x.old[c] + x.new[c], slice(x.first[c], x.first[c] + x.new[c])
        kc = x.rows(x.k, c, n)
        seen = op.sees(x.old[c], x.new[c], x.masks[c])
        want = op.weights(q[r], kc, seen, z[r], scale, w0[c].cpu().numpy(), x.old[c], 0.5)
        ab = (np.abs(kc).sum() and np.abs(q[r]).max() * np.abs(kc).sum(-1).max() * scale) if x.new[c] else 0.0
        arg = 2 * (ab + np.abs(np.where(np.isfinite(z[r]), z[r], 0)).max(initial=0))
        rel = x.D * 2 * E32 * ab + arg * 2.0 ** -22 + 2.0 ** -20 + x.new[c] * (x.Hq // x.Hkv) * E32
        err = np.abs(h[c, :, :n] - want)
        assert (err <= rel * want + 1e-30).all(), (c, float((err / (rel * want + 1e-30)).max()))
        np.testing.assert_array_equal(h[c, :, n:], w0[c, :, n:].cpu().numpy())


def test_weights_of_a_step_sum_to_its_rows(dd):
    x = Case(dd, [33, 1], [500, 900], Hq=8, Hkv=2, page=64, seed=31).fill()
    lse = torch.empty(x.T, x.Hq, device="cuda")
    x.cache.attention(x.q, lse=lse)
    w = torch.zeros(x.C, x.Hkv, x.cache.rows, device="cuda")
    x.cache.weights(x.q, lse, w)
    x.ok()
    want = torch.tensor([33.0, 1.0], device="cuda")[:, None] * 4
    assert ((w.sum(-1) - want).abs() <= want * 2e-4).all()


# ------------------------------------------------------------------------------ evict, commit

def _evict_case(dd, old, budget, sink, recent, dtype="bf16", Hkv=2, D=64, page=16, seed=0, spare_dst=0, values=None):
    x = Case(dd, [0] * len(old), old, S=1, Hq=Hkv, Hkv=Hkv, D=D, page=page, dtype=dtype, seed=seed, ragged=False)
    x.fill()
    pages = -(-budget // page) + spare_dst
    dst = np.arange(x.n_pages, x.n_pages + x.C * pages)
    more = torch.full((x.C * pages, Hkv, page, D), 7.0, device="cuda", dtype=x.k.dtype)
    x.k, x.v = torch.cat([x.k, more]), torch.cat([x.v, more])
    x.dst = x.rng.permutation(dst).reshape(x.C, pages).astype(np.int32)
    x.cache = dd.PagedCache(x.k, x.v, x.table, x.n_ctx, x.Hq, 1)
    w = x.rng.random((x.C, Hkv, x.cache.rows)).astype(np.float32) if values is None else values(x)
    return x, w, torch.from_numpy(x.dst).cuda()


def _check_evict(x, w, r, budget, sink, recent, before_k, before_v):
    keep, n, wo = (r[k].cpu().numpy() for k in ("keep", "n", "weights"))
    k, v = x.host(x.k), x.host(x.v)
    for c in range(x.C):
        assert n[c] == min(x.old[c], budget)
        for g in range(x.Hkv):
            want = op.kept_rows(w[c, g], x.old[c], budget, sink, recent)
            assert keep[c, g].tolist() == want + [-1] * (budget - len(want)), (c, g)
            np.testing.assert_array_equal(wo[c, g, :len(want)], w[c, g, want])
            assert (wo[c, g, len(want):] == 0).all()
            sp, sr = op.place(x.np_table, c, want, x.page)
            dp, dr = op.place(x.dst, c, np.arange(len(want)), x.page)
            for pool, was in ((k, before_k), (v, before_v)):
                was[dp, g, dr] = was[sp, g, sr]
    np.testing.assert_array_equal(k, before_k)      # the kept rows and nothing else
    np.testing.assert_array_equal(v, before_v)


EVICT = [
    dict(old=[100, 16, 17, 0, 5], budget=16, sink=4, recent=4),
    dict(old=[1000, 999], budget=300, sink=0, recent=0, page=64, D=128),
    dict(old=[1000, 40], budget=20, sink=5, recent=15, spare_dst=2),               # no room by weight
    dict(old=[4100], budget=1024, sink=4, recent=256, dtype="f32", Hkv=3, D=128),
    dict(old=[70], budget=1, sink=0, recent=1, dtype="f32"),
    dict(old=[20000, 3], budget=5000, sink=1, recent=7, page=256, Hkv=1),
    dict(old=[33, 33], budget=32, sink=0, recent=0),                               # one row goes
    dict(old=[60000], budget=700, sink=3, recent=5, page=256, Hkv=1),              # more rows than fit on chip
    dict(old=[130, 99], budget=40, sink=13, recent=7),                             # the ranked rows start odd
    # copies of 16 MB and more, the last rows of a budget that no CTA's rows divide
    dict(old=[9000, 4200], budget=4101, sink=4, recent=100, page=64, D=128, Hkv=4),
    dict(old=[5000, 4097, 17], budget=4097, sink=4, recent=100, page=16, D=128, Hkv=4, dtype="f32"),
    dict(old=[8300, 8193], budget=8193, sink=0, recent=1, page=128, D=64, Hkv=4),
]


@pytest.mark.parametrize("i", range(len(EVICT)))
def test_evict_matches_oracle(dd, i):
    kw = dict(EVICT[i])
    x, w, dst = _evict_case(dd, seed=40 + i, **kw)
    bk, bv = x.host(x.k), x.host(x.v)
    r = x.cache.evict(torch.from_numpy(w).cuda(), kw["budget"], dst, kw["sink"], kw["recent"])
    x.ok()
    _check_evict(x, w, r, kw["budget"], kw["sink"], kw["recent"], bk, bv)


SPECIAL = {
    "equal": lambda x: np.ones((x.C, x.Hkv, x.cache.rows), np.float32),
    "two values": lambda x: x.rng.integers(0, 2, (x.C, x.Hkv, x.cache.rows)).astype(np.float32),
    "close": lambda x: (1 + x.rng.integers(0, 5, (x.C, x.Hkv, x.cache.rows)) * 2.0 ** -23).astype(np.float32),
    "nan and infinities": lambda x: x.rng.choice(np.array([np.nan, -np.inf, np.inf, 0, -0.0, 1, -1], np.float32),
                                                 (x.C, x.Hkv, x.cache.rows)),
    "all nan": lambda x: np.full((x.C, x.Hkv, x.cache.rows), np.nan, np.float32),
}


@pytest.mark.parametrize("name", list(SPECIAL))
def test_evict_ties_and_special_weights(dd, name):
    x, w, dst = _evict_case(dd, [1500, 90], 77, 3, 9, seed=50, values=SPECIAL[name], page=32)
    bk, bv = x.host(x.k), x.host(x.v)
    r = x.cache.evict(torch.from_numpy(w).cuda(), 77, dst, 3, 9)
    x.ok()
    _check_evict(x, w, r, 77, 3, 9, bk, bv)


def test_evict_writes_the_lengths_in_place(dd):
    x, w, dst = _evict_case(dd, [100, 9, 64], 32, 1, 2, seed=60)
    r = x.cache.evict(torch.from_numpy(w).cuda(), 32, dst, 1, 2, n_out=x.n_ctx)
    x.ok()
    assert r["n"] is x.n_ctx and x.n_ctx.tolist() == [32, 9, 32]


COMMIT = [
    dict(S=65, L=16, paths=[[1, 2, 3], [5, 9, 30, 64], []], dtype="bf16"),
    dict(S=65, L=64, paths=[list(range(1, 65)), list(range(2, 65))], dtype="f32", Hkv=5),
    dict(S=2, L=1, paths=[[1], []], dtype="bf16", D=64),
    dict(S=20, L=8, paths=[[19], [3, 4, 5, 6, 7, 8, 9, 10]], dtype="f32", D=64, Hkv=1),
    dict(S=128, L=64, paths=[list(range(2, 130, 2))[:63]], dtype="bf16", Hkv=40),
]


@pytest.mark.parametrize("i", range(len(COMMIT)))
@pytest.mark.parametrize("alias", [False, True])
def test_commit_matches_oracle(dd, i, alias):
    kw = dict(COMMIT[i])
    paths, L, S = kw.pop("paths"), kw.pop("L"), kw.pop("S")
    old = [30 + 7 * c for c in range(len(paths))]
    x = Case(dd, [S] * len(paths), old, S=S, seed=70 + i, ragged=False, Hq=kw.get("Hkv", 2), **kw).fill()
    path = np.full((x.C, L), -1, np.int32)
    for c, p in enumerate(paths):
        path[c, :len(p)] = p
    bk, bv = x.host(x.k), x.host(x.v)
    n = x.cache.commit(torch.from_numpy(path).cuda(), torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda(),
                       n_out=x.n_ctx if alias else None)
    x.ok()
    for c, p in enumerate(paths):
        src, dst, end = op.commit_moves(path[c], len(p), old[c])
        assert int(n[c]) == end
        sp, sr = op.place(x.np_table, c, src, x.page)
        dp, dr = op.place(x.np_table, c, dst, x.page)
        for pool in (bk, bv):
            pool[dp, :, dr] = pool[sp, :, sr].copy()
    np.testing.assert_array_equal(x.host(x.k), bk)
    np.testing.assert_array_equal(x.host(x.v), bv)


@pytest.mark.parametrize("i", range(len(COMMIT)))
def test_commit_moves_the_weights_with_the_rows(dd, i):
    """Every row's weight goes where its key goes; all others stay (weights NaN behind the rows held)."""
    kw = dict(COMMIT[i])
    paths, L, S = kw.pop("paths"), kw.pop("L"), kw.pop("S")
    old = [30 + 7 * c for c in range(len(paths))]
    x = Case(dd, [S] * len(paths), old, S=S, seed=170 + i, ragged=False, Hq=kw.get("Hkv", 2), spare=3, **kw).fill()
    path = np.full((x.C, L), -1, np.int32)
    for c, p in enumerate(paths):
        path[c, :len(p)] = p
    w = torch.rand(x.C, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    for c in range(x.C):
        w[c, :, old[c] + S:] = float("nan")
    want, plain = w.cpu().numpy().copy(), (x.k.clone(), x.v.clone())
    acc = torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
    n = x.cache.commit(torch.from_numpy(path).cuda(), acc, weights=w)
    x.ok()
    moved = x.host(x.k), x.host(x.v)
    for c, p in enumerate(paths):
        src, dst, end = op.commit_moves(path[c], len(p), old[c])
        assert int(n[c]) == end
        want[c][:, dst] = want[c][:, src].copy()
    np.testing.assert_array_equal(w.cpu().numpy(), want)
    x.k.copy_(plain[0]), x.v.copy_(plain[1])             # keys and values as without weights
    assert torch.equal(x.cache.commit(torch.from_numpy(path).cuda(), acc), n)
    np.testing.assert_array_equal(x.host(x.k), moved[0])
    np.testing.assert_array_equal(x.host(x.v), moved[1])


def test_weights_follow_a_committed_tree(dd):
    """Two tree steps and a token, each counted, against sums kept row by row for the tokens that stayed."""
    S, C = 17, 2
    x = Case(dd, [17, 9], [140, 33], S=S, tree=True, Hq=8, Hkv=2, page=32, seed=181, spare=40).fill(new_too=False)
    scale = 1 / math.sqrt(x.D)
    w = torch.rand(C, x.Hkv, x.cache.rows, generator=x.gen, device="cuda")
    for c in range(C):
        w[c, :, x.old[c]:] = float("nan")
    kept = [w[c, :, :x.old[c]].cpu().numpy().astype(np.float64) for c in range(C)]
    token = dd.PagedCache(x.k, x.v, x.table, x.n_ctx, x.Hq, 1)
    lse = torch.empty(x.T, x.Hq, device="cuda")
    for last in (False, False, True):
        cache, T, new = (token, C, [1, 1]) if last else (x.cache, x.T, x.new)
        tree, first = (None, [0, 1]) if last else (x.tree, x.first)
        q, z = x.rand(T, x.Hq, x.D), lse[:T]
        qr = cache.append(q, x.rand(T, x.Hkv, x.D), x.rand(T, x.Hkv, x.D), tree=tree)
        cache.attention(qr, tree=tree, lse=z)
        cache.weights(qr, z, w, tree=tree, decay=0.75)
        old = x.n_ctx.tolist()
        path, acc = np.full((C, 16), -1, np.int32), [0, 0]
        hz, hq = z.cpu().numpy().astype(np.float64), x.host(qr).astype(np.float64)
        for c in range(C):
            n, r = old[c] + new[c], slice(first[c], first[c] + new[c])
            seen = op.sees(old[c], new[c], None if last else x.masks[c])
            kc = x.rows(x.k, c, n)
            kept[c] = op.weights(hq[r], kc, seen, hz[r], scale, kept[c], old[c], 0.75)
            if not last:
                slots = np.flatnonzero(x.masks[c][int(np.argmax(x.depth[c]))])[1:]
                path[c, :len(slots)], acc[c] = slots, len(slots)
                kept[c] = kept[c][:, list(range(old[c] + 1)) + [old[c] + int(s) for s in slots]]
        if not last:
            cache.commit(torch.from_numpy(path).cuda(), torch.tensor(acc, dtype=torch.int32).cuda(), n_out=x.n_ctx,
                         weights=w)
        assert dd.read_status(cache.ws) == 0
        for c in range(C):
            m = kept[c].shape[1]
            assert m == old[c] + 1 + acc[c]
            # scale * sum |q_d k_d|, |score| and |lse| lie below 64: a term is off by 128 * 2^-23 * 64 = 2^-10 for
            # the products, 2 * 64 * 2^-22 for the argument, 2^-20 for the exponential, and the sums of at most
            # 3 * 17 * 4 positive ones by 204 * 2^-24 of themselves: together below 2^-9
            np.testing.assert_allclose(w[c, :, :m].cpu().numpy(), kept[c], rtol=2.0 ** -9, atol=0)


# ------------------------------------------------------------------------------ what the device checks

def _status(dd, x):
    torch.cuda.synchronize()
    s = dd.read_status(x.cache.ws)
    dd.clear_status(x.cache.ws)
    return s


@pytest.mark.parametrize("bad", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_a_table_entry_that_is_no_page(dd, bad):
    """Reported; nothing outside the pool is touched, and the other requests are right."""
    x = Case(dd, [3, 4], [40, 300], seed=80).fill()
    good = x.np_table.copy()
    x.table[0, 1] = bad
    k, v = x.rand(x.T, x.Hkv, x.D), x.rand(x.T, x.Hkv, x.D)
    lse = torch.empty(x.T, x.Hq, device="cuda")
    out = x.cache.attention(x.q, lse=lse)
    assert _status(dd, x) == dd.EINTERNAL
    assert torch.isfinite(out.float()).all()
    w = torch.zeros(x.C, x.Hkv, x.cache.rows, device="cuda")
    x.cache.weights(x.q, lse, w)
    assert _status(dd, x) == dd.EINTERNAL
    x.table[0, 1] = int(good[0, 1])
    x.table[0, 2] = bad                                  # the new tokens' page: rows 32..47
    before = x.k.clone()
    x.cache.append(x.q, k, v)
    assert _status(dd, x) == dd.EINTERNAL
    pg = torch.from_numpy(good[0].astype(np.int64)).cuda()
    np.testing.assert_array_equal(x.host(x.k[pg]), x.host(before[pg]))
    x2, wt, dst = _evict_case(dd, [100, 50], 32, 0, 0, seed=81)
    dst[1, 0] = bad
    x2.cache.evict(torch.from_numpy(wt).cuda(), 32, dst)
    assert _status(dd, x2) == dd.EINTERNAL
    y = Case(dd, [9], [10], S=9, seed=82, ragged=False).fill()
    y.table[0, 0] = bad
    y.cache.commit(torch.tensor([[3, 5]], dtype=torch.int32).cuda(), torch.tensor([2], dtype=torch.int32).cuda())
    assert _status(dd, y) == dd.EINTERNAL


def test_lengths_that_do_not_fit_are_reported(dd):
    x = Case(dd, [5, 3], [20, 4], seed=83).fill()
    k, v = x.rand(x.T, x.Hkv, x.D), x.rand(x.T, x.Hkv, x.D)

    def reports(f):
        f()
        assert _status(dd, x) == dd.EINTERNAL

    both = [lambda: x.cache.append(x.q, k, v), lambda: x.cache.attention(x.q)]
    for ctx in (x.cache.rows - 1, x.cache.rows + 5, -1, 2 ** 31 - 1, -2 ** 31):
        x.n_ctx[0] = ctx
        for f in both:
            reports(f)
    x.n_ctx[0] = 20
    was = x.q_start.clone()
    for st in ([0, 9, 8], [-3, 5, 8], [0, 5, 50], [5, 2, 8], [2 ** 31 - 1, -2 ** 31, 8]):
        x.q_start.copy_(torch.tensor(st, dtype=torch.int32))
        for f in both:
            reports(f)
    x.q_start.copy_(was)
    x.cache.append(x.q, k, v)
    assert _status(dd, x) == 0


@pytest.mark.parametrize("Hq", [4, 64, 200])   # rows of a head: few, two tiles, four
def test_attention_of_bad_tables_and_lengths(dd, Hq):
    x = Case(dd, [3, 4], [40, 300], Hq=Hq, seed=85).fill()
    lse = torch.empty(x.T, x.Hq, device="cuda")
    good = int(x.table[0, 1])
    for bad in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        x.table[0, 1] = bad
        out = x.cache.attention(x.q, lse=lse)
        assert _status(dd, x) == dd.EINTERNAL
        assert torch.isfinite(out.float()).all()
    x.table[0, 1] = good
    for ctx in (x.cache.rows - 1, x.cache.rows + 5, -1, 2 ** 31 - 1, -2 ** 31):
        x.n_ctx[0] = ctx
        x.cache.attention(x.q)
        assert _status(dd, x) == dd.EINTERNAL
    x.n_ctx[0] = 40
    was = x.q_start.clone()
    for st in ([0, 9, 8], [-3, 3, 7], [0, 3, 50], [5, 2, 7], [2 ** 31 - 1, -2 ** 31, 7]):
        x.q_start.copy_(torch.tensor(st, dtype=torch.int32))
        x.cache.attention(x.q)
        assert _status(dd, x) == dd.EINTERNAL
    x.q_start.copy_(was)
    out = x.cache.attention(x.q, lse=lse)
    x.ok()
    _check_attention(x, out, lse)


def test_paths_that_name_no_slot_are_reported(dd):
    x = Case(dd, [9], [10], S=9, seed=84, ragged=False).fill()
    one = lambda *a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    for path, acc in (([0, 2], 2), ([3, 9], 2), ([-1, 2], 1), ([1, 2], -1), ([1, 2], 3)):
        before = x.k.clone()
        n = x.cache.commit(one(path), one(acc))
        assert _status(dd, x) == dd.EINTERNAL
        assert 11 <= int(n[0]) <= 13
        assert torch.isnan(before.float()).sum() == torch.isnan(x.k.float()).sum()


# ------------------------------------------------------------------------------ use

def test_offsets_past_32_bits(dd):
    """A pool of more than 2^32 elements, the request's pages at its far end."""
    page, D = 256, 128
    n_pages = (2 ** 32) // (page * D) + 40
    k = torch.zeros(n_pages, 1, page, D, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    table = torch.tensor([[n_pages - 1, n_pages - 3], [5, n_pages - 2]], dtype=torch.int32, device="cuda")
    x = Case(dd, [3, 3], [300, 200], page=page, Hkv=1, Hq=4, seed=90)
    x.k, x.v, x.np_table = k, v, table.cpu().numpy()
    x.cache = dd.PagedCache(k, v, table, x.n_ctx, 4, 3, T=x.T, q_start=x.q_start)
    x.host = lambda t: t.float().cpu().numpy()
    x.fill(new_too=False)
    qr = x.cache.append(x.q, x.rand(6, 1, D), x.rand(6, 1, D))
    lse = torch.empty(6, 4, device="cuda")
    out = x.cache.attention(qr, lse=lse)
    x.ok()
    # the oracle on a small pool of the same pages
    order = [n_pages - 1, n_pages - 3, 5, n_pages - 2]
    x.k, x.v = k[order].contiguous(), v[order].contiguous()
    x.np_table = np.array([[0, 1], [2, 3]])
    x.q = qr
    _check_attention(x, out, lse)
    dst = torch.tensor([[n_pages - 9], [n_pages - 10]], dtype=torch.int32, device="cuda")
    w = torch.rand(2, 1, 512, device="cuda")
    r = x.cache.evict(w, 100, dst, 4, 10)
    x.ok()
    for c in range(2):
        rows = r["keep"][c, 0].long()
        pg = table[c].long()[rows // page]
        assert torch.equal(k[n_pages - 9 - c, 0, :100], k[pg, 0, rows % page])
    del k, v
    torch.cuda.empty_cache()


def test_a_served_tree_step(dd):
    """A step as it is used: append a prompt in two chunks, a tree, its attention, the accepted path
    committed, single tokens behind it, weights, eviction, and a token over the shrunken cache; the
    cache's keys follow the positions throughout."""
    rng = np.random.default_rng(7)
    C, Hq, Hkv, D, page, S = 2, 8, 2, 128, 32, 17
    g = torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    n_pages = 40
    k, v = (torch.full((n_pages, Hkv, page, D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ids = rng.permutation(n_pages).astype(np.int32)
    table = torch.from_numpy(ids[:2 * 12].reshape(2, 12)).cuda()
    n_ctx = torch.zeros(C, dtype=torch.int32, device="cuda")
    gq, gk = rand(D), rand(D)
    host = lambda t: t.float().cpu().numpy()  # noqa: E731
    want_k = [np.zeros((Hkv, 0, D)) for _ in range(C)]
    want_v = [np.zeros((Hkv, 0, D)) for _ in range(C)]
    w = torch.zeros(C, Hkv, 12 * page, device="cuda")

    def step(new, tree=None, base=None):
        """Append and attend `new` tokens per request; checks the outputs against the rows kept here."""
        T = sum(new) if tree is None else C * S
        st = None if tree is not None else torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
        cache = dd.PagedCache(k, v, table, n_ctx, Hq, max(new) if tree is None else S, T=T, q_start=st)
        qi, ki, vi = rand(T, Hq, D), rand(T, Hkv, D), rand(T, Hkv, D)
        b = None if base is None else torch.tensor(base, dtype=torch.int32, device="cuda")
        qr = cache.append(qi, ki, vi, gq, gk, tree=tree, pos_base=b)
        lse = torch.empty(T, Hq, device="cuda")
        out = cache.attention(qr, tree=tree, lse=lse)
        torch.cuda.synchronize()
        assert dd.read_status(cache.ws) == 0
        keys, vals = [], []
        for c in range(C):
            r0 = (0 if c == 0 else new[0]) if tree is None else c * S
            old = want_k[c].shape[1]
            pos = (old if base is None else base[c]) + (np.arange(new[c]) if tree is None else
                                                       tree["pos"][c].cpu().numpy()[:new[c]])
            r = slice(r0, r0 + new[c])
            kk = np.moveaxis(op.append(host(ki)[r], host(gk), pos), 0, 1)
            keys.append(np.concatenate([want_k[c], kk], 1))
            vals.append(np.concatenate([want_v[c], np.moveaxis(host(vi)[r], 0, 1)], 1))
            seen = op.sees(old, new[c], None if tree is None else tree["mask"][c].cpu().numpy())
            q64 = op.append(host(qi)[r], host(gq), pos)
            want, _, mag, ab = op.attention(q64, keys[c], vals[c], seen, 1 / math.sqrt(D))
            # queries and keys are stored in bf16 here: the scores are off by 2 * 2^-8 of their terms
            tol = (E16 + 2 * (2 * E16 + E16 ** 2) * ab[..., None] + 1e-3) * 2 * mag + E16 * np.abs(want)
            assert (np.abs(host(out)[r] - want) <= tol).all()
        return cache, qr, lse, keys, vals

    for new in ([40, 7], [1, 60]):
        cache, qr, lse, want_k, want_v = step(new)
        cache.weights(qr, lse, w)
        n_ctx += torch.tensor(new, dtype=torch.int32, device="cuda")
    trees = [_tree_of(rng, S, n) for n in (17, 11)]
    tree = dict(mask=torch.from_numpy(np.stack([m for m, _ in trees])).cuda(),
                pos=torch.from_numpy(np.stack([d for _, d in trees])).cuda(),
                n_nodes=torch.tensor([17, 11], dtype=torch.int32, device="cuda"))
    cache, qr, lse, keys, vals = step([17, 11], tree)
    # the deepest slot's ancestors are accepted
    path = np.full((C, 16), -1, np.int32)
    acc = []
    for c, (m, d) in enumerate(trees):
        slots = np.flatnonzero(m[int(np.argmax(d))])[1:]
        path[c, :len(slots)] = slots
        acc.append(len(slots))
        rows = list(range(want_k[c].shape[1] + 1)) + [want_k[c].shape[1] + int(s) for s in slots]
        want_k[c], want_v[c] = keys[c][:, rows], vals[c][:, rows]
    cache.commit(torch.from_numpy(path).cuda(), torch.tensor(acc, dtype=torch.int32).cuda(), n_out=n_ctx)
    assert n_ctx.tolist() == [x.shape[1] for x in want_k]
    cache, qr, lse, want_k, want_v = step([1, 1])
    for c in range(C):                                   # the committed rows have no weight yet
        w[c, :, want_k[c].shape[1] - 2 - acc[c]:] = 0
    cache.weights(qr, lse, w)
    n_ctx += 1
    at = n_ctx.tolist()
    dst = torch.from_numpy(ids[24:28].reshape(2, 2)).cuda()
    r = cache.evict(w, 33, dst, sink=2, recent=8, n_out=n_ctx)
    keep = r["keep"].cpu().numpy()
    hw = w.cpu().numpy()
    for c in range(C):
        for h in range(Hkv):
            assert keep[c, h].tolist() == op.kept_rows(hw[c, h], at[c], 33, 2, 8)
        want_k[c] = np.stack([want_k[c][h, keep[c, h]] for h in range(Hkv)])
        want_v[c] = np.stack([want_v[c][h, keep[c, h]] for h in range(Hkv)])
    table = dst
    step([1, 1], base=at)


def test_streams_and_graphs(dd):
    """A side stream, and a captured step replayed on new inputs with changed lengths."""
    x = Case(dd, [1, 1, 1], [100, 30, 260], ragged=False, seed=95, Hq=8, Hkv=2, spare=40).fill()
    lse, out = torch.empty(x.T, x.Hq, device="cuda"), torch.empty_like(x.q)
    k, v, g = x.rand(x.T, x.Hkv, x.D), x.rand(x.T, x.Hkv, x.D), x.rand(x.D)
    q, w = x.rand(x.T, x.Hq, x.D), torch.zeros(x.C, x.Hkv, x.cache.rows, device="cuda")
    qr = torch.empty_like(q)

    def step(stream=None):
        x.cache.append(q, k, v, g, g, out=qr, stream=stream)
        x.cache.attention(qr, out=out, lse=lse, stream=stream)
        x.cache.weights(qr, lse, w, stream=stream)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    step(side)
    side.synchronize()
    x.q = qr
    x.ok()
    _check_attention(x, out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for t in (q, k, v):
            t.copy_(x.rand(*t.shape))
        x.n_ctx += 1
        x.old = [n + 1 for n in x.old]
        graph.replay()
        x.ok()
        _check_attention(x, out, lse)
        assert ((w.sum(-1) - (i + 2) * 4).abs() < 1e-2).all()


@pytest.mark.parametrize("current", [False, True])
def test_a_workspace_is_filled_before_another_stream_uses_it(dd, current):
    """The fill waits behind work of the stream it was made on; a status word that a call on a side stream
    writes meanwhile must not be cleared by it."""
    x = Case(dd, [2], [40], seed=191).fill()
    x.table[0, 0] = -1
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)                        # some 25 ms on the current stream
    cache = dd.PagedCache(x.k, x.v, x.table, x.n_ctx, x.Hq, x.S, T=x.T, q_start=x.q_start)
    if current:
        with torch.cuda.stream(side):
            cache.attention(x.q)
    else:
        cache.attention(x.q, stream=side)
    torch.cuda.synchronize()
    assert dd.read_status(cache.ws) == dd.EINTERNAL


def test_a_workspace_outlives_its_object_on_a_side_stream(dd):
    """Its memory is not given away while a call on a side stream may still use it."""
    x = Case(dd, [2], [40], seed=193).fill()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    cache = dd.PagedCache(x.k, x.v, x.table, x.n_ctx, x.Hq, x.S, T=x.T, q_start=x.q_start)
    at, n = cache.ws.data_ptr(), cache.ws.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    out = cache.attention(x.q, stream=side)
    del cache
    assert all(t.data_ptr() != at for t in [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)])
    side.synchronize()
    assert torch.isfinite(out.float()).all()


def test_binding_refuses_what_it_can_see(dd):
    x = Case(dd, [2, 3], [5, 9], seed=97).fill()
    k = x.rand(x.T, x.Hkv, x.D)
    for bad in (x.q.float(), x.q[:-1], x.q.cpu(), x.q.transpose(0, 1)):
        with pytest.raises((ValueError, TypeError)):
            x.cache.attention(bad)
        with pytest.raises((ValueError, TypeError)):
            x.cache.append(bad, k, k)
    with pytest.raises(ValueError):
        x.cache.append(x.q, k.transpose(1, 2).contiguous().transpose(1, 2), k)
    with pytest.raises(ValueError):
        dd.PagedCache(x.k, x.v[:1], x.table, x.n_ctx, x.Hq, 3, T=5, q_start=x.q_start)
    with pytest.raises(ValueError):
        dd.PagedCache(x.k, x.v, x.table, x.n_ctx, x.Hq, 3, q_start=x.q_start)
    with pytest.raises(dd.DartreeError):
        dd.PagedCache(x.k, x.v, x.table, x.n_ctx, 5, 3, T=5, q_start=x.q_start)
    with pytest.raises(dd.DartreeError):
        x.cache.attention(x.q, scale=-2.0)
    with pytest.raises(dd.DartreeError):
        x.cache.evict(torch.zeros(2, 2, x.cache.rows, device="cuda"), 0, x.table)
