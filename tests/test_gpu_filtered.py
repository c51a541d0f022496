"""Draws under temperature, top-k, top-p and min-p, and the walk of a tree on them, against the float64
oracle, through the binding: tokens, paths and lengths are equal.

The kernel's weights are integers, off by at most one unit of 2^-42 of the largest (half a unit of rounding,
2^-43 of float pairs); a border between tokens is a quotient of sums of at most V of them, the whole sum being at
least one largest weight, so it is off by less than 2 V 2^-42, and the oracle's by far less. A token may
differ only where u lies that near to a border (the oracle reports the distance); inputs are fixed and none does.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import serving as sv  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from diffusion_drafter_draft_gb300 import _build
    _build.build()
    import diffusion_drafter_draft_gb300 as m
    m.lib()
    return m


SETTINGS = [dict(), dict(temperature=0.7, top_k=20, top_p=0.8), dict(top_p=0.95), dict(temperature=1.3, min_p=0.05),
            dict(temperature=0.0), dict(top_k=1), dict(top_p=0.0), dict(temperature=0.4, top_k=300, top_p=0.9, min_p=0.01),
            dict(temperature=2.0, top_k=1000), dict(temperature=3.0, top_p=0.999), dict(top_k=5, min_p=1.0)]


def _check(dd, x, u, dtype, out=None, **kw):
    """x [R, V] float64 values that dtype holds; kw: numbers or arrays [R]."""
    R, V = x.shape
    t = x if isinstance(x, torch.Tensor) else torch.from_numpy(x).to(DT[dtype]).cuda()
    ws = dd.new_workspace(256)
    dev = {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in kw.items()}
    got = dd.sample(t, torch.from_numpy(u).cuda(), ws=ws, **dev).cpu().numpy()
    assert dd.read_status(ws) == 0
    h = t.double().cpu().numpy()
    for r in range(R):
        of = {k: v[r].item() if isinstance(v, np.ndarray) else float(np.float32(v)) if k != "top_k" else v
              for k, v in kw.items()}
        want, near = sv.draw(h[r], float(u[r]), **of)
        assert got[r] == want or near < 2 * V * 2.0 ** -42, (r, int(got[r]), want, near, of)
    return got


def _u(rng, R):
    u = rng.random(R, dtype=np.float32)
    u[u >= 1] = 0.5
    u[:2] = np.array([0.0, 1 - 2.0 ** -24], np.float32)[:R]
    return u


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 255, 1000, 1001, 4099, 20000, 151936])
def test_settings(dd, V, dtype):
    rng = np.random.default_rng(V)
    R = 3 if V > 100000 else 9
    x = rng.standard_normal((R, V)) * 2.5
    for r in range(R):
        x[r, rng.integers(0, V, 5)] += 9 * rng.random(5)
    for kw in SETTINGS:
        _check(dd, x, _u(rng, R), dtype, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sigma", [0.0, 0.02, 1.0, 8.0, 100.0])
def test_spreads_of_logits(dd, sigma, dtype):
    """From all equal to one that holds everything, around a level far from zero."""
    rng = np.random.default_rng(5)
    x = -37.0 + sigma * rng.standard_normal((4, 9001))
    for kw in SETTINGS:
        _check(dd, x, _u(rng, 4), dtype, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_values(dd, dtype):
    """Ties at every border: the lowest tokens are kept, runs longer than the list."""
    rng = np.random.default_rng(6)
    x = np.round(rng.standard_normal((8, 6000)) * 1.2) * 0.5
    x[4:] = np.where(rng.random((4, 6000)) < 0.3, 2.0, -1.0)
    for kw in SETTINGS + [dict(top_k=k) for k in (2, 255, 256, 257, 1024, 5999, 6000, 7000)] + \
            [dict(top_p=p) for p in (1e-6, 0.2, 0.5, 0.9)]:
        _check(dd, x, _u(rng, 8), dtype, **kw)


def test_neighbouring_floats(dd):
    """Thousands of values a last place apart: finer histograms down to single keys."""
    rng = np.random.default_rng(7)
    x = np.stack([1.0 + rng.integers(0, 4000, 8000) * 2.0 ** -23, 8.0 + rng.integers(0, 50, 8000) * 2.0 ** -20,
                  np.where(rng.random(8000) < 0.5, rng.integers(0, 900, 8000) * 2.0 ** -149, 3.0)])
    for kw in SETTINGS + [dict(top_k=4000), dict(top_p=0.5), dict(top_k=3000, top_p=0.3)]:
        _check(dd, x, _u(rng, 3), "f32", **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_infinities_and_nan(dd, dtype):
    rng = np.random.default_rng(8)
    V = 3001
    low = float(torch.finfo(DT[dtype]).min)
    x = rng.standard_normal((9, V))
    x[0] = -np.inf                                             # nothing to draw
    x[1, :] = np.nan
    x[2, :] = -np.inf
    x[2, 2077] = -5.0                                          # one
    x[3, rng.random(V) < 0.9] = -np.inf
    x[4, rng.random(V) < 0.9] = low
    x[5, rng.random(V) < 0.5] = np.nan
    x[6, [3, 500, 2999]] = np.inf                              # they share the weight
    x[7] = low
    x[8, 0], x[8, 1:] = -low, low
    for kw in SETTINGS + [dict(top_k=2500), dict(top_k=2, top_p=0.9)]:
        got = _check(dd, x, _u(rng, 9), dtype, **kw)
        assert got[0] == got[1] == -1 and got[2] == 2077 and got[6] in (3, 500, 2999)


@pytest.mark.parametrize("temperature", [1e-30, 1e-3, 50.0, 1e30])
def test_temperatures(dd, temperature):
    rng = np.random.default_rng(9)
    x = rng.standard_normal((4, 5000)) * 3
    for kw in (dict(), dict(top_p=0.7), dict(top_k=40), dict(min_p=0.5)):
        _check(dd, x, _u(rng, 4), "f32", temperature=temperature, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_settings_of_each_request(dd, dtype):
    rng = np.random.default_rng(10)
    R = 64
    x = rng.standard_normal((R, 12345)) * 2.5
    pick = lambda a, t: rng.choice(np.array(a, t), R)  # noqa: E731
    _check(dd, x, _u(rng, R), dtype, temperature=pick([0, 0.3, 1, 1.5], np.float32),
           top_k=pick([0, 1, 20, 400, 20000], np.int32), top_p=pick([1, 0.9, 0.3, 0], np.float32),
           min_p=pick([0, 0.1, 1], np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,ld,first", [(1000, 1003, 1), (4099, 5000, 3), (777, 778, 5)])
def test_strides_and_alignment(dd, V, ld, first, dtype):
    rng = np.random.default_rng(V)
    big = torch.from_numpy(rng.standard_normal(7 * ld + first) * 2.5).to(DT[dtype]).cuda()
    big[:first] = float("inf")                                 # what lies around the rows is not theirs
    x = big[first:].view(7, ld)
    x[:, V:] = float("inf")
    for kw in SETTINGS[:4]:
        _check(dd, x[:, :V], _u(rng, 7), dtype, **kw)


def test_a_row_does_not_depend_on_its_batch(dd):
    """One, some and many rows: other clusters, the same tokens."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn(300, 30000, generator=gen, device="cuda") * 2).to(torch.bfloat16)
    u = torch.rand(300, generator=gen, device="cuda")
    for kw in SETTINGS[:4]:
        whole = dd.sample(x, u, **kw)
        for n in (1, 3, 40, 120):
            assert torch.equal(dd.sample(x[:n], u[:n], **kw), whole[:n])


def test_large_vocabularies(dd):
    rng = np.random.default_rng(11)
    for V, dtype in ((380001, "f32"), (770000, "bf16")):
        x = rng.standard_normal((2, V)) * 3
        for kw in SETTINGS[:4]:
            _check(dd, x, _u(rng, 2), dtype, **kw)


def test_entries_that_are_no_settings(dd):
    x = torch.randn(5, 100, device="cuda")
    good = dict(u=[0.5] * 5, temperature=[1.0] * 5, top_k=[3] * 5, top_p=[0.9] * 5, min_p=[0.1] * 5)
    dts = dict(u=torch.float32, temperature=torch.float32, top_k=torch.int32, top_p=torch.float32, min_p=torch.float32)
    nan = float("nan")
    for key, bad in (("u", 1.0), ("u", -0.1), ("u", nan), ("temperature", -1.0), ("temperature", nan),
                     ("temperature", float("inf")), ("top_k", -4), ("top_p", 1.5), ("top_p", nan), ("min_p", -0.5),
                     ("min_p", 2.0)):
        ws = dd.new_workspace(256)
        a = {k: torch.tensor(v, dtype=dts[k], device="cuda") for k, v in good.items()}
        a[key][3] = bad
        tok = dd.sample(x, a.pop("u"), ws=ws, **a)
        assert dd.read_status(ws) == dd.EINTERNAL, (key, bad)
        assert ((tok >= 0) & (tok < 100)).all()


def test_refusals(dd):
    x, u = torch.zeros(4, 10, device="cuda"), torch.zeros(4, device="cuda")
    for a in ((x.double(), u), (x.t().contiguous().t(), u), (x[0], u), (x, u[:3]), (x, u.double()), (x.cpu(), u)):
        with pytest.raises(ValueError):
            dd.sample(*a)
    for kw in (dict(top_p=u[:2]), dict(top_k=u), dict(top_k=1.5), dict(out=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            dd.sample(x, u, **kw)
    for kw in (dict(temperature=-1.0), dict(top_k=-1), dict(top_p=2.0), dict(min_p=-1.0)):
        with pytest.raises(dd.DartreeError):
            dd.sample(x, u, **kw)
    assert dd.sample(x[:0], u[:0]).shape == (0,)


# ------------------------------------------------------------------------------------------ trees

def _tree(rng, C, S, L, V, width=4):
    t = {k: np.full((C, S), -1, np.int32) for k in ("tok", "par", "depth")}
    t["n_nodes"] = rng.integers(1, S + 1, C).astype(np.int32)
    t["n_nodes"][0] = S
    for c in range(C):
        t["tok"][c, 0], t["depth"][c, 0] = 0, 0
        for j in range(1, int(t["n_nodes"][c])):
            ok = [i for i in range(max(0, j - width), j) if t["depth"][c, i] < L]
            p = int(rng.choice(ok)) if ok else 0
            t["par"][c, j], t["depth"][c, j] = p, t["depth"][c, p] + 1
            taken = [t["tok"][c, i] for i in range(1, j) if t["par"][c, i] == p]
            t["tok"][c, j] = rng.choice([v for v in range(V) if v not in taken])
    return t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ["node", "position"])
@pytest.mark.parametrize("C,S,L,V", [(1, 20, 6, 8), (7, 33, 16, 50), (80, 12, 5, 9), (2, 65, 16, 3001)])
def test_walk(dd, C, S, L, V, rows, dtype):
    rng = np.random.default_rng(C + S)
    t = _tree(rng, C, S, L, V)
    n = S if rows == "node" else L
    x = torch.from_numpy(rng.standard_normal((C, n, V)) * (1.0 if V < 100 else 0.1))
    for c in range(C):                                         # the target likes the tree
        for j in range(1, int(t["n_nodes"][c])):
            r = int(t["par"][c, j]) if rows == "node" else int(t["depth"][c, t["par"][c, j]])
            if r < n:
                x[c, r, int(t["tok"][c, j])] += 4.0
    x = x.to(DT[dtype]).cuda()
    dev = {k: torch.from_numpy(v).cuda() for k, v in t.items()}
    mode = dd.ROWS_PER_NODE if rows == "node" else dd.ROWS_PER_POSITION
    deepest = 0
    for kw in SETTINGS[:5] + [dict(temperature=rng.choice([0, 0.5, 1], C).astype(np.float32),
                                   top_k=rng.choice([0, 2, 5], C).astype(np.int32))]:
        u = rng.random((C, n), dtype=np.float32).clip(0, 1 - 2.0 ** -24)
        ws = dd.new_workspace(256)
        got = dd.verify_filtered(dev, x, mode, L, torch.from_numpy(u).cuda(), ws=ws, **{
            k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in kw.items()})
        assert dd.read_status(ws) == 0
        want = sv.verify(t, x.double().cpu().numpy(), rows, L, u, lambda c: {
            k: v[c].item() if isinstance(v, np.ndarray) else float(np.float32(v)) if k != "top_k" else v
            for k, v in kw.items()})
        for k in want:
            np.testing.assert_array_equal(got[k].cpu().numpy(), want[k], err_msg=f"{k} {kw}")
        deepest = max(deepest, int(want["accepted_len"].max()))
    assert deepest >= 2


def test_greedy_settings_are_the_greedy_walk(dd):
    rng = np.random.default_rng(3)
    t = _tree(rng, 6, 40, 8, 30)
    x = torch.randn(6, 40, 30, device="cuda") * 0.3
    for c in range(6):
        for j in range(1, int(t["n_nodes"][c])):
            x[c, int(t["par"][c, j]), int(t["tok"][c, j])] += 1.0
    dev = {k: torch.from_numpy(v).cuda() for k, v in t.items()}
    a = dd.verify(dev, x, dd.ROWS_PER_NODE, 8)
    b = dd.verify_filtered(dev, x, dd.ROWS_PER_NODE, 8, torch.rand(6, 40, device="cuda"), temperature=0.0)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_malformed_trees_end(dd):
    """A slot that is its own ancestor's parent: the walk stops after L steps and says so."""
    tok = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    tree = dict(tok=tok, par=torch.tensor([[-1, 0, 1]], dtype=torch.int32, device="cuda"),
                depth=torch.tensor([[0, 0, 0]], dtype=torch.int32, device="cuda"),
                n_nodes=torch.tensor([3], dtype=torch.int32, device="cuda"))
    x = torch.full((1, 1, 4), float("-inf"), device="cuda")
    x[..., 0] = 1.0
    ws = dd.new_workspace(256)
    r = dd.verify_filtered(tree, x, dd.ROWS_PER_POSITION, 1, torch.zeros(1, 1, device="cuda"), ws=ws)
    assert dd.read_status(ws) == dd.EINTERNAL
    assert r["accepted_len"].item() == 1 and r["path"].tolist() == [[1]]
    tree["n_nodes"].fill_(-5)
    r = dd.verify_filtered(tree, x, dd.ROWS_PER_POSITION, 1, torch.zeros(1, 1, device="cuda"))
    assert r["accepted_len"].item() == 0 and r["bonus"].item() == 0


def test_streams_and_graphs(dd):
    """Captured with given buffers and replayed on new inputs; on a side stream."""
    x = torch.randn(3, 5000, device="cuda") * 2
    u, out, ws = torch.rand(3, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), dd.new_workspace(256)
    kw = dict(temperature=0.8, top_k=50, top_p=0.9)
    dd.sample(x, u, out=out, ws=ws, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dd.sample(x, u, out=out, ws=ws, **kw)
    for i in range(3):
        x.copy_(torch.randn(3, 5000, device="cuda") * 2)
        u.copy_(torch.rand(3, device="cuda"))
        g.replay()
        got = out.clone()
        assert torch.equal(dd.sample(x, u, **kw), got)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = dd.sample(x, u, stream=s, **kw)
    s.synchronize()
    assert torch.equal(side, got)


def test_a_row_of_minus_infinity_matches_no_slot(dd):
    """A slot whose token is -1 is not what such a row draws."""
    tree = dict(tok=torch.tensor([[5, -1, 2]], dtype=torch.int32, device="cuda"),
                par=torch.tensor([[-1, 0, 0]], dtype=torch.int32, device="cuda"),
                depth=torch.tensor([[0, 1, 1]], dtype=torch.int32, device="cuda"),
                n_nodes=torch.tensor([3], dtype=torch.int32, device="cuda"))
    x = torch.full((1, 3, 8), float("-inf"), device="cuda")
    r = dd.verify_filtered(tree, x, dd.ROWS_PER_NODE, 4, torch.full((1, 3), 0.5, device="cuda"))
    assert r["accepted_len"].item() == 0 and r["bonus"].item() == -1 and r["path"].tolist() == [[-1] * 4]


def test_draws_on_two_streams_at_once(dd):
    """Calls that run beside one another, each with its own settings, draw what they draw alone."""
    xs = [torch.randn(24, 30011, device="cuda") * (1 + i) for i in range(3)]
    us = [torch.rand(24, device="cuda") for _ in range(3)]
    kw = [dict(top_p=0.9), dict(temperature=0.6, top_k=40), dict(temperature=1.4, top_p=0.99, min_p=0.001)]
    alone = [dd.sample(x, u, **k) for x, u, k in zip(xs, us, kw)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got += [(i, dd.sample(xs[i], us[i], stream=streams[i], **kw[i])) for i in range(3)]
    torch.cuda.synchronize()
    for i, t in got:
        assert torch.equal(t, alone[i])
