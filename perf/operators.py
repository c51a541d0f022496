"""Measured cases of the paged-cache operators: a layer of the target model served over a
key/value cache kept in pages (append with head norms and rotation, attention of new
tokens, accumulated attention weights, eviction by them, commit of a verified tree's path).

`run` computes an operator in its plain form (elementary torch operations in 32 bits, rounded
once at the end) or, with `own` set, makes the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
THETA = 1.0e6
EPS = 1.0e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases

def _case(op, name=None, **kw):
    c = dict(op=op, C=1, S=1, ctx=0, ragged=False, tree=False, Hq=32, Hkv=8, D=128, page=64, dtype="bf16")
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one request's verification tree (65 slots), one layer: latency of the smallest common call
        _case("append", "append tree c1", C=1, S=65, ctx=2048, tree=True),
        # prompt chunks of odd lengths of eight requests, head norms, rotation and store of one layer
        _case("append", "append chunks c8", C=8, S=2047, ctx=1000, ragged=True),
        # single-token step of one request
        _case("attention", "attention token c1", C=1, S=1, ctx=2048),
        # single-token step of a full batch with ragged contexts, bound by the cache it reads
        _case("attention", "attention token c64", C=64, S=1, ctx=8192, ragged=True),
        # verification pass over the pruned trees of four requests
        _case("attention", "attention tree c4", C=4, S=65, ctx=2048, ragged=True, tree=True),
        # a long prompt's second chunk, bound by the tensor cores
        _case("attention", "attention prompt 8192", C=1, S=8192, ctx=8192),
        # weights gathered while sixteen requests step token by token
        _case("weights", "weights token c16", C=16, S=1, ctx=8192, ragged=True),
        # weights gathered from the last part of two prompts, small heads
        _case("weights", "weights chunk c2", C=2, S=511, ctx=8000, ragged=True, Hq=16, Hkv=4, D=64, page=32),
        # a cache of one request that has reached its limit, fp32 pages
        _case("evict", "evict f32 c1", C=1, ctx=4100, budget=1024, sink=4, recent=256, page=16, dtype="f32"),
        # a batch's caches cut to an eighth
        _case("evict", "evict c16", C=16, ctx=16384, ragged=True, budget=2048, sink=4, recent=512),
        # the accepted path of one tree, and of a full batch's trees
        _case("commit", "commit c1", C=1, S=65, L=16, ctx=2048),
        _case("commit", "commit c64", C=64, S=65, L=16, ctx=2000, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "weights", "evict", "commit"])
    D = rng.choice([64, 128, 128])
    Hkv, grp = rng.choice([(1, 8), (2, 5), (4, 4), (8, 4), (8, 1), (4, 7), (2, 16)])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = "bf16" if op in ("attention", "weights") else rng.choice(["bf16", "bf16", "f32"])
    C = _log(rng, 1, 64)
    kw = dict(C=C, D=D, Hq=Hkv * grp, Hkv=Hkv, page=page, dtype=dtype, ragged=rng.random() < 0.7)
    if op == "evict":
        ctx = _log(rng, 64, min(16384, 262144 // C))
        budget = max(1, ctx // rng.choice([2, 4, 8]))
        sink = rng.randint(0, min(4, budget))
        return _case(op, ctx=ctx, budget=budget, sink=sink, recent=rng.randint(0, (budget - sink) // 2), **kw)
    if op == "commit":
        return _case(op, S=rng.randint(2, 128), L=rng.randint(1, 32), ctx=_log(rng, 1, 8192), **kw)
    tree = op != "weights" and rng.random() < 0.3
    S = rng.randint(2, 128) if tree else 1 if rng.random() < 0.3 else _log(rng, 2, 8192 // C)
    return _case(op, S=S, ctx=_log(rng, 1, min(16384 if S == 1 else 8192, 131072 // C)), tree=tree, **kw)


# ------------------------------------------------------------------------------ inputs

def _lengths(case):
    """(new tokens, cached rows) of each request, on the host: what a scheduler has in hand.
    They belong to the case, so that its outputs keep their shapes."""
    C, S, ctx = case["C"], case["S"], case["ctx"]
    rs = np.random.RandomState((C * 1000003 + S * 10007 + ctx) % (2 ** 31))
    new, old = np.full(C, S, np.int64), np.full(C, ctx, np.int64)
    if case["ragged"]:
        old = rs.randint(ctx // 2, ctx + 1, C)
        old[rs.randint(C)] = ctx
        if not case["tree"] and case["op"] != "commit":
            new = rs.randint((S + 1) // 2, S + 1, C)
            new[rs.randint(C)] = S
    return new, old


def _trees(case, rs):
    """Trees of S slots, twelve to a depth: parents, depths and the mask of ancestors."""
    C, S = case["C"], case["S"]
    depth = np.zeros((C, S), np.int32)
    depth[:, 1:] = 1 + np.arange(S - 1) // 12
    mask = np.zeros((C, S, S), np.uint8)
    n = np.full(C, S, np.int32)
    if case["ragged"]:
        n = rs.randint((S + 1) // 2, S + 1, C).astype(np.int32)
    for c in range(C):
        mask[c, 0, 0] = 1
        for j in range(1, n[c]):
            d = depth[c, j]
            lo, hi = (0, 1) if d == 1 else (1 + 12 * (d - 2), 1 + 12 * (d - 1))
            mask[c, j] = mask[c, rs.randint(lo, hi)]
            mask[c, j, j] = 1
        depth[c, n[c]:] = -1
    return mask, depth, n


def prepare(case, seed):
    rs = np.random.RandomState(seed % (2 ** 31))
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    C, S, Hq, Hkv, D, page = (case[k] for k in ("C", "S", "Hq", "Hkv", "D", "page"))
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    new, old = _lengths(case)
    dev = lambda a, t=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(t)  # noqa: E731
    rand = lambda *s, t=dt: torch.randn(s, generator=gen, device=DEV).to(t)  # noqa: E731
    s = dict(case=case, new=new, old=old, tree=None, q_start=None)
    if case["tree"]:
        mask, depth, n = _trees(case, rs)
        s["tree"] = dict(mask=dev(mask, torch.uint8), pos=dev(depth), n_nodes=dev(n))
        s["depth"], new = depth, n.astype(np.int64)
        s["new"] = new
        T = C * S
    else:
        T = int(new.sum())
        if case["ragged"] and op != "commit":
            s["q_start"] = dev(np.concatenate([[0], np.cumsum(new)]))
    s["T"] = T
    # pages: every request's rows in pages scattered over the pool
    rows = case["ctx"] + S
    most = -(-rows // page)
    spare = -(-case["budget"] // page) if op == "evict" else 0
    pool = C * (most + spare)
    order = rs.permutation(pool).astype(np.int32)
    s["table"] = dev(order[:C * most].reshape(C, most))
    s["n_ctx"] = dev(old)
    s["k"], s["v"] = rand(pool, Hkv, page, D), rand(pool, Hkv, page, D)
    if op == "append":
        # one projection's output: queries, keys and values of a token side by side
        qkv = rand(T, (Hq + 2 * Hkv) * D)
        s["q_in"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k_in"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["v_in"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["gq"] = (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(dt)
        s["gk"] = (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(dt)
        s["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device=DEV)
    if op in ("attention", "weights"):
        s["q"] = rand(T, Hq, D)
        s["out"] = torch.zeros(T, Hq, D, dtype=dt, device=DEV)
        s["lse"] = torch.zeros(T, Hq, dtype=torch.float32, device=DEV)
    if op == "weights":
        _attention(s, s["out"], s["lse"])       # the step's attention gave the rows' sums
        s["w"] = torch.rand(C, Hkv, most * page, generator=gen, device=DEV)
    if op == "evict":
        # sums of attention weights: a few rows hold most of the mass
        s["w"] = torch.randn(C, Hkv, most * page, generator=gen, device=DEV).mul_(1.5).exp_()
        s["dst"] = dev(order[C * most:].reshape(C, spare))
        s["keep"] = torch.zeros(C, Hkv, case["budget"], dtype=torch.int32, device=DEV)
        s["n_out"] = torch.zeros(C, dtype=torch.int32, device=DEV)
        s["w_out"] = torch.zeros(C, Hkv, spare * page, device=DEV)
    if op == "commit":
        L = case["L"]
        acc = rs.randint(0, min(L, S - 1) + 1, C)
        path = np.full((C, L), -1, np.int64)
        for c in range(C):
            path[c, :acc[c]] = 1 + np.sort(rs.choice(S - 1, acc[c], replace=False))
        s["path"], s["acc"] = dev(path), dev(acc)
        s["host_path"], s["host_acc"] = path, acc
        s["n_out"] = torch.zeros(C, dtype=torch.int32, device=DEV)
    if own:
        import diffusion_drafter_draft_gb300 as dd
        s["cache"] = dd.PagedCache(s["k"], s["v"], s["table"], s["n_ctx"], Hq, S, T=T, q_start=s["q_start"])
    return s


# ------------------------------------------------------------------------------ plain forms

def _starts(s):
    """First row of q of each request."""
    return np.arange(len(s["new"])) * s["case"]["S"] if s["tree"] is not None else np.concatenate([[0], np.cumsum(s["new"])[:-1]])


def _rows(s, c, n, table=None):
    """(page, row in it) of the first n cached rows of request c."""
    page = s["case"]["page"]
    j = torch.arange(n, device=DEV)
    return (s["table"] if table is None else table)[c][j // page].long(), j % page


def _gather(s, pool, c, n):
    """The first n cached rows of request c, [Hkv, n, D]."""
    p, r = _rows(s, c, n)
    return pool[p, :, r].transpose(0, 1)


def _visible(s, c, i0, i1):
    """Which of the request's rows the new tokens i0 .. i1 - 1 see, [i1 - i0, n]."""
    old, new = int(s["old"][c]), int(s["new"][c])
    j = torch.arange(old + new, device=DEV)
    if s["tree"] is None:
        return j[None, :] <= old + torch.arange(i0, i1, device=DEV)[:, None]
    seen = torch.ones(i1 - i0, old + new, dtype=torch.bool, device=DEV)
    seen[:, old:] = s["tree"]["mask"][c, i0:i1, :new] != 0
    return seen


def _blocks(s, c):
    """Row ranges of a request whose scores fit a gigabyte or so."""
    n, new = int(s["old"][c] + s["new"][c]), int(s["new"][c])
    step = max(1, (1 << 28) // (n * s["case"]["Hq"]))
    return [(i, min(new, i + step)) for i in range(0, new, step)]


def _scores(s, q, kc):
    """Scaled scores [Hkv, grp, rows, n] of q [rows, Hq, D] against kc [Hkv, n, D], in kc's type."""
    rows, Hq, D = q.shape
    Hkv = kc.shape[0]
    g = q.to(kc.dtype).view(rows, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
    return (g @ kc.transpose(1, 2) * (1.0 / math.sqrt(D))).view(Hkv, Hq // Hkv, rows, -1)


def _attention(s, out, lse):
    Hq, D = s["case"]["Hq"], s["case"]["D"]
    for c, r0 in enumerate(_starts(s)):
        n = int(s["old"][c] + s["new"][c])
        kc, vc = _gather(s, s["k"], c, n).float(), _gather(s, s["v"], c, n).float()
        for i0, i1 in _blocks(s, c):
            x = _scores(s, s["q"][r0 + i0:r0 + i1], kc).masked_fill_(~_visible(s, c, i0, i1), float("-inf"))
            m = x.amax(-1, keepdim=True)
            x = x.sub_(m).exp_()
            l = x.sum(-1, keepdim=True)
            o = (x.flatten(1, 2) @ vc).view(*x.shape[:3], D) / l
            out[r0 + i0:r0 + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, Hq, D).to(out.dtype)
            lse[r0 + i0:r0 + i1] = (m + l.log()).squeeze(-1).permute(2, 0, 1).reshape(i1 - i0, Hq)


def _append(s):
    case = s["case"]
    D, page = case["D"], case["page"]
    dt = s["q_out"].dtype
    rows, pos, pages, at = [], [], [], []
    for c, r0 in enumerate(_starts(s)):
        i = torch.arange(int(s["new"][c]), device=DEV)
        j = int(s["old"][c]) + i
        rows.append(int(r0) + i)
        pos.append(j if s["tree"] is None else int(s["old"][c]) + s["tree"]["pos"][c, :len(i)])
        pages.append(s["table"][c][j // page].long())
        at.append(j % page)
    rows, pos, pages, at = (torch.cat(x) for x in (rows, pos, pages, at))
    inv = THETA ** (-2.0 * torch.arange(D // 2, device=DEV, dtype=torch.float64) / D)
    ang = pos.double()[:, None] * inv
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def turned(x, g):
        x = x[rows].float()
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * g.float()
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(dt)

    s["q_out"][rows] = turned(s["q_in"], s["gq"])
    s["k"][pages, :, at] = turned(s["k_in"], s["gk"])
    s["v"][pages, :, at] = s["v_in"][rows]


def _weights(s):
    for c, r0 in enumerate(_starts(s)):
        old, n = int(s["old"][c]), int(s["old"][c] + s["new"][c])
        kc = _gather(s, s["k"], c, n).float()
        w = torch.zeros(kc.shape[:2], device=DEV)
        for i0, i1 in _blocks(s, c):
            x = _scores(s, s["q"][r0 + i0:r0 + i1], kc)
            l = s["lse"][r0 + i0:r0 + i1].t().reshape(x.shape[:3])
            x = x.sub_(l[..., None]).exp_().masked_fill_(~_visible(s, c, i0, i1), 0.0)
            w += x.sum((1, 2))
        s["w"][c, :, :old] = s["w"][c, :, :old] * 0.9 + w[:, :old]
        s["w"][c, :, old:n] = w[:, old:]


def _evict(s):
    case = s["case"]
    B, sink, recent, Hkv = case["budget"], case["sink"], case["recent"], case["Hkv"]
    s["keep"].fill_(-1)
    for c in range(case["C"]):
        n = int(s["old"][c])
        w = s["w"][c, :, :n]
        if n <= B:
            idx = torch.arange(n, device=DEV).expand(Hkv, n)
        else:
            rank = w.clone()
            rank[:, :sink] = float("inf")
            rank[:, n - recent:] = float("inf")
            # ties go to the lowest row: a stable sort keeps their order
            idx = rank.sort(dim=1, descending=True, stable=True).indices[:, :B].sort(dim=1).values
        k = idx.shape[1]
        h = torch.arange(Hkv, device=DEV)[:, None]
        p, r = s["table"][c][idx // case["page"]].long(), idx % case["page"]
        dp, dr = _rows(s, c, k, s["dst"])
        s["k"][dp, h, dr] = s["k"][p, h, r]
        s["v"][dp, h, dr] = s["v"][p, h, r]
        s["w_out"][c, :, :k] = w.gather(1, idx)
        s["keep"][c, :, :k] = idx.int()
    s["n_out"].copy_(s["n_ctx"].clamp(max=B))


def _commit(s):
    page = s["case"]["page"]
    for c in range(s["case"]["C"]):
        a, old = int(s["host_acc"][c]), int(s["old"][c])
        if a == 0:
            continue
        j = old + s["path"][c, :a].long()
        d = old + 1 + torch.arange(a, device=DEV)
        t = s["table"][c].long()
        for pool in (s["k"], s["v"]):
            pool[t[d // page], :, d % page] = pool[t[j // page], :, j % page]
    torch.add(s["n_ctx"], s["acc"] + 1, out=s["n_out"])


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if op == "append":
        if own:
            s["cache"].append(s["q_in"], s["k_in"], s["v_in"], s["gq"], s["gk"], eps=EPS, theta=THETA, tree=s["tree"],
                              out=s["q_out"])
        else:
            _append(s)
        return dict(q=s["q_out"], k=s["k"], v=s["v"])
    if op == "attention":
        if own:
            s["cache"].attention(s["q"], tree=s["tree"], out=s["out"], lse=s["lse"])
        else:
            _attention(s, s["out"], s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    if op == "weights":
        if own:
            s["cache"].weights(s["q"], s["lse"], s["w"], tree=s["tree"], decay=0.9)
        else:
            _weights(s)
        return dict(w=s["w"])
    if op == "evict":
        if own:
            s["cache"].evict(s["w"], case["budget"], s["dst"], sink=case["sink"], recent=case["recent"], keep=s["keep"],
                             n_out=s["n_out"], weights_out=s["w_out"])
        else:
            _evict(s)
        return dict(keep=s["keep"], n=s["n_out"], w=s["w_out"], k=s["k"], v=s["v"])
    if own:
        s["cache"].commit(s["path"], s["acc"], n_out=s["n_out"])
    else:
        _commit(s)
    return dict(n=s["n_out"], k=s["k"], v=s["v"])


# ------------------------------------------------------------------------------ work

def work(case):
    """Mean lengths of a ragged batch stand for its requests (three quarters of the most)."""
    C, S, ctx, Hq, Hkv, D = (case[k] for k in ("C", "S", "ctx", "Hq", "Hkv", "D"))
    e = 2 if case["dtype"] == "bf16" else 4
    part = 0.75 if case["ragged"] else 1.0
    old, op = ctx * part, case["op"]
    new = S * part if op != "commit" else S
    if op == "append":
        x = C * new * (Hq + 2 * Hkv) * D
        return dict(bytes=2 * x * e, flops=8 * x)
    # new tokens see the context and about half of one another
    pairs = C * Hq * new * (old + (new + 1) / 2)
    rows = C * Hkv * (old + new)
    if op == "attention":
        return dict(bytes=2 * rows * D * e + 2 * C * new * Hq * D * e + 4 * C * new * Hq, flops=4 * D * pairs)
    if op == "weights":
        return dict(bytes=rows * D * e + C * new * Hq * (D * e + 4) + 8 * rows, flops=2 * D * pairs)
    if op == "evict":
        kept = C * Hkv * min(case["budget"], old)
        return dict(bytes=4 * C * Hkv * old + kept * (4 * D * e + 8), flops=0)
    moved = C * Hkv * min(case["L"], S - 1) / 2
    return dict(bytes=moved * 4 * D * e + 8 * C, flops=0)


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """From the definitions in 64 bits: outputs of copied or chosen values have no entry."""
    s = prepare(case, seed)
    op, D, Hq, Hkv, page = case["op"], case["D"], case["Hq"], case["Hkv"], case["page"]
    grp = Hq // Hkv
    if op in ("evict", "commit"):
        return None
    tree = s["tree"]
    first = 0
    if op == "append":
        q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
        freq = torch.exp(torch.arange(D // 2, device=DEV, dtype=torch.float64) * (-2.0 / D * math.log(THETA)))
    elif op == "attention":
        o = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=DEV)
        z = torch.zeros(s["T"], Hq, dtype=torch.float64, device=DEV)
    else:
        acc = s["w"].double()
    for c in range(case["C"]):
        old, new = int(s["old"][c]), int(s["new"][c])
        n = old + new
        if op == "append":
            for t in range(0, new, 512):
                e = min(new, t + 512)
                i = torch.arange(t, e, device=DEV)
                j = old + i
                v[s["table"][c, j // page].long(), :, j % page] = s["v_in"][first + t:first + e].double()
                p = old + (i if tree is None else tree["pos"][c, t:e].long())
                turn = torch.polar(torch.ones(e - t, 1, D // 2, dtype=torch.float64, device=DEV),
                                   (p.double()[:, None] * freq)[:, None])
                for src, gain, dst in ((s["q_in"], s["gq"], None), (s["k_in"], s["gk"], k)):
                    x = src[first + t:first + e].double()
                    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.double()
                    y = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * turn
                    y = torch.cat([y.real, y.imag], -1)
                    if dst is None:
                        q[first + t:first + e] = y
                    else:
                        dst[s["table"][c, j // page].long(), :, j % page] = y
        else:
            j = torch.arange(n, device=DEV)
            kc = s["k"][s["table"][c, j // page].long(), :, j % page].double()      # [n, Hkv, D]
            vc = s["v"][s["table"][c, j // page].long(), :, j % page].double() if op == "attention" else None
            step = max(1, (1 << 26) // (n * grp))
            if op == "weights":
                acc[c, :, :old] *= 0.9
                acc[c, :, old:n] = 0
            for t in range(0, new, step):
                e = min(new, t + step)
                i = torch.arange(t, e, device=DEV)
                hidden = j[None, :] > (old + i)[:, None]
                if tree is not None:
                    hidden = torch.cat([torch.zeros(e - t, old, dtype=torch.bool, device=DEV),
                                        tree["mask"][c, t:e, :new] == 0], 1)
                for g in range(Hkv):
                    x = torch.einsum("thd,nd->thn", s["q"][first + t:first + e, g * grp:(g + 1) * grp].double(),
                                     kc[:, g]) / math.sqrt(D)
                    x.masked_fill_(hidden[:, None, :], -math.inf)
                    if op == "attention":
                        z[first + t:first + e, g * grp:(g + 1) * grp] = torch.logsumexp(x, -1)
                        o[first + t:first + e, g * grp:(g + 1) * grp] = torch.softmax(x, -1) @ vc[:, g]
                    else:
                        l = s["lse"][first + t:first + e, g * grp:(g + 1) * grp].double()
                        acc[c, g, :n] += torch.exp(x - l[..., None]).sum((0, 1))
        first += case["S"] if tree is not None else new
    if op == "append":
        return dict(q=q, k=k, v=v)
    return dict(out=o, lse=z) if op == "attention" else dict(w=acc)
