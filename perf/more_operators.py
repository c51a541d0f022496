"""Measured cases of a serving step around the paged cache: pages and rows for the step's new
tokens from the requests' lengths (and pages given back), attention of a batch whose requests
share a long prefix, tokens drawn under temperature, top-k, top-p and min-p from given random
numbers, and a tree's verification by such draws.

`run` computes an operator in its plain form (elementary torch operations; draws in 64 bits,
where a token hangs on a sum's last digits) or, with `own` set, makes the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases

def _pages(op, name=None, C=64, S=1, ctx=2048, page=64, tree=False, short=False):
    c = dict(op=op, C=C, S=S, ctx=ctx, page=page, tree=tree, short=short)
    return dict(c, name=name) if name else c


def _shared(name=None, C=64, S=1, G=1, shared=4096, rest=512, ragged=True, tree=False, Hq=32, Hkv=8, D=128, page=64):
    c = dict(op="attention", C=C, S=S, G=G, shared=shared, rest=rest, ragged=ragged, tree=tree, Hq=Hq, Hkv=Hkv, D=D,
             page=page)
    return dict(c, name=name) if name else c


def _draws(op, name=None, C=1, V=151936, dtype="bf16", settings="topk", S=65, L=16, rows="node"):
    c = dict(op=op, C=C, V=V, dtype=dtype, settings=settings)
    if op == "verify":
        c.update(S=S, L=L, rows=rows)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a verification step of a full batch: every request asks for a tree's slots
        _pages("reserve", "reserve trees c64", C=64, S=65, tree=True),
        # a large batch of prompt parts and single tokens, the pool too small for all
        _pages("reserve", "reserve chunks c512", C=512, S=128, ctx=4096, page=16, short=True),
        # after the commit: the pages that the rejected slots held go back
        _pages("release", "release trees c64", C=64, S=65, tree=True),
        # a few requests of one short system prompt, token by token: latency
        _shared("shared tokens c8", C=8, shared=2048, rest=128),
        # a full batch behind one long document, token by token
        _shared("shared tokens c64", C=64, shared=16384, rest=512),
        # verification trees of sixteen requests behind one document
        _shared("shared trees c16", C=16, S=65, shared=8192, rest=512, tree=True),
        # drafts of a few tokens, five documents, small heads, pages of 32
        _shared("shared groups c48", C=48, S=3, G=5, shared=6000, rest=700, Hq=16, Hkv=4, D=64, page=32),
        # one request's next token under the settings that its model is published with
        _draws("sample", "sample c1", C=1),
        # a batch in which every request has settings of its own, some of them greedy
        _draws("sample", "sample mixed c64", C=64, settings="mixed"),
        # a large batch, fp32 logits, nucleus alone
        _draws("sample", "sample nucleus f32 c256", C=256, dtype="f32", settings="nucleus"),
        # one tree verified by draws, a row of logits for each slot
        _draws("verify", "verify c1", C=1),
        # a batch of trees, a row for each position, mixed settings
        _draws("verify", "verify position c32", C=32, settings="mixed", rows="position"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["reserve", "release", "attention", "attention", "attention", "sample", "sample", "verify"])
    if op in ("reserve", "release"):
        C, tree = _log(rng, 1, 512), rng.random() < 0.5
        S = rng.randint(2, 128) if tree else _log(rng, 1, 65536 // C)
        return _pages(op, C=C, S=S, ctx=_log(rng, 1, 8192), page=rng.choice([16, 32, 64, 128, 256]), tree=tree,
                      short=op == "reserve" and rng.random() < 0.3)
    if op == "attention":
        Hkv, grp = rng.choice([(1, 8), (2, 5), (4, 4), (8, 4), (8, 1), (4, 7), (2, 16)])
        C, tree = _log(rng, 2, 64), rng.random() < 0.3
        S = rng.randint(2, 128) if tree else 1 if rng.random() < 0.5 else rng.randint(2, 16)
        most = min(16384, 280000000 // (C * S * Hkv * grp))
        return _shared(C=C, S=S, G=rng.choice([1, 1, min(C, 3), min(C, rng.randint(2, 8))]),
                       shared=_log(rng, 64, max(64, most)), rest=_log(rng, 1, 1024), ragged=rng.random() < 0.7,
                       tree=tree, Hq=Hkv * grp, Hkv=Hkv, D=rng.choice([64, 128, 128]),
                       page=rng.choice([16, 32, 64, 128, 256]))
    dtype, V = rng.choice(["bf16", "bf16", "f32"]), _log(rng, 1000, 151936)
    settings = rng.choice(["mixed", "topk", "nucleus", "min_p", "plain"])
    if op == "sample":
        return _draws(op, C=_log(rng, 1, 256), V=V, dtype=dtype, settings=settings)
    rows = rng.choice(["node", "position"])
    L = rng.randint(1, 16)
    S = rng.randint(2, min(65, 12 * L + 1))
    return _draws(op, C=_log(rng, 1, 32 if rows == "position" else 8), V=V, dtype=dtype, settings=settings, S=S, L=L,
                  rows=rows)


# ------------------------------------------------------------------------------ inputs

def _dev(a, t=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(t)


def _host_rng(case):
    """Lengths belong to the case, so that its outputs keep their shapes."""
    words = [v for v in case.values() if type(v) is int]
    return np.random.RandomState(sum(v * 1000003 ** i for i, v in enumerate(words)) % (2 ** 31))


def prepare(case, seed):
    if case["op"] in ("reserve", "release"):
        return _prepare_pages(case, seed)
    if case["op"] == "attention":
        return _prepare_attention(case, seed)
    return _prepare_draws(case, seed)


def _prepare_pages(case, seed):
    C, S, ctx, page, op = (case[k] for k in ("C", "S", "ctx", "page", "op"))
    rl, rs = _host_rng(case), np.random.RandomState(seed % (2 ** 31))
    old = rl.randint(0, ctx + 1, C)
    new = rl.randint(1, S + 1, C)
    new[rl.rand(C) < (0.0 if case["tree"] else 0.4)] = 1       # single tokens among the prompt parts
    most = -(-(ctx + S) // page) + 1
    held = -(-old // page)
    want = -(-(old + new) // page) - held
    spare = int(want.sum()) * 3 // 4 if case["short"] else int(want.sum()) + 7
    pool = int(held.sum() + want.sum()) + 7
    order = rs.permutation(pool).astype(np.int32)
    table = np.full((C, most), -1, np.int32)
    at = 0
    for c in range(C):
        n = held[c] + (want[c] if op == "release" else 0)
        table[c, :n] = order[at:at + n]
        at += n
    s = dict(case=case, old=old.astype(np.int64), new=new.astype(np.int64), n_ctx=_dev(old))
    free = np.zeros(pool, np.int32)
    if op == "reserve":
        free[:spare] = order[at:at + spare]
        s["n_free"] = _dev([spare])
    else:
        free[:pool - at] = order[at:]
        s["n_free"] = _dev([pool - at])
        s["keep"] = np.minimum(old + 1 + rl.randint(0, 5, C), old + new)
        s["shared"] = np.minimum(old, rl.randint(0, ctx + 1, C) * (rl.rand(C) < 0.5)) // page * page
        s["held"] = old + new
        for k in ("keep", "shared", "held"):
            s["d_" + k] = _dev(s[k])
    s.update(h_table=table, h_free=free, h_n=int(s["n_free"].item()), table=_dev(table), free=_dev(free), pool=pool)
    s["T"] = T = C * S if case["tree"] else int(new.sum())
    s["d_new"] = _dev(new)
    s["n_out"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if op == "reserve":
        s["q_start"] = None if case["tree"] else torch.zeros(C + 1, dtype=torch.int32, device=DEV)
        s["out"] = dict(granted=torch.zeros(C, dtype=torch.int32, device=DEV),
                        slot=torch.zeros(T, dtype=torch.int64, device=DEV),
                        pos=torch.zeros(T, dtype=torch.int32, device=DEV),
                        request=torch.zeros(T, dtype=torch.int32, device=DEV), n_free=s["n_out"])
    if own:
        import diffusion_drafter_draft_gb300 as dd
        pages = torch.zeros(pool, 1, page, 64, dtype=torch.bfloat16, device=DEV)
        s["cache"] = dd.PagedCache(pages, pages.clone(), s["table"], s["n_ctx"], 1, S, T=T, q_start=s.get("q_start"))
    return s


def _prepare_attention(case, seed):
    C, S, G, Hq, Hkv, D, page = (case[k] for k in ("C", "S", "G", "Hq", "Hkv", "D", "page"))
    rl, rs = _host_rng(case), np.random.RandomState(seed % (2 ** 31))
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    start = np.concatenate([[0], np.sort(rl.choice(C - 1, G - 1, replace=False) + 1) if G > 1 else [], [C]])
    start = start.astype(np.int64)
    rows = np.full(G, case["shared"], np.int64)
    rest, new = np.full(C, case["rest"], np.int64), np.full(C, S, np.int64)
    if case["ragged"]:
        if G > 1:
            rows = rl.randint(max(1, case["shared"] // 4), case["shared"] + 1, G)
        rest = rl.randint(0, case["rest"] + 1, C)
        new = rl.randint((S + 1) // 2, S + 1, C)
        new[rl.randint(C)] = S
    group = np.repeat(np.arange(G), np.diff(start))
    old = rows[group] + rest
    s = dict(case=case, new=new, old=old, tree=None, q_start=None, rows=_dev(rows), start=_dev(start))
    most = -(-int(old.max() + S) // page)
    whole = rows // page                                       # pages that a group's requests have in common
    own_pages = -(-(old + S) // page) - whole[group]
    pool = int(whole.sum() + own_pages.sum())
    order = rs.permutation(pool).astype(np.int32)
    table = np.zeros((C, most), np.int32)
    common = np.concatenate([[0], np.cumsum(whole)])
    at = int(common[-1])
    for c in range(C):
        g, w = group[c], whole[group[c]]
        table[c, :w] = order[common[g]:common[g] + w]
        table[c, w:w + own_pages[c]] = order[at:at + own_pages[c]]
        at += int(own_pages[c])
    if case["tree"]:
        mask = np.zeros((C, S, S), np.uint8)
        for c in range(C):
            mask[c, 0, 0] = 1
            for j in range(1, int(new[c])):
                d = (j + 11) // 12
                lo, hi = (0, 1) if d == 1 else (1 + 12 * (d - 2), 1 + 12 * (d - 1))
                mask[c, j] = mask[c, rs.randint(lo, hi)]
                mask[c, j, j] = 1
        s["tree"] = dict(mask=_dev(mask, torch.uint8), n_nodes=_dev(new))
        s["T"] = C * S
    else:
        s["T"] = int(new.sum())
        if case["ragged"]:
            s["q_start"] = _dev(np.concatenate([[0], np.cumsum(new)]))
    s["table"], s["n_ctx"] = _dev(table), _dev(old)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=DEV).to(torch.bfloat16)

    s["k"], s["v"] = rand(pool, Hkv, page, D), rand(pool, Hkv, page, D)
    s["q"] = rand(s["T"], Hq, D)
    s["out"] = torch.zeros(s["T"], Hq, D, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros(s["T"], Hq, device=DEV)
    if own:
        import diffusion_drafter_draft_gb300 as dd
        s["cache"] = dd.PagedCache(s["k"], s["v"], s["table"], s["n_ctx"], Hq, S, T=s["T"], q_start=s["q_start"])
        # (behind the shared pages: what a prefix has in its last page, the rest and the new tokens)
        s["shared"] = s["cache"].shared(s["start"], s["rows"], most_rows=case["shared"],
                                        most_rest=case["rest"] + S + page - 1)
    return s


def _settings(case, R, rs):
    """Scalars of a batch with one setting, or arrays of a value for each request."""
    kind = case["settings"]
    if kind == "topk":
        return dict(temperature=0.7, top_k=20, top_p=0.8, min_p=0.0)
    if kind == "nucleus":
        return dict(temperature=1.0, top_k=0, top_p=0.95, min_p=0.0)
    if kind == "min_p":
        return dict(temperature=1.2, top_k=0, top_p=1.0, min_p=0.05)
    if kind == "plain":
        return dict(temperature=0.9, top_k=0, top_p=1.0, min_p=0.0)
    pick = lambda a, t: _dev(np.array(a)[rs.randint(0, len(a), R)], t)  # noqa: E731
    return dict(temperature=pick([0.0, 0.3, 0.7, 1.0, 1.3], torch.float32), top_k=pick([0, 0, 1, 20, 50, 400], torch.int32),
                top_p=pick([1.0, 0.95, 0.8, 0.5], torch.float32), min_p=pick([0.0, 0.0, 0.05, 0.2], torch.float32))


def _prepare_draws(case, seed):
    C, V, op = case["C"], case["V"], case["op"]
    rs = np.random.RandomState(seed % (2 ** 31))
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    n = 1 if op == "sample" else case["S"] if case["rows"] == "node" else case["L"]
    # a model's logits: a broad floor and a few tokens far above it
    x = torch.randn((C * n, V), generator=gen, device=DEV).mul_(2.5)
    step = V // 20
    at = torch.randint(0, V, (C * n, 1), generator=gen, device=DEV) + step * torch.arange(20, device=DEV)
    x.scatter_(1, at % V, 15.0 * torch.rand((C * n, 20), generator=gen, device=DEV))
    s = dict(case=case, set=_settings(case, C, rs))
    u = torch.rand((C * n,), generator=gen, device=DEV)
    if op == "sample":
        s["logits"], s["u"] = x.to(DTYPES[case["dtype"]]), u
        s["out"] = torch.zeros(C, dtype=torch.int32, device=DEV)
    else:
        S, L = case["S"], case["L"]
        x = x.view(C, n, V)
        tok, par = np.full((C, S), -1, np.int64), np.full((C, S), -1, np.int64)
        depth, nodes = np.full((C, S), -1, np.int64), rs.randint((S + 1) // 2, S + 1, C)
        put = []
        for c in range(C):
            m = int(nodes[c])
            tok[c, :m] = rs.choice(V, m, replace=False)
            depth[c, 0] = 0
            j = np.arange(1, m)
            depth[c, 1:m] = 1 + (j - 1) // 12
            for i in j:
                d = depth[c, i]
                par[c, i] = 0 if d == 1 else rs.randint(1 + 12 * (d - 2), 1 + 12 * (d - 1))
            cur = 0                                            # the target likes one path of the tree
            while True:
                kids = np.flatnonzero(par[c] == cur)
                if not len(kids):
                    break
                kid = int(kids[rs.randint(len(kids))])
                put.append((c, cur if case["rows"] == "node" else int(depth[c, cur]), int(tok[c, kid]),
                            22.0 if rs.rand() < 0.75 else 10.0))
                cur = kid
        if put:
            i = [_dev([p[k] for p in put], torch.int64) for k in range(3)]
            x[i[0], i[1], i[2]] = _dev([p[3] for p in put], torch.float32)
        s["target"], s["u"] = x.to(DTYPES[case["dtype"]]), u.view(C, n)
        s["tree"] = dict(tok=_dev(tok), par=_dev(par), depth=_dev(depth), n_nodes=_dev(nodes))
        s["out"] = dict(accepted_len=torch.zeros(C, dtype=torch.int32, device=DEV),
                        path=torch.zeros(C, L, dtype=torch.int32, device=DEV),
                        bonus=torch.zeros(C, dtype=torch.int32, device=DEV))
    if own:
        import diffusion_drafter_draft_gb300 as dd
        s["ws"] = dd.new_workspace(256)
    return s


# ------------------------------------------------------------------------------ plain forms

def _reserve(s):
    """The lengths are the scheduler's own, on the host; what the kernels read goes to the GPU."""
    case = s["case"]
    C, S, page, T = case["C"], case["S"], case["page"], s["T"]
    table, free, n, rows = s["h_table"].copy(), s["h_free"], s["h_n"], T
    granted, q = np.zeros(C, np.int64), np.zeros(C + 1, np.int64)
    slot, pos, req = np.full(T, -1, np.int64), np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    for c in range(C):
        o, m = int(s["old"][c]), int(s["new"][c])
        held = -(-o // page)
        need = -(-(o + m) // page) - held
        first = c * S if case["tree"] else int(q[c])
        if o + m <= table.shape[1] * page and need <= n and (case["tree"] or m <= rows):
            table[c, held:held + need] = free[n - need:n][::-1]
            n -= need
            rows -= m
            granted[c] = m
            j = o + np.arange(m)
            slot[first:first + m] = table[c, j // page].astype(np.int64) * page + j % page
            pos[first:first + m] = j
            req[first:first + m] = c
        q[c + 1] = q[c] + granted[c]
    out = s["out"]
    s["table"].copy_(_dev(table))
    if s["q_start"] is not None:
        s["q_start"].copy_(_dev(q))
    for k, v in (("granted", granted), ("slot", slot), ("pos", pos), ("request", req), ("n_free", [n])):
        out[k].copy_(_dev(v, out[k].dtype))


def _release(s):
    page, free, n = s["case"]["page"], s["h_free"].copy(), s["h_n"]
    for c in range(s["case"]["C"]):
        lo = max(-(-int(s["keep"][c]) // page), -(-int(s["shared"][c]) // page))
        give = s["h_table"][c, lo:max(lo, -(-int(s["held"][c]) // page))]
        free[n:n + len(give)] = give
        n += len(give)
    s["free"].copy_(_dev(free))
    s["n_out"].copy_(_dev([n]))


def _starts(s):
    """First row of q of each request."""
    new = s["new"]
    fixed = s["tree"] is not None or s["q_start"] is None
    return np.arange(len(new)) * s["case"]["S"] if fixed else np.concatenate([[0], np.cumsum(new)[:-1]])


def _attention(s):
    case = s["case"]
    Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    if s["tree"] is not None:
        s["out"].zero_()
        s["lse"].zero_()
    for c, r0 in enumerate(_starts(s)):
        old, new = int(s["old"][c]), int(s["new"][c])
        n = old + new
        j = torch.arange(n, device=DEV)
        p, r = s["table"][c][j // page].long(), j % page
        kc, vc = s["k"][p, :, r].transpose(0, 1).float(), s["v"][p, :, r].transpose(0, 1).float()
        q = s["q"][r0:r0 + new].float().view(new, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
        x = (q @ kc.transpose(1, 2) * (1.0 / math.sqrt(D))).view(Hkv, Hq // Hkv, new, n)
        if s["tree"] is None:
            seen = j[None, :] <= old + torch.arange(new, device=DEV)[:, None]
        else:
            seen = torch.ones(new, n, dtype=torch.bool, device=DEV)
            seen[:, old:] = s["tree"]["mask"][c, :new, :new] != 0
        x.masked_fill_(~seen, float("-inf"))
        m = x.amax(-1, keepdim=True)
        x = x.sub_(m).exp_()
        l = x.sum(-1, keepdim=True)
        o = (x.flatten(1, 2) @ vc).view(*x.shape[:3], D) / l
        s["out"][r0:r0 + new] = o.permute(2, 0, 1, 3).reshape(new, Hq, D).to(torch.bfloat16)
        s["lse"][r0:r0 + new] = (m + l.log()).squeeze(-1).permute(2, 0, 1).reshape(new, Hq)


def _setting(s, key, rows, n):
    """A setting of logit rows `rows`, n of them to a request, as a column in 64 bits."""
    v = s["set"][key]
    if not torch.is_tensor(v):
        # (the settings are float32 where they are numbers of the call, too)
        return torch.full((len(rows), 1), float(np.float32(v)), dtype=torch.float64, device=DEV)
    return v.double()[rows // n][:, None]


def _drawn(s, logits, u, n=1):
    """The token of each row of logits [R, V], n rows to a request."""
    R, V = logits.shape
    out = torch.empty(R, dtype=torch.int64, device=DEV)
    step = max(1, (1 << 23) // V)
    for r0 in range(0, R, step):
        rows = torch.arange(r0, min(R, r0 + step), device=DEV)
        x = logits[rows].double()
        T, k, p, least = (_setting(s, key, rows, n) for key in ("temperature", "top_k", "top_p", "min_p"))
        y, order = x.sort(dim=1, descending=True, stable=True)      # ties: the lowest token first
        w = ((y - y[:, :1]) / torch.where(T > 0, T, torch.ones_like(T))).exp()
        rank = torch.arange(V, device=DEV)[None]
        keep = (rank < k) | (k <= 0)
        wk = w * keep
        before = wk.cumsum(1) - wk
        keep &= (before < p * wk.sum(1, keepdim=True)) | (p >= 1) | (rank == 0)
        keep &= (w >= least) | (rank == 0)
        keep &= (rank == 0) | (T > 0)                               # temperature 0: the largest
        kept = torch.zeros_like(w).scatter_(1, order, w * keep)
        c = kept.cumsum(1)
        goal = u[rows].double()[:, None] * c[:, -1:]
        out[rows] = (c <= goal).sum(1).clamp(max=V - 1)
    return out


def _verify(s):
    case, t = s["case"], s["tree"]
    C, L, S = case["C"], case["L"], case["S"]
    x = s["target"]
    n = x.shape[1]
    tok = _drawn(s, x.flatten(0, 1), s["u"].flatten(), n).view(C, n)
    cur = torch.zeros(C, dtype=torch.int64, device=DEV)
    live = torch.ones(C, dtype=torch.bool, device=DEV)
    out = s["out"]
    out["accepted_len"].zero_()
    out["path"].fill_(-1)
    out["bonus"].fill_(-1)
    slots = torch.arange(S, device=DEV)[None]
    at = torch.arange(C, device=DEV)
    for step in range(L + 1):
        row = cur if case["rows"] == "node" else t["depth"][at, cur].long()
        has = live & (row < n)                                      # no row at the last depth: no bonus token
        d = tok[at, row.clamp(max=n - 1)]
        hit = (t["par"] == cur[:, None]) & (t["tok"] == d[:, None]) & (slots < t["n_nodes"][:, None]) & (slots > 0)
        found = hit.any(1) & has
        kid = torch.where(hit, slots, torch.full_like(slots, S)).amin(1)
        out["bonus"].copy_(torch.where(has & ~found, d, out["bonus"].long()))
        if step < L:
            out["path"][:, step] = torch.where(found, kid, torch.full_like(kid, -1)).int()
        out["accepted_len"] += found.int()
        cur = torch.where(found, kid, cur)
        live = found


def run(state):
    s, op = state, state["case"]["op"]
    if op == "reserve":
        if own:
            s["cache"].reserve(s["d_new"], s["free"], s["n_free"], out=s["out"])
        else:
            _reserve(s)
        got = dict(s["out"], table=s["table"])
        return got if s["q_start"] is None else dict(got, q_start=s["q_start"])
    if op == "release":
        if own:
            s["cache"].release(s["d_held"], s["d_keep"], s["free"], s["n_free"], n_shared=s["d_shared"], n_out=s["n_out"])
        else:
            _release(s)
        return dict(free=s["free"], n_free=s["n_out"])
    if op == "attention":
        if own:
            s["cache"].attention(s["q"], tree=s["tree"], shared=s["shared"], out=s["out"], lse=s["lse"])
        else:
            _attention(s)
        return dict(out=s["out"], lse=s["lse"])
    if op == "sample":
        if own:
            import diffusion_drafter_draft_gb300 as dd
            dd.sample(s["logits"], s["u"], **s["set"], out=s["out"], ws=s["ws"])
        else:
            s["out"].copy_(_drawn(s, s["logits"], s["u"]))
        return s["out"]
    if own:
        import diffusion_drafter_draft_gb300 as dd
        rows = dd.ROWS_PER_NODE if s["case"]["rows"] == "node" else dd.ROWS_PER_POSITION
        dd.verify_filtered(s["tree"], s["target"], rows, s["case"]["L"], s["u"], **s["set"], out=s["out"], ws=s["ws"])
    else:
        _verify(s)
    return s["out"]


# ------------------------------------------------------------------------------ work

def work(case):
    """Means stand for ragged lengths; a walk reads about three rows of logits."""
    op, C = case["op"], case["C"]
    if op in ("reserve", "release"):
        S, page = case["S"], case["page"]
        new = C * (S + 1) / 2 * (1.0 if case["tree"] else 0.6)
        if op == "release":
            return dict(bytes=16 * C + 8 * new / page, flops=0)
        return dict(bytes=16 * (C * S if case["tree"] else new) + 20 * C + 8 * new / page, flops=0)
    if op == "attention":
        S, G, Hq, Hkv, D = (case[k] for k in ("S", "G", "Hq", "Hkv", "D"))
        part = 0.5 if case["ragged"] else 1.0
        new = S * (0.75 if case["ragged"] else 1.0)
        shared = case["shared"] * (0.625 if case["ragged"] and G > 1 else 1.0)
        rest = case["rest"] * part
        rows = Hkv * (G * shared + C * (rest + new))
        pairs = C * Hq * new * (shared + rest + (new + 1) / 2)
        return dict(bytes=4 * rows * D + 4 * C * new * Hq * D + 4 * C * new * Hq, flops=4 * D * pairs)
    e = 2 if case["dtype"] == "bf16" else 4
    rows = C if op == "sample" else 3 * C
    return dict(bytes=rows * (case["V"] * e + 24), flops=4 * rows * case["V"])


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """From the definitions in 64 bits: tables, slots and page lists are chosen, not computed."""
    if case["op"] in ("reserve", "release"):
        return None
    if case["op"] == "attention":
        return _exact_attention(case, seed)
    rows = case["C"] * (1 if case["op"] == "sample" else 4)
    if rows * case["V"] > 300 * 151936:
        return None
    s = prepare(case, seed)
    u = s["u"].double().cpu().numpy()

    def token(c, row, v):
        of = {k: float(a[c].item()) if torch.is_tensor(a) else float(np.float32(a)) for k, a in s["set"].items()}
        x = row.double().cpu().numpy()
        if of["temperature"] == 0:
            return int(np.flatnonzero(x == x.max())[0])
        p = np.exp((x - x.max()) / of["temperature"])
        order = np.lexsort((np.arange(len(x)), -x))
        if of["top_k"] > 0:
            order = order[:int(of["top_k"])]
        if of["top_p"] < 1:
            q = np.cumsum(p[order])
            order = order[:int(np.searchsorted(q, of["top_p"] * q[-1], side="left")) + 1]
        order = np.sort(order[(p[order] >= of["min_p"]) | (order == order[0])])
        q = np.cumsum(p[order])
        return int(order[min(int(np.searchsorted(q, v * q[-1], side="right")), len(order) - 1)])

    if case["op"] == "sample":
        return np.array([token(c, s["logits"][c], u[c]) for c in range(case["C"])], np.int32)
    C, L = case["C"], case["L"]
    t = {k: v.cpu().numpy() for k, v in s["tree"].items()}
    acc, path, bonus = np.zeros(C, np.int32), np.full((C, L), -1, np.int32), np.full(C, -1, np.int32)
    for c in range(C):
        kids = {}
        for j in range(int(t["n_nodes"][c]) - 1, 0, -1):
            kids[int(t["par"][c, j]), int(t["tok"][c, j])] = j
        cur = 0
        while True:
            r = cur if case["rows"] == "node" else int(t["depth"][c, cur])
            if r >= s["target"].shape[1]:
                break
            d = token(c, s["target"][c, r], u[c, r])
            if (cur, d) not in kids:
                bonus[c] = d
                break
            cur = kids[cur, d]
            path[c, acc[c]] = cur
            acc[c] += 1
    return dict(accepted_len=acc, path=path, bonus=bonus)


def _exact_attention(case, seed):
    s = prepare(case, seed)
    S, Hq, Hkv, D, page = (case[k] for k in ("S", "Hq", "Hkv", "D", "page"))
    grp = Hq // Hkv
    o = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    z = torch.zeros(s["T"], Hq, dtype=torch.float64, device=DEV)
    first = 0
    for c in range(case["C"]):
        old, new = int(s["old"][c]), int(s["new"][c])
        n = old + new
        j = torch.arange(n, device=DEV)
        at, row = s["table"][c, j // page].long(), j % page
        i = torch.arange(new, device=DEV)
        hidden = j[None, :] > (old + i)[:, None]
        if s["tree"] is not None:
            hidden = torch.cat([torch.zeros(new, old, dtype=torch.bool, device=DEV),
                                s["tree"]["mask"][c, :new, :new] == 0], 1)
        for g in range(Hkv):
            kc, vc = s["k"][at, g, row].double(), s["v"][at, g, row].double()
            x = torch.einsum("thd,nd->thn", s["q"][first:first + new, g * grp:(g + 1) * grp].double(), kc) / math.sqrt(D)
            x.masked_fill_(hidden[:, None, :], -math.inf)
            z[first:first + new, g * grp:(g + 1) * grp] = torch.logsumexp(x, -1)
            o[first:first + new, g * grp:(g + 1) * grp] = torch.softmax(x, -1) @ vc
        first += S if s["q_start"] is None else new
    return dict(out=o, lse=z)
