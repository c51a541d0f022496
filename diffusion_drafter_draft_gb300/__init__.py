"""Python binding of libdartree.so, the sm_103a DARTree draft-tree build and verify step.

Argument marshalling only: every step runs in the library's CUDA kernels. Tensors
are torch CUDA tensors (PyTorch supplies device memory and the current stream);
they are passed to the C ABI as raw device pointers. There is no CPU fallback:
if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "DartreeError", "lib", "library_path", "F32", "BF16", "ROWS_PER_POSITION", "ROWS_PER_NODE",
    "workspace_bytes", "new_workspace", "topk", "expand", "prune", "tree_mask", "build_tree",
    "verify", "read_status", "clear_status", "Round", "EXPORTS", "heap_build", "HeapRound",
    "verify_sample", "adaptive_budget", "lm_head_topk", "tree_attention", "AttnParams", "HostRounds",
    "HostInputs", "HostOutputs", "PagedCache",
]

F32, BF16 = 0, 1
ROWS_PER_POSITION, ROWS_PER_NODE = 0, 1
OK, EINVAL, EDTYPE, EWORKSPACE, ECUDA, ETIMEOUT, EINTERNAL, EUNSUPPORTED = 0, -1, -2, -3, -4, -5, -6, -7

EXPORTS = ("dartree_head_init", "dartree_workspace_bytes", "dartree_topk", "dartree_expand", "dartree_prune",
           "dartree_tree_mask", "dartree_build_tree", "dartree_verify", "dartree_read_status",
           "dartree_clear_status", "dartree_status_string", "dartree_verify_static", "dartree_gemm_bf16",
           "dartree_head_prepare", "dartree_round", "dartree_selftest_wait", "dartree_timing",
           "dartree_timing_read", "dartree_kernel_name", "dartree_heap_workspace_bytes", "dartree_heap_build",
           "dartree_verify_sample", "dartree_adaptive_budget", "dartree_lm_head_workspace_bytes",
           "dartree_lm_head_topk", "dartree_tree_attention_workspace_bytes", "dartree_tree_attention", "dartree_host_session_create",
           "dartree_host_session_destroy", "dartree_host_stage", "dartree_host_round", "dartree_host_input_bytes",
           "dartree_paged_workspace_bytes", "dartree_paged_attention_plan", "dartree_paged_append",
           "dartree_paged_attention", "dartree_paged_weights", "dartree_paged_evict", "dartree_paged_commit", "dartree_paged_commit_weights")


class DartreeError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {code} ({status_string(code)})")


class Head(ctypes.Structure):
    _fields_ = [("E", ctypes.c_void_p), ("Wq", ctypes.c_void_p), ("V", ctypes.c_int), ("H", ctypes.c_int),
                ("dtype", ctypes.c_int), ("WqT", ctypes.c_void_p)]


class Params(ctypes.Structure):
    _fields_ = [("C", ctypes.c_int), ("L", ctypes.c_int), ("K", ctypes.c_int), ("W", ctypes.c_int),
                ("B", ctypes.c_int), ("beta", ctypes.c_float)]


class Candidates(ctypes.Structure):
    _fields_ = [("tok", ctypes.c_void_p), ("logit", ctypes.c_void_p)]


class Supertree(ctypes.Structure):
    _fields_ = [("tok", ctypes.c_void_p), ("par", ctypes.c_void_p), ("score", ctypes.c_void_p),
                ("n", ctypes.c_void_p)]


class AttnParams(ctypes.Structure):
    _fields_ = [("C", ctypes.c_int), ("S", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("D", ctypes.c_int), ("N", ctypes.c_int), ("theta", ctypes.c_float)]


class PagedParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("C", "T", "S", "Hq", "Hkv", "D", "page", "n_pages", "max_pages", "dtype")]


class PagedCacheDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "table", "n_ctx", "q_start")]


class PagedPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("few", "tiles_per_cta", "chunks", "cluster", "alone")] + \
        [("part_bytes", ctypes.c_size_t)]


class PagedTokens(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ldq", ctypes.c_int64),
                ("ldk", ctypes.c_int64), ("ldv", ctypes.c_int64), ("gq", ctypes.c_void_p), ("gk", ctypes.c_void_p),
                ("pos_base", ctypes.c_void_p), ("eps", ctypes.c_float), ("theta", ctypes.c_float)]


class Tree(ctypes.Structure):
    _fields_ = [("tok", ctypes.c_void_p), ("par", ctypes.c_void_p), ("depth", ctypes.c_void_p),
                ("score", ctypes.c_void_p), ("n_nodes", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("pos", ctypes.c_void_p)]


_LIB = None


def library_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdartree.so")


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with diffusion_drafter_draft_gb300._build.build()")
    L = ctypes.CDLL(path)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    P = ctypes.POINTER
    sig = {
        "dartree_head_init": (i, [P(Head), vp, vp, i, i, i]),
        "dartree_round": (i, [P(Head), P(Params), vp, vp, vp, vp, i, P(Tree), vp, vp, vp, vp, sz, vp]),
        "dartree_selftest_wait": (i, [vp, sz, i, ctypes.c_uint, vp]),
        "dartree_timing": (i, [i]),
        "dartree_timing_read": (i, [i, P(ctypes.c_int), P(ctypes.c_double)]),
        "dartree_kernel_name": (ctypes.c_char_p, [i]),
        "dartree_head_prepare": (i, [P(Head), vp, vp]),
        "dartree_heap_workspace_bytes": (sz, [P(Params), i, i, i]),
        "dartree_heap_build": (i, [P(Head), P(Params), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "dartree_workspace_bytes": (sz, [P(Params), i, i, i]),
        "dartree_topk": (i, [vp, i, i, i, i, vp, vp, vp, sz, vp]),
        "dartree_expand": (i, [P(Head), P(Params), vp, vp, P(Candidates), P(Supertree), vp, sz, vp]),
        "dartree_prune": (i, [P(Params), P(Supertree), vp, P(Tree), vp]),
        "dartree_tree_mask": (i, [P(Params), P(Tree), vp]),
        "dartree_build_tree": (i, [P(Head), P(Params), vp, vp, vp, P(Tree), P(Supertree), P(Candidates), vp, sz,
                                   vp]),
        "dartree_verify": (i, [P(Params), P(Tree), vp, i, i, i, vp, vp, vp, vp, sz, vp]),
        "dartree_verify_static": (i, [P(Params), P(Tree), vp, i, i, i, vp, vp, vp, vp]),
        "dartree_verify_sample": (i, [P(Params), P(Tree), vp, i, i, i, ctypes.c_float, ctypes.c_uint64, vp, vp, vp,
                                      vp, sz, vp]),
        "dartree_adaptive_budget": (i, [i, P(ctypes.c_int), P(ctypes.c_int)]),
        "dartree_lm_head_workspace_bytes": (sz, [i, i, i, i]),
        "dartree_tree_attention_workspace_bytes": (sz, [P(AttnParams)]),
        "dartree_tree_attention": (i, [P(AttnParams), vp, vp, vp, vp, vp, vp, P(Tree), vp, vp, sz, vp]),
        "dartree_lm_head_topk": (i, [vp, vp, i, i, i, i, i, vp, vp, vp, sz, vp]),
        "dartree_gemm_bf16": (i, [vp, vp, vp, i, i, i, vp, vp]),
        "dartree_read_status": (i, [vp, P(ctypes.c_int32), vp]),
        "dartree_clear_status": (i, [vp, vp]),
        "dartree_status_string": (ctypes.c_char_p, [i]),
        "dartree_host_session_create": (i, [P(Head), P(Params), i, P(vp)]),
        "dartree_host_session_destroy": (None, [vp]),
        "dartree_host_stage": (i, [vp, P(HostInputs)]),
        "dartree_host_round": (i, [vp, P(HostOutputs), vp]),
        "dartree_host_input_bytes": (sz, [vp, i]),
        "dartree_paged_workspace_bytes": (sz, [P(PagedParams)]),
        "dartree_paged_attention_plan": (i, [P(PagedParams), P(PagedPlan)]),
        "dartree_paged_append": (i, [P(PagedParams), P(PagedTokens), P(PagedCacheDesc), P(Tree), vp, vp, sz, vp]),
        "dartree_paged_attention": (i, [P(PagedParams), vp, P(PagedCacheDesc), P(Tree), ctypes.c_float, vp, vp, vp, sz,
                                        vp]),
        "dartree_paged_weights": (i, [P(PagedParams), vp, vp, P(PagedCacheDesc), P(Tree), ctypes.c_float,
                                      ctypes.c_float, vp, vp, sz, vp]),
        "dartree_paged_evict": (i, [P(PagedParams), P(PagedCacheDesc), vp, i, i, i, vp, i, vp, vp, vp, vp, sz, vp]),
        "dartree_paged_commit": (i, [P(PagedParams), P(PagedCacheDesc), vp, vp, i, vp, vp, sz, vp]),
        "dartree_paged_commit_weights": (i, [P(PagedParams), P(PagedCacheDesc), vp, vp, i, vp, vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _LIB = L
    return L


def status_string(code: int) -> str:
    try:
        return lib().dartree_status_string(code).decode()
    except Exception:  # library missing while formatting an error
        return "?"


def _call(name: str, *args) -> None:
    rc = getattr(lib(), name)(*args)
    if rc != OK:
        raise DartreeError(rc, name)


# --------------------------------------------------------------------------- tensors

_DT = {torch.float32: F32, torch.bfloat16: BF16}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _need(t: torch.Tensor, name: str, dtype=None, shape=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _stream(stream=None) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _keep(stream, *tensors) -> None:
    """Tensors allocated here and used by work enqueued on a side stream are not
    reused by the caching allocator before that work is done."""
    if stream is None or stream == torch.cuda.current_stream():
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _params(C, L, K, W, B, beta) -> Params:
    return Params(int(C), int(L), int(K), int(W), int(B), float(beta))


def workspace_bytes(C, L, K, W, B, beta, V, H, dtype_code) -> int:
    n = lib().dartree_workspace_bytes(ctypes.byref(_params(C, L, K, W, B, beta)), int(V), int(H), int(dtype_code))
    if n == 0:
        raise DartreeError(EINVAL, "dartree_workspace_bytes")
    return int(n)


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    ws = torch.zeros(int(nbytes), dtype=torch.uint8, device=device or "cuda")
    if ws.data_ptr() % 256:
        raise RuntimeError("workspace is not 256-byte aligned")
    return ws


def read_status(ws: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int32(0)
    _call("dartree_read_status", ctypes.c_void_p(ws.data_ptr()), ctypes.byref(v), _stream(stream))
    return int(v.value)


def selftest_wait(ws: torch.Tensor, which: int, limit_us: int, stream=None) -> None:
    """Enqueues a bounded wait on something never signalled (0: mbarrier, 1: grid
    barrier); it must end after limit_us with DARTREE_ETIMEOUT in ws's status word."""
    _call("dartree_selftest_wait", ctypes.c_void_p(ws.data_ptr()), ws.numel(), int(which), int(limit_us),
          _stream(stream))


def num_kernel_ids() -> int:
    """Kernel families the library times (ids 0 .. n-1; the last one is "other")."""
    n = 0
    while lib().dartree_kernel_name(n).decode() != "unknown":
        n += 1
    return n


def timing(enable: bool) -> None:
    """Starts (clearing earlier records) or stops per-kernel launch timing."""
    _call("dartree_timing", int(bool(enable)))


def kernel_times() -> dict:
    """{kernel family: (launches, total device ms)} recorded since timing(True)."""
    out = {}
    for k in range(num_kernel_ids()):
        n, ms = ctypes.c_int(0), ctypes.c_double(0.0)
        _call("dartree_timing_read", k, ctypes.byref(n), ctypes.byref(ms))
        if n.value:
            out[lib().dartree_kernel_name(k).decode()] = (int(n.value), float(ms.value))
    return out


def clear_status(ws: torch.Tensor, stream=None) -> None:
    _call("dartree_clear_status", ctypes.c_void_p(ws.data_ptr()), _stream(stream))


def _head(E: torch.Tensor, Wq: torch.Tensor, prepare: bool = False, stream=None):
    """(head description, W_q^T tensor or None). With prepare, bf16 heads get W_q^T
    for the small-batch path; the caller keeps the returned tensor alive while the
    head is used."""
    V, H = E.shape
    _need(E, "E")
    _need(Wq, "Wq", E.dtype, (H, H))
    h = Head()
    _call("dartree_head_init", ctypes.byref(h), ctypes.c_void_p(E.data_ptr()), ctypes.c_void_p(Wq.data_ptr()),
          int(V), int(H), _dtype_code(E))
    wqt = None
    if prepare and E.dtype == torch.bfloat16:
        wqt = torch.empty((H, H), dtype=E.dtype, device=E.device)
        _call("dartree_head_prepare", ctypes.byref(h), ctypes.c_void_p(wqt.data_ptr()), _stream(stream))
    return h, wqt


# --------------------------------------------------------------------------- steps

def topk(logits: torch.Tensor, K: int, ws: torch.Tensor | None = None, stream=None):
    """S1: top-K of every row of logits [rows, V] -> (tok int32 [rows, K], val float32 [rows, K])."""
    rows, V = logits.shape
    _need(logits, "logits")
    dev = logits.device
    tok = torch.empty((rows, K), dtype=torch.int32, device=dev)
    val = torch.empty((rows, K), dtype=torch.float32, device=dev)
    ws = ws if ws is not None else new_workspace(256, dev)
    _call("dartree_topk", ctypes.c_void_p(logits.data_ptr()), int(rows), int(V), int(K), _dtype_code(logits),
          ctypes.c_void_p(tok.data_ptr()), ctypes.c_void_p(val.data_ptr()), ctypes.c_void_p(ws.data_ptr()),
          ws.numel(), _stream(stream))
    return tok, val


def _alloc_supertree(C, L, W, dev):
    return dict(tok=torch.empty((C, L, W), dtype=torch.int32, device=dev),
                par=torch.empty((C, L, W), dtype=torch.int32, device=dev),
                score=torch.empty((C, L, W), dtype=torch.float32, device=dev),
                n=torch.empty((C, L), dtype=torch.int32, device=dev))


def _st_struct(st) -> Supertree:
    return Supertree(st["tok"].data_ptr(), st["par"].data_ptr(), st["score"].data_ptr(), st["n"].data_ptr())


def _alloc_tree(C, B, dev, with_mask=True):
    S = B + 1
    t = dict(tok=torch.empty((C, S), dtype=torch.int32, device=dev),
             par=torch.empty((C, S), dtype=torch.int32, device=dev),
             depth=torch.empty((C, S), dtype=torch.int32, device=dev),
             score=torch.empty((C, S), dtype=torch.float32, device=dev),
             n_nodes=torch.empty((C,), dtype=torch.int32, device=dev))
    if with_mask:
        t["mask"] = torch.empty((C, S, S), dtype=torch.uint8, device=dev)
        t["pos"] = torch.empty((C, S), dtype=torch.int32, device=dev)
    return t


def _tree_struct(t) -> Tree:
    g = lambda k: t[k].data_ptr() if k in t and t[k] is not None else None  # noqa: E731
    return Tree(g("tok"), g("par"), g("depth"), g("score"), g("n_nodes"), g("mask"), g("pos"))


def expand(E, Wq, hidden, anchor, cand_tok, cand_val, W, beta, ws=None, stream=None):
    """S2-S7 from a candidate table -> supertree dict (tok, par, score, n)."""
    C, L, H = hidden.shape
    K = cand_tok.shape[-1]
    head, wqt = _head(E, Wq, prepare=True, stream=stream)
    _need(hidden, "hidden", E.dtype, (C, L, H))
    _need(anchor, "anchor", torch.int32, (C,))
    _need(cand_tok, "cand_tok", torch.int32, (C, L, K))
    _need(cand_val, "cand_val", torch.float32, (C, L, K))
    p = _params(C, L, K, W, 1, beta)
    ws = ws if ws is not None else new_workspace(workspace_bytes(C, L, K, W, 1, beta, E.shape[0], H, head.dtype),
                                                 hidden.device)
    st = _alloc_supertree(C, L, W, hidden.device)
    cand = Candidates(cand_tok.data_ptr(), cand_val.data_ptr())
    sts = _st_struct(st)
    _call("dartree_expand", ctypes.byref(head), ctypes.byref(p), ctypes.c_void_p(hidden.data_ptr()),
          ctypes.c_void_p(anchor.data_ptr()), ctypes.byref(cand), ctypes.byref(sts), ctypes.c_void_p(ws.data_ptr()),
          ws.numel(), _stream(stream))
    _keep(stream, ws, wqt)
    return st


def prune(st, anchor, B, stream=None):
    """S8: deferred pruning of a supertree -> tree dict (tok, par, depth, score, n_nodes)."""
    C, L, W = st["tok"].shape
    for k in ("tok", "par", "n"):
        _need(st[k], k, torch.int32)
    _need(st["score"], "score", torch.float32)
    _need(anchor, "anchor", torch.int32, (C,))
    t = _alloc_tree(C, B, anchor.device, with_mask=False)
    p = _params(C, L, 1, W, B, 0.0)
    ts, sts = _tree_struct(t), _st_struct(st)
    _call("dartree_prune", ctypes.byref(p), ctypes.byref(sts), ctypes.c_void_p(anchor.data_ptr()), ctypes.byref(ts),
          _stream(stream))
    return t


def tree_mask(tree, L, stream=None):
    """S9: adds mask and pos to a tree dict (in place) and returns it."""
    C, S = tree["par"].shape
    for k in ("par", "depth", "n_nodes"):
        _need(tree[k], k, torch.int32)
    tree["mask"] = torch.empty((C, S, S), dtype=torch.uint8, device=tree["par"].device)
    tree["pos"] = torch.empty((C, S), dtype=torch.int32, device=tree["par"].device)
    p = _params(C, L, 1, 1, S - 1, 0.0)
    ts = _tree_struct(tree)
    _call("dartree_tree_mask", ctypes.byref(p), ctypes.byref(ts), _stream(stream))
    return tree


def verify(tree, target, rows: int, L: int, ws=None, stream=None):
    """S10: greedy longest accepted prefix -> dict(accepted_len, path, bonus)."""
    C, S = tree["tok"].shape
    V = target.shape[-1]
    _need(target, "target", None, (C, L, V) if rows == ROWS_PER_POSITION else (C, S, V))
    dev = target.device
    out = dict(accepted_len=torch.empty((C,), dtype=torch.int32, device=dev),
               path=torch.empty((C, L), dtype=torch.int32, device=dev),
               bonus=torch.empty((C,), dtype=torch.int32, device=dev))
    if ws is None:
        ws = new_workspace(256 + 8 * C * max(L, S), dev)
    p = _params(C, L, 1, 1, S - 1, 0.0)
    ts = _tree_struct(tree)
    _call("dartree_verify", ctypes.byref(p), ctypes.byref(ts), ctypes.c_void_p(target.data_ptr()), int(rows), int(V),
          _dtype_code(target), ctypes.c_void_p(out["accepted_len"].data_ptr()), ctypes.c_void_p(out["path"].data_ptr()),
          ctypes.c_void_p(out["bonus"].data_ptr()), ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(stream))
    return out


def verify_sample(tree, target, rows: int, L: int, temperature: float, seed: int, ws=None, stream=None):
    """S10 at temperature T > 0 (Gumbel-max draws, Philox4x32-10 noise keyed by seed)
    -> dict(accepted_len, path, bonus)."""
    C, S = tree["tok"].shape
    V = target.shape[-1]
    _need(target, "target", None, (C, L, V) if rows == ROWS_PER_POSITION else (C, S, V))
    dev = target.device
    out = dict(accepted_len=torch.empty((C,), dtype=torch.int32, device=dev),
               path=torch.empty((C, L), dtype=torch.int32, device=dev),
               bonus=torch.empty((C,), dtype=torch.int32, device=dev))
    if ws is None:
        ws = new_workspace(256 + 8 * C * max(L, S), dev)
    p = _params(C, L, 1, 1, S - 1, 0.0)
    ts = _tree_struct(tree)
    _call("dartree_verify_sample", ctypes.byref(p), ctypes.byref(ts), ctypes.c_void_p(target.data_ptr()), int(rows),
          int(V), _dtype_code(target), float(temperature), int(seed) & 0xFFFFFFFFFFFFFFFF,
          ctypes.c_void_p(out["accepted_len"].data_ptr()), ctypes.c_void_p(out["path"].data_ptr()),
          ctypes.c_void_p(out["bonus"].data_ptr()), ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(stream))
    return out


def adaptive_budget(C: int) -> tuple[int, int]:
    """(B, W) for C concurrent requests (dartree_adaptive_budget)."""
    B, W = ctypes.c_int(), ctypes.c_int()
    _call("dartree_adaptive_budget", int(C), ctypes.byref(B), ctypes.byref(W))
    return B.value, W.value


def lm_head_topk(hidden, W_lm, K: int, ws=None, stream=None):
    """The drafter's LM head fused with S1: hidden [R, H] x W_lm[V, H]^T -> per-row
    top-K (tok [R, K] int32, val [R, K] fp32), logits never written."""
    R, H = hidden.shape
    V = W_lm.shape[0]
    _need(hidden, "hidden", torch.bfloat16, (R, H))
    _need(W_lm, "W_lm", torch.bfloat16, (V, H))
    dev = hidden.device
    tok = torch.empty((R, K), dtype=torch.int32, device=dev)
    val = torch.empty((R, K), dtype=torch.float32, device=dev)
    need = lib().dartree_lm_head_workspace_bytes(R, V, H, K)
    if need == 0:
        raise DartreeError(EUNSUPPORTED, "dartree_lm_head_workspace_bytes")
    if ws is None:
        ws = new_workspace(need, dev)
    _call("dartree_lm_head_topk", ctypes.c_void_p(hidden.data_ptr()), ctypes.c_void_p(W_lm.data_ptr()), R, V, H,
          int(K), BF16, ctypes.c_void_p(tok.data_ptr()), ctypes.c_void_p(val.data_ptr()),
          ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(stream))
    return tok, val


def tree_attention(q, k_tree, v_tree, k_cache, vt_cache, n_ctx, tree, theta: float = 1.0e6, ws=None,
                   stream=None):
    """One attention layer of the verification pass over the tree (dartree_tree_attention):
    q [C, S, Hq, D], k_tree/v_tree [C, S, Hkv, D], k_cache [C, Hkv, N, D], vt_cache
    [C, Hkv, D, N] (bf16), n_ctx [C] int32, tree with mask/pos/n_nodes -> out [C, S, Hq, D]."""
    C, S, Hq, D = q.shape
    Hkv = k_tree.shape[2]
    N = k_cache.shape[2]
    for name, x, shp in (("q", q, (C, S, Hq, D)), ("k_tree", k_tree, (C, S, Hkv, D)),
                         ("v_tree", v_tree, (C, S, Hkv, D)), ("k_cache", k_cache, (C, Hkv, N, D)),
                         ("vt_cache", vt_cache, (C, Hkv, D, N))):
        _need(x, name, torch.bfloat16, shp)
    _need(n_ctx, "n_ctx", torch.int32, (C,))
    _need(tree["mask"], "mask", torch.uint8, (C, S, S))
    _need(tree["pos"], "pos", torch.int32, (C, S))
    _need(tree["n_nodes"], "n_nodes", torch.int32, (C,))
    p = AttnParams(C, S, Hq, Hkv, D, N, float(theta))
    need = lib().dartree_tree_attention_workspace_bytes(ctypes.byref(p))
    if need == 0:
        raise DartreeError(EUNSUPPORTED, "dartree_tree_attention_workspace_bytes")
    if ws is None:
        ws = new_workspace(need, q.device)
    out = torch.empty((C, S, Hq, D), dtype=torch.bfloat16, device=q.device)
    ts = _tree_struct({k: tree[k] for k in ("mask", "pos", "n_nodes")})
    _call("dartree_tree_attention", ctypes.byref(p), *(ctypes.c_void_p(x.data_ptr()) for x in
                                                       (q, k_tree, v_tree, k_cache, vt_cache, n_ctx)),
          ctypes.byref(ts), ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
          _stream(stream))
    return out


def verify_static(tree, target, rows: int, L: int, stream=None):
    """S10 through dartree_verify_static (no workspace; scratch in a fixed device array)."""
    C, S = tree["tok"].shape
    V = target.shape[-1]
    _need(target, "target", None, (C, L, V) if rows == ROWS_PER_POSITION else (C, S, V))
    dev = target.device
    out = dict(accepted_len=torch.empty((C,), dtype=torch.int32, device=dev),
               path=torch.empty((C, L), dtype=torch.int32, device=dev),
               bonus=torch.empty((C,), dtype=torch.int32, device=dev))
    p = _params(C, L, 1, 1, S - 1, 0.0)
    ts = _tree_struct(tree)
    _call("dartree_verify_static", ctypes.byref(p), ctypes.byref(ts), ctypes.c_void_p(target.data_ptr()), int(rows),
          int(V), _dtype_code(target), ctypes.c_void_p(out["accepted_len"].data_ptr()),
          ctypes.c_void_p(out["path"].data_ptr()), ctypes.c_void_p(out["bonus"].data_ptr()), _stream(stream))
    return out


def gemm_bf16(A, B, status=None, stream=None):
    """Building block: D = A . B^T (bf16 in, fp32 out) through the tcgen05 GEMM."""
    M, K = A.shape
    N = B.shape[0]
    _need(A, "A", torch.bfloat16)
    _need(B, "B", torch.bfloat16, (N, K))
    D = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _call("dartree_gemm_bf16", ctypes.c_void_p(A.data_ptr()), ctypes.c_void_p(B.data_ptr()),
          ctypes.c_void_p(D.data_ptr()), int(M), int(N), int(K),
          ctypes.c_void_p(status.data_ptr()) if status is not None else None, _stream(stream))
    return D


def build_tree(E, Wq, base, hidden, anchor, K, W, B, beta, ws=None, keep_intermediates=False, stream=None):
    """S1-S9: one tree build -> tree dict (+ 'cand_tok', 'cand_val', 'st' when keep_intermediates)."""
    C, L, V = base.shape
    H = E.shape[1]
    head, wqt = _head(E, Wq, prepare=True, stream=stream)
    _need(base, "base", E.dtype, (C, L, V))
    _need(hidden, "hidden", E.dtype, (C, L, H))
    _need(anchor, "anchor", torch.int32, (C,))
    dev = base.device
    p = _params(C, L, K, W, B, beta)
    ws = ws if ws is not None else new_workspace(workspace_bytes(C, L, K, W, B, beta, V, H, head.dtype), dev)
    t = _alloc_tree(C, B, dev)
    ts = _tree_struct(t)
    st_p = cand_p = None
    if keep_intermediates:
        st = _alloc_supertree(C, L, W, dev)
        t["st"] = st
        t["cand_tok"] = torch.empty((C, L, K), dtype=torch.int32, device=dev)
        t["cand_val"] = torch.empty((C, L, K), dtype=torch.float32, device=dev)
        st_p = ctypes.byref(_st_struct(st))
        cand_p = ctypes.byref(Candidates(t["cand_tok"].data_ptr(), t["cand_val"].data_ptr()))
    _call("dartree_build_tree", ctypes.byref(head), ctypes.byref(p), ctypes.c_void_p(base.data_ptr()),
          ctypes.c_void_p(hidden.data_ptr()), ctypes.c_void_p(anchor.data_ptr()), ctypes.byref(ts), st_p, cand_p,
          ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(stream))
    _keep(stream, ws, wqt)
    return t


class Round:
    """One draft round (build + verify) with every buffer allocated once.

    run() enqueues dartree_build_tree and dartree_verify on the current stream and
    allocates nothing, so it can be timed, repeated or captured in a CUDA graph.
    """

    def __init__(self, E, Wq, C, L, K, W, B, beta, rows, device=None):
        self.E, self.Wq = E, Wq
        self.V, self.H = E.shape
        self.C, self.L, self.K, self.W, self.B, self.beta, self.rows = C, L, K, W, B, beta, rows
        dev = device or E.device
        self.head, self.wqt = _head(E, Wq, prepare=True)
        self.p = _params(C, L, K, W, B, beta)
        self.ws = new_workspace(workspace_bytes(C, L, K, W, B, beta, self.V, self.H, self.head.dtype), dev)
        self.tree = _alloc_tree(C, B, dev)
        self._ts = _tree_struct(self.tree)
        self.out = dict(accepted_len=torch.empty((C,), dtype=torch.int32, device=dev),
                        path=torch.empty((C, L), dtype=torch.int32, device=dev),
                        bonus=torch.empty((C,), dtype=torch.int32, device=dev))
        self.dtype_code = self.head.dtype

    def run(self, base, hidden, anchor, target, stream=None):
        """dartree_round: build + verify in one call."""
        _call("dartree_round", ctypes.byref(self.head), ctypes.byref(self.p), ctypes.c_void_p(base.data_ptr()),
              ctypes.c_void_p(hidden.data_ptr()), ctypes.c_void_p(anchor.data_ptr()),
              ctypes.c_void_p(target.data_ptr()), int(self.rows), ctypes.byref(self._ts),
              ctypes.c_void_p(self.out["accepted_len"].data_ptr()), ctypes.c_void_p(self.out["path"].data_ptr()),
              ctypes.c_void_p(self.out["bonus"].data_ptr()), ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel(),
              _stream(stream))
        return self.out

    def run_two_calls(self, base, hidden, anchor, target, stream=None):
        """The same round as dartree_build_tree followed by dartree_verify."""
        s = _stream(stream)
        _call("dartree_build_tree", ctypes.byref(self.head), ctypes.byref(self.p), ctypes.c_void_p(base.data_ptr()),
              ctypes.c_void_p(hidden.data_ptr()), ctypes.c_void_p(anchor.data_ptr()), ctypes.byref(self._ts), None,
              None, ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel(), s)
        _call("dartree_verify", ctypes.byref(self.p), ctypes.byref(self._ts), ctypes.c_void_p(target.data_ptr()),
              int(self.rows), int(self.V), int(self.dtype_code), ctypes.c_void_p(self.out["accepted_len"].data_ptr()),
              ctypes.c_void_p(self.out["path"].data_ptr()), ctypes.c_void_p(self.out["bonus"].data_ptr()),
              ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel(), s)
        return self.out


class HostInputs(ctypes.Structure):
    _fields_ = [("base_logits", ctypes.c_void_p), ("block_hidden", ctypes.c_void_p), ("anchor", ctypes.c_void_p),
                ("target", ctypes.c_void_p)]


class HostOutputs(ctypes.Structure):
    _fields_ = [("accepted_len", ctypes.c_void_p), ("path", ctypes.c_void_p), ("bonus", ctypes.c_void_p)]


class HostRounds:
    """Rounds fed from host buffers through the library's host session
    (dartree_host_session_create / dartree_host_stage / dartree_host_round): the
    session holds two device sets of the inputs, and round i runs from set i % 2
    while round i + 1's inputs are copied into the other set on the session's copy
    stream. Each round's results are copied into the caller's host buffers on the
    current stream right after the round, complete once that stream is synchronised.
    Host tensors should be pinned for the copies to overlap the rounds.
    """

    KEYS = ("base", "hidden", "anchor", "target")

    def __init__(self, rnd: "Round", like: dict = None):
        self.rnd = rnd
        h = ctypes.c_void_p()
        _call("dartree_host_session_create", ctypes.byref(rnd.head), ctypes.byref(rnd.p), int(rnd.rows),
              ctypes.byref(h))
        self._s = h
        self._keep = []  # host tensors of the rounds in flight

    def __del__(self):
        s = getattr(self, "_s", None)
        if s is not None and s.value and _LIB is not None:
            _LIB.dartree_host_session_destroy(s)
            self._s = None

    def h2d_bytes(self) -> int:
        return sum(int(lib().dartree_host_input_bytes(self._s, k)) for k in range(4))

    @staticmethod
    def _host(t: torch.Tensor, name: str) -> int:
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
        return t.data_ptr()

    def copy_in(self, i: int, host: dict):
        """Stage round i's inputs (host tensors, pinned for overlap): dartree_host_stage."""
        x = HostInputs(*(self._host(host[k], k) for k in self.KEYS))
        _call("dartree_host_stage", self._s, ctypes.byref(x))
        self._keep = (self._keep + [host])[-2:]

    def run(self, i: int, host_out: dict, stream=None):
        """Round i on the current stream from its staged inputs, results into host_out
        (host int32 tensors shaped like Round.out): dartree_host_round."""
        o = HostOutputs(*(self._host(host_out[k], k) for k in ("accepted_len", "path", "bonus")))
        _call("dartree_host_round", self._s, ctypes.byref(o), _stream(stream))
        return host_out


class HeapRound:
    """Node-by-node best-first drafting (one head evaluation per popped node), the
    baseline the deferred search replaces; every buffer allocated once, run()
    allocates nothing (it can be timed or captured in a CUDA graph)."""

    def __init__(self, E, Wq, C, L, K, B, beta, device=None):
        self.V, self.H = E.shape
        self.C, self.L, self.K, self.B, self.beta = C, L, K, B, beta
        dev = device or E.device
        self.head, self.wqt = _head(E, Wq, prepare=True)
        self.p = _params(C, L, K, 1, B, beta)
        n = lib().dartree_heap_workspace_bytes(ctypes.byref(self.p), int(self.V), int(self.H), int(self.head.dtype))
        if n == 0:
            raise DartreeError(EUNSUPPORTED, "dartree_heap_workspace_bytes")
        self.ws = new_workspace(n, dev)
        self.out = dict(tok=torch.empty((C, B), dtype=torch.int32, device=dev),
                        parent=torch.empty((C, B), dtype=torch.int32, device=dev),
                        depth=torch.empty((C, B), dtype=torch.int32, device=dev),
                        score=torch.empty((C, B), dtype=torch.float32, device=dev))

    def run(self, base, hidden, anchor, stream=None):
        o = self.out
        _call("dartree_heap_build", ctypes.byref(self.head), ctypes.byref(self.p), ctypes.c_void_p(base.data_ptr()),
              ctypes.c_void_p(hidden.data_ptr()), ctypes.c_void_p(anchor.data_ptr()),
              ctypes.c_void_p(o["tok"].data_ptr()), ctypes.c_void_p(o["parent"].data_ptr()),
              ctypes.c_void_p(o["depth"].data_ptr()), ctypes.c_void_p(o["score"].data_ptr()),
              ctypes.c_void_p(self.ws.data_ptr()), self.ws.numel(), _stream(stream))
        return o


def heap_build(E, Wq, base, hidden, anchor, K, B, beta, stream=None):
    """dartree_heap_build on fresh buffers -> dict(tok, parent, depth, score) [C, B] in pop order."""
    C, L, _ = base.shape
    h = HeapRound(E, Wq, C, L, K, B, beta, device=base.device)
    out = h.run(base, hidden, anchor, stream)
    _keep(stream, h.ws, h.wqt)
    out["_keep"] = (h.ws, h.wqt)
    return out


class PagedCache:
    """One layer's key/value cache kept in pages and the calls on it (dartree_paged_*):
    append, attention and weights for a step's new tokens, evict, commit.

      k_pages, v_pages  [n_pages, Hkv, page, D], bf16 or float32 (keys rotated)
      table             [C, max_pages] int32, the page of each run of `page` rows
      n_ctx             [C] int32, rows cached before the step's new tokens
      Hq, S             query heads; most new tokens of a request
      q_start           [C + 1] int32 first rows of q (T rows in all); None: S tokens of
                        every request, or a tree's S slots
      ws                a workspace to use (shared by calls that follow one another on
                        the device; the one of a larger batch will do; cleared, and ordered
                        between streams, by the caller); allocated when None

    The tensors are read at every call: a serving loop changes table, n_ctx and q_start
    in place. Nothing is allocated by a call that is given its outputs, so it can be
    captured into a CUDA graph (the object is kept as long as the graph). read_status(cache.ws)
    tells what the kernels found wrong in lengths and tables. Calls run on `stream` (default:
    the current stream of the pages' device) and outputs they allocate belong to it; the
    workspace is made on the stream that is current when the object is, and the first call on
    another stream waits for that and keeps the memory until the work there is done (calls
    that are captured on another stream do not wait: torch.cuda.graph has waited for the
    device). An object is used by one host thread at a time.
    """

    def __init__(self, k_pages, v_pages, table, n_ctx, Hq, S, T=None, q_start=None, ws=None):
        _need(k_pages, "k_pages")
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [n_pages, Hkv, page, D]")
        self.n_pages, self.Hkv, self.page, self.D = k_pages.shape
        self.device, self.dtype = k_pages.device, k_pages.dtype
        self.Hq, self.S = int(Hq), int(S)
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table must be [C, max_pages]")
        self.C, self.max_pages = table.shape
        if T is None:
            if q_start is not None:
                raise ValueError("T (rows of q) is needed with q_start")
            T = self.C * self.S
        self.T = int(T)
        self._need(v_pages, "v_pages", self.dtype, k_pages.shape)
        self._need(table, "table", torch.int32)
        self._need(n_ctx, "n_ctx", torch.int32, (self.C,))
        if q_start is not None:
            self._need(q_start, "q_start", torch.int32, (self.C + 1,))
        self.k_pages, self.v_pages, self.table, self.n_ctx, self.q_start = k_pages, v_pages, table, n_ctx, q_start
        self.p = PagedParams(self.C, self.T, self.S, self.Hq, self.Hkv, self.D, self.page, self.n_pages,
                             self.max_pages, _dtype_code(k_pages))
        self._m = PagedCacheDesc(k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), n_ctx.data_ptr(),
                                 q_start.data_ptr() if q_start is not None else None)
        n = lib().dartree_paged_workspace_bytes(ctypes.byref(self.p))
        if n == 0:
            raise DartreeError(EUNSUPPORTED, "dartree_paged_workspace_bytes")
        self._made, self._known = None, None            # end of the workspace's fill, streams that know it
        if ws is None:
            # (only its status word has to start at zero; the calls fill the rest themselves)
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
            s = torch._C._cuda_getCurrentRawStream(self.device.index)
            self._known = {s}
            self._made = self._on_device(lambda: self._clear(ws, s))
        else:
            self._need(ws, "ws", torch.uint8)
        self.ws = ws
        self._wsp = (ws.data_ptr(), ws.numel())
        self.rows = self.max_pages * self.page
        L = lib()
        self._fn = {n: getattr(L, "dartree_paged_" + n)
                    for n in ("append", "attention", "weights", "evict", "commit", "commit_weights")}
        self._pp, self._mp = ctypes.byref(self.p), ctypes.byref(self._m)
        self._t = Tree()
        self._tp = ctypes.byref(self._t)
        self._x = PagedTokens()
        self._xp = ctypes.byref(self._x)
        self._shapes = dict(q=torch.Size((self.T, self.Hq, self.D)), k=torch.Size((self.T, self.Hkv, self.D)),
                            lse=torch.Size((self.T, self.Hq)),
                            mask=torch.Size((self.C, self.S, self.S)), pos=torch.Size((self.C, self.S)),
                            C=torch.Size((self.C,)), D=torch.Size((self.D,)),
                            w=torch.Size((self.C, self.Hkv, self.rows)))

    def _need(self, t, name, dtype=None, shape=None) -> int:
        """Address of a contiguous tensor on the pages' device; raises for any other."""
        if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == self.device \
                and t.is_contiguous():
            return t.data_ptr()
        ptr = _need(t, name, dtype, shape)
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        return ptr

    def _on_device(self, f):
        if torch.cuda.current_device() == self.device.index:
            return f()
        with torch.cuda.device(self.device):
            return f()

    _cleared = {}   # (device, stream): an event behind the last workspace cleared there

    def _clear(self, ws, s):
        """Clears the workspace's status word on the current stream s; an event behind that, None while s is
        captured (others cannot wait for that)."""
        _call("dartree_clear_status", ctypes.c_void_p(ws.data_ptr()), ctypes.c_void_p(s))
        if torch.cuda.is_current_stream_capturing():
            return None
        e = self._cleared.setdefault((self.device.index, s), torch.cuda.Event())
        e.record(torch.cuda.current_stream(self.device))
        return e

    def _meet(self, stream):
        """A stream other than the one that filled the workspace is about to use it."""
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        with torch.cuda.stream(stream):
            self.ws.record_stream(stream)
            if not torch.cuda.is_current_stream_capturing():
                if self._made is not None:
                    stream.wait_event(self._made)
                self._known.add(stream.cuda_stream)

    def _run(self, name, stream, *args):
        # (the current stream as its handle: a torch.cuda.Stream object costs more than the launch)
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(self.device.index)
        if self._known is not None and s not in self._known:
            self._meet(stream)
        if torch.cuda.current_device() == self.device.index:
            rc = self._fn[name](*args, *self._wsp, s)
        else:
            with torch.cuda.device(self.device):
                rc = self._fn[name](*args, *self._wsp, s)
        if rc != OK:
            raise DartreeError(rc, "dartree_paged_" + name)

    def _new(self, make, shape, dtype, stream):
        """An output tensor that belongs to the stream of the call that fills it."""
        if stream is None:
            return make(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return make(shape, dtype=dtype, device=self.device)

    def _tree(self, tree, key):
        """The tree's n_nodes and its mask or pos, or None."""
        if tree is None:
            return None
        self._t.n_nodes = self._need(tree["n_nodes"], "tree['n_nodes']", torch.int32, self._shapes["C"])
        setattr(self._t, key, self._need(tree[key], f"tree[{key!r}]", torch.uint8 if key == "mask" else torch.int32,
                                         self._shapes[key]))
        return self._tp

    def _heads(self, t, name, shape):
        """A [T, heads, D] tensor whose tokens may lie further apart: (address, elements between tokens)."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.shape != shape or t.dtype is not self.dtype or t.device != self.device:
            raise ValueError(f"{name} must be {self.dtype} {tuple(shape)} on {self.device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        ld, h, one = t.stride()
        if one != 1 or (h != self.D and shape[1] > 1):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        return t.data_ptr(), (ld if self.T > 1 else shape[1] * self.D)

    def append(self, q, k, v, q_gain=None, k_gain=None, eps=1e-6, theta=1.0e6, tree=None, pos_base=None, out=None,
               stream=None):
        """Head norms (with gains [D]), rotation and store of the new tokens (dartree_paged_append):
        q [T, Hq, D], k and v [T, Hkv, D], parts of one tensor or not -> rotated queries [T, Hq, D]."""
        sh, x = self._shapes, self._x
        x.q, x.ldq = self._heads(q, "q", sh["q"])
        x.k, x.ldk = self._heads(k, "k", sh["k"])
        x.v, x.ldv = self._heads(v, "v", sh["k"])
        x.gq = None if q_gain is None else self._need(q_gain, "q_gain", self.dtype, sh["D"])
        x.gk = None if k_gain is None else self._need(k_gain, "k_gain", self.dtype, sh["D"])
        x.pos_base = None if pos_base is None else self._need(pos_base, "pos_base", torch.int32, sh["C"])
        x.eps, x.theta = eps, theta
        if out is None:
            out = self._new(torch.empty, self._shapes["q"], self.dtype, stream)
        op = self._need(out, "out", self.dtype, self._shapes["q"])
        self._run("append", stream, self._pp, self._xp, self._mp, self._tree(tree, "pos"), op)
        return out

    def attention(self, q, tree=None, scale=None, out=None, lse=None, stream=None):
        """Attention of the new tokens, already appended, over the pages (dartree_paged_attention):
        q [T, Hq, D] rotated -> out [T, Hq, D], not q itself; lse [T, Hq] float32 is filled when given.
        scale: None or 0 for 1 / sqrt(D)."""
        qp = self._need(q, "q", self.dtype, self._shapes["q"])
        if out is None:
            out = self._new(torch.empty, self._shapes["q"], self.dtype, stream)
        op = self._need(out, "out", self.dtype, self._shapes["q"])
        lp = None if lse is None else self._need(lse, "lse", torch.float32, self._shapes["lse"])
        self._run("attention", stream, self._pp, qp, self._mp, self._tree(tree, "mask"), scale or 0.0, op, lp)
        return out

    def weights(self, q, lse, weights, tree=None, scale=None, decay=1.0, stream=None):
        """weights [C, Hkv, max_pages * page] float32 decayed and increased by the attention weight each
        cached row receives from the new tokens (dartree_paged_weights). The new rows' weights start from 0;
        rows that were appended without this call keep what lay there. A tree's rows move with the
        accepted path when commit is given the weights."""
        qp = self._need(q, "q", self.dtype, self._shapes["q"])
        lp = self._need(lse, "lse", torch.float32, self._shapes["lse"])
        wp = self._need(weights, "weights", torch.float32, self._shapes["w"])
        self._run("weights", stream, self._pp, qp, lp, self._mp, self._tree(tree, "mask"), scale or 0.0, decay, wp)
        return weights

    def evict(self, weights, budget, dst_table, sink=0, recent=0, keep=None, n_out=None, weights_out=None,
              stream=None):
        """The first `sink`, the last `recent` and the heaviest other rows of every request and key/value
        head, `budget` in all, copied into the pages of dst_table [C, dst_pages], none of them pages of
        the cache's table (dartree_paged_evict) ->
        dict(keep [C, Hkv, budget], n [C], weights [C, Hkv, dst_pages * page])."""
        budget = int(budget)
        wp = self._need(weights, "weights", torch.float32, self._shapes["w"])
        if not isinstance(dst_table, torch.Tensor) or dst_table.dim() != 2:
            raise ValueError("dst_table must be [C, dst_pages]")
        pages = dst_table.shape[1]
        dp = self._need(dst_table, "dst_table", torch.int32, (self.C, pages))

        def output(t, name, dtype, shape, new):
            if t is None:
                t = self._new(new, shape, dtype, stream)
            self._need(t, name, dtype, shape)
            return t

        keep = output(keep, "keep", torch.int32, (self.C, self.Hkv, max(budget, 0)), torch.empty)
        n_out = output(n_out, "n_out", torch.int32, (self.C,), torch.empty)
        weights_out = output(weights_out, "weights_out", torch.float32, (self.C, self.Hkv, pages * self.page),
                             torch.zeros)
        self._run("evict", stream, self._pp, self._mp, wp, budget, int(sink), int(recent), dp, pages, keep.data_ptr(),
                  n_out.data_ptr(), weights_out.data_ptr())
        return dict(keep=keep, n=n_out, weights=weights_out)

    def commit(self, path, accepted_len, n_out=None, stream=None, weights=None):
        """The accepted path [C, L] of each request's tree moved behind the root's row
        (dartree_paged_commit) -> rows cached then [C] (n_out may be the cache's n_ctx).
        weights [C, Hkv, max_pages * page], when given, moves with the rows
        (dartree_paged_commit_weights)."""
        if not isinstance(path, torch.Tensor) or path.dim() != 2:
            raise ValueError("path must be [C, L]")
        L = path.shape[1]
        pp = self._need(path, "path", torch.int32, (self.C, L))
        ap = self._need(accepted_len, "accepted_len", torch.int32, self._shapes["C"])
        if n_out is None:
            n_out = self._new(torch.empty, (self.C,), torch.int32, stream)
        op = self._need(n_out, "n_out", torch.int32, self._shapes["C"])
        if weights is None:
            self._run("commit", stream, self._pp, self._mp, pp, ap, L, op)
        else:
            wp = self._need(weights, "weights", torch.float32, self._shapes["w"])
            self._run("commit_weights", stream, self._pp, self._mp, pp, ap, L, wp, op)
        return n_out
