"""Lengths without a tree (pos and mask both NULL) pass the checks of the paged calls; a tree that lacks the one that the
call needs does not (no GPU needed; the fake pointers are never dereferenced: every call ends at its workspace)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dd():
    from diffusion_drafter_draft_gb300 import _build
    _build.build()
    import diffusion_drafter_draft_gb300 as m
    m.lib()
    return m


def test_lengths_are_taken_and_half_trees_refused(dd):
    L = dd.lib()
    p = dd.PagedParams(2, 6, 3, 8, 2, 128, 64, 8, 4, 1)
    m, F = dd.PagedCacheDesc(256, 256, 256, 256, None), ctypes.c_void_p(256)
    ragged = dd.PagedCacheDesc(256, 256, 256, 256, 256)
    x = dd.PagedTokens(256, 1 << 16, 1 << 17, 1024, 256, 256, None, None, None, 1e-6, 1e6)
    g = dd.PagedGroups(1, 0, 0, 1, 256, 256)

    def calls(mask, pos, nodes=256, m=m):
        t = dd.Tree(None, None, None, None, nodes, mask, pos)
        a = ctypes.byref(p), ctypes.byref(m), ctypes.byref(t)
        return (L.dartree_paged_append(a[0], ctypes.byref(x), a[1], a[2], ctypes.c_void_p(1 << 20), F, 0, None),
                L.dartree_paged_attention(a[0], F, a[1], a[2], 0.0, ctypes.c_void_p(1 << 20), None, F, 0, None),
                L.dartree_paged_weights(a[0], F, F, a[1], a[2], 0.0, 1.0, F, F, 0, None),
                L.dartree_paged_shared_attention(a[0], F, a[1], a[2], ctypes.byref(g), 0.0, ctypes.c_void_p(1 << 20), None,
                                                 F, 0, None))

    assert calls(None, None) == (dd.EWORKSPACE,) * 4
    assert calls(256, 256) == (dd.EWORKSPACE,) * 4
    assert calls(None, 256) == (dd.EWORKSPACE,) + (dd.EINVAL,) * 3       # a tree without its mask
    assert calls(256, None) == (dd.EINVAL,) + (dd.EWORKSPACE,) * 3       # without its positions
    assert calls(None, None, nodes=None) == (dd.EINVAL,) * 4
    assert calls(None, None, m=ragged) == (dd.EINVAL,) * 4               # lengths are q_start's there
