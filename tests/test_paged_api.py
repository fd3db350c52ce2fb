"""Refusals of the paged-cache calls that the host makes: nothing here reaches a kernel."""
import copy
import ctypes
import pickle

import pytest
import torch

from block_sparse_causal_bsa_b200 import binding as bb
from block_sparse_causal_bsa_b200 import paged

P16, P256 = 16, 256                        # stand-ins for aligned device pointers


def _cs(**kw):
    f = dict(n_pages=100, Hkv=8, page=64, d=128, dtype=bb.BSA_BF16)
    f.update(kw)
    return bb.CacheShape(*[f[n] for n, _ in bb.CacheShape._fields_])


def _attend(s, slots=4, max_pages=20, Hq=32, T=1, q=P16, k=P16, out=P16, scale=0.1, st=P16, ws=P256, nb=1 << 40,
            W=None, idx=P16):
    L = bb.lib()
    if W is None:
        return L.bsa_attend_tree(ctypes.byref(s), slots, max_pages, Hq, T, q, k, P16, P16, P16, None, None, scale,
                                 out, None, st, ws, nb, None)
    return L.bsa_attend_pages(ctypes.byref(s), slots, max_pages, Hq, T, q, k, P16, P16, P16, None, idx, P16, W,
                              scale, out, None, st, ws, nb, None)


REFUSED = (bb.BSA_ERR_INVALID_ARG, bb.BSA_ERR_UNSUPPORTED)


@pytest.mark.parametrize("bad", [dict(n_pages=0), dict(Hkv=0), dict(page=48), dict(page=256), dict(d=96),
                                 dict(dtype=bb.BSA_F32), dict(dtype=9), dict(n_pages=1 << 24, Hkv=8)])
def test_cache_shapes(bad):
    s, L = _cs(**bad), bb.lib()
    assert _attend(s) in REFUSED and _attend(s, W=4) in REFUSED
    assert bb.lib().bsa_attend_paged_workspace_bytes(ctypes.byref(s), 4, 20, 32, 1) == 0
    assert L.bsa_select_pages_workspace_bytes(ctypes.byref(s), 4, 20, 32, 1) == 0
    assert L.bsa_pages_copy(ctypes.byref(s), P16, P16, P16, P16, 4, P16, None) in REFUSED
    assert L.bsa_cache_append(ctypes.byref(s), 4, 20, 1, P16, P16, P16, P16, P16, P16, P16, None, P16, None) in REFUSED
    assert L.bsa_cache_compact(ctypes.byref(s), 4, 20, 1, P16, P16, P16, P16, P16, P16, P16, None, P16,
                               None) in REFUSED
    assert L.bsa_last_error()


@pytest.mark.parametrize("bad", [dict(slots=0), dict(max_pages=0), dict(Hq=12), dict(Hq=8 * 17), dict(T=0),
                                 dict(T=1025), dict(slots=5000), dict(max_pages=40000), dict(q=None), dict(k=None),
                                 dict(out=None), dict(st=None), dict(ws=None), dict(q=P16 + 2), dict(out=P16 + 4),
                                 dict(ws=P256 + 16), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                 dict(scale=float("inf")), dict(nb=1000)])
def test_attend_arguments(bad):
    assert _attend(_cs(), **bad) in REFUSED
    assert _attend(_cs(), W=4, **bad) in REFUSED
    assert bb.lib().bsa_last_error()


def test_attend_pages_lists():
    assert _attend(_cs(), W=0) == bb.BSA_ERR_INVALID_ARG
    assert _attend(_cs(), W=32769) == bb.BSA_ERR_UNSUPPORTED
    assert _attend(_cs(), W=4, idx=None) == bb.BSA_ERR_INVALID_ARG


@pytest.mark.parametrize("k,a,b", [(0, 0, 1), (4, -1, 1), (4, 0, 0), (4, 3, 2), (4, 2 ** 31 - 1, 2 ** 31 - 1), (32769, 1, 1)])
def test_select_params(k, a, b):
    p, s = bb.PageSelectParams(k, a, b), _cs()
    assert bb.lib().bsa_select_pages(ctypes.byref(s), ctypes.byref(p), 4, 20, 32, 1, P16, P16, P16, P16, None, P16,
                                     P16, None, P16, P256, 1 << 40, None) in REFUSED


def test_select_workspace():
    p, s, L = bb.PageSelectParams(4, 1, 1), _cs(), bb.lib()
    nb = L.bsa_select_pages_workspace_bytes(ctypes.byref(s), 4, 20, 32, 3)
    assert nb >= 4 * 8 * 3 * 20 * 4
    call = lambda ws, n: L.bsa_select_pages(ctypes.byref(s), ctypes.byref(p), 4, 20, 32, 3, P16, P16, P16, P16, None,
                                            P16, P16, None, P16, ws, n, None)
    assert call(None, nb) == bb.BSA_ERR_INVALID_ARG
    assert call(P256, nb - 1) == bb.BSA_ERR_INVALID_ARG
    assert call(P256 + 8, nb) == bb.BSA_ERR_INVALID_ARG


def test_bookkeeping_arguments():
    L = bb.lib()
    for slots, mp, n, page in [(0, 4, 9, 16), (4, 0, 9, 16), (4, 4, 0, 16), (4, 4, 9, 24), (4097, 4, 9, 16),
                               (4, 32769, 9, 16), (4, 4, 1 << 27, 16)]:
        assert L.bsa_pages_fork(slots, mp, n, page, P16, P16, P16, P16, P16, None) in REFUSED
        assert L.bsa_pages_resize(slots, mp, n, page, P16, P16, P16, P16, P16, None, P16, None) in REFUSED
    for hole in range(5):
        a = [None if i == hole else P16 for i in range(5)]
        assert L.bsa_pages_fork(4, 4, 9, 16, *a, None) == bb.BSA_ERR_INVALID_ARG
    assert L.bsa_pages_resize(4, 4, 9, 16, P16, P16, P16 + 4, P16, P16, None, P16, None) == bb.BSA_ERR_INVALID_ARG
    s = _cs()
    assert L.bsa_pages_copy(ctypes.byref(s), P16, P16, P16, P16, -1, P16, None) == bb.BSA_ERR_INVALID_ARG
    assert L.bsa_pages_copy(ctypes.byref(s), P16, P16, P16, P16 + 4, 1, P16, None) == bb.BSA_ERR_INVALID_ARG
    assert L.bsa_tree_mask(0, 4, P16, None, P16, P16, None) == bb.BSA_ERR_INVALID_ARG
    assert L.bsa_tree_mask(1, 1025, P16, None, P16, P16, None) == bb.BSA_ERR_UNSUPPORTED
    assert L.bsa_tree_mask(1, 4, None, None, P16, P16, None) == bb.BSA_ERR_INVALID_ARG


def _cache(**kw):
    f = dict(layers=2, n_pages=10, Hkv=2, page=16, d=64, slots=3, max_pages=4, device="cpu")
    f.update(kw)
    return paged.PagedCache.create(**f)


def test_wrappers_refuse_wrong_tensors():
    c = _cache()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q = bf(3, 4, 2, 64)
    bad = [
        lambda: paged.fork(c, i32(4)), lambda: paged.fork(c, torch.zeros(3, dtype=torch.int64)),
        lambda: paged.resize(c, i32(6)[::2]), lambda: paged.copy_pages(c, i32(3, 3)),
        lambda: paged.copy_pages(c, i32(3, 2), layer=2), lambda: paged.append(c, bf(3, 2, 5, 32), bf(3, 2, 5, 64)),
        lambda: paged.append(c, bf(3, 2, 5, 64), bf(3, 2, 4, 64)),
        lambda: paged.append(c, bf(3, 2, 64, 5).transpose(2, 3), bf(3, 2, 5, 64)),
        lambda: paged.compact(c, i32(3, 4), i32(2)), lambda: paged.compact(c, i32(3), i32(3)),
        lambda: paged.attend_tree(q.float(), c), lambda: paged.attend_tree(q[:2], c),
        lambda: paged.attend_tree(q, c, mask=torch.zeros(3, 2, 2, dtype=torch.int64)),
        lambda: paged.attend_tree(q, c, q_len=i32(2)), lambda: paged.attend_tree(q, c, out=bf(3, 4, 2, 32)),
        lambda: paged.attend_tree(q, c, lse=bf(3, 4, 2)), lambda: paged.attend_tree(bf(3, 2, 4, 64).transpose(1, 2), c),
        lambda: paged.attend_pages(q, c, i32(3, 2, 2), i32(3, 2, 2)),
        lambda: paged.attend_pages(q, c, i32(3, 2, 2, 4), i32(3, 4, 2)),
        lambda: paged.select_pages(q, _cache(bounds=False), paged.PageSelectConfig(2)),
        lambda: paged.tree_mask(i32(4)), lambda: paged.tree_mask(i32(2, 4), q_len=i32(3)),
        lambda: paged.PagedCache(c.k.float(), c.v.float(), None, c.page_table, c.seq_len, c.refs),
        lambda: paged.PagedCache(c.k, c.v[:1], None, c.page_table, c.seq_len, c.refs),
        lambda: paged.PagedCache(c.k, c.v, c.bounds, c.page_table, c.seq_len[:2], c.refs),
        lambda: paged.PagedCache(c.k, c.v, c.bounds, c.page_table, c.seq_len, c.refs[:4]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(bb.BsaError):
            f()
            print("accepted", i)
    # right in every other way, but there is no kernel for the CPU
    with pytest.raises(bb.BsaError, match="GPU"):
        paged.attend_tree(q, c)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))])
def test_caches_can_be_copied_and_pickled(how):
    c = paged.PagedCache.create(layers=1, n_pages=4, Hkv=1, page=16, d=64, slots=2, max_pages=2, device="cpu")
    c.refs[1] = 3
    n = c.workspace_bytes("attend_paged", 2, 1)
    other = how(c)
    assert torch.equal(other.refs, c.refs) and other.k.shape == c.k.shape
    other.page_table = torch.full((3, 2), -1, dtype=torch.int32)       # what is derived follows its own tensors
    other.seq_len = torch.zeros(3, dtype=torch.int32)
    assert other.workspace_bytes("attend_paged", 2, 1) == n and other.slots == 3 and c.slots == 2
    other.shape()
    c.shape()
