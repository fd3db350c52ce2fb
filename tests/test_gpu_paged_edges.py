"""Corners of the paged-cache calls: lengths that are garbage, tables of mostly idle slots, the
longest trees and chunks."""
import random

import numpy as np
import pytest
import torch

from block_sparse_causal_bsa_b200 import binding as bb
from block_sparse_causal_bsa_b200 import paged
from oracle import paged_oracle as O
from paged_util import check, f8, lse_tolerance, make_cache, out_tolerance, scale_of, words

pytestmark = pytest.mark.gpu

LO, HI = -2**31, 2**31 - 1


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


# seq_len, q_len (None: T for every slot) of slots 1 .. 4; a difference of the first two pairs, taken in
# 32 bits, wraps around to a length that is none
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("wild_len,wild_ql", [([LO, LO + 2, -1, HI], None),
                                              ([LO, 50, HI, 60], [3, LO, HI, -1])])
def test_wild_lengths_are_left_out(T, wild_len, wild_ql):
    page, d, Hkv, Hq = 16, 64, 2, 4
    lens = [70, 60, 60, 60, 60]
    cache = make_cache(1, lens=lens, max_pages=6, page=page, Hkv=Hkv, d=d)
    cache.seq_len[1:] = _i32(wild_len)
    ql = None if wild_ql is None else _i32([T] + wild_ql)
    q = _randn(2, 5, Hq, T, d)
    out, out2 = torch.full_like(q, 3.0), torch.full_like(q, 3.0)
    _, _, st = paged.attend_tree(q, cache, q_len=ql, out=out)
    assert int(st) == bb.BSA_DEV_BAD_INDEX
    sel = paged.select_pages(q, cache, paged.PageSelectConfig(3, 1, 1), q_len=ql)
    sel2 = paged.select_pages(q, cache, paged.PageSelectConfig(3, 1, 1), q_len=ql, want_scores=True)
    assert int(sel["dev_status"]) == int(sel2["dev_status"]) == bb.BSA_DEV_BAD_INDEX
    assert (sel["kv_cnt"][1:] == 0).all() and (sel["kv_idx"][1:] == -1).all()
    assert torch.equal(sel["kv_idx"], sel2["kv_idx"]) and torch.isneginf(sel2["scores"][1:]).all()
    _, _, st = paged.attend_pages(q, cache, sel["kv_idx"], sel["kv_cnt"], q_len=ql, out=out2)
    assert int(st) == bb.BSA_DEV_BAD_INDEX
    for o in (out, out2):
        assert (o[1:] == 3.0).all() and torch.isfinite(o.float()).all() and not (o[0] == 3.0).all()
    # the writers: slot 0's rows alone
    k0 = cache.k.clone()
    kn = _randn(3, 5, Hkv, T, d)
    assert int(paged.append(cache, kn, kn, q_len=ql)) == bb.BSA_DEV_BAD_INDEX
    tab = cache.page_table.cpu()
    for t in range(T):
        k0[0, tab[0, (70 - T + t) // page], :, (70 - T + t) % page] = kn[0, :, t]
    assert torch.equal(cache.k, k0)
    keep = torch.arange(T, dtype=torch.int32, device="cuda").expand(5, T).contiguous()
    st = paged.compact(cache, keep, _i32([T, LO, HI, T, T]), q_len=ql)
    assert int(st) == bb.BSA_DEV_BAD_INDEX and torch.equal(cache.k, k0)
    # the bookkeeping: slots with such lengths stay as they are
    table, refs = cache.page_table.clone(), cache.refs.clone()
    bad = [not 0 <= n <= 6 * page for n in wild_len]
    _, _, st = paged.resize(cache, _i32([LO] + [HI if b else -1 for b in bad]))
    assert int(st) == bb.BSA_DEV_BAD_INDEX
    assert cache.seq_len.tolist() == [70] + wild_len
    assert torch.equal(cache.page_table, table) and torch.equal(cache.refs, refs)


@pytest.mark.parametrize("T", [63, 64, 65, 200, 1000, 1024])
def test_masks_of_long_trees(T):
    rng = random.Random(T)
    par = [[t - 1 for t in range(T)],                                          # a chain
           [-1 if t == 0 else rng.randint(max(0, t - 90), t - 1) for t in range(T)],
           [-1 if t < 3 else rng.randint(0, t - 1) for t in range(T)]]
    ql = [T, T, T - 17]
    mask, st = paged.tree_mask(_i32(par), q_len=_i32(ql))
    assert int(st) == 0
    want = words(np.stack([O.ancestors(p) for p in par]))
    for b in range(3):
        assert torch.equal(mask[b, :ql[b]].cpu(), want[b, :ql[b]]) and (mask[b, ql[b]:] == 0).all()


def _check_slot(go, gl, qn, cache, b, n, ql, see, dtype, p_bits):
    """Rows [Hq, ql, d] of a slot against the formula in 64 bits."""
    Hkv, page, d = cache.k.shape[2:]
    pages = cache.page_table[b, :-(-n // page)].cpu().long()
    G = qn.shape[0] // Hkv
    vis = np.ones((ql, n), bool)
    vis[:, n - ql:] = see
    for h in range(Hkv):
        kr, vr = (f8(x[0, pages.to(x.device), h].reshape(-1, d)[:n]) for x in (cache.k, cache.v))
        qh = qn[h * G:(h + 1) * G, :ql].reshape(G * ql, d)
        ro, rl = O.softmax_rows(qh, kr, vr, np.tile(vis, (G, 1)), scale_of(d))
        km, vm = np.abs(kr).max(), np.abs(vr).max()
        check(go[h * G:(h + 1) * G, :ql].reshape(-1, d), ro,
              out_tolerance(ro, qh, km, vm, d, scale_of(d), dtype, p_bits), (b, h))
        check(gl[h * G:(h + 1) * G, :ql].reshape(-1), rl, lse_tolerance(rl, qh, km, d, scale_of(d), n), (b, h))


@pytest.mark.parametrize("T,Hq,Hkv,page,d,tree", [(1024, 2, 1, 128, 128, False), (1000, 3, 1, 16, 64, True),
                                                  (257, 16, 1, 64, 128, True), (300, 1, 1, 32, 64, False)])
def test_long_chunks_and_trees(T, Hq, Hkv, page, d, tree):
    """Several row tiles per item of one KV head, up to sixteen mask words."""
    rng = random.Random(T)
    qls = [T, T - 1, 129]
    lens = [T, T + 777, 140]
    cache = make_cache(5, lens=lens, max_pages=-(-max(lens) // page), page=page, Hkv=Hkv, d=d,
                       garbage=float("nan"))
    par = [[-1 if t == 0 else rng.randint(max(0, t - 70), t - 1) for t in range(T)] for _ in lens]
    see = np.stack([O.ancestors(p) for p in par]) if tree else np.broadcast_to(np.tril(np.ones((T, T), bool)), (3, T, T))
    q = _randn(6, 3, Hq, T, d)
    out, lse, st = paged.attend_tree(q, cache, mask=words(see).cuda() if tree else None, q_len=_i32(qls))
    assert int(st) == 0
    for b, (n, ql) in enumerate(zip(lens, qls)):
        _check_slot(f8(out[b]), f8(lse[b]), f8(q[b]), cache, b, n, ql, see[b, :ql, :ql], "bf16", 8)
        assert (out[b, :, ql:] == 0).all() and torch.isneginf(lse[b, :, ql:]).all()


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 2), (12, 4, 2)])
def test_a_table_of_mostly_idle_slots(T, Hq, Hkv):
    slots, page, d = 4096, 16, 64
    lens, qls = [0] * slots, [0] * slots
    for s, n in [(0, 33), (31, 70), (32, T), (1999, 500), (4095, 129)]:
        lens[s], qls[s] = n, T
    lens[77] = 64                                          # rows, but no token in the call
    cache = make_cache(9, lens=lens, max_pages=32, page=page, Hkv=Hkv, d=d)
    q = _randn(10, slots, Hq, T, d)
    out, lse, st = paged.attend_tree(q, cache, q_len=_i32(qls))
    sel = paged.select_pages(q, cache, paged.PageSelectConfig(32, 1, 1), q_len=_i32(qls))
    out2, lse2, st2 = paged.attend_pages(q, cache, sel["kv_idx"], sel["kv_cnt"], q_len=_i32(qls))
    assert int(st) == int(st2) == int(sel["dev_status"]) == 0
    see = np.tril(np.ones((T, T), bool))
    for s in range(slots):
        if qls[s]:
            for o, l, p_bits in ((out, lse, 16 if Hq // Hkv * T <= 16 else 8), (out2, lse2, 16)):
                _check_slot(f8(o[s]), f8(l[s]), f8(q[s]), cache, s, lens[s], T, see, "bf16", p_bits)
    idle = torch.tensor([n == 0 for n in qls])
    for o, l in ((out, lse), (out2, lse2)):
        assert (o.cpu()[idle] == 0).all() and torch.isneginf(l.cpu()[idle]).all()
    # nobody takes part
    none = _i32([0] * slots)
    out, lse, st = paged.attend_tree(q, cache, q_len=none)
    assert int(st) == 0 and (out == 0).all() and torch.isneginf(lse).all()


def test_a_list_as_long_as_it_may_be():
    """32768 entries for a table of 40 pages: the row's count says how many of them are read."""
    page, d = 16, 64
    cache = make_cache(11, lens=[600, 9], max_pages=40, page=page, Hkv=1, d=d)
    W = 32768
    idx = torch.full((2, 1, 1, W), 12345, dtype=torch.int32, device="cuda")
    idx[0, 0, 0, :38] = torch.randperm(38, generator=torch.Generator().manual_seed(1)).int().cuda()
    idx[1, 0, 0, 0] = 0
    cnt = _i32([38, 1]).view(2, 1, 1)
    q = _randn(12, 2, 3, 1, d)
    out, lse, st = paged.attend_pages(q, cache, idx, cnt)
    assert int(st) == 0
    for b, n in enumerate([600, 9]):
        _check_slot(f8(out[b]), f8(lse[b]), f8(q[b]), cache, b, n, 1, np.ones((1, 1), bool), "bf16", 16)
    # all of them the same page past the end, the count as large as it may be: all skipped
    out, lse, st = paged.attend_pages(q, cache, torch.full_like(idx, 39), _i32([W, W]).view(2, 1, 1))
    assert int(st) == bb.BSA_DEV_BAD_INDEX and (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("T,Hq,d,dtype", [(1, 4, 128, "bf16"), (2, 8, 128, "fp16"), (1, 3, 64, "fp16"),
                                          (4, 4, 64, "bf16"), (20, 4, 64, "bf16")])
def test_one_item_shared_by_every_cta(T, Hq, d, dtype):
    """One sequence, one KV head: all CTAs leave partial results of one item."""
    n, page = 90001, 128
    cache = make_cache(13, lens=[n], max_pages=-(-n // page), page=page, Hkv=1, d=d, dtype=dtype)
    q = _randn(14, 1, Hq, T, d).to(cache.k.dtype)
    out, lse, st = paged.attend_tree(q, cache)
    again, lse2, _ = paged.attend_tree(q, cache)
    assert int(st) == 0 and torch.equal(out, again) and torch.equal(lse, lse2)
    see = np.tril(np.ones((T, T), bool))
    p_bits = 16 if Hq * T <= 16 else 8
    _check_slot(f8(out[0]), f8(lse[0]), f8(q[0]), cache, 0, n, T, see, dtype, p_bits)
    # the same as a list of all its pages
    if T == 1:
        W = cache.max_pages
        idx = torch.arange(W, dtype=torch.int32, device="cuda").view(1, 1, 1, W)
        out, lse, st = paged.attend_pages(q, cache, idx, _i32([W]).view(1, 1, 1))
        assert int(st) == 0
        _check_slot(f8(out[0]), f8(lse[0]), f8(q[0]), cache, 0, n, T, see, dtype, 16)
