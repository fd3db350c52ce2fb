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
