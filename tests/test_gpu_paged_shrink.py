"""Sequences cut back inside a page and grown again: the bounds are those of the rows that are there, after the
append that follows, and the pages selected are the definition's."""
import numpy as np
import pytest
import torch

from block_sparse_causal_bsa_b200 import paged
from oracle import paged_oracle as O
from paged_util import DT, f8

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _check_bounds(cache, layer, but=()):
    """Every page of every slot, but the slots' last page in `but`: minimum and maximum of its filled rows."""
    page, table, lens = cache.k.shape[3], cache.page_table.cpu().tolist(), cache.seq_len.cpu().tolist()
    for s, n in enumerate(lens):
        for j in range(-(-n // page)):
            if s in but and j == (n - 1) // page:
                continue
            rows = cache.k[layer, table[s][j], :, :min(page, n - j * page)].float()
            got = cache.bounds[layer, table[s][j]].float()
            assert torch.equal(got[:, 0], rows.amin(1)) and torch.equal(got[:, 1], rows.amax(1)), (s, j)


@pytest.mark.parametrize("page,d,dtype,T", [(16, 64, "bf16", 1), (32, 128, "fp16", 3), (64, 128, "bf16", 1), (128, 64, "fp16", 40),
                                            (128, 128, "bf16", 2)])
def test_shrink_and_append(page, d, dtype, T):
    """Rows far out of range (and NaN) are appended, dropped again by a resize alone, and other rows take
    their place; several times, to lengths all over the pages."""
    slots, Hkv, layers = 6, 2, 2
    g = torch.Generator().manual_seed(page)
    cache = paged.PagedCache.create(layers=layers, n_pages=6 * slots, Hkv=Hkv, page=page, d=d, slots=slots, max_pages=6,
                                    dtype=DT[dtype])
    n0 = [1, page - 1, page, page + 1, 2 * page + page // 2, 3]

    def append(lens, q, mul, nan=False):
        qs = [b - a for a, b in zip(cache.seq_len.tolist(), lens)]
        _, _, st = paged.resize(cache, _i32(lens))
        assert int(st) == 0
        k = (torch.randn(slots, Hkv, q, d, generator=g) * mul).to(DT[dtype])
        if nan:
            k[:, :, 0, 3] = float("nan")
        for layer in range(layers):
            assert int(paged.append(cache, k.cuda(), k.cuda(), q_len=_i32(qs), layer=layer)) == 0

    append(n0, max(n0), 1.0)
    for step in range(3):
        more = [n + page // 2 + 1 + step for n in n0]
        append(more, page // 2 + 1 + step, 50.0, nan=step == 1)
        assert int(paged.resize(cache, _i32(n0))[2]) == 0
        append([n + T for n in n0], T, 1.0)
        for layer in range(layers):
            _check_bounds(cache, layer)
        assert int(paged.resize(cache, _i32(n0))[2]) == 0
        for layer in range(layers):
            _check_bounds(cache, layer, but=range(slots))


def test_a_fork_cut_back_and_grown():
    """A child that drops rows of the shared last page gets a copy when it grows: its bounds are of
    its own rows. And where all holders grow, the last one keeps the page."""
    page, d, Hkv = 64, 64, 1
    g = torch.Generator().manual_seed(5)
    cache = paged.PagedCache.create(layers=1, n_pages=20, Hkv=Hkv, page=page, d=d, slots=3, max_pages=5)
    r = lambda T, mul: (torch.randn(3, Hkv, T, d, generator=g) * mul).to(torch.bfloat16).cuda()
    paged.resize(cache, _i32([0, 100, 0]))
    paged.append(cache, x := r(100, 1.0), x, q_len=_i32([0, 100, 0]))
    paged.resize(cache, _i32([0, 110, 0]))
    paged.append(cache, x := r(10, 30.0), x, q_len=_i32([0, 10, 0]))
    assert int(paged.fork(cache, _i32([1, -1, 1]))) == 0
    paged.resize(cache, _i32([99, 110, 104]))
    pairs, _, st = paged.resize(cache, _i32([101, 111, 105]))
    assert int(st) == 0 and pairs.tolist()[2] == [-1, -1] and pairs.tolist()[0][0] >= 0 and pairs.tolist()[1][0] >= 0
    assert int(paged.copy_pages(cache, pairs)) == 0
    assert int(paged.append(cache, x := r(2, 1.0), x, q_len=_i32([2, 1, 1]))) == 0
    _check_bounds(cache, 0)


def test_selection_after_a_rejected_chain():
    """The page of a rejected chain with huge keys is ranked by the rows that replaced it."""
    page, d, Hkv, n = 16, 64, 1, 20 * 16 + 5
    g = torch.Generator().manual_seed(6)
    r = lambda T, mul: (torch.randn(1, Hkv, T, d, generator=g) * mul).to(torch.bfloat16).cuda()
    cache = paged.PagedCache.create(layers=1, n_pages=32, Hkv=Hkv, page=page, d=d, slots=1, max_pages=30)
    paged.resize(cache, _i32([n]))
    paged.append(cache, x := r(n, 1.0), x)
    paged.resize(cache, _i32([n + 8]))
    paged.append(cache, x := r(8, 100.0), x)
    paged.resize(cache, _i32([n]))
    paged.resize(cache, _i32([n + 60]))
    paged.append(cache, x := r(60, 1.0), x)
    q = torch.randn(1, 2, 1, d, generator=g).to(torch.bfloat16)
    for want_scores in (False, True):
        sel = paged.select_pages(q.cuda(), cache, paged.PageSelectConfig(6, 1, 1), want_scores=want_scores)
        table, own = cache.page_table.tolist()[0], (n + 59) // page
        k = f8(cache.k[0])
        ref = []
        for j in range(own + 1):
            rows = k[table[j], 0, :min(page, n + 60 - j * page)]
            ref.append(O.page_score(f8(q)[0, :, 0], rows.min(0), rows.max(0)))
        assert int(sel["dev_status"]) == 0
        assert sel["kv_idx"][0, 0, 0].tolist() == O.select(ref, own, 6, 1, 1)
        if want_scores:
            assert np.array_equal(sel["scores"].cpu().numpy()[0, 0, 0, :own + 1], np.array(ref, np.float32))
