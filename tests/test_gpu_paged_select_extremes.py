"""Selection where the screening of the scores says nothing: queries that are not finite, sums that overflow in
32 bits (in one head of a group, too), magnitudes over the whole range, together with pages that cannot be ranked.
With and without returned scores the lists and the status are the definition's: what has no finite score
ranks last, lower pages first."""
import numpy as np
import pytest
import torch

from block_sparse_causal_bsa_b200 import binding as bb
from block_sparse_causal_bsa_b200 import paged
from oracle import paged_oracle as O
from paged_util import DT, f8, make_cache

pytestmark = pytest.mark.gpu
PAGES, PAGE = 30, 16


def _cache(dtype="bf16", d=64, pages=PAGES, seed=94):
    return make_cache(seed, lens=[pages * PAGE], max_pages=pages, page=PAGE, Hkv=1, d=d, dtype=dtype)


def _set_bounds(cache, j, lo, hi):
    pg = cache.page_table[0, j].item()
    cache.bounds[0, pg, 0, 0] = lo
    cache.bounds[0, pg, 0, 1] = hi


def _definition(q, cache, cfg):
    """The list and the status bits, from 64-bit scores rounded to 32."""
    table, bd, qn, n_pages = cache.page_table[0].tolist(), f8(cache.bounds[0]), f8(q)[0, :, 0], cache.k.shape[1]
    vis = cache.max_pages
    scores, bits = [], 0
    for j in range(vis):
        ranked = cfg.n_first <= j < vis - cfg.n_last and vis > cfg.k > cfg.n_first + cfg.n_last
        if not 0 <= table[j] < n_pages:
            scores.append(-np.inf)
            bits |= bb.BSA_DEV_BAD_INDEX if ranked else 0
            continue
        lo, hi = bd[table[j], 0]
        with np.errstate(invalid="ignore", over="ignore"):
            s = O.page_score(qn, lo, hi) if np.isfinite(qn).all() and np.isfinite(lo + hi).all() else np.float32(np.nan)
        if not np.isfinite(s):
            bits |= bb.BSA_DEV_BAD_SCORE if ranked else 0
            s = -np.inf
        scores.append(s)
    return O.select(scores, vis - 1, cfg.k, cfg.n_first, cfg.n_last), bits


def _check(q, cache, cfg, what):
    want, bits = _definition(q, cache, cfg)
    for want_scores in (True, False):
        sel = paged.select_pages(q.cuda(), cache, cfg, want_scores=want_scores)
        got = sel["kv_idx"][0, 0, 0].tolist()
        assert got == want + [-1] * (cfg.k - len(want)), (what, want_scores)
        assert int(sel["dev_status"]) == bits, (what, want_scores)


def _q(G, d=64, seed=4, dtype="bf16"):
    return torch.randn(1, G, 1, d, generator=torch.Generator().manual_seed(seed)).to(DT[dtype])


@pytest.mark.parametrize("k", [3, 8, 20, 27, 28, 29])
@pytest.mark.parametrize("val", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_nonfinite_query_beside_pages_that_cannot_be_ranked(k, val, dtype):
    for holes in ([], [2], [7, 8, 20], [1, 28], list(range(3, 27))):
        cache = _cache(dtype)
        for j in holes:
            cache.page_table[0, j] = -1
        _set_bounds(cache, 11, float("inf"), float("inf"))
        q = _q(2, dtype=dtype)
        q[0, 1, 0, 9] = val
        _check(q, cache, paged.PageSelectConfig(k, 1, 1), (k, val, holes))


@pytest.mark.parametrize("k", [3, 8, 20, 27, 29])
def test_finite_query_beside_pages_that_cannot_be_ranked(k):
    for holes in ([2], [7, 8, 20], list(range(1, 20)), list(range(3, 29))):
        cache = _cache()
        _set_bounds(cache, 21, -1.0, float("nan"))
        for j in holes:
            cache.page_table[0, j] = cache.k.shape[1]
        _check(_q(2), cache, paged.PageSelectConfig(k, 1, 1), (k, holes))


@pytest.mark.parametrize("k", [3, 8, 20])
def test_an_infinite_query_value_against_keys_of_the_other_sign(k):
    """Head 0 is infinitely bad, head 1 has finite scores: still no page has a finite score."""
    cache = _cache()
    cache.bounds[0, :, 0, 0, 5] = -3.0
    cache.bounds[0, :, 0, 1, 5] = -1.0
    q = _q(2)
    q[0, 0, 0, 5] = float("inf")
    cache.page_table[0, 3] = -1
    _check(q, cache, paged.PageSelectConfig(k, 1, 1), k)


@pytest.mark.parametrize("k", [3, 8, 20])
def test_one_heads_sum_overflows_on_the_way(k):
    """Head 0: negative products that overflow 32 bits, then positive ones: the sum is finite, and larger
    than head 1's, on every third page."""
    cache = _cache(d=64)
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    q[0, 0, 0, :8] = -2.0 ** 64
    q[0, 0, 0, 56:] = 2.0 ** 64
    q[0, 1, 0, 30] = 2.0 ** 64
    for j in range(PAGES):
        a = torch.zeros(64)
        a[:8] = 2.0 ** 62                                   # -2^126 each: -2^129
        a[56:] = 2.0 ** 62
        a[60:] *= 1 + 0.125 * (j % 3)                       # 2^129 + (j % 3) 2^125
        a[30] = 2.0 ** 56 * j                               # head 1: 2^120 j
        _set_bounds(cache, j, a.to(torch.bfloat16), a.to(torch.bfloat16))
    _check(q, cache, paged.PageSelectConfig(k, 1, 1), k)


@pytest.mark.parametrize("dtype,span", [("bf16", 120), ("bf16", 64), ("bf16", 20), ("fp16", 14), ("fp16", 4)])
@pytest.mark.parametrize("G,d", [(1, 64), (2, 128), (5, 64), (16, 128)])
def test_magnitudes_over_the_whole_range(dtype, span, G, d):
    """Pages and query channels of very different magnitudes: whether the screen can be used or not, the
    lists are the definition's. (Magnitudes differ between pages by powers of two and are alike within one, so that
    64-bit sums are exact.)"""
    for seed in range(6):
        g = torch.Generator().manual_seed(100 * span + seed)
        cache = _cache(dtype, d, pages=200, seed=seed)
        e = torch.randint(-span, span // 2, (1, cache.k.shape[1], 1, 1, 1), generator=g).double()
        b = cache.bounds.cpu().double() * 2.0 ** e
        top = torch.finfo(DT[dtype]).max
        cache.bounds.copy_(b.clamp(-top, top).to(DT[dtype]))
        if dtype == "bf16" or span < 10:
            q = (_q(G, d, seed, dtype).double() * 2.0 ** [0, span // 2, -span // 2][seed % 3]).to(DT[dtype])
        else:
            q = _q(G, d, seed, dtype)
        if seed == 5:
            cache.page_table[0, 50] = -1
        _check(q, cache, paged.PageSelectConfig([9, 60, 150][seed % 3], 1, 2), (dtype, span, seed))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("val", [float("nan"), float("inf"), float("-inf")])
def test_bounds_that_are_not_finite_are_bad_scores(dtype, val):
    """... and not pages that the table lacks."""
    for chan in (0, 9, 63):
        cache = _cache(dtype)
        pg = cache.page_table[0, 12].item()
        cache.bounds[0, pg, 0, 1, chan] = val
        _check(_q(2, dtype=dtype), cache, paged.PageSelectConfig(8, 1, 1), (dtype, val, chan))


@pytest.mark.parametrize("k", [5, 64, 300])
@pytest.mark.parametrize("G,d,dtype", [(4, 128, "bf16"), (2, 64, "fp16"), (16, 64, "bf16")])
@pytest.mark.parametrize("lean", [0.0, 0.4, 0.7, 1.0])
def test_scores_of_both_signs(k, G, d, dtype, lean):
    """Keys with channel offsets and a query against them: scores around zero, where few or many 32-bit keys lie
    between two pages; with pages missing, too."""
    pages = 700
    cache = _cache(dtype, d, pages=pages, seed=int(10 * lean) + G)
    off = 3 * torch.sign(torch.randn(d, generator=torch.Generator().manual_seed(d)))
    cache.bounds += off.to(DT[dtype]).cuda()
    q = (_q(G, d, k, dtype).float() - lean * off).to(DT[dtype])
    cfg = paged.PageSelectConfig(k, 1, 2)
    _check(q, cache, cfg, (lean, k))
    for j in (0, 17, 400, 699):
        cache.page_table[0, j] = -1
    _check(q, cache, cfg, (lean, k, "missing"))
