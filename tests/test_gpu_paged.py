"""The paged-cache operators against the plain fp64 oracle: attention of drafted trees and chains
over the cache, selection of pages and attention over them, appending, compacting, forking,
growing, copying and freeing, one by one and as a serving step."""
import random

import numpy as np
import pytest
import torch

from block_sparse_causal_bsa_b200 import binding as bb
from block_sparse_causal_bsa_b200 import paged
from oracle import paged_oracle as O
from paged_util import (DT, check, f8, lse_tolerance, make_cache, out_tolerance, scale_of, words)

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _random_tree(rng, T, n_roots=1):
    return [-1 if t < n_roots else rng.randint(max(0, t - 5), t - 1) for t in range(T)]


def _run_tree(seed, *, lens, qls, T, Hq, Hkv, d, page, dtype="bf16", see=None, garbage=None, max_pages=None,
              cache=None, expect=0):
    """attend_tree against the oracle; see [B, T, T] bool or None (a chain)."""
    max_pages = max_pages or max(1, max(-(-n // page) for n in lens))
    cache = cache or make_cache(seed, lens=lens, max_pages=max_pages, page=page, Hkv=Hkv, d=d, dtype=dtype,
                                garbage=garbage)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(len(lens), Hq, T, d, generator=g).to(DT[dtype])
    mask = None if see is None else words(see).cuda()
    mark = 7.0
    out = torch.full((len(lens), Hq, T, d), mark, dtype=DT[dtype], device="cuda")
    lse = torch.full((len(lens), Hq, T), mark, device="cuda")
    _, _, st = paged.attend_tree(q.cuda(), cache, mask=mask, q_len=_i32(qls), out=out, lse=lse)
    torch.cuda.synchronize()
    assert int(st) == expect
    go, gl = f8(out), f8(lse)
    k, v, table, qn = f8(cache.k[0]), f8(cache.v[0]), cache.page_table.cpu().tolist(), f8(q)
    for b, (n, ql) in enumerate(zip(lens, qls)):
        assert (go[b, :, ql:] == mark).all() and (gl[b, :, ql:] == mark).all()      # left as they were
        if ql == 0:
            continue
        sd = np.tril(np.ones((ql, ql), bool)) if see is None else see[b, :ql, :ql]
        with np.errstate(invalid="ignore"):
            ro, rl = O.attend_tree(qn[b, :, :ql], k, v, table[b], n, ql, page, sd, scale_of(d))
        pages = table[b][:-(-n // page)]
        kr, vr = k[pages], v[pages]
        km, vm = np.abs(kr[np.isfinite(kr)]).max(), np.abs(vr[np.isfinite(vr)]).max()
        p_bits = 16 if Hq // Hkv * T <= 16 else 8
        check(gl[b, :, :ql], rl, lse_tolerance(rl, qn[b], km, d, scale_of(d), n), ("lse", b))
        fin = np.isfinite(ro)
        assert np.array_equal(np.isnan(go[b, :, :ql]), np.isnan(ro)), ("nan", b)
        check(np.where(np.isnan(ro), 0, go[b, :, :ql]), np.where(np.isnan(ro), 0, ro),
              out_tolerance(np.where(fin, ro, 0), qn[b], km, vm, d, scale_of(d), dtype, p_bits), ("out", b))
    return go, gl, cache, q


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16"), (64, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (5, 1)])
def test_decode_one_token(d, dtype, page, Hq, Hkv):
    lens = [1, 15, 16, 17, 63, 64, 65, 128, 129, 400]
    _run_tree(11, lens=lens, qls=[1] * len(lens), T=1, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype,
              garbage=float("nan"))


@pytest.mark.parametrize("T,Hq,Hkv,page,d,dtype", [
    (2, 4, 1, 16, 128, "bf16"), (5, 6, 2, 32, 64, "fp16"), (8, 8, 2, 64, 128, "bf16"), (16, 16, 1, 128, 64, "bf16"),
    (33, 4, 2, 16, 128, "fp16"), (64, 8, 2, 64, 128, "bf16"), (65, 2, 2, 64, 64, "bf16"), (130, 3, 1, 32, 128, "bf16")])
def test_tree(T, Hq, Hkv, page, d, dtype):
    rng = random.Random(T)
    lens, qls = [], []
    for i in range(5):
        ql = [T, 1, max(1, T // 2), T, 0][i]
        lens.append(ql + [0, 3, 70, 333, 90][i])
        qls.append(ql)
    par = [_random_tree(rng, T, n_roots=1 + i % 2) for i in range(5)]
    see = np.stack([O.ancestors(p) for p in par])
    _run_tree(21, lens=lens, qls=qls, T=T, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype, see=see,
              garbage=float("inf"))
    mask, st = paged.tree_mask(_i32(par), q_len=_i32(qls))
    assert int(st) == 0
    want = words(see).cuda()
    for b, ql in enumerate(qls):
        assert torch.equal(mask[b, :ql], want[b, :ql]) and (mask[b, ql:] == 0).all()


@pytest.mark.parametrize("T", [1, 7, 64, 100])
def test_chain(T):
    _run_tree(31, lens=[T, T + 1, T + 500], qls=[T, min(T, 3), T], T=T, Hq=8, Hkv=2, d=128, page=64)


@pytest.mark.parametrize("T,Hq,Hkv,page,d,dtype,B", [
    (1, 8, 4, 16, 128, "bf16", 40), (6, 4, 2, 16, 64, "fp16", 40), (24, 4, 2, 64, 128, "bf16", 40),
    (70, 8, 4, 32, 64, "bf16", 20), (70, 4, 2, 128, 128, "fp16", 20), (9, 8, 4, 16, 64, "bf16", 30)])
def test_many_tiles_per_share(T, Hq, Hkv, page, d, dtype, B):
    """Enough work that every SM walks many tiles and several items: the rings wrap, and segments
    begin and end inside shares. Sampled sequences against the oracle, the status for all."""
    rng = random.Random(7)
    qls = [rng.choice([T, T, max(1, T // 2), 1]) for _ in range(B)]
    lens = [ql + rng.choice([0, 900, 2500, 4000]) + rng.randint(0, 130) for ql in qls]
    cache = make_cache(33, lens=lens, max_pages=-(-max(lens) // page), page=page, Hkv=Hkv, d=d, dtype=dtype,
                       garbage=float("nan"))
    q = torch.randn(B, Hq, T, d, generator=torch.Generator().manual_seed(34)).to(DT[dtype])
    out, lse, st = paged.attend_tree(q.cuda(), cache, q_len=_i32(qls))
    out2, lse2, st2 = paged.attend_tree(q.cuda(), cache, q_len=_i32(qls))
    assert int(st) == 0 and int(st2) == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)              # bit for bit
    assert torch.isfinite(out.float()).all()
    k, v, table, qn = cache.k[0].cpu(), cache.v[0].cpu(), cache.page_table.cpu().tolist(), f8(q)
    go, gl = f8(out), f8(lse)
    for b in range(0, B, 4):
        n, ql, G = lens[b], qls[b], Hq // Hkv
        pages = torch.tensor(table[b][:-(-n // page)])
        for h in range(Hkv):
            kr, vr = (f8(x[pages, h].reshape(-1, d)[:n]) for x in (k, v))
            qh = qn[b, h * G:(h + 1) * G, :ql].reshape(G * ql, d)
            see = np.ones((ql, n), bool)
            see[:, n - ql:] = np.tril(np.ones((ql, ql), bool))
            z = np.where(np.tile(see, (G, 1)), qh @ kr.T * scale_of(d), -np.inf)
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            ro, rl = p @ vr / p.sum(1, keepdims=True), (m + np.log(p.sum(1, keepdims=True)))[:, 0]
            km, vm = np.abs(kr).max(), np.abs(vr).max()
            check(go[b, h * G:(h + 1) * G, :ql].reshape(-1, d), ro,
                  out_tolerance(ro, qh, km, vm, d, scale_of(d), dtype, 16 if G * T <= 16 else 8), (b, h))
            check(gl[b, h * G:(h + 1) * G, :ql].reshape(-1), rl, lse_tolerance(rl, qh, km, d, scale_of(d), n), (b, h))


def test_mask_that_leaves_rows_empty():
    see = np.zeros((2, 6, 6), bool)
    see[0, 2, 4] = see[0, 3, 0] = True          # any mask, not ancestors alone; other rows see nothing
    go, gl, _, _ = _run_tree(41, lens=[6, 40], qls=[6, 6], T=6, Hq=4, Hkv=2, d=64, page=16, see=see)
    assert (go[0, :, 0] == 0).all() and np.isneginf(gl[0, :, 0]).all()


@pytest.mark.parametrize("T", [6, 40])
def test_nonfinite_drafts_reach_only_rows_that_see_them(T):
    lens, page, d = [T + 77, T], 16, 128
    rng = random.Random(5)
    par = [_random_tree(rng, T) for _ in lens]
    see = np.stack([O.ancestors(p) for p in par])
    cache = make_cache(51, lens=lens, max_pages=16, page=page, Hkv=2, d=d)
    tab = cache.page_table.cpu()
    for b in range(2):
        for t, val in [(T - 1, float("nan")), (T - 2, float("inf")), (3, float("-inf"))]:
            pos = lens[b] - T + t
            cache.v[0, tab[b, pos // page], :, pos % page, t % d] = val
    pos = lens[0] - 1
    cache.k[0, tab[0, pos // page], 0, pos % page, 5] = float("nan")       # seen by the last draft alone
    go, gl, cache2, q = _run_tree_nan(52, cache, lens, T, see, page, d)


def _run_tree_nan(seed, cache, lens, T, see, page, d):
    Hq = 8
    q = torch.randn(len(lens), Hq, T, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    out, lse, st = paged.attend_tree(q.cuda(), cache, mask=words(see).cuda())
    assert int(st) == 0
    go, gl = f8(out), f8(lse)
    k, v, table, qn = f8(cache.k[0]), f8(cache.v[0]), cache.page_table.cpu().tolist(), f8(q)
    for b, n in enumerate(lens):
        with np.errstate(invalid="ignore"):
            ro, rl = O.attend_tree(qn[b], k, v, table[b], n, T, page, see[b], scale_of(d))
        assert np.array_equal(np.isnan(go[b]), np.isnan(ro)) and np.array_equal(np.isinf(go[b]), np.isinf(ro))
        assert np.array_equal(np.isnan(gl[b]), np.isnan(rl))
        fin = np.isfinite(ro)
        km = np.nanmax(np.abs(k[np.isfinite(k)]))
        vm = np.abs(v[np.isfinite(v)]).max()
        check(np.where(fin, go[b], 0), np.where(fin, ro, 0),
              out_tolerance(np.where(fin, ro, 0), qn[b], km, vm, d, scale_of(d), "bf16", 16 if T * 4 <= 16 else 8), b)
    return go, gl, cache, q


def test_bad_table_entries_and_lengths_are_reported_and_skipped():
    lens, page, d = [100, 50, 80], 16, 64
    cache = make_cache(61, lens=lens, max_pages=8, page=page, Hkv=2, d=d)
    good = cache.page_table.clone()
    cache.page_table[0, 2] = cache.k.shape[1]             # no such page: its rows are not seen
    cache.page_table[2, 1] = -5
    q = torch.randn(3, 4, 2, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out, lse, st = paged.attend_tree(q.cuda(), cache)
    assert int(st) == bb.BSA_DEV_BAD_INDEX
    k, v, table = f8(cache.k[0]), f8(cache.v[0]), good.cpu().tolist()
    for b, hole in [(0, range(32, 48)), (1, ()), (2, range(16, 32))]:
        n = lens[b]
        for g in range(4):
            kr, vr = O.rows_of(k, table[b], n, page, g // 2), O.rows_of(v, table[b], n, page, g // 2)
            see = np.tril(np.ones((n, n), bool))[n - 2:]
            see[:, list(hole)] = False
            ro, rl = O.softmax_rows(f8(q)[b, g], kr, vr, see, scale_of(d))
            check(f8(out)[b, g], ro, out_tolerance(ro, f8(q), np.abs(k).max(), np.abs(v).max(), d, scale_of(d),
                                                   "bf16", 16), (b, g))
            check(f8(lse)[b, g], rl, lse_tolerance(rl, f8(q), np.abs(k).max(), d, scale_of(d), n), (b, g))
    # lengths that do not fit: the slot is left out, the others are served
    cache.page_table.copy_(good)
    cache.seq_len[1] = 1
    out2 = torch.full_like(out, 3.0)
    _, _, st = paged.attend_tree(q.cuda(), cache, out=out2)
    assert int(st) == bb.BSA_DEV_BAD_INDEX and (out2[1] == 3.0).all() and torch.isfinite(out2).all()
    cache.seq_len[1] = 8 * page + 1
    _, _, st = paged.attend_tree(q.cuda(), cache, out=out2)
    assert int(st) == bb.BSA_DEV_BAD_INDEX and (out2[1] == 3.0).all()


# ---------------------------------------------------------------------------------------------
# selection and attention over lists

def _scores(qn, bounds, table, own_page, G, h):
    return [O.page_score(qn[h * G:(h + 1) * G], bounds[table[j], h, 0], bounds[table[j], h, 1])
            for j in range(own_page + 1)]


def _run_sparse(seed, *, lens, qls, T, Hq, Hkv, d, page, cfg, dtype="bf16", garbage=None, cache=None, q=None):
    max_pages = max(cfg.k, max(-(-n // page) for n in lens))
    cache = cache or make_cache(seed, lens=lens, max_pages=max_pages, page=page, Hkv=Hkv, d=d, dtype=dtype,
                                garbage=garbage)
    if q is None:
        q = torch.randn(len(lens), Hq, T, d, generator=torch.Generator().manual_seed(seed + 1)).to(DT[dtype])
    ql = _i32(qls)
    sel = paged.select_pages(q.cuda(), cache, cfg, q_len=ql, want_scores=True)
    sel2 = paged.select_pages(q.cuda(), cache, cfg, q_len=ql)
    assert torch.equal(sel["kv_idx"], sel2["kv_idx"]) and torch.equal(sel["kv_cnt"], sel2["kv_cnt"])
    mark = 5.0
    out = torch.full((len(lens), Hq, T, d), mark, dtype=DT[dtype], device="cuda")
    lse = torch.full((len(lens), Hq, T), mark, device="cuda")
    _, _, st = paged.attend_pages(q.cuda(), cache, sel["kv_idx"], sel["kv_cnt"], q_len=ql, out=out, lse=lse)
    assert int(st) == 0 and int(sel["dev_status"]) == 0
    idx, cnt, sc = sel["kv_idx"].cpu().numpy(), sel["kv_cnt"].cpu().numpy(), sel["scores"].cpu().numpy()
    k, v, bd = f8(cache.k[0]), f8(cache.v[0]), f8(cache.bounds[0])
    table, qn, go, gl = cache.page_table.cpu().tolist(), f8(q), f8(out), f8(lse)
    G = Hq // Hkv
    fin = lambda x: np.abs(x[np.isfinite(x)]).max()
    for b, (n, ql_) in enumerate(zip(lens, qls)):
        assert (go[b, :, ql_:] == mark).all() and (gl[b, :, ql_:] == mark).all()
        assert (idx[b, :, ql_:] == -1).all() and (cnt[b, :, ql_:] == 0).all()
        assert np.isneginf(sc[b, :, ql_:]).all()
        for t in range(ql_):
            pos = n - ql_ + t
            own = pos // page
            for h in range(Hkv):
                ref = _scores(qn[b, :, t], bd, table[b], own, G, h)
                assert np.array_equal(sc[b, h, t, :own + 1], np.array(ref, np.float32)), (b, t, h)
                assert np.isneginf(sc[b, h, t, own + 1:]).all()
                want = O.select(ref, own, cfg.k, cfg.n_first, cfg.n_last)
                assert cnt[b, h, t] == len(want)
                assert idx[b, h, t].tolist() == want + [-1] * (cfg.k - len(want)), (b, t, h)
                hs = slice(h * G, (h + 1) * G)
                ro, rl = O.attend_list(qn[b, hs, t], k[:, h], v[:, h], table[b], pos, page, want, scale_of(d))
                check(go[b, hs, t], ro, out_tolerance(ro, qn[b], fin(k), fin(v), d, scale_of(d), dtype, 16), (b, t, h))
                check(gl[b, hs, t], rl, lse_tolerance(rl, qn[b], fin(k), d, scale_of(d), n), (b, t, h))
    return sel, cache, q


@pytest.mark.parametrize("Hq,Hkv,d,page,dtype", [
    (8, 2, 128, 64, "bf16"), (2, 2, 64, 16, "fp16"), (3, 1, 128, 16, "bf16"), (4, 2, 64, 32, "bf16"),
    (16, 2, 128, 32, "fp16"), (12, 1, 64, 16, "bf16"), (16, 1, 128, 16, "bf16"), (5, 1, 64, 128, "fp16")])
def test_select_and_attend(Hq, Hkv, d, page, dtype):
    lens = [1, page, page + 1, 5 * page + 3, 23 * page - 1]
    cfg = paged.PageSelectConfig(6, 1, 2)
    _run_sparse(71, lens=lens, qls=[1] * 5, T=1, Hq=Hq, Hkv=Hkv, d=d, page=page, cfg=cfg, dtype=dtype,
                garbage=float("nan"))


@pytest.mark.parametrize("k,n_first,n_last", [(1, 0, 1), (3, 1, 2), (2, 0, 1), (9, 3, 3), (40, 1, 1)])
def test_select_budgets_chain(k, n_first, n_last):
    _run_sparse(81, lens=[40, 333, 700, 9], qls=[4, 3, 0, 4], T=4, Hq=4, Hkv=2, d=64, page=16,
                cfg=paged.PageSelectConfig(k, n_first, n_last))


def test_budget_beyond_the_table():
    """k past the pages that the table has room for: lists of every page, padded."""
    lens, page = [100, 16, 1], 16
    cache = make_cache(82, lens=lens, max_pages=7, page=page, Hkv=2, d=64)
    q = torch.randn(3, 4, 1, 64, generator=torch.Generator().manual_seed(83)).to(torch.bfloat16).cuda()
    sel = paged.select_pages(q, cache, paged.PageSelectConfig(50, 1, 1))
    for b, n in enumerate(lens):
        m = -(-n // page)
        assert sel["kv_idx"][b, 1, 0].tolist() == list(range(m)) + [-1] * (50 - m)
    out, lse, st = paged.attend_pages(q, cache, sel["kv_idx"], sel["kv_cnt"])
    full, lsef, st2 = paged.attend_tree(q, cache)
    assert int(st) == 0 and int(st2) == 0
    assert torch.equal(out, full) and torch.allclose(lse, lsef, atol=1e-5)


def test_select_ties_go_to_the_lower_page():
    """Copies of pages, and q = 0 (every score equal): the lowest indexes win."""
    lens, page = [64 * 16], 16
    cache = make_cache(91, lens=lens, max_pages=64, page=page, Hkv=1, d=64)
    cache.bounds[0] = cache.bounds[0][torch.arange(cache.k.shape[1], device="cuda") % 3]
    _run_sparse(91, lens=lens, qls=[1], T=1, Hq=2, Hkv=1, d=64, page=page,
                cfg=paged.PageSelectConfig(17, 1, 1), cache=cache)
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    sel, _, _ = _run_sparse(92, lens=lens, qls=[1], T=1, Hq=2, Hkv=1, d=64, page=page,
                            cfg=paged.PageSelectConfig(17, 1, 1), cache=cache, q=q)
    assert sel["kv_idx"][0, 0, 0].tolist() == list(range(16)) + [63]


def test_select_wide_range_of_magnitudes():
    """Bounds and queries from subnormals to the largest finite values: the fp64 sums are the
    definition's (all terms of a page kept within 2^30 of each other, so the sum is exact)."""
    g = torch.Generator().manual_seed(3)
    for dtype, lo, hi in [("bf16", -126, 110), ("fp16", -20, 3)]:
        cache = make_cache(93, lens=[40 * 16], max_pages=40, page=16, Hkv=1, d=128, dtype=dtype)
        e = torch.randint(lo, hi, (1, cache.k.shape[1], 1, 1, 1), generator=g).double()
        cache.bounds.copy_((cache.bounds.cpu().double() * 2.0 ** e).to(DT[dtype]))
        # no rank depends on a value that overflowed: fp32 scores must stay finite
        q = (torch.randn(1, 4, 1, 128, generator=g) * 0.01).to(DT[dtype])
        sel = paged.select_pages(q.cuda(), cache, paged.PageSelectConfig(9, 1, 1), want_scores=True)
        assert int(sel["dev_status"]) == 0
        table = cache.page_table.cpu().tolist()[0]
        ref = _scores(f8(q)[0, :, 0], f8(cache.bounds[0]), table, 39, 4, 0)
        assert np.array_equal(sel["scores"].cpu().numpy()[0, 0, 0], np.array(ref, np.float32)), dtype
        assert sel["kv_idx"][0, 0, 0].tolist() == O.select(ref, 39, 9, 1, 1)


def test_select_reports_nonfinite_and_missing_pages():
    lens, page = [30 * 16], 16
    cfg = paged.PageSelectConfig(8, 1, 1)
    q = torch.randn(1, 2, 1, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    for what, bit in [("nan", bb.BSA_DEV_BAD_SCORE), ("inf", bb.BSA_DEV_BAD_SCORE), ("page", bb.BSA_DEV_BAD_INDEX)]:
        cache = make_cache(94, lens=lens, max_pages=30, page=page, Hkv=1, d=64)
        if what == "page":
            cache.page_table[0, 7] = 10 ** 6
        else:
            cache.bounds[0, cache.page_table[0, 7].item(), 0, 1, 9] = float(what)
        sel = paged.select_pages(q, cache, cfg)
        assert int(sel["dev_status"]) == bit
        got = sel["kv_idx"][0, 0, 0].tolist()
        assert got == sorted(got) and len(set(got)) == 8 and 7 not in got
    # forced pages are not ranked, so theirs is not reported
    cache = make_cache(94, lens=lens, max_pages=30, page=page, Hkv=1, d=64)
    cache.bounds[0, cache.page_table[0, 0].item()] = float("nan")
    assert int(paged.select_pages(q, cache, cfg)["dev_status"]) == 0
    # a NaN query: every score is NaN, the list is still a valid one
    q2 = q.clone()
    q2[0, 0, 0, 3] = float("nan")
    sel = paged.select_pages(q2, cache, cfg)
    got = sel["kv_idx"][0, 0, 0].tolist()
    assert int(sel["dev_status"]) == bb.BSA_DEV_BAD_SCORE and got == sorted(set(got)) and len(got) == 8


def test_attend_pages_bad_entries_counts_and_empty_lists():
    lens, page, d = [200, 200, 200, 200], 16, 64
    cache = make_cache(95, lens=lens, max_pages=13, page=page, Hkv=1, d=d)
    q = torch.randn(4, 2, 1, d, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    idx = _i32([[3, 99, 12, -4, 0], [1, 2, 3, 4, 5], [9, 1, 13, 0, 0], [7, 7, 7, 7, 7]]).reshape(4, 1, 1, 5)
    cnt = _i32([5, 0, 9, 1]).reshape(4, 1, 1)
    out, lse, st = paged.attend_pages(q.cuda(), cache, idx, cnt)
    assert int(st) == bb.BSA_DEV_BAD_INDEX
    k, v, table = f8(cache.k[0]), f8(cache.v[0]), cache.page_table.cpu().tolist()
    for b, pages in enumerate([[3, 12, 0], [], [9, 1, 0, 0], [7]]):
        rows = [(p, o) for p in pages for o in range(page) if p * page + o <= 199]
        kr = np.array([k[table[b][p], 0, o] for p, o in rows]).reshape(-1, d)
        vr = np.array([v[table[b][p], 0, o] for p, o in rows]).reshape(-1, d)
        ro, rl = O.softmax_rows(f8(q)[b, :, 0], kr, vr, np.ones((2, len(rows)), bool), scale_of(d))
        check(f8(out)[b, :, 0], ro, out_tolerance(ro, f8(q), np.abs(k).max(), np.abs(v).max(), d, scale_of(d),
                                                  "bf16", 16), b)
        check(f8(lse)[b, :, 0], rl, lse_tolerance(rl, f8(q), np.abs(k).max(), d, scale_of(d), 200), b)


# ---------------------------------------------------------------------------------------------
# rows and pages

def _same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def _bounds_ref(kpool, table, n, page, j, layer=0):
    rows = kpool[layer, table[j], :, :min(page, n - j * page)].float()
    return rows.amin(1), rows.amax(1)


@pytest.mark.parametrize("T,page,d,dtype,Hkv", [(1, 16, 128, "bf16", 2), (1, 64, 64, "fp16", 3), (5, 16, 64, "bf16", 1),
                                               (40, 32, 128, "fp16", 2), (130, 64, 128, "bf16", 2),
                                               (300, 128, 64, "bf16", 1), (1024, 16, 128, "bf16", 1)])
def test_append(T, page, d, dtype, Hkv):
    qls = [T, 1, 0, max(1, T // 3), T]
    lens = [T, 1 + 2 * page, 10, max(1, T // 3) + page - 1, T + 3 * page + 5]
    mp = max(-(-n // page) for n in lens) + 1
    cache = make_cache(101, lens=lens, max_pages=mp, page=page, Hkv=Hkv, d=d, dtype=dtype, layers=2)
    # the bounds as they are before the call: of the rows before it
    for s, (n, ql) in enumerate(zip(lens, qls)):
        base = n - ql
        if base % page and ql:
            pg = cache.page_table[s, base // page]
            cache.bounds[1, pg, :, 0] = cache.k[1, pg, :, :base % page].amin(1)
            cache.bounds[1, pg, :, 1] = cache.k[1, pg, :, :base % page].amax(1)
    g = torch.Generator().manual_seed(102)
    kn = torch.randn(5, Hkv, T, d, generator=g).to(DT[dtype]).cuda()
    vn = torch.randn(5, Hkv, T, d, generator=g).to(DT[dtype]).cuda()
    want = [cache.k.clone(), cache.v.clone(), cache.bounds.clone()]
    tab = cache.page_table.cpu().tolist()
    for s, (n, ql) in enumerate(zip(lens, qls)):
        for t in range(ql):
            pos = n - ql + t
            want[0][1, tab[s][pos // page], :, pos % page] = kn[s, :, t]
            want[1][1, tab[s][pos // page], :, pos % page] = vn[s, :, t]
        if ql:
            for j in range((n - ql) // page, (n - 1) // page + 1):
                lo, hi = _bounds_ref(want[0], tab[s], n, page, j, 1)
                want[2][1, tab[s][j], :, 0], want[2][1, tab[s][j], :, 1] = lo.to(DT[dtype]), hi.to(DT[dtype])
    st = paged.append(cache, kn, vn, q_len=_i32(qls), layer=1)
    assert int(st) == 0
    for a, b in zip((cache.k, cache.v, cache.bounds), want):
        assert _same_bits(a, b)


def test_append_without_bounds_and_with_bad_slots():
    lens, page = [20, 20, 20], 16
    cache = make_cache(103, lens=lens, max_pages=2, page=page, Hkv=1, d=64)
    cache.bounds = None
    cache.page_table[1, 1] = 77
    cache.seq_len[2] = 3                                   # fewer than the call's tokens
    kn = torch.ones(3, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
    before = cache.k.clone()
    tab = cache.page_table.cpu()
    assert int(paged.append(cache, kn, kn)) == bb.BSA_DEV_BAD_INDEX
    for pos in range(12, 20):
        before[0, tab[0, pos // 16], :, pos % 16] = 1
    for pos in range(12, 16):                              # the page that the table holds is written
        before[0, tab[1, 0], :, pos] = 1
    assert _same_bits(cache.k, before)


def test_append_nan_makes_the_bounds_nan():
    cache = make_cache(104, lens=[20], max_pages=2, page=16, Hkv=1, d=64)
    kn = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    kn[0, 0, 2, 7] = float("nan")
    assert int(paged.append(cache, kn, kn)) == 0
    b = cache.bounds[0, cache.page_table[0, 1].item(), 0].float()
    assert torch.isnan(b[:, 7]).all() and int(torch.isnan(b).sum()) == 2


@pytest.mark.parametrize("T,page,d,dtype", [(1, 16, 64, "bf16"), (6, 16, 128, "fp16"), (33, 16, 128, "bf16"),
                                            (64, 64, 64, "bf16"), (200, 32, 128, "bf16"), (512, 128, 64, "fp16")])
def test_compact(T, page, d, dtype):
    rng = random.Random(T)
    Hkv = 2
    qls = [T, T, max(1, T // 2), 0, T, T]
    lens = [T, T + 37, max(1, T // 2) + 64, 5, T + 200, T + 15]
    keep, nk = [], []
    for i, ql in enumerate(qls):
        n = [rng.randint(0, ql), ql, rng.randint(0, ql), 0, 0, 1][i]
        kp = sorted(rng.sample(range(ql), n)) if i != 5 else [ql - 1]
        keep.append(kp + [99999] * (T - n))
        nk.append(n)
    cache = make_cache(111, lens=lens, max_pages=-(-max(lens) // page), page=page, Hkv=Hkv, d=d, dtype=dtype)
    want = [cache.k.clone(), cache.v.clone(), cache.bounds.clone()]
    tab = cache.page_table.cpu().tolist()
    for s in range(6):
        base = lens[s] - qls[s]
        for i in range(nk[s]):
            a, b = base + keep[s][i], base + i
            for w in want[:2]:
                w[0, tab[s][b // page], :, b % page] = w[0, tab[s][a // page], :, a % page]
        end = base + nk[s]
        if qls[s]:
            for j in range(base // page, -(-end // page)):
                lo, hi = _bounds_ref(want[0], tab[s], end, page, j)
                want[2][0, tab[s][j], :, 0], want[2][0, tab[s][j], :, 1] = lo.to(DT[dtype]), hi.to(DT[dtype])
    st = paged.compact(cache, _i32(keep), _i32(nk), q_len=_i32(qls))
    assert int(st) == 0
    for a, b in zip((cache.k, cache.v, cache.bounds), want):
        assert _same_bits(a, b)


def test_compact_bad_lists_leave_the_slot_alone():
    lens = [30] * 5
    cache = make_cache(112, lens=lens, max_pages=2, page=16, Hkv=1, d=64)
    keep = _i32([[0, 2, 2, 3], [3, 1, 0, 0], [1, 4, 0, 0], [-1, 0, 0, 0], [0, 1, 2, 3]])
    nk = _i32([3, 2, 2, 1, 5])
    before = [cache.k.clone(), cache.v.clone(), cache.bounds.clone()]
    assert int(paged.compact(cache, keep, nk)) == bb.BSA_DEV_BAD_INDEX
    for a, b in zip((cache.k, cache.v, cache.bounds), before):
        assert _same_bits(a, b)


def _book_of(cache, page):
    bk = O.Book(cache.slots, cache.max_pages, cache.refs.numel(), page)
    bk.table, bk.len, bk.refs = cache.page_table.cpu().tolist(), cache.seq_len.cpu().tolist(), cache.refs.cpu().tolist()
    return bk


def _check_book(cache, bk):
    assert cache.page_table.cpu().tolist() == bk.table
    assert cache.seq_len.cpu().tolist() == bk.len
    assert cache.refs.cpu().tolist() == bk.refs


@pytest.mark.parametrize("seed,slots,n_pages,page", [(1, 6, 40, 16), (2, 33, 300, 32), (3, 7, 13, 64), (4, 130, 2000, 16),
                                                     (5, 1, 9, 128), (6, 40, 97, 16)])
def test_fork_resize_random_sequences_of_calls(seed, slots, n_pages, page):
    rng = random.Random(seed)
    max_pages = 12
    cache = paged.PagedCache.create(layers=1, n_pages=n_pages, Hkv=1, page=page, d=64, slots=slots,
                                    max_pages=max_pages)
    bk = O.Book(slots, max_pages, n_pages, page)
    short_seen = False
    for step in range(40):
        new = []
        for s in range(slots):
            r = rng.random()
            n = bk.len[s]
            if r < 0.3:
                new.append(-1)
            elif r < 0.6:
                new.append(n + rng.choice([1, 1, 2, page, 3 * page + 1]))
            elif r < 0.75:
                new.append(rng.randint(0, n))
            elif r < 0.85:
                new.append(0)
            else:
                new.append(rng.randint(0, max_pages * page))
        new = [min(n, max_pages * page) if rng.random() < 0.98 else n for n in new]
        pairs, n_free, st = paged.resize(cache, _i32(new))
        wp, wf, short, bad = bk.resize(new)
        assert pairs.cpu().tolist() == [list(p) for p in wp], step
        assert int(n_free) == wf
        assert int(st) == (bb.BSA_DEV_NO_PAGES if short else 0) | (bb.BSA_DEV_BAD_INDEX if bad else 0)
        _check_book(cache, bk)
        short_seen |= short
        if slots > 1 and rng.random() < 0.7:
            parent = [-1] * slots
            for c in range(slots):
                if rng.random() < 0.4:
                    parent[c] = rng.randrange(slots) if rng.random() < 0.97 else slots + 3
            ok = bk.fork(parent)
            assert (int(paged.fork(cache, _i32(parent))) == 0) == ok
            _check_book(cache, bk)
    if n_pages < 3 * slots:
        assert short_seen


def test_resize_large_pool():
    """More pages than threads, and more slots than a pass of them."""
    slots, page, n_pages = 2500, 16, 50001
    cache = paged.PagedCache.create(layers=1, n_pages=n_pages, Hkv=1, page=page, d=64, slots=slots, max_pages=40)
    bk = O.Book(slots, 40, n_pages, page)
    rng = random.Random(9)
    for step in range(3):
        new = [rng.choice([-1, 0, rng.randint(0, 640)]) for _ in range(slots)]
        pairs, n_free, st = paged.resize(cache, _i32(new))
        wp, wf, short, bad = bk.resize(new)
        assert int(st) == (bb.BSA_DEV_NO_PAGES if short else 0) and int(n_free) == wf
        _check_book(cache, bk)


@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("fp16", 64, 128)])
def test_copy_pages(dtype, d, page):
    cache = make_cache(121, lens=[page * 20], max_pages=20, page=page, Hkv=3, d=d, dtype=dtype, layers=2)
    pairs = [[0, 10], [0, 11], [-1, -1], [3, 12], [5, 13]]
    want = [cache.k.clone(), cache.v.clone(), cache.bounds.clone()]
    for s, t in pairs:
        if s >= 0:
            for w in want:
                w[1, t] = w[1, s]
    assert int(paged.copy_pages(cache, _i32(pairs), layer=1)) == 0
    for a, b in zip((cache.k, cache.v, cache.bounds), want):
        assert _same_bits(a, b)
    # conflicts: a destination that is a source, the same destination twice, out of range
    pairs = [[1, 2], [2, 14], [4, 15], [6, 15], [7, 7], [8, 24], [99, 3], [-1, 9], [9, -1], [9, 16]]
    for s, t in [(2, 14), (4, 15), (9, 16)]:
        for w in want:
            w[1, t] = w[1, s]
    assert int(paged.copy_pages(cache, _i32(pairs), layer=1)) == bb.BSA_DEV_BAD_INDEX
    for a, b in zip((cache.k, cache.v, cache.bounds), want):
        assert _same_bits(a, b)
    assert int(paged.copy_pages(cache, _i32([]).reshape(0, 2))) == 0


def test_tree_mask_bad_parents():
    mask, st = paged.tree_mask(_i32([[-1, 0, 2, 1, 7]]))
    assert int(st) == bb.BSA_DEV_BAD_INDEX
    assert mask[0, :, 0].tolist() == [1, 3, 4, 8 + 3, 16]
