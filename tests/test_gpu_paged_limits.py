"""The largest table that the calls take, full: 32768 pages of one sequence."""
import numpy as np
import pytest
import torch

from block_sparse_causal_bsa_b200 import paged
from oracle import paged_oracle as O
from paged_tight import Rows
from paged_util import f8, make_cache, scale_of

pytestmark = pytest.mark.gpu
PAGES, PAGE, D = 32768, 16, 64


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def cache():
    return make_cache(7, lens=[PAGES * PAGE], max_pages=PAGES, page=PAGE, Hkv=1, d=D)


def _q(seed, G, T):
    return torch.randn(1, G, T, D, generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("G,T", [(2, 1), (1, 18)])
def test_attention(cache, G, T):
    n = PAGES * PAGE
    q = _q(T, G, T)
    out, lse, st = paged.attend_tree(q.cuda(), cache)
    assert int(st) == 0
    pages = cache.page_table[0].long()
    k, v = (f8(x[0, pages, 0].reshape(-1, D)) for x in (cache.k, cache.v))
    see = np.ones((G * T, n), bool)
    see[:, n - T:] = np.tile(np.tril(np.ones((T, T), bool)), (G, 1))
    ref = Rows(f8(q)[0].reshape(-1, D), k, v, see, scale_of(D), "bf16", G * T)
    assert ref.problem(f8(out)[0].reshape(-1, D), f8(lse)[0].reshape(-1)) is None


@pytest.mark.parametrize("k", [7, 64, 2000, 32767, 32768])
def test_selection_and_its_attention(cache, k):
    q = _q(k, 4, 2)
    cfg = paged.PageSelectConfig(k, 2, 3)
    exact, fast = (paged.select_pages(q.cuda(), cache, cfg, want_scores=w) for w in (True, False))
    assert int(exact["dev_status"]) == int(fast["dev_status"]) == 0
    assert torch.equal(exact["kv_idx"], fast["kv_idx"]) and torch.equal(exact["kv_cnt"], fast["kv_cnt"])
    table, bd = cache.page_table[0].cpu().numpy(), f8(cache.bounds[0])[:, 0]
    for t in range(2):
        own = PAGES - 1
        lo, hi = bd[table, 0], bd[table, 1]
        sc = np.max([np.maximum(x * lo, x * hi).sum(1) for x in f8(q)[0, :, t]], 0).astype(np.float32)
        assert np.array_equal(sc, exact["scores"][0, 0, t].cpu().numpy())
        order = np.lexsort((np.arange(own + 1), -sc))
        must = np.r_[0, 1, own - 2, own - 1, own]
        want = np.r_[must, [j for j in order if j not in set(must)][:k - 5]]
        assert fast["kv_idx"][0, 0, t, :len(want)].tolist() == sorted(want.tolist())
    out, lse, st = paged.attend_pages(q.cuda(), cache, fast["kv_idx"], fast["kv_cnt"])
    assert int(st) == 0
    if k <= 64 or k == PAGES:                          # (PAGES: every page, in other shares than attend_tree's)
        for t in range(2):
            at = [p * PAGE + o for p in fast["kv_idx"][0, 0, t].tolist() for o in range(PAGE)
                  if p * PAGE + o <= PAGES * PAGE - 2 + t]
            kr, vr = (f8(x[0, cache.page_table[0, torch.tensor(at).cuda() // PAGE].long(), 0, torch.tensor(at).cuda() % PAGE])
                      for x in (cache.k, cache.v))
            ref = Rows(f8(q)[0, :, t], kr, vr, None, scale_of(D), "bf16", 4)
            assert ref.problem(f8(out)[0, :, t], f8(lse)[0, :, t]) is None


def test_rows_written_and_moved_at_the_end(cache):
    T, n = 1024, PAGES * PAGE
    g = torch.Generator().manual_seed(3)
    k, v, b = cache.k.clone(), cache.v.clone(), cache.bounds.clone()
    c = paged.PagedCache(k, v, b, cache.page_table.clone(), cache.seq_len.clone(), cache.refs.clone())
    kn, vn = (torch.randn(1, 1, T, D, generator=g).bfloat16().cuda() for _ in range(2))
    assert int(paged.append(c, kn, vn)) == 0
    keep = list(range(1, T, 2))
    assert int(paged.compact(c, _i32([keep + [0] * (T - len(keep))]), _i32([len(keep)]))) == 0
    pages = c.page_table[0, PAGES - T // PAGE:].long()
    got = c.k[0, pages, 0].reshape(T, D)
    assert torch.equal(got[:len(keep)], kn[0, 0, keep]) and torch.equal(c.v[0, pages, 0].reshape(T, D)[:len(keep)], vn[0, 0, keep])
    assert torch.equal(c.k[0, c.page_table[0, :PAGES - T // PAGE].long()], cache.k[0, c.page_table[0, :PAGES - T // PAGE].long()])
    done = len(keep) // PAGE
    rows = c.k[0, pages[:done], 0]
    assert torch.equal(c.bounds[0, pages[:done], 0, 0], rows.amin(1)) and torch.equal(c.bounds[0, pages[:done], 0, 1], rows.amax(1))
    # the sequence given back, and taken again
    pairs, n_free, st = paged.resize(c, _i32([0]))
    assert int(st) == 0 and int(n_free) == c.refs.numel() and not c.refs.any() and (c.page_table == -1).all()
    pairs, n_free, st = paged.resize(c, _i32([n]))
    assert int(st) == 0 and c.page_table[0].tolist() == list(range(PAGES)) and int(n_free) == c.refs.numel() - PAGES
