"""NaN and infinities in queries, keys and values that a token sees reach its result, whatever the number of
query rows and however its keys are split: an empty result (0, -inf) means that it sees nothing. Rows
beside them are not touched."""
import numpy as np
import pytest
import torch

from block_sparse_causal_bsa_b200 import paged
from paged_tight import Rows
from paged_util import DT, f8, make_cache, scale_of, words

pytestmark = pytest.mark.gpu

# query rows per KV head 1, 16 (warp-level MMAs), 17, 128, 129, 256 (tcgen05, one and two groups of rows), 320
ROWS = [(1, 1), (4, 4), (1, 17), (4, 32), (3, 43), (8, 32), (4, 80)]
LENS = [90, 3000]                 # keys of one or two tiles in one share; split over many


def _setup(G, T, n, d, dtype, seed=3):
    cache = make_cache(seed, lens=[n, n], max_pages=-(-n // 32), page=32, Hkv=2, d=d, dtype=dtype)
    q = torch.randn(2, 2 * G, T, d, generator=torch.Generator().manual_seed(seed + 1)).to(DT[dtype])
    return cache, q


def _at(cache, b, pos):
    return cache.page_table[b, pos // 32].item(), pos % 32


def _check(cache, q, G, T, n, poisoned, see=None):
    """poisoned bool [2, Hq, T]: rows that have to be NaN, output and lse; the others as in 64 bits."""
    mask = None if see is None else words(np.stack([see, see])).cuda()
    out, lse, st = paged.attend_tree(q.cuda(), cache, mask=mask)
    assert int(st) == 0
    d = q.shape[-1]
    dtype = "bf16" if q.dtype == torch.bfloat16 else "fp16"
    go, gl, qn = f8(out), f8(lse), f8(q)
    k, v, table = cache.k[0].cpu(), cache.v[0].cpu(), cache.page_table.cpu()
    rows = np.ones((T, n), bool)
    rows[:, n - T:] = np.tril(np.ones((T, T), bool)) if see is None else see
    for b in range(2):
        pages = table[b, :-(-n // 32)].long()
        for h in range(2):
            kr, vr = (f8(x[pages, h].reshape(-1, d)[:n]) for x in (k, v))
            for g in range(h * G, (h + 1) * G):
                bad = poisoned[b, g]
                assert np.isnan(go[b, g][bad]).all() and np.isnan(gl[b, g][bad]).all(), (b, g)
                if bad.all():
                    continue
                kf, vf = np.nan_to_num(kr, nan=0.0, posinf=0.0, neginf=0.0), np.nan_to_num(vr, nan=0.0, posinf=0.0, neginf=0.0)
                ref = Rows(qn[b, g][~bad], kf, vf, rows[~bad], scale_of(d), dtype, G * T)
                assert ref.problem(go[b, g][~bad], gl[b, g][~bad]) is None, (b, g)


@pytest.mark.parametrize("n", LENS)
@pytest.mark.parametrize("G,T", ROWS)
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_nan_queries(G, T, n, d, dtype):
    cache, q = _setup(G, T, n, d, dtype)
    bad = np.zeros((2, 2 * G, T), bool)
    for b, g, t in [(0, 0, 0), (1, 2 * G - 1, T - 1), (1, G, T // 2)]:
        q[b, g, t, (5 * t) % d] = float("nan")
        bad[b, g, t] = True
    _check(cache, q, G, T, n, bad)


@pytest.mark.parametrize("n", LENS)
@pytest.mark.parametrize("G,T", ROWS)
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_a_channel_of_all_keys_nan(G, T, n, d, dtype):
    cache, q = _setup(G, T, n, d, dtype)
    bad = np.zeros((2, 2 * G, T), bool)
    for j in range(-(-n // 32)):
        cache.k[0, cache.page_table[0, j].item(), 1, :, 7] = float("nan")
    bad[0, G:] = True
    _check(cache, q, G, T, n, bad)


@pytest.mark.parametrize("lo,hi", [(0, 64), (64, 320), (1024, 2048), (2880, 2912)])
@pytest.mark.parametrize("G,T", ROWS)
def test_a_stretch_of_keys_nan(G, T, lo, hi):
    """Whole shares of the split hold nothing but NaN scores."""
    n = 3000
    cache, q = _setup(G, T, n, 128, "bf16")
    for pos in range(lo, hi):
        pg, r = _at(cache, 1, pos)
        cache.k[0, pg, 0, r] = float("nan")
    bad = np.zeros((2, 2 * G, T), bool)
    bad[1, :G] = True
    _check(cache, q, G, T, n, bad)


@pytest.mark.parametrize("G,T", [r for r in ROWS if r[1] > 1])
@pytest.mark.parametrize("what", ["nan", "empty"])
def test_a_token_that_sees_one_nan_key_or_none(G, T, what):
    """A call without earlier positions; token 1 sees token 0 alone, whose key is NaN, or nothing."""
    n = T
    cache, q = _setup(G, T, n, 64, "bf16")
    see = np.tril(np.ones((T, T), bool))
    see[:, 0] = False
    see[0, 0] = what == "nan"
    see[1] = False
    see[1, 0] = what == "nan"
    bad = np.zeros((2, 2 * G, T), bool)
    for b in range(2):
        pg, r = _at(cache, b, 0)
        cache.k[0, pg, :, r, 3] = float("nan")
    if what == "nan":
        bad[:, :, :2] = True
    _check(cache, q, G, T, n, bad, see)


@pytest.mark.parametrize("n", LENS)
@pytest.mark.parametrize("G,T", ROWS)
def test_an_infinite_value_that_weighs_nothing(G, T, n):
    """The weight underflows to 0 in 32 bits: 0 x inf, as in the plain form; the channel is never finite."""
    cache, q = _setup(G, T, n, 64, "bf16")
    q = q.abs() + 1
    for pos in range(32):
        pg, r = _at(cache, 0, pos)
        cache.k[0, pg, 0, r] = -60.0
    pg, r = _at(cache, 0, 5)
    if n - T <= 5:
        pytest.skip("the key is a drafted one")
    cache.v[0, pg, 0, r, 9] = float("inf")
    out, lse, st = paged.attend_tree(q.cuda(), cache)
    assert int(st) == 0
    o = out.float().cpu()
    assert not torch.isfinite(o[0, :G, :, 9]).any()
    o[0, :G, :, 9] = 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
