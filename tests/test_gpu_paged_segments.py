"""Attention of more than 16 query rows per KV head where a CTA's share falls into many short segments: items of one
tile, which the two groups of the kernel take in turn, and items of 129 rows and more, whose tile
begins in one share and ends in the next. Against the 64-bit result."""
import numpy as np
import pytest
import torch

from block_sparse_causal_bsa_b200 import paged
from paged_tight import Rows
from paged_util import DT, f8, make_cache, scale_of

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_chain(seed, *, lens, qls, T, Hq, Hkv, d, page, dtype, sample):
    cache = make_cache(seed, lens=lens, max_pages=max(1, max(-(-n // page) for n in lens)), page=page, Hkv=Hkv, d=d,
                       dtype=dtype, garbage=float("nan"))
    q = torch.randn(len(lens), Hq, T, d, generator=torch.Generator().manual_seed(seed + 1)).to(DT[dtype])
    out, lse, st = paged.attend_tree(q.cuda(), cache, q_len=_i32(qls))
    again, lse2, st2 = paged.attend_tree(q.cuda(), cache, q_len=_i32(qls))
    assert int(st) == 0 and int(st2) == 0
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    G = Hq // Hkv
    k, v, table, qn, go, gl = cache.k[0].cpu(), cache.v[0].cpu(), cache.page_table.cpu(), f8(q), f8(out), f8(lse)
    assert np.isfinite(go).all()
    for b in sample:
        n, ql = lens[b], qls[b]
        if ql == 0:
            continue
        pages = table[b, :-(-n // page)].long()
        see = np.ones((ql, n), bool)
        see[:, n - ql:] = np.tril(np.ones((ql, ql), bool))
        for h in range(Hkv):
            kr, vr = (f8(x[pages, h].reshape(-1, d)[:n]) for x in (k, v))
            hs = slice(h * G, (h + 1) * G)
            ref = Rows(qn[b, hs, :ql].reshape(G * ql, d), kr, vr, np.tile(see, (G, 1)), scale_of(d), dtype, G * T)
            assert ref.problem(go[b, hs, :ql].reshape(G * ql, d), gl[b, hs, :ql].reshape(-1)) is None, (b, h)


def segments(lens, qls, G, Hkv, n_cta=148):
    """(tiles, shared) of every segment of every share, as the kernel lays them out."""
    items = []
    for n, ql in zip(lens, qls):
        rows = G * ql
        if ql:
            items += [(-(-n // 64), 2 if rows > 128 else 1, min(256, rows - r0) <= 128)
                      for _ in range(Hkv) for r0 in range(0, rows, 256)]
    total = sum(t * w for t, w, _ in items)
    per = max(-(-total // n_cta), 2)
    out, at = {}, 0
    for t, w, share in items:
        for c in range(at // per, (at + t * w - 1) // per + 1):
            a, b = max(at, c * per) - at, min(at + t * w, (c + 1) * per) - at
            out.setdefault(c, []).append((-(-b // w) - -(-a // w), share))
        at += t * w
    return list(out.values())


@pytest.mark.parametrize("B,T,qls,G,Hkv,d,dtype", [
    (300, 20, [20, 17, 20, 9], 1, 2, 64, "bf16"),           # one shared tile after the other
    (230, 33, [33, 9, 33, 33, 20], 4, 2, 128, "fp16"),      # ... with items of 132 rows between them
    (190, 40, [40], 4, 1, 64, "bf16"),                      # 160 rows: tiles that begin and end in other shares
    (193, 64, [64, 1, 32, 0, 5], 8, 1, 128, "bf16")])        # up to two row tiles of 256
def test_short_segments(B, T, qls, G, Hkv, d, dtype):
    qls = [qls[i % len(qls)] for i in range(B)]
    lens = [max(ql + (i * 7) % 30, 1) for i, ql in enumerate(qls)]
    shares = segments(lens, qls, G, Hkv)
    pairs = [(x, y) for s in shares for x, y in zip(s, s[1:])]
    # what the case is for: shared segments of one tile in a row, or segments without a tile
    assert any(x == (1, True) and y == (1, True) for x, y in pairs) or any(x[0] == 0 for s in shares for x in s)
    run_chain(B, lens=lens, qls=qls, T=T, Hq=G * Hkv, Hkv=Hkv, d=d, page=16, dtype=dtype, sample=range(0, B, 7))
