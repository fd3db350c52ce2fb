"""Attention outputs against bounds that shrink with them (paged_tight): long sequences shared by every CTA,
prompt chunks, drafted tokens at every kind of row count, page lists."""
import random

import numpy as np
import pytest
import torch

from block_sparse_causal_bsa_b200 import paged
from oracle import paged_oracle as O
from paged_tight import Rows
from paged_util import DT, f8, make_cache, scale_of, words

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _heads(cache, b, n):
    """Per KV head of slot b: (head, K rows, V rows) in 64 bits."""
    page, d = cache.k.shape[3:]
    pages = cache.page_table[b, :-(-n // page)].long()
    for h in range(cache.k.shape[2]):
        yield h, *(f8(x[0, pages, h].reshape(-1, d)[:n]) for x in (cache.k, cache.v))


def _check_tree(seed, *, lens, qls, T, G, Hkv, d, page, dtype, tree=False):
    rng = random.Random(seed)
    cache = make_cache(seed, lens=lens, max_pages=max(1, max(-(-n // page) for n in lens)), page=page, Hkv=Hkv, d=d,
                       dtype=dtype, garbage=float("nan"))
    q = torch.randn(len(lens), G * Hkv, T, d, generator=torch.Generator().manual_seed(seed + 1)).to(DT[dtype])
    see = np.stack([O.ancestors([-1 if t == 0 else rng.randint(max(0, t - 6), t - 1) for t in range(T)]) if tree else
                    np.tril(np.ones((T, T), bool)) for _ in lens])
    out, lse, st = paged.attend_tree(q.cuda(), cache, mask=words(see).cuda() if tree else None, q_len=_i32(qls))
    assert int(st) == 0
    go, gl, qn = f8(out), f8(lse), f8(q)
    for b, (n, ql) in enumerate(zip(lens, qls)):
        if ql == 0:
            continue
        vis = np.ones((ql, n), bool)
        vis[:, n - ql:] = see[b, :ql, :ql]
        for h, kr, vr in _heads(cache, b, n):
            hs = slice(h * G, (h + 1) * G)
            ref = Rows(qn[b, hs, :ql].reshape(G * ql, d), kr, vr, np.tile(vis, (G, 1)), scale_of(d), dtype, G * T)
            assert ref.problem(go[b, hs, :ql].reshape(G * ql, d), gl[b, hs, :ql].reshape(-1)) is None, (b, h)


@pytest.mark.parametrize("T,G,d,dtype", [(1, 4, 128, "bf16"), (2, 8, 128, "fp16"), (1, 16, 64, "fp16"), (1, 1, 128, "bf16"),
                                         (4, 4, 64, "bf16"), (20, 1, 64, "bf16"), (33, 4, 128, "bf16"), (20, 4, 64, "fp16")])
@pytest.mark.parametrize("n", [3968, 20011, 90001])
def test_one_sequence_shared_by_every_cta(n, T, G, d, dtype):
    _check_tree(n + T, lens=[n], qls=[T], T=T, G=G, Hkv=1, d=d, page=128, dtype=dtype)


@pytest.mark.parametrize("T,G,Hkv,d,dtype,tree", [
    (2, 4, 2, 128, "bf16", False), (4, 4, 2, 64, "fp16", True), (3, 5, 1, 128, "fp16", True), (16, 1, 2, 128, "bf16", True),
    (17, 1, 2, 128, "bf16", True), (5, 8, 1, 128, "bf16", True), (8, 16, 1, 64, "fp16", True), (33, 4, 2, 128, "fp16", True),
    (64, 4, 2, 128, "bf16", True), (9, 16, 1, 128, "bf16", False), (43, 3, 1, 64, "bf16", True)])
def test_ragged_drafts(T, G, Hkv, d, dtype, tree):
    qls = [T, max(1, T // 2), T, 1, T, 0, T]
    lens = [ql + [0, 37, 900, 5000, 2048, 3, 7777][i] for i, ql in enumerate(qls)]
    _check_tree(T + G, lens=lens, qls=qls, T=T, G=G, Hkv=Hkv, d=d, page=32, dtype=dtype, tree=tree)


@pytest.mark.parametrize("T,G,d,dtype,lens,qls", [
    (1024, 2, 128, "bf16", [1024, 2500], [1024, 1024]), (777, 4, 64, "fp16", [777, 1200, 700], [777, 1, 500]),
    (513, 3, 128, "fp16", [4000, 513], [513, 300]), (256, 8, 128, "bf16", [256, 1111], [256, 255])])
def test_prompt_chunks(T, G, d, dtype, lens, qls):
    _check_tree(T, lens=lens, qls=qls, T=T, G=G, Hkv=1, d=d, page=64, dtype=dtype)


@pytest.mark.parametrize("G,Hkv,T,page,d,dtype,lens,W", [
    (4, 2, 1, 64, 128, "bf16", [40000, 100, 64], 64), (2, 1, 5, 16, 64, "fp16", [24007, 130, 5], 96),
    (16, 1, 2, 32, 128, "fp16", [9001, 33], 200), (1, 2, 3, 128, 128, "bf16", [7000, 3], 20)])
def test_page_lists(G, Hkv, T, page, d, dtype, lens, W):
    """Lists of random pages, in any order, of every length."""
    rng = random.Random(W)
    cache = make_cache(W, lens=lens, max_pages=-(-max(lens) // page), page=page, Hkv=Hkv, d=d, dtype=dtype,
                       garbage=float("nan"))
    B = len(lens)
    q = torch.randn(B, G * Hkv, T, d, generator=torch.Generator().manual_seed(W + 1)).to(DT[dtype])
    idx, cnt = np.full((B, Hkv, T, W), -1), np.zeros((B, Hkv, T), int)
    for b, h, t in np.ndindex(B, Hkv, T):
        pages = rng.sample(range((lens[b] - T + t) // page + 1), min(W, (lens[b] - T + t) // page + 1))
        pages = pages[:max(1, len(pages) - rng.choice([0, 0, 3, len(pages) // 2]))]
        idx[b, h, t, :len(pages)], cnt[b, h, t] = pages, len(pages)
    out, lse, st = paged.attend_pages(q.cuda(), cache, _i32(idx.tolist()), _i32(cnt.tolist()))
    assert int(st) == 0
    go, gl, qn = f8(out), f8(lse), f8(q)
    for b, n in enumerate(lens):
        for h, kr, vr in _heads(cache, b, n):
            for t in range(T):
                at = [p * page + o for p in idx[b, h, t, :cnt[b, h, t]] for o in range(page) if p * page + o <= n - T + t]
                hs = slice(h * G, (h + 1) * G)
                ref = Rows(qn[b, hs, t], kr[at], vr[at], None, scale_of(d), dtype, G)
                assert ref.problem(go[b, hs, t], gl[b, hs, t]) is None, (b, h, t)
