"""Cases and tolerances shared by the tests of the paged-cache operators."""
import math

import numpy as np
import torch

from block_sparse_causal_bsa_b200 import paged

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f8(t):
    return t.detach().cpu().double().numpy()


def make_cache(seed, *, lens, max_pages, page, Hkv, d, dtype="bf16", layers=1, spare=4, device="cuda",
               garbage=None):
    """A cache whose slots hold lens[s] random rows each on randomly placed pages. garbage: what
    every row that belongs to no sequence holds (None: random values)."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    need = sum(-(-n // page) for n in lens)
    P = need + spare
    dt = DT[dtype]
    k = torch.randn(layers, P, Hkv, page, d, generator=g).to(dt)
    v = torch.randn(layers, P, Hkv, page, d, generator=g).to(dt)
    k += (0.7 * torch.randn(layers, P, Hkv, 1, d, generator=g)).to(dt)
    perm = torch.randperm(P, generator=g)
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    refs = torch.zeros(P, dtype=torch.int32)
    bounds = torch.zeros(layers, P, Hkv, 2, d, dtype=dt)
    live = torch.zeros(P, page, dtype=torch.bool)
    at = 0
    for s, n in enumerate(lens):
        m = -(-n // page)
        table[s, :m] = perm[at:at + m].int()
        refs[perm[at:at + m]] = 1
        for j in range(m):
            fill = min(page, n - j * page)
            pg = perm[at + j]
            live[pg, :fill] = True
            bounds[:, pg, :, 0] = k[:, pg, :, :fill].amin(2)
            bounds[:, pg, :, 1] = k[:, pg, :, :fill].amax(2)
        at += m
    if garbage is not None:
        dead = ~live[None, :, None, :, None].expand_as(k)
        k[dead] = garbage
        v[dead] = garbage
    return paged.PagedCache(k=k.to(device), v=v.to(device), bounds=bounds.to(device),
                            page_table=table.to(device), seq_len=torch.tensor(lens, dtype=torch.int32, device=device),
                            refs=refs.to(device))


def out_tolerance(ref, q, k_rows_max, v_max, d, scale, dtype, p_bits):
    """|out - ref| allowed: half a step of the output type, and what the weights can be off by.
    A logit: d products summed in fp32, each addition off by 2^-24 relative to the sum of
    magnitudes, at most d |q| |k| scale. A weight: twice that (it and the denominator), the
    exponential's 2^-22 twice, and its rounding to p_bits bits before the product. A value of
    magnitude v_max is weighted by it."""
    dl = (d + 2) * 2.0 ** -24 * float(np.abs(q).max()) * k_rows_max * scale * d
    w = 2 * dl + 2 * 2.0 ** -22 + 2.0 ** -p_bits + 64 * 2.0 ** -24
    eps = torch.finfo(DT[dtype]).eps
    tiny = torch.finfo(DT[dtype]).smallest_normal * eps
    return eps / 2 * np.abs(ref) + w * v_max * (1 + eps) + tiny


def lse_tolerance(ref, q, k_rows_max, d, scale, n):
    dl = (d + 2) * 2.0 ** -24 * float(np.abs(q).max()) * k_rows_max * scale * d
    return dl + 2.0 ** -21 + (n / 64 + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(np.isfinite(ref), ref, 0))


def check(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    inf = np.isinf(ref)
    assert np.array_equal(np.isinf(got) & inf, inf) and np.array_equal(np.sign(got[inf]), np.sign(ref[inf])), what
    err = np.abs(np.where(inf, 0, got) - np.where(inf, 0, ref))
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(err.max()), np.argwhere(bad)[:4].tolist())


def words(see):
    """bool [B, T, T] -> int64 mask words [B, T, ceil(T/64)]."""
    B, T, _ = see.shape
    W = -(-T // 64)
    out = np.zeros((B, T, W), np.uint64)
    for w in range(W):
        for i in range(min(64, T - 64 * w)):
            out[:, :, w] |= see[:, :, 64 * w + i].astype(np.uint64) << np.uint64(i)
    return torch.from_numpy(out.view(np.int64))


def scale_of(d):
    return 1.0 / math.sqrt(d)
