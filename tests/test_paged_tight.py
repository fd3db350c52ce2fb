"""The bounds of paged_tight: correctly rounded results pass them, planted mistakes (in the oracle, on
the CPU) do not."""
import numpy as np
import pytest
import torch

from paged_tight import Rows
from paged_util import DT, scale_of


def _rows(n, R, d, dtype, rows_per_head, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dtype]).double().numpy()
    page_mean = torch.randn(-(-n // 64), d, generator=g).repeat_interleave(64, 0)[:n] * 0.7
    k = (torch.randn(n, d, generator=g) + page_mean).to(DT[dtype]).double().numpy()
    see = np.ones((R, n), bool)
    see[:, n - min(n, R):] = np.tril(np.ones((R, min(n, R)), bool))
    return Rows(r(R, d), k, r(n, d), see, scale_of(d), dtype, rows_per_head)


CASES = [(90001, 20, 64, "bf16", 20), (90001, 1, 128, "bf16", 1), (3968, 32, 128, "bf16", 32), (3968, 8, 64, "fp16", 8),
         (700, 40, 64, "fp16", 40), (500, 4, 128, "bf16", 4), (130, 17, 128, "bf16", 17)]


@pytest.mark.parametrize("n,R,d,dtype,rows", CASES)
def test_rounded_results_pass(n, R, d, dtype, rows):
    for seed in range(3):
        x = _rows(n, R, d, dtype, rows, seed)
        assert x.problem(x.rounded(), x.lse.astype(np.float32).astype(np.float64)) is None


@pytest.mark.parametrize("n,R,d,dtype,rows", CASES)
def test_planted_mistakes_are_found(n, R, d, dtype, rows):
    x = _rows(n, R, d, dtype, rows, 7)
    zero = np.zeros_like(x.out)
    assert x.problem(zero)
    tiles = np.add.reduceat((x.w ** 2).sum(0), np.arange(0, n, 64))
    # a tile of 64 keys that counts as much as the average, or most: without its values, or with another tile's
    for t0 in (64 * int(np.argmax(tiles >= tiles.mean())), 64 * int(tiles.argmax())):
        v = x.v.copy()
        v[t0:t0 + 64] = 0
        assert x.problem(x.rounded(v=v)), t0
        v = x.v.copy()
        other = 64 if t0 == 0 else 0
        m = min(64, n - t0, n - other)
        v[t0:t0 + m] = x.v[other:other + m]
        assert x.problem(x.rounded(v=v)), t0
    for parts in (4, 148):                             # a part's output lost, its sum kept
        per = max(128, n // parts)
        w = x.w.copy()
        w[:, per:2 * per] = 0
        if n > per:
            assert x.problem(x.rounded(w=w)), parts
    w = x.w.copy()                                     # half of the keys' weights off by two percent
    w[:, :n // 2] *= 1.02
    assert x.problem(x.rounded(w=w))
    assert x.problem(x.rounded() * (1 + 2 * torch.finfo(DT[dtype]).eps)), "two steps"
    lse = x.lse.copy()
    lse[-1] += 1e-2
    assert x.problem(x.rounded(), lse)
