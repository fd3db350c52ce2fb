"""The paged-cache operators together, as a serving loop uses them: drafted trees grown, verified
and compacted over several steps with forks in between, against plain Python lists of rows and the
fp64 oracle; the same step captured in a CUDA graph; two streams at once; pools past 2^31 elements."""
import random

import numpy as np
import pytest
import torch

from block_sparse_causal_bsa_b200 import binding as bb
from block_sparse_causal_bsa_b200 import paged
from oracle import paged_oracle as O
from paged_util import DT, check, f8, lse_tolerance, make_cache, out_tolerance, scale_of, words

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("seed,page,d,dtype,Hq,Hkv", [(1, 16, 64, "bf16", 4, 2), (2, 32, 128, "fp16", 3, 1),
                                                      (3, 64, 128, "bf16", 16, 1)])
def test_speculative_serving_loop(seed, page, d, dtype, Hq, Hkv):
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    slots, T, max_pages, layers = 7, 9, 20, 2
    cache = paged.PagedCache.create(layers=layers, n_pages=160, Hkv=Hkv, page=page, d=d, slots=slots,
                                    max_pages=max_pages, dtype=DT[dtype])
    cache.k.fill_(float("nan"))                       # what no sequence holds is never looked at
    cache.v.fill_(float("nan"))
    rows = [[([], []) for _ in range(slots)] for _ in range(layers)]       # [layer][slot] -> K rows, V rows
    G = Hq // Hkv
    for step in range(7):
        # forks: copies of a random slot into empty ones
        parent = [-1] * slots
        empty = [s for s in range(slots) if not rows[0][s][0]]
        full = [s for s in range(slots) if rows[0][s][0]]
        for s in empty:
            if full and rng.random() < 0.7:
                parent[s] = rng.choice(full)
        assert int(paged.fork(cache, _i32(parent))) == 0
        for s, p in enumerate(parent):
            if p >= 0:
                for lay in range(layers):
                    rows[lay][s] = (list(rows[lay][p][0]), list(rows[lay][p][1]))
        # the step's tokens: a chunk of a prompt, a tree, one token, or none
        ql = [rng.choice([0, 1, T, T]) if rows[0][s][0] else rng.choice([0, T, T]) for s in range(slots)]
        base = [len(rows[0][s][0]) for s in range(slots)]
        pairs, _, st = paged.resize(cache, _i32([b + q for b, q in zip(base, ql)]))
        assert int(st) == 0
        par = [[-1 if t == 0 else rng.randint(max(0, t - 3), t - 1) for t in range(T)] for _ in range(slots)]
        mask, st = paged.tree_mask(_i32(par), q_len=_i32(ql))
        assert int(st) == 0
        see = np.stack([O.ancestors(p) for p in par])
        n_keep = [rng.randint(0, q) for q in ql]
        if step == 0:
            n_keep = list(ql)
        keep = [sorted(rng.sample(range(q), n)) for q, n in zip(ql, n_keep)]
        cfg = paged.PageSelectConfig(3, 1, 1)
        for lay in range(layers):
            assert int(paged.copy_pages(cache, pairs, layer=lay)) == 0
            q = torch.randn(slots, Hq, T, d, generator=g).to(DT[dtype])
            kn, vn = (torch.randn(slots, Hkv, T, d, generator=g).to(DT[dtype]) for _ in range(2))
            assert int(paged.append(cache, kn.cuda(), vn.cuda(), q_len=_i32(ql), layer=lay)) == 0
            out, lse, st = paged.attend_tree(q.cuda(), cache, mask=mask, q_len=_i32(ql), layer=lay)
            sel = paged.select_pages(q.cuda(), cache, cfg, q_len=_i32(ql), layer=lay)
            outp, lsep, st2 = paged.attend_pages(q.cuda(), cache, sel["kv_idx"], sel["kv_cnt"], q_len=_i32(ql),
                                                 layer=lay)
            assert int(st) == 0 and int(st2) == 0 and int(sel["dev_status"]) == 0
            go, gl, gp, gpl, qn = f8(out), f8(lse), f8(outp), f8(lsep), f8(q)
            idx, cnt = sel["kv_idx"].cpu().numpy(), sel["kv_cnt"].cpu().numpy()
            p_bits = 16 if G * T <= 16 else 8
            for s in range(slots):
                if ql[s] == 0:
                    continue
                K = rows[lay][s][0] + [f8(kn)[s, :, t] for t in range(ql[s])]     # rows of [Hkv, d]
                V = rows[lay][s][1] + [f8(vn)[s, :, t] for t in range(ql[s])]
                K, V = np.stack(K, 1), np.stack(V, 1)                            # [Hkv, n, d]
                n = K.shape[1]
                vis = np.concatenate([np.ones((ql[s], base[s]), bool), see[s, :ql[s], :ql[s]]], 1)
                km, vm = np.abs(K).max(), np.abs(V).max()
                for h in range(Hq):
                    ro, rl = O.softmax_rows(qn[s, h, :ql[s]], K[h // G], V[h // G], vis, scale_of(d))
                    tol = out_tolerance(ro, qn[s], km, vm, d, scale_of(d), dtype, p_bits)
                    check(go[s, h, :ql[s]], ro, tol, ("tree", step, lay, s, h))
                    check(gl[s, h, :ql[s]], rl, lse_tolerance(rl, qn[s], km, d, scale_of(d), n), ("lse", step, s, h))
                for t in range(ql[s]):
                    own = (base[s] + t) // page
                    for hk in range(Hkv):
                        # bounds of the pages' filled rows, drafts of the step among them
                        sc = []
                        for j in range(own + 1):
                            r = K[hk, j * page:min(n, (j + 1) * page)]
                            sc.append(O.page_score(qn[s, hk * G:(hk + 1) * G, t], r.min(0), r.max(0)))
                        want = O.select(sc, own, cfg.k, cfg.n_first, cfg.n_last)
                        assert idx[s, hk, t].tolist() == want + [-1] * (3 - len(want)), (step, lay, s, t, hk)
                        at = [p * page + o for p in want for o in range(page) if p * page + o <= base[s] + t]
                        ro, rl = O.softmax_rows(qn[s, hk * G:(hk + 1) * G, t], K[hk][at], V[hk][at],
                                                np.ones((G, len(at)), bool), scale_of(d))
                        tol = out_tolerance(ro, qn[s], km, vm, d, scale_of(d), dtype, 16)
                        check(gp[s, hk * G:(hk + 1) * G, t], ro, tol, ("pages", step, lay, s, t))
            assert int(paged.compact(cache, _i32([k + [-1] * (T - len(k)) for k in keep]), _i32(n_keep),
                                     q_len=_i32(ql), layer=lay)) == 0
            for s in range(slots):
                for t in keep[s]:
                    rows[lay][s][0].append(f8(kn)[s, :, t])
                    rows[lay][s][1].append(f8(vn)[s, :, t])
        # accepted lengths; one slot ends now and then
        new = [len(rows[0][s][0]) for s in range(slots)]
        if step >= 2:
            end = rng.randrange(slots)
            new[end] = 0
            for lay in range(layers):
                rows[lay][end] = ([], [])
        _, n_free, st = paged.resize(cache, _i32(new))
        assert int(st) == 0
        refs = cache.refs.cpu()
        held = cache.page_table[cache.page_table >= 0].cpu().long()
        assert torch.equal(torch.bincount(held, minlength=160).int(), refs)
        assert int(n_free) == int((refs == 0).sum())


def _step(cache, new_len, kn, vn, q, mask, ql, cfg):
    pairs, n_free, st0 = paged.resize(cache, new_len)
    st1 = paged.copy_pages(cache, pairs)
    st2 = paged.append(cache, kn, vn, q_len=ql)
    out, lse, st3 = paged.attend_tree(q, cache, mask=mask, q_len=ql)
    sel = paged.select_pages(q, cache, cfg, q_len=ql)
    outp, lsep, st4 = paged.attend_pages(q, cache, sel["kv_idx"], sel["kv_cnt"], q_len=ql)
    return [out, lse, outp, lsep, sel["kv_idx"], sel["kv_cnt"], st0, st1, st2, st3, sel["dev_status"], st4, n_free]


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (12, 8, 2), (40, 8, 1)])
def test_captured_step_replays(T, Hq, Hkv):
    """A whole step in a CUDA graph, replayed with other inputs and on grown sequences: bit for bit
    what the calls give one by one, with an eager step in between."""
    B, page, d = 5, 16, 64
    lens = [100, 3, 257, 64, 1]
    cfg = paged.PageSelectConfig(5, 1, 1)
    mk = lambda: make_cache(7, lens=lens, max_pages=60, page=page, Hkv=Hkv, d=d, spare=200)
    a, b = mk(), mk()
    g = torch.Generator().manual_seed(8)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    see = np.stack([O.ancestors([-1 if t == 0 else random.Random(t + s).randint(0, t - 1) for t in range(T)])
                    for s in range(B)])
    mask, ql = words(see).cuda(), _i32([T] * B)
    ins = [_i32([n + T for n in lens]), rand(B, Hkv, T, d), rand(B, Hkv, T, d), rand(B, Hq, T, d)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                     # first calls load the kernels
        warm = mk()
        _step(warm, ins[0], *ins[1:], mask, ql, cfg)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _step(a, ins[0], *ins[1:], mask, ql, cfg)
    n = list(lens)
    for rep in range(3):
        n = [x + T for x in n]
        ins[0].copy_(_i32(n))
        for t in ins[1:]:
            t.copy_(rand(*t.shape))
        graph.replay()
        want = _step(b, ins[0], *ins[1:], mask, ql, cfg)
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y), rep
        for x, y in ((a.k, b.k), (a.v, b.v), (a.bounds, b.bounds), (a.page_table, b.page_table),
                     (a.seq_len, b.seq_len), (a.refs, b.refs)):
            assert torch.equal(x, y), rep


def test_two_streams_at_once_and_a_given_stream():
    lens, page, d = [5000, 3000, 800, 4097], 16, 128
    cache = make_cache(17, lens=lens, max_pages=320, page=page, Hkv=2, d=d)
    g = torch.Generator().manual_seed(18)
    cfg = paged.PageSelectConfig(20, 1, 2)
    cases = []
    for T in (1, 5, 24, 70):
        q = torch.randn(4, 8, T, d, generator=g).to(torch.bfloat16).cuda()
        ref = paged.attend_tree(q, cache)
        sel = paged.select_pages(q, cache, cfg)
        refp = paged.attend_pages(q, cache, sel["kv_idx"], sel["kv_cnt"])
        cases.append((q, ref, sel, refp))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for rep in range(6):
        for i, (q, _, _, _) in enumerate(cases):
            s = streams[(rep + i) % 3]
            o = paged.attend_tree(q, cache, stream=s)
            sel = paged.select_pages(q, cache, cfg, stream=s.cuda_stream if rep % 2 else s)
            p = paged.attend_pages(q, cache, sel["kv_idx"], sel["kv_cnt"], stream=s)
            got.append((i, o, sel, p))
    torch.cuda.synchronize()
    for i, o, sel, p in got:
        _, ref, rsel, refp = cases[i]
        for x, y in zip(o + p, ref + refp):
            assert torch.equal(x, y)
        assert torch.equal(sel["kv_idx"], rsel["kv_idx"]) and torch.equal(sel["kv_cnt"], rsel["kv_cnt"])


def test_offsets_past_32_bits():
    """Pools of more than 2^31 elements, the sequences on the last pages."""
    P, Hkv, page, d, B = 17000, 8, 128, 128, 2
    assert P * Hkv * page * d > 2 ** 31
    cache = paged.PagedCache.create(layers=1, n_pages=P, Hkv=Hkv, page=page, d=d, slots=B, max_pages=5)
    g = torch.Generator().manual_seed(19)
    lens, T = [500, 130], 3
    pages = [[P - 1, P - 3, P - 2, P - 7], [P - 5, P - 4]]
    for s in range(B):
        cache.page_table[s, :len(pages[s])] = _i32(pages[s])
        cache.refs[pages[s]] = 1
    rowsK = torch.randn(B, Hkv, 500, d, generator=g).to(torch.bfloat16)
    rowsV = torch.randn(B, Hkv, 500, d, generator=g).to(torch.bfloat16)
    cache.seq_len.copy_(_i32(lens))
    assert int(paged.append(cache, rowsK.cuda(), rowsV.cuda(), q_len=_i32(lens))) == 0
    for s in range(B):
        for j, pg in enumerate(pages[s]):
            n = min(page, lens[s] - j * page)
            assert torch.equal(cache.k[0, pg, :, :n].cpu(), rowsK[s, :, j * page:j * page + n])
    q = torch.randn(B, 16, T, d, generator=g).to(torch.bfloat16)
    out, _, st = paged.attend_tree(q.cuda(), cache)
    outw, _, stw = paged.attend_tree(q.cuda().repeat(1, 1, 4, 1), cache)     # 24 rows per KV head: tcgen05
    sel = paged.select_pages(q.cuda(), cache, paged.PageSelectConfig(3, 1, 1))
    outp, _, st2 = paged.attend_pages(q.cuda(), cache, sel["kv_idx"], sel["kv_cnt"])
    assert int(st) == 0 and int(stw) == 0 and int(st2) == 0 and int(sel["dev_status"]) == 0
    qn = f8(q)
    for s in range(B):
        for h in range(16):
            K, V = f8(rowsK)[s, h // 2, :lens[s]], f8(rowsV)[s, h // 2, :lens[s]]
            km, vm = np.abs(K).max(), np.abs(V).max()
            see = np.tril(np.ones((lens[s], lens[s]), bool))
            ro, _ = O.softmax_rows(qn[s, h], K, V, see[-T:], scale_of(d))
            check(f8(out)[s, h], ro, out_tolerance(ro, qn[s], km, vm, d, scale_of(d), "bf16", 16), (s, h))
            ro, _ = O.softmax_rows(np.tile(qn[s, h], (4, 1)), K, V, see[-4 * T:], scale_of(d))
            check(f8(outw)[s, h], ro, out_tolerance(ro, qn[s], km, vm, d, scale_of(d), "bf16", 8), (s, h))
            for t in range(T):
                at = [x for p in sel["kv_idx"][s, h // 2, t].tolist() if p >= 0
                      for x in range(p * page, (p + 1) * page) if x <= lens[s] - T + t]
                ro, _ = O.softmax_rows(qn[s, h, t:t + 1], K[at], V[at], np.ones((1, len(at)), bool), scale_of(d))
                check(f8(outp)[s, h, t:t + 1], ro, out_tolerance(ro, qn[s], km, vm, d, scale_of(d), "bf16", 16), (s, h, t))
    assert int(paged.copy_pages(cache, _i32([[P - 1, P - 10]]))) == 0
    assert torch.equal(cache.k[0, P - 1], cache.k[0, P - 10]) and torch.equal(cache.v[0, P - 1], cache.v[0, P - 10])
    assert int(paged.compact(cache, _i32([[0, 2, -1], [1, 2, -1]]), _i32([2, 2]))) == 0
    assert torch.equal(cache.k[0, P - 7, :, 498 - 384].cpu(), rowsK[0, :, 499])
    _, n_free, st = paged.resize(cache, _i32([0, 0]))
    assert int(st) == 0 and int(n_free) == P
    _, n_free, st = paged.resize(cache, _i32([600, 640]))
    assert int(st) == 0 and cache.page_table.cpu().tolist() == [[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]]


def test_results_do_not_depend_on_the_batch():
    """The same sequence alone and among others (another split over the SMs): equal within the
    tolerance of either, and each repeats bit for bit."""
    page, d, T = 32, 128, 20
    lens = [3000, 7000, 50, 64]
    cache = make_cache(27, lens=lens, max_pages=220, page=page, Hkv=2, d=d)
    q = torch.randn(4, 8, T, d, generator=torch.Generator().manual_seed(28)).to(torch.bfloat16).cuda()
    a, la, _ = paged.attend_tree(q, cache)
    b, lb, _ = paged.attend_tree(q, cache)
    assert torch.equal(a, b) and torch.equal(la, lb)
    for s in range(4):
        one, l1, st = paged.attend_tree(q, cache, q_len=_i32([T if i == s else 0 for i in range(4)]))
        assert int(st) == 0
        km = float(cache.k.float().abs().max())
        vm = float(cache.v.float().abs().max())
        tol = out_tolerance(f8(a)[s], f8(q), km, vm, d, scale_of(d), "bf16", 8)
        assert (np.abs(f8(one)[s] - f8(a)[s]) <= 2 * tol).all()
        assert (one[[i for i in range(4) if i != s]] == 0).all()
        assert torch.isneginf(l1[[i for i in range(4) if i != s]]).all()
