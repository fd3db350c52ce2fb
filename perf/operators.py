"""Cases of the paged-cache operators: attention for a tree of drafted tokens, attention over
the pages a cheap score selects for each query, appending / compacting cache rows, and
forking / growing / copying / freeing pages.

``own = False`` computes each case in plain torch operations; ``own = True`` makes the calls of
``block_sparse_causal_bsa_b200.paged``. The cache is a pool of pages [P, Hkv, page, d] per
tensor, with the per-page channel bounds of the keys [P, Hkv, 2, d] (minimum, maximum), a page
table [slots, max_pages] (-1 where there is no page), lengths [slots] and reference counts [P].
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # --- attention for a tree of drafted tokens (one token: plain decode) over the cache
        # one user, a short prompt, eight drafted tokens: the latency of a call
        dict(name="tree_one_user", kind="tree", B=1, Hq=32, Hkv=8, d=128, page=64, T=8, T_lo=8,
             len_lo=1003, len_hi=1003, chain=False, dtype="bf16"),
        # sixteen users decoding one token each over 64k tokens (the decode workload's shape)
        dict(name="tree_decode_64k", kind="tree", B=16, Hq=32, Hkv=8, d=128, page=128, T=1, T_lo=1,
             len_lo=65536, len_hi=65536, chain=True, dtype="bf16"),
        # a ragged batch, drafts of 9 to 33 tokens, small pages, fp16, small heads
        dict(name="tree_ragged", kind="tree", B=24, Hq=16, Hkv=4, d=64, page=16, T=33, T_lo=9,
             len_lo=700, len_hi=18001, chain=False, dtype="fp16"),
        # wide trees over long contexts: 256 query rows per KV head, bound by the products
        dict(name="tree_wide_32k", kind="tree", B=8, Hq=32, Hkv=8, d=128, page=64, T=64, T_lo=64,
             len_lo=32768, len_hi=32768, chain=False, dtype="bf16"),
        # --- selection of pages by their key bounds, then attention over the selected pages
        # one user at 128k tokens, one token: the latency of the two calls
        dict(name="sparse_one_user_128k", kind="sparse", B=1, Hq=32, Hkv=8, d=128, page=64, T=1,
             T_lo=1, len_lo=131072, len_hi=131072, k=64, n_first=1, n_last=2, dtype="bf16"),
        # the decode workload's batch at 64k tokens, a budget of 64 pages of 64 tokens
        dict(name="sparse_decode_64k", kind="sparse", B=16, Hq=32, Hkv=8, d=128, page=64, T=1,
             T_lo=1, len_lo=65536, len_hi=65536, k=64, n_first=1, n_last=2, dtype="bf16"),
        # up to five tokens a user (a drafted chain), ragged lengths, small pages and heads, fp16
        dict(name="sparse_chain_ragged", kind="sparse", B=12, Hq=16, Hkv=4, d=64, page=16, T=5,
             T_lo=2, len_lo=130, len_hi=24007, k=96, n_first=2, n_last=3, dtype="fp16"),
        # --- appending rows to the cache, and compacting the accepted rows of a draft
        # one new token for each of 64 users: every layer of every decode step
        dict(name="append_token", kind="append", B=64, Hq=32, Hkv=8, d=128, page=64, T=1, T_lo=1,
             len_lo=500, len_hi=2000, compact=False, dtype="bf16"),
        # a prompt chunk of up to 1024 tokens for 32 users
        dict(name="append_chunk", kind="append", B=32, Hq=32, Hkv=8, d=128, page=64, T=1024,
             T_lo=513, len_lo=1500, len_hi=4000, compact=False, dtype="bf16"),
        # drafts of up to 33 tokens appended, and the accepted ones moved together
        dict(name="append_accept", kind="append", B=48, Hq=32, Hkv=8, d=128, page=16, T=33, T_lo=9,
             len_lo=100, len_hi=2500, compact=True, dtype="bf16"),
        # --- forking sequences, growing them with copies of the shared last pages, freeing them
        # four samples of each of four prompts
        dict(name="fork_few", kind="fork", parents=4, fan=3, Hq=32, Hkv=8, d=128, page=64,
             len_lo=900, len_hi=2100, grow=1, dtype="bf16"),
        # eight more samples of each of 56 prompts
        dict(name="fork_many", kind="fork", parents=56, fan=8, Hq=32, Hkv=8, d=128, page=128,
             len_lo=1000, len_hi=6000, grow=3, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "sparse", "sparse", "append", "fork"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    c = dict(kind=kind, Hq=Hkv * G, Hkv=Hkv, d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if kind == "fork":
        c.update(parents=rng.randint(1, 48), fan=rng.randint(1, 8), grow=rng.randint(1, 40))
        c["len_lo"] = _log_int(rng, 1, 2000)
        c["len_hi"] = c["len_lo"] + _log_int(rng, 1, 3000)
        return c
    c["B"] = _log_int(rng, 1, 48)
    if kind == "tree":
        c["T"] = rng.choice([1, _log_int(rng, 1, 64)])
        c["chain"] = rng.random() < 0.3
        top = min(65536, 2 ** 21 // (c["B"] * max(1, Hkv // 4)) // max(1, G * c["T"] // 64))
    elif kind == "sparse":
        c["T"] = rng.choice([1, 1, rng.randint(2, 6)])
        c["k"] = _log_int(rng, 4, 128)
        c["n_first"], c["n_last"] = rng.randint(0, 2), rng.randint(1, 2)
        top = min(131072, 2 ** 20 // c["B"])
    else:
        c["T"] = rng.choice([1, _log_int(rng, 2, 500)])
        c["compact"] = c["T"] <= 128 and rng.random() < 0.6
        top = 4000
    c["T_lo"] = rng.randint(1, c["T"])
    c["len_hi"] = max(c["T"], _log_int(rng, 1, max(2, top)))
    c["len_lo"] = rng.randint(max(c["T"], c["len_hi"] // 8), c["len_hi"])
    return c


# --------------------------------------------------------------------------------------------
# sizes that follow from the case alone

def _lens(case):
    """Lengths (after the call's own tokens) and query lengths of the sequences."""
    n = case["parents"] if case["kind"] == "fork" else case["B"]
    out, ql = [], []
    for i in range(n):
        f = (i * 0.6180339887) % 1.0
        out.append(case["len_lo"] + int(round((case["len_hi"] - case["len_lo"]) * f)))
        if case["kind"] != "fork":
            g = (i * 0.7548776662) % 1.0
            ql.append(case["T_lo"] + int(round((case["T"] - case["T_lo"]) * g)))
    if ql:
        ql[0] = case["T"]
    return out, ql


def _n_keep(ql):
    return [max(1, (2 * t + i) // 5) if t > 1 else 1 for i, t in enumerate(ql)]


def _listed_pages(case, length, ql, t):
    return min(case["k"], (length - ql + t) // case["page"] + 1)


def work(case):
    lens, ql = _lens(case)
    d, page, Hkv, G = case["d"], case["page"], case["Hkv"], case["Hq"] // case["Hkv"]
    row = d * 2
    if case["kind"] == "tree":
        rows = sum(ql) * case["Hq"]
        return dict(bytes=2 * Hkv * sum(lens) * row + rows * (2 * row + 4),
                    flops=sum(4 * d * case["Hq"] * q * n for n, q in zip(lens, ql)))
    if case["kind"] == "sparse":
        rows = sum(ql) * case["Hq"]
        pages = sum(-(-n // page) for n in lens)
        b, f = 2 * pages * Hkv * row + rows * (2 * row + 4), 0
        for n, q in zip(lens, ql):
            keys = [min(_listed_pages(case, n, q, t) * page, n - q + t + 1) for t in range(q)]
            # the tokens of one sequence may share pages: the longest list is what must be read
            b += 2 * Hkv * max(keys) * row + q * Hkv * (case["k"] + 1) * 4
            f += 4 * d * case["Hq"] * sum(keys) + 2 * d * case["Hq"] * q * (n // page + 1)
        return dict(bytes=b, flops=f)
    if case["kind"] == "append":
        rows = sum(ql) * Hkv
        touched = sum((n - 1) // page - (n - q) // page + 1 for n, q in zip(lens, ql)) * Hkv
        b = 4 * rows * row + 2 * touched * row
        if case["compact"]:
            nk = sum(_n_keep(ql)) * Hkv
            b += 4 * nk * row + touched * 2 * row
        return dict(bytes=b, flops=2 * rows * d)
    pairs = sum(case["fan"] for n in lens if n % page)
    table = sum(-(-n // page) for n in lens) * (1 + case["fan"])
    return dict(bytes=pairs * 2 * Hkv * (2 * page + 2) * row + 12 * table, flops=0)


# --------------------------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    pr = random.Random(seed * 1000003 + 17)
    dt, d, page, Hkv, Hq = DT[case["dtype"]], case["d"], case["page"], case["Hkv"], case["Hq"]
    lens, ql = _lens(case)
    fork = case["kind"] == "fork"
    if fork:
        # children in the low slots, parents in the high ones
        n_child = case["parents"] * case["fan"]
        slots = n_child + case["parents"]
        lens = [0] * n_child + lens
        parent = [n_child + i % case["parents"] for i in range(n_child)] + [-1] * case["parents"]
        grown = [lens[p] + case["grow"] for p in parent[:n_child]] + [n + case["grow"] for n in lens[n_child:]]
        need = sum(-(-n // page) for n in lens)
        extra = sum(case["grow"] // page + 2 for _ in range(slots))
        P, max_pages = need + extra + 5, -(-max(grown) // page) + 1
    else:
        slots = case["B"]
        need = sum(-(-n // page) for n in lens)
        P, max_pages = need + 3, -(-max(lens) // page) + 1

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=dt)

    k, v = normal(P, Hkv, page, d), normal(P, Hkv, page, d)
    # keys share a direction within a page, as neighbouring tokens do: pages differ in score
    k.add_(normal(P, Hkv, 1, d))
    perm = torch.randperm(P, generator=g, device=dev)
    table = torch.full((slots, max_pages), -1, dtype=torch.int32, device=dev)
    refs = torch.zeros(P, dtype=torch.int32, device=dev)
    bounds = torch.empty(P, Hkv, 2, d, dtype=dt, device=dev)
    bounds[:, :, 0], bounds[:, :, 1] = k.amin(2), k.amax(2)
    at = 0
    for s, n in enumerate(lens):
        m = -(-n // page)
        pages = perm[at:at + m]
        table[s, :m] = pages.int()
        refs[pages] = 1
        if n % page:        # the last page's bounds cover its filled rows alone
            part = k[pages[-1], :, :n % page]
            bounds[pages[-1], :, 0], bounds[pages[-1], :, 1] = part.amin(1), part.amax(1)
        at += m
    i32 = dict(dtype=torch.int32, device=dev)
    st = dict(case=case, lens=lens, ql=ql, k=k, v=v, bounds=bounds, table=table, refs=refs,
              seq_len=torch.tensor(lens, **i32))
    if fork:
        st.update(parent=torch.tensor(parent, **i32), grown=torch.tensor(grown, **i32),
                  back=torch.tensor(lens, **i32), n_child=n_child, parent_h=parent, grown_h=grown)
    else:
        T = case["T"]
        st["q_len"] = torch.tensor(ql, **i32)
        if case["kind"] == "append":
            st["k_new"], st["v_new"] = normal(slots, Hkv, T, d), normal(slots, Hkv, T, d)
            if case["compact"]:
                nk = _n_keep(ql)
                keep = [sorted(pr.sample(range(q), n)) + [-1] * (T - n) for q, n in zip(ql, nk)]
                st.update(nk=nk, keep=torch.tensor(keep, **i32), n_keep=torch.tensor(nk, **i32))
            # the first pass's bounds are those of the passes after it: the rows before the call
            for s, (n, q) in enumerate(zip(lens, ql)):
                base = n - q
                for j in range(base // page, (n - 1) // page + 1):
                    m = max(0, min(base - j * page, page))
                    if m:
                        part = k[table[s, j], :, :m]
                        bounds[table[s, j], :, 0], bounds[table[s, j], :, 1] = part.amin(1), part.amax(1)
        else:
            st["q"] = normal(slots, Hq, T, d)
            st["out"] = torch.zeros(slots, Hq, T, d, dtype=dt, device=dev)
            st["lse"] = torch.zeros(slots, Hq, T, dtype=torch.float32, device=dev)
        if case["kind"] == "tree" and not case["chain"]:
            par = [[-1 if t == 0 else pr.randint(max(0, t - 6), t - 1) for t in range(T)] for _ in range(slots)]
            st["parents"] = torch.tensor(par, **i32)
            words = -(-T // 64)
            bits = [[0] * T for _ in range(slots)]
            for s in range(slots):
                for t in range(T):
                    bits[s][t] = (bits[s][par[s][t]] if par[s][t] >= 0 else 0) | (1 << t)
            signed = lambda x: x - (1 << 64) if x >> 63 else x
            st["mask"] = torch.tensor([[[signed((bits[s][t] >> (64 * w)) & (2 ** 64 - 1)) for w in range(words)]
                                        for t in range(T)] for s in range(slots)], dtype=torch.int64, device=dev)
    if own:
        from block_sparse_causal_bsa_b200 import paged
        st["cache"] = paged.PagedCache(k=k.unsqueeze(0), v=v.unsqueeze(0), bounds=bounds.unsqueeze(0),
                                       page_table=table, seq_len=st["seq_len"], refs=refs)
    return st


# --------------------------------------------------------------------------------------------
# one pass

def run(st):
    kind = st["case"]["kind"]
    if own:
        return _OWN[kind](st)
    return _PLAIN[kind](st)


def _own_tree(st):
    from block_sparse_causal_bsa_b200 import paged
    out, lse, _ = paged.attend_tree(st["q"], st["cache"], mask=st.get("mask"), q_len=st["q_len"],
                                    out=st["out"], lse=st["lse"])
    return out, lse


def _own_sparse(st):
    from block_sparse_causal_bsa_b200 import paged
    c = st["case"]
    sel = paged.select_pages(st["q"], st["cache"], paged.PageSelectConfig(c["k"], c["n_first"], c["n_last"]),
                             q_len=st["q_len"])
    out, lse, _ = paged.attend_pages(st["q"], st["cache"], sel["kv_idx"], sel["kv_cnt"], q_len=st["q_len"],
                                     out=st["out"], lse=st["lse"])
    return sel["kv_idx"], sel["kv_cnt"], out, lse


def _own_append(st):
    from block_sparse_causal_bsa_b200 import paged
    paged.append(st["cache"], st["k_new"], st["v_new"], q_len=st["q_len"])
    if st["case"]["compact"]:
        paged.compact(st["cache"], st["keep"], st["n_keep"], q_len=st["q_len"])
    return st["k"], st["v"], st["bounds"]


def _own_fork(st):
    from block_sparse_causal_bsa_b200 import paged
    c = st["cache"]
    paged.fork(c, st["parent"])
    pairs, _, _ = paged.resize(c, st["grown"])
    paged.copy_pages(c, pairs)
    step_table = c.page_table.clone()       # what a sampler keeps of the step
    paged.resize(c, st["back"])
    return pairs, step_table, c.page_table, c.seq_len, c.refs, st["k"], st["v"], st["bounds"]


_OWN = dict(tree=_own_tree, sparse=_own_sparse, append=_own_append, fork=_own_fork)


def _softmax_av(s, keep, v):
    """s [..., rows, keys] fp32 logits, keep the visible pairs, v [..., keys, d] fp32: the
    attention output and the natural log of the softmax denominator (0 and -inf for a row that
    sees no key)."""
    s = torch.where(keep, s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, 1.0, l)
    return o, (m + torch.log(l)).squeeze(-1)


def _tree_keep(mask_b, q, dev):
    """[q, q] visibility of the drafted tokens from the mask words of one sequence."""
    j = torch.arange(q, device=dev)
    if mask_b is None:
        return j[None, :] <= j[:, None]
    return ((mask_b[:q][:, j // 64] >> (j % 64)) & 1).bool()


def _plain_tree(st):
    c, k, v = st["case"], st["k"], st["v"]
    d, page, Hkv, G = c["d"], c["page"], c["Hkv"], c["Hq"] // c["Hkv"]
    out = torch.zeros_like(st["q"])
    lse = torch.zeros_like(st["lse"])
    for b, (n, q) in enumerate(zip(st["lens"], st["ql"])):
        pages = st["table"][b, :-(-n // page)].long()
        kb = k[pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].float()
        vb = v[pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].float()
        qb = st["q"][b, :, :q].float().reshape(Hkv, G * q, d)
        s = torch.matmul(qb, kb.transpose(1, 2)) / math.sqrt(d)
        keep = torch.ones(q, n, dtype=torch.bool, device=k.device)
        keep[:, n - q:] = _tree_keep(st["mask"][b] if "mask" in st else None, q, k.device)
        o, ls = _softmax_av(s, keep.repeat(G, 1), vb)
        out[b, :, :q] = o.reshape(Hkv * G, q, d).to(out.dtype)
        lse[b, :, :q] = ls.reshape(Hkv * G, q)
    return out, lse


def _plain_sparse(st):
    c, k, v, dev = st["case"], st["k"], st["v"], st["k"].device
    d, page, Hkv, G, T, K = c["d"], c["page"], c["Hkv"], c["Hq"] // c["Hkv"], c["T"], c["k"]
    out = torch.zeros_like(st["q"])
    lse = torch.zeros_like(st["lse"])
    idx = torch.full((c["B"], Hkv, T, K), -1, dtype=torch.int32, device=dev)
    cnt = torch.zeros(c["B"], Hkv, T, dtype=torch.int32, device=dev)
    for b, (n, q) in enumerate(zip(st["lens"], st["ql"])):
        npg = -(-n // page)
        pages = st["table"][b, :npg].long()
        bd = st["bounds"][pages].double()                                   # [npg, Hkv, 2, d]
        qb = st["q"][b, :, :q].double().reshape(Hkv, G * q, d)
        sc = torch.matmul(qb.clamp(min=0), bd[:, :, 1].permute(1, 2, 0)) + \
            torch.matmul(qb.clamp(max=0), bd[:, :, 0].permute(1, 2, 0))
        sc = sc.reshape(Hkv, G, q, npg).amax(1).float()
        j = torch.arange(npg, device=dev)
        last = (n - q + torch.arange(q, device=dev)) // page               # each token's own page
        forced = (j[None] < c["n_first"]) | (j[None] > last[:, None] - c["n_last"])
        sc = torch.where(forced, float("inf"), sc)
        sc = torch.where(j[None] > last[:, None], float("-inf"), sc)
        order = torch.sort(sc, dim=-1, descending=True, stable=True).indices
        kk = min(K, npg)
        ct = torch.clamp(last + 1, max=K)                                   # [q]
        sel = torch.where(torch.arange(kk, device=dev)[None] < ct[:, None], order[..., :kk], npg)
        sel = torch.sort(sel, dim=-1).values                                # [Hkv, q, kk]
        idx[b, :, :q, :kk] = torch.where(sel < npg, sel, -1).int()
        cnt[b, :, :q] = ct.int()
        pg = pages[sel.clamp(max=npg - 1)]
        h = torch.arange(Hkv, device=dev)[:, None, None]
        ks = k[pg, h].reshape(Hkv, q, kk * page, d).float()
        vs = v[pg, h].reshape(Hkv, q, kk * page, d).float()
        pos = (sel[..., None] * page + torch.arange(page, device=dev)).reshape(Hkv, q, 1, kk * page)
        keep = pos <= (n - q + torch.arange(q, device=dev))[:, None, None]
        qs = st["q"][b, :, :q].float().reshape(Hkv, G, q, d).transpose(1, 2)
        o, ls = _softmax_av(torch.matmul(qs, ks.transpose(2, 3)) / math.sqrt(d), keep, vs)
        out[b, :, :q] = o.transpose(1, 2).reshape(Hkv * G, q, d).to(out.dtype)
        lse[b, :, :q] = ls.transpose(1, 2).reshape(Hkv * G, q)
    return idx, cnt, out, lse


def _plain_append(st):
    c, k, v, bounds, dev = st["case"], st["k"], st["v"], st["bounds"], st["k"].device
    page = c["page"]
    for b, (n, q) in enumerate(zip(st["lens"], st["ql"])):
        base = n - q
        pos = base + torch.arange(q, device=dev)
        pg, off = st["table"][b].long()[pos // page], pos % page
        k[pg, :, off] = st["k_new"][b, :, :q].transpose(0, 1)
        v[pg, :, off] = st["v_new"][b, :, :q].transpose(0, 1)
        if c["compact"]:
            m = st["nk"][b]
            src, dst = base + st["keep"][b, :m].long(), base + torch.arange(m, device=dev)
            tb = st["table"][b].long()
            kr, vr = k[tb[src // page], :, src % page], v[tb[src // page], :, src % page]
            k[tb[dst // page], :, dst % page] = kr
            v[tb[dst // page], :, dst % page] = vr
        end = base + (st["nk"][b] if c["compact"] else q)
        for j in range(base // page, (end - 1) // page + 1):
            rows = k[st["table"][b, j].long(), :, :min(end - j * page, page)].float()
            bounds[st["table"][b, j].long()] = torch.stack((rows.amin(1), rows.amax(1)), 1).to(k.dtype)
        for j in range((end - 1) // page + 1, (n - 1) // page + 1):
            # pages of rejected drafts alone keep the bounds of the rows appended to them
            rows = st["k_new"][b, :, max(0, j * page - base):min(q, (j + 1) * page - base)]
            new = torch.stack((rows.amin(1), rows.amax(1)), 1)
            bounds[st["table"][b, j].long()] = new
    return k, v, bounds


def _plain_resize(st, new_len):
    """Grow or shrink every slot to new_len: pages past the new length lose a reference; then,
    in slot order, the lowest free pages are taken, first for a copy of a partly filled last
    page that others still hold (the last slot that grows it keeps it when all holders grow),
    then for the new pages."""
    page, table, seq, refs, dev = st["case"]["page"], st["table"], st["seq_len"], st["refs"], st["k"].device
    S, MP = table.shape
    P = refs.numel()
    j = torch.arange(MP, device=dev)[None]
    have, want = (seq + page - 1) // page, (new_len + page - 1) // page
    drop = (j >= want[:, None]) & (j < have[:, None])
    idx = torch.where(drop, table, P).long().reshape(-1)
    less = torch.zeros(P + 1, dtype=torch.int32, device=dev).scatter_add_(0, idx, torch.ones_like(idx, dtype=torch.int32))
    refs -= less[:P]
    table[drop] = -1
    # shared last pages of the growing slots
    grows = new_len > seq
    tail = torch.where(seq % page != 0, table.gather(1, (seq // page).clamp(max=MP - 1).long()[:, None])[:, 0], -1)
    cand = grows & (tail >= 0) & (refs[tail.clamp(min=0).long()] > 1)
    same = (tail[:, None] == tail[None]) & cand[:, None] & cand[None]
    holders = same.sum(1)
    after = (same & (torch.arange(S, device=dev)[None] > torch.arange(S, device=dev)[:, None])).any(1)
    cow = cand & ~((holders == refs[tail.clamp(min=0).long()]) & ~after)
    need = torch.where(grows, want - have, 0) + cow
    first = torch.cumsum(need, 0) - need
    free = refs == 0
    rank = torch.where(free, torch.cumsum(free, 0) - 1, P).long()
    pool = torch.full((P + 1,), -1, dtype=torch.int32, device=dev).scatter_(
        0, rank, torch.arange(P, device=dev, dtype=torch.int32))
    new_tail = pool[first.clamp(max=P).long()]
    pairs = torch.stack((torch.where(cow, tail, -1), torch.where(cow, new_tail, -1)), 1).int()
    fresh = (j >= have[:, None]) & (j < want[:, None]) & grows[:, None]
    at = (first + cow)[:, None] + j - have[:, None]
    table.copy_(torch.where(fresh, pool[at.clamp(0, P).long()], table))
    table.copy_(torch.where(cow[:, None] & (j == (seq // page)[:, None]), new_tail[:, None], table))
    taken = torch.zeros(P + 1, dtype=torch.int32, device=dev)
    taken.scatter_add_(0, torch.where(fresh, table, P).long().reshape(-1),
                       torch.ones(S * MP, dtype=torch.int32, device=dev))
    taken.scatter_add_(0, torch.where(cow, new_tail, P).long(), torch.ones(S, dtype=torch.int32, device=dev))
    left = torch.zeros(P + 1, dtype=torch.int32, device=dev).scatter_add_(
        0, torch.where(cow, tail, P).long(), torch.ones(S, dtype=torch.int32, device=dev))
    refs += taken[:P] - left[:P]
    seq.copy_(new_len)
    return pairs


def _plain_fork(st):
    table, seq, refs, k = st["table"], st["seq_len"], st["refs"], st["k"]
    P, page, dev = refs.numel(), st["case"]["page"], k.device
    par = st["parent"]
    is_child = par >= 0
    src = par.clamp(min=0).long()
    j = torch.arange(table.shape[1], device=dev)[None]
    rows = torch.where(is_child[:, None] & (j < ((seq[src] + page - 1) // page)[:, None]), table[src], -1)
    table.copy_(torch.where(is_child[:, None], rows, table))
    more = torch.zeros(P + 1, dtype=torch.int32, device=dev)
    more.scatter_add_(0, torch.where(rows >= 0, rows, P).long().reshape(-1),
                      torch.ones(rows.numel(), dtype=torch.int32, device=dev))
    refs += more[:P]
    seq.copy_(torch.where(is_child, seq[src], seq))
    pairs = _plain_resize(st, st["grown"])
    # pairs of (-1, -1) copy a spare page (the last one) onto itself
    frm = torch.where(pairs[:, 0] >= 0, pairs[:, 0], P - 1).long()
    to = torch.where(pairs[:, 1] >= 0, pairs[:, 1], P - 1).long()
    for t in (st["k"], st["v"], st["bounds"]):
        t[to] = t[frm]
    step_table = table.clone()
    _plain_resize(st, st["back"])
    return pairs, step_table, table, seq, refs, st["k"], st["v"], st["bounds"]


_PLAIN = dict(tree=_plain_tree, sparse=_plain_sparse, append=_plain_append, fork=_plain_fork)


# --------------------------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    """Attention and selection from their definition in 64 bits, one (sequence, KV head) at a
    time. Cases that only move data have no computed numbers."""
    if case["kind"] not in ("tree", "sparse"):
        return None
    st = prepare(case, seed)
    d, page, Hkv, G, T = case["d"], case["page"], case["Hkv"], case["Hq"] // case["Hkv"], case["T"]
    dev = st["k"].device
    f8 = torch.float64
    out = torch.zeros(st["q"].shape, dtype=f8, device=dev)
    lse = torch.zeros(st["lse"].shape, dtype=f8, device=dev)
    sparse = case["kind"] == "sparse"
    if sparse:
        idx = torch.full((case["B"], Hkv, T, case["k"]), -1, dtype=torch.int32)
        cnt = torch.zeros(case["B"], Hkv, T, dtype=torch.int32)
    for b, (n, q) in enumerate(zip(st["lens"], st["ql"])):
        npg = -(-n // page)
        pages = st["table"][b, :npg].long()
        for h in range(Hkv):
            kb = st["k"][pages, h].reshape(-1, d)[:n].to(f8)
            vb = st["v"][pages, h].reshape(-1, d)[:n].to(f8)
            qh = st["q"][b, h * G:(h + 1) * G, :q].to(f8)                    # [G, q, d]
            see = torch.zeros(q, n, dtype=torch.bool, device=dev)
            if sparse:
                lo, hi = st["bounds"][pages, h, 0].to(f8), st["bounds"][pages, h, 1].to(f8)
                for t in range(q):
                    own_page = (n - q + t) // page
                    sc = torch.stack([torch.maximum(qh[g, t] * lo, qh[g, t] * hi).sum(1) for g in range(G)]
                                     ).amax(0).float().tolist()
                    must = [x for x in range(own_page + 1) if x < case["n_first"] or x > own_page - case["n_last"]]
                    rest = sorted((x for x in range(own_page + 1) if x not in set(must)), key=lambda x: (-sc[x], x))
                    # forced pages fill the budget first (the earliest of them if there are too many)
                    chosen = sorted((must + rest)[:case["k"]])
                    idx[b, h, t, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
                    cnt[b, h, t] = len(chosen)
                    lists = torch.tensor(chosen, device=dev)
                    pos = (lists[:, None] * page + torch.arange(page, device=dev)).reshape(-1)
                    see[t, pos[pos <= n - q + t]] = True
            else:
                see[:, :n - q] = True
                for t in range(q):
                    if case["chain"]:
                        see[t, n - q:n - q + t + 1] = True
                        continue
                anc = None if case["chain"] else st["parents"][b].tolist()
                if anc is not None:
                    rows, cols = [], []
                    for t in range(q):
                        x = t
                        while x >= 0:
                            rows.append(t)
                            cols.append(n - q + x)
                            x = anc[x]
                    see[torch.tensor(rows, device=dev), torch.tensor(cols, device=dev)] = True
            if sparse:
                for t in range(q):
                    at = see[t].nonzero()[:, 0]
                    z = qh[:, t] @ kb[at].T / math.sqrt(d)
                    out[b, h * G:(h + 1) * G, t] = torch.softmax(z, -1) @ vb[at]
                    lse[b, h * G:(h + 1) * G, t] = torch.logsumexp(z, -1)
                continue
            for g in range(G):
                z = (qh[g] @ kb.T / math.sqrt(d)).masked_fill(~see, float("-inf"))
                out[b, h * G + g, :q] = torch.softmax(z, -1) @ vb
                lse[b, h * G + g, :q] = torch.logsumexp(z, -1)
    if sparse:
        return idx.to(dev), cnt.to(dev), out, lse
    return out, lse
