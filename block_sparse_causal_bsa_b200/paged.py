"""Serving from a paged cache: pages of many sequences in one pool, several query tokens a step.

A step, for the sequences ("slots") of a :class:`PagedCache`::

    pairs, n_free, st = paged.resize(cache, new_len)      # pages for the step's tokens
    for layer in ...:
        paged.copy_pages(cache, pairs, layer=layer)       # only after a fork: shared last pages
        paged.append(cache, k_new, v_new, q_len=q_len, layer=layer)
        out, lse, st = paged.attend_tree(q, cache, mask=mask, q_len=q_len, layer=layer)
        # or: sel = paged.select_pages(q, cache, cfg, q_len=q_len, layer=layer)
        #     out, lse, st = paged.attend_pages(q, cache, sel["kv_idx"], sel["kv_cnt"], ...)
    # after the drafts are verified, per layer (a chain of which the first ones are accepted needs none):
        paged.compact(cache, keep, n_keep, q_len=q_len, layer=layer)
    paged.resize(cache, cache.seq_len - q_len + n_keep)   # the rejected drafts' pages

The calls run on the current stream of the cache's device (or on ``stream``) and return at once.
Arguments that the host can check raise :class:`BsaError`; what only the device sees is in the
status tensors returned. ``include/bsa.h`` ("paged cache") says what each call does. Output rows of
tokens that a call leaves out (past q_len, or of a slot whose lengths do not fit) are not written: in tensors
made here they are 0 (lse: -inf) when q_len is given, and undefined when it is not.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
from typing import NamedTuple, Optional

import torch

from .binding import (BSA_BF16, BSA_ERR_INVALID_ARG, BSA_ERR_UNSUPPORTED, BSA_F16, BsaError, CacheShape,
                      PageSelectParams, _check, lib)

_DTYPES = {torch.bfloat16: BSA_BF16, torch.float16: BSA_F16}


def _bad(msg: str, status: int = BSA_ERR_INVALID_ARG):
    raise BsaError(status, msg)


class _Plan(NamedTuple):
    """What a cache's tensors say, read once (a step makes several calls per layer)."""
    shape: object
    layers: int
    Hkv: int
    page: int
    d: int
    dtype: torch.dtype
    device: torch.device
    index: Optional[int]
    slots: int
    max_pages: int
    row_bytes: int                   # of one row per page of a layer


@dataclasses.dataclass
class PagedCache:
    """The pools of all layers, and the bookkeeping they share (device tensors, contiguous).

    k, v [layers, n_pages, Hkv, page, d] (bf16 or fp16); bounds [layers, n_pages, Hkv, 2, d] of the
    same type or None; page_table [slots, max_pages], seq_len [slots], refs [n_pages] int32."""
    k: torch.Tensor
    v: torch.Tensor
    bounds: Optional[torch.Tensor]
    page_table: torch.Tensor
    seq_len: torch.Tensor
    refs: torch.Tensor

    @classmethod
    def create(cls, *, layers: int, n_pages: int, Hkv: int, page: int, d: int, slots: int, max_pages: int,
               dtype: torch.dtype = torch.bfloat16, device="cuda", bounds: bool = True) -> "PagedCache":
        """An empty cache."""
        i32 = dict(dtype=torch.int32, device=device)
        shape = (layers, n_pages, Hkv, page, d)
        return cls(k=torch.zeros(shape, dtype=dtype, device=device),
                   v=torch.zeros(shape, dtype=dtype, device=device),
                   bounds=(torch.zeros(layers, n_pages, Hkv, 2, d, dtype=dtype, device=device) if bounds
                           else None),
                   page_table=torch.full((slots, max_pages), -1, **i32),
                   seq_len=torch.zeros(slots, **i32), refs=torch.zeros(n_pages, **i32))

    def __post_init__(self):
        self.shape()

    def _check(self):
        if self.k.dim() != 5 or self.k.shape != self.v.shape:
            _bad("k and v must be [layers, n_pages, Hkv, page, d]")
        L, P, H, page, d = self.k.shape
        if self.k.dtype not in _DTYPES:
            _bad("the paged cache takes bf16 and fp16", BSA_ERR_UNSUPPORTED)
        _tensor("v", self.v, self.k.shape, self.k.dtype, self.device)
        _tensor("k", self.k, self.k.shape, self.k.dtype, self.device)
        if self.bounds is not None:
            _tensor("bounds", self.bounds, (L, P, H, 2, d), self.k.dtype, self.device)
        if self.page_table.dim() != 2:
            _bad("page_table must be [slots, max_pages]")
        _tensor("page_table", self.page_table, self.page_table.shape, torch.int32, self.device)
        _tensor("seq_len", self.seq_len, (self.slots,), torch.int32, self.device)
        _tensor("refs", self.refs, (P,), torch.int32, self.device)

    @property
    def device(self):
        return self.k.device

    @property
    def slots(self) -> int:
        return self.page_table.shape[0]

    @property
    def max_pages(self) -> int:
        return self.page_table.shape[1]

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if not name.startswith("_"):             # what is derived from the tensors is derived anew
            object.__setattr__(self, "_plan", None)
            object.__setattr__(self, "_bytes", {})

    def __getstate__(self):                      # copies and pickles hold the tensors alone
        return {f.name: getattr(self, f.name) for f in dataclasses.fields(self)}

    def __setstate__(self, state):
        for name, value in state.items():
            setattr(self, name, value)

    def shape(self):
        """The C shape (by reference), kept until a tensor of the cache is replaced."""
        return (self._plan or self._make_plan()).shape

    def _make_plan(self):
        self._check()
        L, P, H, page, d = self.k.shape
        dev = self.k.device
        self._plan = _Plan(ctypes.byref(CacheShape(P, H, page, d, _DTYPES[self.k.dtype])), L, H, page, d,
                           self.k.dtype, dev, dev.index if dev.type == "cuda" else None,
                           self.page_table.shape[0], self.page_table.shape[1], P * H * d * 2)
        return self._plan

    def workspace_bytes(self, call: str, Hq: int, T: int) -> int:
        n = self._bytes.get((call, Hq, T))
        if n is None:
            n = getattr(lib(), f"bsa_{call}_workspace_bytes")(self.shape(), self.slots, self.max_pages, Hq, T)
            if n == 0:
                _bad(lib().bsa_last_error().decode(), BSA_ERR_UNSUPPORTED)
            self._bytes[(call, Hq, T)] = n
        return n

    def _layer(self, p, layer: int):
        if not 0 <= layer < p.layers:
            _bad(f"layer {layer} of {p.layers}")
        step = layer * p.row_bytes
        return (self.k.data_ptr() + step * p.page, self.v.data_ptr() + step * p.page,
                self.bounds.data_ptr() + 2 * step if self.bounds is not None else None)


@dataclasses.dataclass
class PageSelectConfig:
    """Pages per token (k), of which the first n_first and the last n_last are always kept."""
    k: int
    n_first: int = 1
    n_last: int = 1


def _tensor(name: str, t, shape, dtype, device):
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        _bad(f"{name} must be a tensor")
    if t.device != device:
        _bad(f"{name} is on {t.device}, the cache on {device}")
    if t.dtype != dtype:
        _bad(f"{name} must be {dtype}, is {t.dtype}")
    if t.shape != shape:
        _bad(f"{name} must be {list(shape)}, is {list(t.shape)}")
    _bad(f"{name} must be contiguous")


def _stream(p, stream):
    """The handle of the current stream, when the call is to run there; None: it needs _elsewhere."""
    if p.index is None:
        _bad(f"the cache is on {p.device}; the kernels need a GPU")
    if stream is None and torch._C._cuda_getDevice() == p.index:
        return torch._C._cuda_getCurrentRawStream(p.index)
    return None


def _elsewhere(p, stream, call, *args, **kw):
    """call(*args, **kw) with the cache's device and `stream` current, so that outputs and
    workspaces are allocated for the stream that uses them."""
    with contextlib.ExitStack() as st:
        st.enter_context(torch.cuda.device(p.device))
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=p.device)
            if stream.device != p.device:
                _bad(f"the stream is on {stream.device}, the cache on {p.device}")
            st.enter_context(torch.cuda.stream(stream))
        return call(*args, **kw)


def _qlen(cache, p, q_len):
    return None if q_len is None else _tensor("q_len", q_len, (p.slots,), torch.int32, p.device)


def fork(cache: PagedCache, parent: torch.Tensor, *, stream=None) -> torch.Tensor:
    """Slots c with parent[c] >= 0 (int32 [slots]) become copies of their parents, sharing their
    pages. Returns the status."""
    p = cache._plan or cache._make_plan()
    pp = _tensor("parent", parent, (p.slots,), torch.int32, p.device)
    s = _stream(p, stream)
    if s is None:
        return _elsewhere(p, stream, fork, cache, parent)
    refs = cache.refs
    st = refs.new_empty(1)
    _check(lib().bsa_pages_fork(p.slots, p.max_pages, refs.shape[0], p.page, cache.page_table.data_ptr(),
                                cache.seq_len.data_ptr(), refs.data_ptr(), pp, st.data_ptr(), s))
    return st


def resize(cache: PagedCache, new_len: torch.Tensor, *, stream=None):
    """Sets the slots' lengths (int32 [slots]; negative: as it is, 0: freed), taking and giving up
    pages. Returns (pairs [slots, 2] for copy_pages, free pages left, status)."""
    p = cache._plan or cache._make_plan()
    n = _tensor("new_len", new_len, (p.slots,), torch.int32, p.device)
    s = _stream(p, stream)
    if s is None:
        return _elsewhere(p, stream, resize, cache, new_len)
    refs = cache.refs
    st, n_free, pairs = refs.new_empty(1), refs.new_empty(1), refs.new_empty(p.slots, 2)
    _check(lib().bsa_pages_resize(p.slots, p.max_pages, refs.shape[0], p.page, cache.page_table.data_ptr(),
                                  cache.seq_len.data_ptr(), refs.data_ptr(), n, pairs.data_ptr(),
                                  n_free.data_ptr(), st.data_ptr(), s))
    return pairs, n_free, st


def copy_pages(cache: PagedCache, pairs: torch.Tensor, *, layer: int = 0, stream=None) -> torch.Tensor:
    """Copies one layer's pages pairs[i, 0] to pairs[i, 1] (int32 [n, 2]; (-1, -1) is skipped).
    Returns the status."""
    p = cache._plan or cache._make_plan()
    if not isinstance(pairs, torch.Tensor) or pairs.dim() != 2:
        _bad("pairs must be [n, 2]")
    pp = _tensor("pairs", pairs, (pairs.shape[0], 2), torch.int32, p.device)
    k, v, b = cache._layer(p, layer)
    s = _stream(p, stream)
    if s is None:
        return _elsewhere(p, stream, copy_pages, cache, pairs, layer=layer)
    st = cache.refs.new_empty(1)
    if pairs.shape[0] == 0:
        return st.zero_()
    _check(lib().bsa_pages_copy(p.shape, k, v, b, pp, pairs.shape[0], st.data_ptr(), s))
    return st


def append(cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, *, q_len=None, layer: int = 0,
           stream=None) -> torch.Tensor:
    """Writes k_new, v_new [slots, Hkv, T, d] to the last q_len positions of the slots (resize
    comes first) and sets their pages' bounds. Returns the status."""
    p = cache._plan or cache._make_plan()
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 4:
        _bad("k_new must be [slots, Hkv, T, d]")
    T = k_new.shape[2]
    shape = (p.slots, p.Hkv, T, p.d)
    kn = _tensor("k_new", k_new, shape, p.dtype, p.device)
    vn = _tensor("v_new", v_new, shape, p.dtype, p.device)
    ql = _qlen(cache, p, q_len)
    k, v, b = cache._layer(p, layer)
    s = _stream(p, stream)
    if s is None:
        return _elsewhere(p, stream, append, cache, k_new, v_new, q_len=q_len, layer=layer)
    st = cache.refs.new_empty(1)
    _check(lib().bsa_cache_append(p.shape, p.slots, p.max_pages, T, kn, vn, k, v, b, cache.page_table.data_ptr(),
                                  cache.seq_len.data_ptr(), ql, st.data_ptr(), s))
    return st


def compact(cache: PagedCache, keep: torch.Tensor, n_keep: torch.Tensor, *, q_len=None, layer: int = 0,
            stream=None) -> torch.Tensor:
    """Moves the rows keep[s, :n_keep[s]] (ascending, int32 [slots, T]) of the last q_len positions
    of each slot together. Resize to seq_len - q_len + n_keep afterwards. Returns the status."""
    p = cache._plan or cache._make_plan()
    if not isinstance(keep, torch.Tensor) or keep.dim() != 2:
        _bad("keep must be [slots, T]")
    T = keep.shape[1]
    kp = _tensor("keep", keep, (p.slots, T), torch.int32, p.device)
    nk = _tensor("n_keep", n_keep, (p.slots,), torch.int32, p.device)
    ql = _qlen(cache, p, q_len)
    k, v, b = cache._layer(p, layer)
    s = _stream(p, stream)
    if s is None:
        return _elsewhere(p, stream, compact, cache, keep, n_keep, q_len=q_len, layer=layer)
    st = cache.refs.new_empty(1)
    _check(lib().bsa_cache_compact(p.shape, p.slots, p.max_pages, T, kp, nk, k, v, b, cache.page_table.data_ptr(),
                                   cache.seq_len.data_ptr(), ql, st.data_ptr(), s))
    return st


def tree_mask(parents: torch.Tensor, *, q_len=None, stream=None):
    """Ancestor masks of drafted trees: parents int32 [B, T], -1 for a root. Returns (mask int64
    [B, T, ceil(T/64)], status)."""
    if not isinstance(parents, torch.Tensor) or parents.dim() != 2:
        _bad("parents must be [B, T]")
    B, T = parents.shape
    dev = parents.device
    pp = _tensor("parents", parents, (B, T), torch.int32, dev)
    ql = None if q_len is None else _tensor("q_len", q_len, (B,), torch.int32, dev)
    where = _Where(dev, dev.index if dev.type == "cuda" else None)
    s = _stream(where, stream)
    if s is None:
        return _elsewhere(where, stream, tree_mask, parents, q_len=q_len)
    st = parents.new_empty(1)
    mask = parents.new_empty(B, T, (T + 63) // 64, dtype=torch.int64)
    _check(lib().bsa_tree_mask(B, T, pp, ql, mask.data_ptr(), st.data_ptr(), s))
    return mask, st


class _Where(NamedTuple):
    device: torch.device
    index: Optional[int]


def _query(q, p):
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        _bad("q must be [slots, Hq, T, d]")
    _, Hq, T, _ = q.shape
    return Hq, T, _tensor("q", q, (p.slots, Hq, T, p.d), p.dtype, p.device)


def _attend(call, q, query, cache, p, extra, q_len, layer, scale, out, lse, s):
    Hq, T, qp = query
    ql = _qlen(cache, p, q_len)
    k, v, _ = cache._layer(p, layer)
    if scale is None:
        scale = p.d ** -0.5
    nb = cache.workspace_bytes("attend_paged", Hq, T)
    # rows past q_len are not written: 0 and -inf in tensors made here
    if out is None:
        out = torch.empty_like(q) if q_len is None else torch.zeros_like(q)
        op = out.data_ptr()
    else:
        op = _tensor("out", out, q.shape, q.dtype, p.device)
    if lse is None:
        lse = q.new_empty(q.shape[:3], dtype=torch.float32)
        if q_len is not None:
            lse.fill_(float("-inf"))
        lp = lse.data_ptr()
    else:
        lp = _tensor("lse", lse, q.shape[:3], torch.float32, p.device)
    refs = cache.refs
    st, ws = refs.new_empty(1), refs.new_empty((nb + 3) // 4)
    _check(call(p.shape, p.slots, p.max_pages, Hq, T, qp, k, v, cache.page_table.data_ptr(),
                cache.seq_len.data_ptr(), ql, *extra, scale, op, lp, st.data_ptr(), ws.data_ptr(), nb, s))
    return out, lse, st


def attend_tree(q: torch.Tensor, cache: PagedCache, *, mask=None, q_len=None, layer: int = 0,
                scale: Optional[float] = None, out=None, lse=None, stream=None):
    """Attention of the last q_len positions (q [slots, Hq, T, d]) over the whole cache of their
    slots; mask int64 [slots, T, ceil(T/64)] says which drafted tokens see each other (None: a
    chain). Returns (out, lse, status)."""
    p = cache._plan or cache._make_plan()
    query = _query(q, p)
    m = None
    if mask is not None:
        T = query[1]
        m = _tensor("mask", mask, (p.slots, T, (T + 63) // 64), torch.int64, p.device)
    s = _stream(p, stream)
    if s is None:
        return _elsewhere(p, stream, attend_tree, q, cache, mask=mask, q_len=q_len, layer=layer, scale=scale,
                          out=out, lse=lse)
    return _attend(lib().bsa_attend_tree, q, query, cache, p, (m,), q_len, layer, scale, out, lse, s)


def attend_pages(q: torch.Tensor, cache: PagedCache, kv_idx: torch.Tensor, kv_cnt: torch.Tensor, *,
                 q_len=None, layer: int = 0, scale: Optional[float] = None, out=None, lse=None, stream=None):
    """Attention of each token over its listed pages (kv_idx [slots, Hkv, T, W], kv_cnt [slots, Hkv,
    T], int32). Returns (out, lse, status)."""
    p = cache._plan or cache._make_plan()
    query = _query(q, p)
    T = query[1]
    if not isinstance(kv_idx, torch.Tensor) or kv_idx.dim() != 4:
        _bad("kv_idx must be [slots, Hkv, T, W]")
    W = kv_idx.shape[3]
    i = _tensor("kv_idx", kv_idx, (p.slots, p.Hkv, T, W), torch.int32, p.device)
    c = _tensor("kv_cnt", kv_cnt, (p.slots, p.Hkv, T), torch.int32, p.device)
    s = _stream(p, stream)
    if s is None:
        return _elsewhere(p, stream, attend_pages, q, cache, kv_idx, kv_cnt, q_len=q_len, layer=layer,
                          scale=scale, out=out, lse=lse)
    return _attend(lib().bsa_attend_pages, q, query, cache, p, (i, c, W), q_len, layer, scale, out, lse, s)


def select_pages(q: torch.Tensor, cache: PagedCache, cfg: PageSelectConfig, *, q_len=None, layer: int = 0,
                 want_scores: bool = False, stream=None):
    """Pages for each token by the K-min/K-max bound of their keys. Returns a dict: kv_idx [slots,
    Hkv, T, k], kv_cnt [slots, Hkv, T], scores [slots, Hkv, T, max_pages] (None unless
    want_scores), dev_status."""
    p = cache._plan or cache._make_plan()
    Hq, T, qp = _query(q, p)
    ql = _qlen(cache, p, q_len)
    b = cache._layer(p, layer)[2]
    if b is None:
        _bad("the cache has no bounds")
    if cfg.k < 1:
        _bad("k must be >= 1")
    s = _stream(p, stream)
    if s is None:
        return _elsewhere(p, stream, select_pages, q, cache, cfg, q_len=q_len, layer=layer, want_scores=want_scores)
    nb = cache.workspace_bytes("select_pages", Hq, T)
    refs = cache.refs
    idx, cnt, st = refs.new_empty(p.slots, p.Hkv, T, cfg.k), refs.new_empty(p.slots, p.Hkv, T), refs.new_empty(1)
    scores = ws = None
    if want_scores:
        scores = refs.new_empty((p.slots, p.Hkv, T, p.max_pages), dtype=torch.float32)
    else:
        ws = refs.new_empty((nb + 3) // 4)
    _check(lib().bsa_select_pages(p.shape, ctypes.byref(PageSelectParams(cfg.k, cfg.n_first, cfg.n_last)), p.slots,
                                  p.max_pages, Hq, T, qp, b, cache.page_table.data_ptr(),
                                  cache.seq_len.data_ptr(), ql, idx.data_ptr(), cnt.data_ptr(),
                                  scores.data_ptr() if want_scores else None, st.data_ptr(),
                                  None if want_scores else ws.data_ptr(), nb, s))
    return dict(kv_idx=idx, kv_cnt=cnt, scores=scores, dev_status=st)
