"""Serving operators over torch CUDA tensors (C ABI in include/mk_serve.h):
pages of a K/V cache, decode attention over a shared prefix, token
probabilities and the verification of drafted tokens.

Argument checks and marshalling only; the work runs in libmk.so.  Every call
is asynchronous on the current stream of its tensors' device (or on `stream`),
takes its scratch from torch's allocator on that stream, and can be captured
into a CUDA graph.  With `stream`, the caller orders it with the streams that
make the inputs and use the outputs, and keeps the inputs until the call has
run.  Tensors of one call are on one device, which need not be the current one.
Arguments that do not fit raise ValueError, codes of the library MkError.  An
empty list or batch is a call without work: it returns its (empty) outputs and
launches nothing.  There are no backward passes: tensors that require gradients
are refused where gradients are recorded.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import (MK_OK, MkError, load, mk_attn_shared_args, mk_kv_pool, mk_kv_state, mk_verify_args)

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _no_grad(what: str) -> None:
    """For tensors that require gradients: a result without its gradient is refused rather than returned."""
    if torch.is_grad_enabled():
        raise ValueError(f"{what} has no backward pass: call it under torch.no_grad(), or with detached tensors")


def _ints(t, n: int, name: str, dev) -> int:
    """The address of a contiguous int32 tensor of at least n words on `dev`."""
    if not (t.dtype is torch.int32 and t.is_contiguous() and t.numel() >= n and t.device == dev):
        raise ValueError(f"{name}: a contiguous int32 tensor of at least {n} words on {dev}")
    return t.data_ptr()


def _status(t, dev):
    return None if t is None else _ints(t, 1, "status", dev)


_current_device = torch.cuda.current_device


class _On:
    """The device and stream of a call: makes them current where they are not, so that launches and scratch go there."""

    __slots__ = ("raw", "ctx")

    def __init__(self, dev, stream):
        if dev.type != "cuda":
            raise ValueError("tensors must be CUDA tensors")
        self.ctx = None
        if stream is not None:
            _need(stream.device == dev, "the stream is another device's")
            self.ctx = torch.cuda.stream(stream)
            self.raw = stream.cuda_stream
        else:
            if dev.index != _current_device():
                self.ctx = torch.cuda.device(dev)
            self.raw = torch._C._cuda_getCurrentRawStream(dev.index)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.raw

    def __exit__(self, *e):
        if self.ctx is not None:
            self.ctx.__exit__(*e)


def _check(rc: int, where: str) -> None:
    if rc != MK_OK:
        raise MkError(rc, where)


# ------------------------------------------------------------------ cache pages

class KvPool:
    """A pool of K/V pages over two tensors [layers][pages][kv heads][page][head_dim] (contiguous, of the same shape
    and type).  An engine's cache tensors are one, with a page per sequence slot."""

    def __init__(self, k, v):
        _need(k.dim() == 5 and k.shape == v.shape and k.dtype == v.dtype and k.device == v.device,
              "k and v: tensors [layers][pages][kv heads][page][head_dim] of one shape, type and device")
        _need(k.is_contiguous() and v.is_contiguous(), "k and v must be contiguous")
        self.k, self.v, self.device = k, v, k.device
        self.n_layers, self.n_pages, self.n_kv_heads, self.page, self.head_dim = k.shape
        self._c = mk_kv_pool(k.data_ptr(), v.data_ptr(), *k.shape, k.element_size())
        self._ref = ctypes.byref(self._c)


class KvState:
    """The bookkeeping of a paged cache: which pages each sequence holds (include/mk_serve.h has the layout of
    `buffer`).  With `buffer`, the bookkeeping that it holds; otherwise every page is free."""

    def __init__(self, n_seqs: int, n_pages: int, max_pages: int, buffer=None, device="cuda", stream=None):
        self.n_seqs, self.n_pages, self.max_pages = n_seqs, n_pages, max_pages
        words = load().mk_kv_state_words(n_seqs, max_pages, n_pages)
        _need(words > 0, "sizes must be positive")
        new = buffer is None
        if new:
            dev = torch.device(device)
            if stream is not None:
                with torch.cuda.stream(stream):
                    buffer = torch.empty(words, dtype=torch.int32, device=dev)
            else:
                buffer = torch.empty(words, dtype=torch.int32, device=dev)
        self.device = buffer.device
        self.buffer = buffer
        self._c = mk_kv_state(_ints(buffer, words, "buffer", buffer.device), n_seqs, max_pages, n_pages)
        self._ref = ctypes.byref(self._c)
        if new:
            with _On(self.device, stream) as s:
                _check(load().mk_kv_init(self._ref, s), "mk_kv_init")

    def _part(self, a: int, n: int):
        return self.buffer[a:a + n]

    @property
    def n_free(self):
        """Pages free (one word on the device)."""
        return self._part(0, 1)

    @property
    def status_word(self):
        return self._part(1, 1)

    @property
    def lens(self):
        """Length of each sequence."""
        return self._part(4, self.n_seqs)

    @property
    def refs(self):
        """References to each page."""
        return self._part(4 + self.n_seqs, self.n_pages)

    @property
    def table(self):
        """Pages of each sequence, [n_seqs][max_pages], -1 where there is none."""
        a = 4 + self.n_seqs + 2 * self.n_pages
        return self.buffer[a:a + self.n_seqs * self.max_pages].view(self.n_seqs, self.max_pages)

    def status(self) -> int:
        """The first device-side error since the last call of this method (synchronises)."""
        code = int(self.status_word.item())
        if code:
            self.status_word.zero_()
        return code


def _kv_call(pool: KvPool, state: KvState, n: int, stream, what: str, call) -> None:
    _need(pool.device == state.device and pool.n_pages == state.n_pages,
          "the state is another pool's (device or number of pages)")
    with _On(pool.device, stream) as s:
        if n == 0:
            return
        ws = torch.empty(load().mk_kv_workspace_bytes(pool.n_pages, n), dtype=torch.uint8, device=pool.device)
        _check(call(ws.data_ptr(), s), what)


def kv_resize(pool: KvPool, state: KvState, seqs, lens, stream=None) -> None:
    """Set the lengths of the sequences `seqs` to `lens` (int32 tensors): pages past the new length are given back,
    growing sequences take pages, and a shared last page is copied before a sequence grows in it.  Length 0 frees."""
    n = seqs.numel()
    a, b = _ints(seqs, n, "seqs", pool.device), _ints(lens, n, "lens", pool.device)
    _kv_call(pool, state, n, stream, "mk_kv_resize",
             lambda ws, s: load().mk_kv_resize(pool._ref, state._ref, a, b, n, ws, s))


def kv_fork(pool: KvPool, state: KvState, parents, children, stream=None) -> None:
    """Make the empty sequences `children` copies of `parents` (int32 tensors): full pages are shared, a last page
    that is not full is copied."""
    n = parents.numel()
    _need(children.numel() == n, "a child for each parent")
    a, b = _ints(parents, n, "parents", pool.device), _ints(children, n, "children", pool.device)
    _kv_call(pool, state, n, stream, "mk_kv_fork",
             lambda ws, s: load().mk_kv_fork(pool._ref, state._ref, a, b, n, ws, s))


def kv_compact(pool: KvPool, state: KvState, stream=None) -> None:
    """Move the pages in use to the low end of the pool."""
    _kv_call(pool, state, 1, stream, "mk_kv_compact",
             lambda ws, s: load().mk_kv_compact(pool._ref, state._ref, ws, s))


def kv_copy(src: KvPool, dst: KvPool, items, status=None, stream=None) -> None:
    """Copy rows between pages of two pools, all layers and heads: `items` is an int32 tensor [n][5] of source page,
    source row, destination page, destination row, rows."""
    _need(items.dim() == 2 and items.shape[1] == 5, "items: [n][5]")
    _need(src.device == dst.device and src.k.dtype == dst.k.dtype, "the pools differ in device or type")
    n = items.shape[0]
    p = _ints(items, 5 * n, "items", src.device)
    with _On(src.device, stream) as s:
        if n == 0:
            return
        L = load()
        ws = torch.empty(L.mk_kv_workspace_bytes(1, n), dtype=torch.uint8, device=src.device)
        _check(L.mk_kv_copy(src._ref, dst._ref, p, n, _status(status, src.device), ws.data_ptr(), s), "mk_kv_copy")


# ------------------------------------------------------------------ shared-prefix attention

def shared_attention(q, k, v, table, lens, prefix_pages=None, prefix_len=None, scale=None, out=None, return_lse=False,
                     lse=None, status=None, stream=None):
    """Decode attention of a batch whose sequences share their first `prefix_len` positions.

    q: [batch][tokens][q heads][head_dim] bf16 / fp16 (tokens: the last positions of each sequence); k, v: one layer of
    a pool, [pages][kv heads][page][head_dim]; table: int32 [batch][pages of a sequence]; lens: int32 [batch], prefix
    included (negative: the sequence is unused and its output rows stay as they are); prefix_pages: int32 pages of the
    prefix; prefix_len: int32, one word.  Returns out like q, or (out, lse) with lse float [batch][tokens][q heads].
    Sums are 32-bit; a softmax weight is rounded to q's type where prefix_pages has room for 1024 positions or more."""
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
        raise ValueError("q: [batch][tokens][heads][head_dim]; k and v: [pages][kv heads][page][head_dim] of one shape "
                         "and strides")
    if q.requires_grad or k.requires_grad or v.requires_grad:
        _no_grad("shared_attention")
    B, T, nq, d = q.shape
    n_pages, nkv, page, dk = k.shape
    dev, dtype = q.device, q.dtype
    qs, ks = q.stride(), k.stride()
    code = DTYPES.get(dtype)
    if d != dk or code is None or dtype is not k.dtype or dtype is not v.dtype or k.device != dev or v.device != dev:
        raise ValueError("q, k and v agree in head_dim, type and device")
    if qs[3] != 1 or ks[3] != 1:
        raise ValueError("the last dimension must be contiguous")
    if table.dim() != 2 or table.shape[0] != B:
        raise ValueError("table: [batch][pages]")
    if out is not None:
        _need(out.shape == q.shape and out.dtype is dtype and out.device == dev and out.stride(3) == 1,
              "out: like q, its last dimension contiguous")
    if lse is not None:
        _need(lse.shape == (B, T, nq) and lse.dtype is torch.float32 and lse.is_contiguous() and lse.device == dev,
              "lse: a contiguous float tensor [batch][tokens][heads]")
    n_prefix = prefix_pages.numel() if prefix_pages is not None else 0
    if n_prefix:
        _need(prefix_len is not None, "prefix_pages without prefix_len")
        pp, pl = _ints(prefix_pages, n_prefix, "prefix_pages", dev), _ints(prefix_len, 1, "prefix_len", dev)
    else:
        pp = pl = None
    with _On(dev, stream) as s:
        if out is None:
            out = q.new_empty((B, T, nq, d))
        if lse is None and return_lse:
            lse = q.new_empty((B, T, nq), dtype=torch.float32)
        if B == 0:
            return (out, lse) if return_lse else out
        os = out.stride()
        a = mk_attn_shared_args(
            B, T, nq, nkv, d, code, page, n_pages, n_prefix, table.shape[1],
            1.0 / math.sqrt(d) if scale is None else scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
            lse.data_ptr() if lse is not None else None, pp, pl, _ints(table, 1, "table", dev),
            _ints(lens, B, "lens", dev), None if status is None else _ints(status, 1, "status", dev),
            # (a dimension of size 1 may come with any stride)
            qs[0] if B > 1 else 8, qs[1] if T > 1 else 8, qs[2] if nq > 1 else 8,
            os[0] if B > 1 else 8, os[1] if T > 1 else 8, os[2] if nq > 1 else 8,
            ks[0] if n_pages > 1 else 8, ks[1] if nkv > 1 else 8, ks[2] if page > 1 else 8)
        L, ref = load(), ctypes.byref(a)
        n = L.mk_attn_shared_workspace_bytes(ref)
        ws = table.new_empty(max(n, 256) // 4 + 1)
        _check(L.mk_attn_shared(ref, ws.data_ptr(), s), "mk_attn_shared")
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ probabilities and verification

def token_probs(logits, temperature=None, out=None, stream=None):
    """softmax(logits / temperature) in 32 bits: logits [rows][vocab] (float, bf16 or fp16), temperature float [rows]
    or None (1).  Temperature 0 puts everything on the first of the largest logits."""
    _need(logits.dim() == 2 and logits.stride(1) == 1 and logits.dtype in DTYPES, "logits: [rows][vocab], rows contiguous")
    if logits.requires_grad or (temperature is not None and temperature.requires_grad):
        _no_grad("token_probs")
    n, V = logits.shape
    dev = logits.device
    t = None
    if temperature is not None:
        _need(temperature.dtype is torch.float32 and temperature.is_contiguous() and temperature.numel() == n and
              temperature.device == dev, "temperature: a contiguous float tensor [rows]")
        t = temperature.data_ptr()
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty((n, V), dtype=torch.float32, device=dev)
        else:
            _need(out.shape == logits.shape and out.dtype is torch.float32 and out.stride(1) == 1 and out.device == dev,
                  "out: float [rows][vocab], rows contiguous")
        if n == 0:
            return out
        _check(load().mk_token_probs(logits.data_ptr(), DTYPES[logits.dtype], logits.stride(0), t, out.data_ptr(),
                                     out.stride(0), n, V, s), "mk_token_probs")
    return out


def verify(target, draft, tokens, u, n_drafted=None, status=None, stream=None):
    """How many drafted tokens stand against the target's probabilities, and the token sampled after them.

    target: float [batch][drafted + 1][vocab]; draft: float [batch][drafted][vocab] or None (a drafter without
    probabilities); tokens: int32 [batch][drafted]; u: float [batch][drafted + 1] in [0, 1); n_drafted: int32 [batch]
    or None (all).  Returns (tokens int32 [batch][drafted + 1], -1 after the sampled one; accepted int32 [batch])."""
    _need(target.dim() == 3 and target.dtype is torch.float32 and target.stride(2) == 1,
          "target: float [batch][drafted + 1][vocab], rows contiguous")
    if target.requires_grad or (draft is not None and draft.requires_grad):
        _no_grad("verify")
    B, T, V = target.shape
    T -= 1
    dev = target.device
    _need(T >= 0 and u.shape == (B, T + 1) and u.dtype is torch.float32 and u.is_contiguous() and u.device == dev,
          "u: a contiguous float tensor [batch][drafted + 1]")
    _need(tokens.dim() != 2 or T == 0 or tokens.shape[1] == T, "tokens: [batch][drafted]")  # (or the words in a row)
    d, ds = None, (0, 0)
    if draft is not None and T > 0:
        _need(draft.shape == (B, T, V) and draft.dtype is torch.float32 and draft.stride(2) == 1 and draft.device == dev,
              "draft: float [batch][drafted][vocab], rows contiguous")
        d, ds = draft.data_ptr(), draft.stride()
    x = _ints(tokens, B * T, "tokens", dev) if T > 0 else None
    n = None if n_drafted is None else _ints(n_drafted, B, "n_drafted", dev)
    with _On(dev, stream) as s:
        out = torch.empty((B, T + 1), dtype=torch.int32, device=dev)
        acc = torch.empty(B, dtype=torch.int32, device=dev)
        if B == 0:
            return out, acc
        ts = target.stride()
        a = mk_verify_args(B, T, V, target.data_ptr(), d, x, n, u.data_ptr(), out.data_ptr(), acc.data_ptr(),
                           _status(status, dev), ts[0], ts[1], ds[0], ds[1])
        _check(load().mk_verify(ctypes.byref(a), s), "mk_verify")
    return out, acc
