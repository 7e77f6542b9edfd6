"""Serving over the paged cache: torch conveniences over
``include/moe_attn_serve.h``, in the manner of ``attention.py`` (whose checks,
streams and memory pools hold here too).

A step of a server that drafts tokens: ``page_plan`` (pages, slots and
positions of the step's tokens), ``qk_rope_append``, ``attn_tree``, sampling
(the caller's), ``kv_accept``, and the lengths less what was not accepted.
"""
from __future__ import annotations

import quantized_moe_expert_align_gb300 as _moe

from . import attention as _attn
from .attention import (AttnWorkspace, _gpu, _i32, _lse, _need_torch, _on, _p, _pool_of, _result,  # noqa: F401
                        _rows, _rows_out, _window, _workspace, _wrong)

MOE_TREE_TOKENS = 64


def moe_page_plan_workspace_size(B):
    return _moe.load().moe_page_plan_workspace_size(B)


def moe_attn_tree_workspace_size(B, T, Hq, Hkv, D):
    return _moe.load().moe_attn_tree_workspace_size(B, T, Hq, Hkv, D)


class PagePool:
    """The free pages of a cache, on the GPU: ``ring`` [n] int32, of whose
    places ``state[1]`` from place ``state[0]`` on hold free page numbers."""

    def __init__(self, ring, state):
        _need_torch()
        _i32(ring, "ring", (ring.numel(),), ring.get_device())
        _i32(state, "state", (2,), ring.get_device())
        if not ring.is_cuda or ring.numel() < 1:
            raise ValueError("PagePool: ring is a contiguous int32 [n] on a GPU, n at least 1")
        self.ring, self.state = ring, state

    @classmethod
    def full(cls, num_pages, device="cuda"):
        """All pages of a cache are free."""
        _need_torch()
        torch = _attn.torch
        return cls(torch.arange(num_pages, dtype=torch.int32, device=device),
                   torch.tensor([0, num_pages], dtype=torch.int32, device=device))


class PagePlan:
    """What page_plan writes: ``seq_lens`` [B], ``cu_q`` and ``cu_k`` [B+1],
    ``positions`` and ``slots`` [rows], ``kept`` [B] (None without windows),
    ``state`` [2] (the pool's, unless set to a tensor of its own); all int32."""

    def __init__(self, seq_lens, cu_q, cu_k, positions, slots, kept=None, state=None):
        self.seq_lens, self.cu_q, self.cu_k = seq_lens, cu_q, cu_k
        self.positions, self.slots, self.kept, self.state = positions, slots, kept, state

    @classmethod
    def empty(cls, B, rows, windows=False, device="cuda", stream=None):
        _need_torch()
        new = lambda n: _result((n,), _attn.torch.int32, device, stream)  # noqa: E731
        return cls(new(B), new(B + 1), new(B + 1), new(rows), new(rows), new(B) if windows else None)


def page_plan(pool, page_table, seq_lens, new_lens, page_size, rows, window=0, sinks=0, kept=None,
              offsets=None, out=None, workspace=None, stream=None):
    """Pages, slots and positions of one step: sequence b has seq_lens[b]
    cached tokens and gets new_lens[b] more (-1: it has finished; its pages go
    back to the pool).  page_table [B][n] gets the new pages; ``rows`` is the
    number of rows of the step's buffers, at least the new tokens.  With a
    ``window``, pages behind it go back too, ``kept`` [B] saying how far that
    has come (zeros at first).  offsets [rows]: positions are seq_lens[b] +
    offsets[row] instead of seq_lens[b] + i (depths of drafted tokens).

    Returns ``out``, a PagePlan (a new one by default); any of its seq_lens and
    kept may be the tensor passed in.  The pool's state moves on in place unless
    out.state is a tensor of its own.  If the pages do not suffice or a number is
    out of range, nothing moves, no row has a slot, and the workspace's status
    says so."""
    if _attn.torch is None:
        _need_torch()
    (B, n), dev = page_table.shape, _gpu(page_table, "page_table")
    _i32(page_table, "page_table", (B, n), dev)
    _i32(pool.ring, "ring", (pool.ring.numel(),), dev)
    _i32(pool.state, "state", (2,), dev)
    _i32(seq_lens, "seq_lens", (B,), dev)
    _i32(new_lens, "new_lens", (B,), dev)
    if offsets is not None:
        _i32(offsets, "offsets", (rows,), dev)
    if window:
        if kept is None:
            raise ValueError("window: kept [B] is needed")
        _i32(kept, "kept", (B,), dev)
    elif sinks:
        raise ValueError("sinks: only with a window")
    if out is None:
        out = PagePlan.empty(B, rows, bool(window), page_table.device, stream)
    if out.state is None:
        out.state = pool.state
    _i32(out.state, "out.state", (2,), dev)
    _i32(out.seq_lens, "out.seq_lens", (B,), dev)
    _i32(out.cu_q, "out.cu_q", (B + 1,), dev)
    if out.cu_k is not None:
        _i32(out.cu_k, "out.cu_k", (B + 1,), dev)
    _i32(out.positions, "out.positions", (rows,), dev)
    _i32(out.slots, "out.slots", (rows,), dev)
    if window:
        if out.kept is None:
            raise ValueError("window: out.kept [B] is needed")
        _i32(out.kept, "out.kept", (B,), dev)
    ws = workspace
    if ws is None or ws._gpu != dev:
        ws = _workspace(ws, stream, dev, "pages", B)
    w, s = _window(window, sinks)
    _moe._check((_moe._lib or _moe.load()).moe_page_plan(
        pool.ring.data_ptr(), pool.ring.numel(), pool.state.data_ptr(), out.state.data_ptr(),
        page_table.data_ptr(), n, page_size, seq_lens.data_ptr(), new_lens.data_ptr(),
        kept.data_ptr() if w else None, _p(offsets), w, s, B, rows, out.seq_lens.data_ptr(),
        out.kept.data_ptr() if w else None, out.cu_q.data_ptr(), _p(out.cu_k), out.positions.data_ptr(),
        out.slots.data_ptr(), ws._ptr, ws.nbytes, _on(stream, dev)), "moe_page_plan")
    return out


def attn_tree(q, cache, page_table, seq_lens, cu_q, tree, scale=None, out=None, lse=None,
              workspace=None, stream=None):
    """Attention of drafted tokens over the paged cache: q [T][Hq][D], of
    which sequence b has the rows [cu_q[b], cu_q[b+1]) (64 at most), its last
    cached tokens.  tree [T] int64: bit j of a row's is set where it sees drafted
    token j of its sequence ((2 << i) - 1 for row i: plain causal order); it sees
    all tokens before the drafted ones.  page_table [B][n], seq_lens [B] and cu_q
    [B+1] int32; scale defaults to D^-1/2.  Returns out [T][Hq][D]; ``lse`` True
    or a float32 [T][Hq] tensor also returns the logsumexp, as (out, lse)."""
    if _attn.torch is None:
        _need_torch()
    T, Hq, D = q.shape
    if D != cache.D:
        raise ValueError(f"q has heads of {D}, the cache of {cache.D}")
    (B, n), dev = page_table.shape, _gpu(q, "q")
    if cache._gpu != dev:
        raise _wrong(cache.data, "cache", "data", dev)
    _i32(page_table, "page_table", (B, n), dev)
    _i32(seq_lens, "seq_lens", (B,), dev)
    _i32(cu_q, "cu_q", (B + 1,), dev)
    if (tree.dtype is not _attn.torch.int64 or tree.shape != (T,) or not tree.is_contiguous() or
            tree.get_device() != dev):
        raise _wrong(tree, "tree", f"contiguous int64 {(T,)}", dev)
    sq = _rows(q, "q", T, Hq, D, dev)
    if out is None:
        out = _rows_out(T, Hq, D, q.device, stream)
    so = _rows(out, "out", T, Hq, D, dev)
    lse = _lse(lse, T, Hq, q.device, dev, stream)
    ws = workspace
    if ws is None or ws._gpu != dev:
        ws = _workspace(ws, stream, dev, "tree", B, T, Hq, cache.Hkv, D)
    _moe._check((_moe._lib or _moe.load()).moe_attn_tree(
        q.data_ptr(), sq, cache._ref, page_table.data_ptr(), n, seq_lens.data_ptr(), cu_q.data_ptr(),
        tree.data_ptr(), D ** -0.5 if scale is None else scale, out.data_ptr(), so, _p(lse), B, T, Hq,
        ws._ptr, ws.nbytes, _on(stream, dev)), "moe_attn_tree")
    return out if lse is None else (out, lse)


def kv_accept(cache, page_table, base, accept, workspace=None, stream=None):
    """Accepted tokens to their places: cached token base[b] + accept[b][i] of
    sequence b becomes token base[b] + i.  accept [B][P] int32 holds rising
    numbers, ended by -1 (P at most 64); page_table [B][n] and base [B] int32."""
    if _attn.torch is None:
        _need_torch()
    (B, n), dev = page_table.shape, _gpu(page_table, "page_table")
    _i32(page_table, "page_table", (B, n), dev)
    if cache._gpu != dev:
        raise _wrong(cache.data, "cache", "data", dev)
    _i32(base, "base", (B,), dev)
    P = accept.shape[1]
    _i32(accept, "accept", (B, P), dev)
    ws = workspace
    if ws is None or ws._gpu != dev:
        ws = _workspace(ws, stream, dev)
    _moe._check((_moe._lib or _moe.load()).moe_kv_accept(
        cache._ref, page_table.data_ptr(), n, base.data_ptr(), accept.data_ptr(), B, P, ws._ptr, ws.nbytes,
        _on(stream, dev)), "moe_kv_accept")
