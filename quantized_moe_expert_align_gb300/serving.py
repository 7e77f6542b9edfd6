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
        dev = ring.get_device()
        _i32(ring, "ring", (ring.numel(),), dev)
        _i32(state, "state", (2,), dev)
        if not ring.is_cuda or ring.numel() < 1:
            raise ValueError("PagePool: ring is a contiguous int32 [n] on a GPU, n at least 1")
        self.ring, self.state = ring, state
        self._gpu, self._size = dev, ring.numel()
        self._ptrs = ring.data_ptr(), state.data_ptr()

    @classmethod
    def full(cls, num_pages, device="cuda"):
        """All pages of a cache are free."""
        _need_torch()
        torch = _attn.torch
        return cls(torch.arange(num_pages, dtype=torch.int32, device=device),
                   torch.tensor([0, num_pages], dtype=torch.int32, device=device))


class PagePlan:
    """What page_plan writes: ``seq_lens`` [B], ``cu_q`` and ``cu_k`` [B+1]
    (cu_k None: not written), ``positions`` and ``slots`` [rows], ``kept`` [B]
    (None without windows), ``state`` [2] (None: the pool's own; it may be set);
    all contiguous int32 on one GPU.  Its tensors are looked at when it is made:
    another set of tensors is another plan."""

    def __init__(self, seq_lens, cu_q, cu_k, positions, slots, kept=None, state=None):
        _need_torch()
        B, rows, dev = seq_lens.numel(), positions.numel(), seq_lens.get_device()
        for name, t, n in (("seq_lens", seq_lens, B), ("cu_q", cu_q, B + 1), ("cu_k", cu_k, B + 1),
                           ("positions", positions, rows), ("slots", slots, rows), ("kept", kept, B),
                           ("state", state, 2)):
            if t is not None or name in ("seq_lens", "cu_q", "positions", "slots"):
                _i32(t, name, (n,), dev)
        self._all = seq_lens, cu_q, cu_k, positions, slots, kept, state
        self._B, self._rows, self._gpu = B, rows, dev
        self._ptrs = tuple(_p(t) for t in self._all)

    seq_lens = property(lambda self: self._all[0])
    cu_q = property(lambda self: self._all[1])
    cu_k = property(lambda self: self._all[2])
    positions = property(lambda self: self._all[3])
    slots = property(lambda self: self._all[4])
    kept = property(lambda self: self._all[5])

    @property
    def state(self):
        return self._all[6]

    @state.setter
    def state(self, t):
        if t is not None:
            _i32(t, "state", (2,), self._gpu)
        self._all = self._all[:6] + (t,)
        self._ptrs = self._ptrs[:6] + (_p(t),)

    @classmethod
    def empty(cls, B, rows, windows=False, device="cuda", stream=None, seq_lens=None, kept=None, state=None):
        """New tensors for those that are not given."""
        _need_torch()
        new = lambda n: _result((n,), _attn.torch.int32, device, stream)  # noqa: E731
        return cls(new(B) if seq_lens is None else seq_lens, new(B + 1), new(B + 1), new(rows), new(rows),
                   new(B) if windows and kept is None else kept, state)


def page_plan(pool, page_table, seq_lens, new_lens, page_size, rows, window=0, sinks=0, kept=None,
              offsets=None, out=None, workspace=None, stream=None, dropped=None):
    """Pages, slots and positions of one step: sequence b has seq_lens[b]
    cached tokens and gets new_lens[b] more (-1: it has finished; its pages go
    back to the pool).  page_table [B][n] gets the new pages; ``rows`` is the
    number of rows of the step's buffers, at least the new tokens.  With a
    ``window``, pages behind it go back too, ``kept`` [B] saying how far that
    has come (zeros at first); from then on the row is for attention through that
    window alone (of the new tokens over what kv_gather brings, too).  offsets [rows]: positions are seq_lens[b] +
    offsets[row] instead of seq_lens[b] + i (depths of drafted tokens).  dropped
    [B]: tokens that sequence b has lost since its last step (rejected drafts),
    whose pages are still in its table: they are used first, or go back (a step
    that drops tokens of a page that has gone back is refused).

    Returns ``out``, a PagePlan (a new one by default); any of its seq_lens and
    kept may be the tensor passed in.  The pool's state moves on in place unless
    out.state is a tensor of its own.  If the pages do not suffice or a number is
    out of range, nothing moves, no row has a slot, and the workspace's status
    says so."""
    if _attn.torch is None:
        _need_torch()
    (B, n), dev = page_table.shape, _gpu(page_table, "page_table")
    _i32(page_table, "page_table", (B, n), dev)
    if pool._gpu != dev:
        raise _wrong(pool.ring, "pool", "a ring", dev)
    _i32(seq_lens, "seq_lens", (B,), dev)
    _i32(new_lens, "new_lens", (B,), dev)
    if offsets is not None:
        _i32(offsets, "offsets", (rows,), dev)
    if dropped is not None:
        _i32(dropped, "dropped", (B,), dev)
    if window:
        if kept is None:
            raise ValueError("window: kept [B] is needed")
        _i32(kept, "kept", (B,), dev)
    elif sinks:
        raise ValueError("sinks: only with a window")
    if out is None:
        out = PagePlan.empty(B, rows, bool(window), page_table.device, stream)
    if out._B != B or out._rows != rows or out._gpu != dev:
        raise ValueError(f"out: a plan for {B} sequences and {rows} rows on cuda:{dev} expected, got "
                         f"{out._B} and {out._rows} on cuda:{out._gpu}")
    if window and out.kept is None:
        raise ValueError("window: out.kept [B] is needed")
    ws = workspace
    if ws is None or ws._gpu != dev:
        ws = _workspace(ws, stream, dev, "pages", B)
    w, s = _window(window, sinks) if window else (0, 0)
    ring, state = pool._ptrs
    lens_out, cu_q, cu_k, positions, slots, kept_out, state_out = out._ptrs
    _moe._check((_moe._lib or _moe.load()).moe_page_plan(
        ring, pool._size, state, state_out or state, page_table.data_ptr(), n, page_size, seq_lens.data_ptr(),
        new_lens.data_ptr(), _p(dropped), kept.data_ptr() if w else None, _p(offsets), w, s, B, rows, lens_out, kept_out, cu_q,
        cu_k, positions, slots, ws._ptr, ws.nbytes, _on(stream, dev)), "moe_page_plan")
    return out


def attn_tree(q, cache, page_table, seq_lens, cu_q, tree, scale=None, out=None, lse=None,
              workspace=None, stream=None):
    """Attention of drafted tokens over the paged cache: q [T][Hq][D], of
    which sequence b has the rows [cu_q[b], cu_q[b+1]) (64 at most), its last
    cached tokens.  tree [T] int64: bit j of a row's is set where it sees drafted
    token j of its sequence ((2 << i) - 1 for row i: plain causal order); it sees
    all tokens before the drafted ones (none of whose pages may have gone back behind
    a window).  page_table [B][n], seq_lens [B] and cu_q
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
