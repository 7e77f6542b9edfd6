"""Attention half of a decoder layer: torch conveniences over ``include/moe_attn.h``.

Each function checks shapes and types, allocates what the caller did not
pass, calls the C entry point of the same name and raises ``MoeError`` on a
host-side error.  Errors found on the device are in the workspace's status
word (``moe_w4a16_get_device_status(workspace.buf)``).

Rows may be strided between tokens (the three parts of one fused projection);
the heads of a token and the values of a head are contiguous.  Tensors have
to live on the current device (others are refused: the library launches there)
and be ready on the stream of the call (the current stream unless ``stream`` is
given).  What a call allocates comes from the memory pool of that stream.
"""
from __future__ import annotations

import ctypes
import math

import quantized_moe_expert_align_gb300 as _moe

# Bound by the first call: importing this package does not import torch.
torch = _BF16 = _I32 = _F32 = _raw_stream = _this_gpu = None


def _need_torch():
    global torch, _BF16, _I32, _F32, _raw_stream, _this_gpu
    if torch is None:
        import torch as t
        _BF16, _I32, _F32 = t.bfloat16, t.int32, t.float32
        _raw_stream, _this_gpu = t._C._cuda_getCurrentRawStream, t._C._cuda_getDevice
        torch = t

MOE_KV_BF16 = 0
MOE_KV_FP8 = 1
MOE_ATTN_STATUS_BYTES = 256


def moe_kv_cache_size(type, num_pages, page_size, Hkv, D):
    """(status, data bytes, scale bytes) of a cache."""
    d, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = _moe.load().moe_kv_cache_size(type, num_pages, page_size, Hkv, D, ctypes.byref(d),
                                       ctypes.byref(s))
    return st, d.value, s.value


def moe_attn_decode_workspace_size(B, Hq, Hkv, D):
    return _moe.load().moe_attn_decode_workspace_size(B, Hq, Hkv, D)


def moe_attn_prefill_workspace_size(B, Tq, Hq, Hkv, D):
    return _moe.load().moe_attn_prefill_workspace_size(B, Tq, Hq, Hkv, D)


def rope_table(max_pos, rot, base=10000.0, factor=1.0, original_max=None, beta_fast=32.0,
               beta_slow=1.0, magnitude=None, device="cuda"):
    """cos_sin [max_pos][rot] fp32 (rot/2 cosines, then rot/2 sines), from
    angles computed in 64 bits.

    Pair i turns by pos * f_i with f_i = base^(-2i/rot).  For contexts longer
    than the model was trained on, ``factor`` > 1:
    * ``original_max`` None: every f_i is divided by ``factor`` (positions
      interpolated linearly);
    * ``original_max`` given: by parts.  A pair that makes at least
      ``beta_fast`` turns within ``original_max`` positions keeps f_i, one
      that makes at most ``beta_slow`` turns has it divided by ``factor``, and
      in between the two are blended linearly in the pair's index, between
      whole indexes in [0, rot - 1] (no pair is divided in full where the blend
      ends past the last one, rot/2 - 1).
    ``magnitude`` multiplies cosines and sines (by parts, default
    0.1 ln(factor) + 1; else 1), which scales q and k and so the attention's
    scores by its square.
    """
    _need_torch()
    if rot % 2 or rot < 0 or max_pos < 1 or factor < 1.0:
        raise ValueError("rope_table: rot even, max_pos >= 1, factor >= 1")
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    f = base ** (-2.0 * i / max(rot, 1))
    if factor > 1.0 and original_max is None:
        f = f / factor
    elif factor > 1.0:
        def index_of(turns):   # the (real) pair index that makes `turns` turns
            return rot / 2 * math.log(original_max / (2 * math.pi * turns)) / math.log(base)
        lo = max(math.floor(index_of(beta_fast)), 0)
        hi = min(math.ceil(index_of(beta_slow)), rot - 1)
        blend = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - blend) + f / factor * blend
        if magnitude is None:
            magnitude = 0.1 * math.log(factor) + 1.0
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * f
    return (torch.cat([a.cos(), a.sin()], 1) * (1.0 if magnitude is None else magnitude)).float()


class KVCache:
    """A paged key/value cache over caller-owned tensors: ``data``
    [num_pages][Hkv][2][page_size][D] bfloat16 or float8_e4m3fn and, for the
    latter, ``scales`` [num_pages][Hkv][2][page_size] float32."""

    def __init__(self, data, scales=None):
        _need_torch()
        if (data.dim() != 5 or data.shape[2] != 2 or not data.is_contiguous() or
                not data.is_cuda):
            raise ValueError("KVCache: data is a contiguous [num_pages][Hkv][2][page_size][D] "
                             "on a GPU")
        if data.dtype == torch.bfloat16 and scales is None:
            kind = MOE_KV_BF16
        elif data.dtype == torch.float8_e4m3fn and scales is not None:
            kind = MOE_KV_FP8
            if (scales.dtype != torch.float32 or scales.shape != data.shape[:4] or
                    not scales.is_contiguous() or scales.device != data.device):
                raise ValueError("KVCache: scales is a contiguous float32 "
                                 "[num_pages][Hkv][2][page_size] on data's device")
        else:
            raise ValueError("KVCache: bfloat16 data, or float8_e4m3fn data with scales")
        self.data, self.scales = data, scales
        self.num_pages, self.Hkv, _, self.page_size, self.D = data.shape
        self._c = _moe.moe_kv_cache_t(data.data_ptr(), None if scales is None else scales.data_ptr(),
                                      kind, self.num_pages, self.page_size, self.Hkv, self.D)
        self._ref = ctypes.byref(self._c)
        self._gpu = data.get_device()

    @classmethod
    def empty(cls, num_pages, Hkv, D, page_size=64, fp8=True, device="cuda"):
        """A new cache (contents undefined until tokens are appended)."""
        _need_torch()
        shape = (num_pages, Hkv, 2, page_size, D)
        if fp8:
            return cls(torch.empty(shape, dtype=torch.float8_e4m3fn, device=device),
                       torch.empty(shape[:4], dtype=torch.float32, device=device))
        return cls(torch.empty(shape, dtype=torch.bfloat16, device=device))


class AttnWorkspace:
    """A reusable workspace: ``op`` "decode", "prefill" or "tree" sized for up
    to B sequences and ``rows`` query rows in all, "pages" (page_plan) for up to
    B sequences; without ``op``, for qk_rope_append, kv_gather and kv_accept.
    ``buf`` is what the status call takes."""

    def __init__(self, device, op=None, B=0, rows=0, Hq=1, Hkv=1, D=128):
        if op is None:
            n = MOE_ATTN_STATUS_BYTES
        elif op == "decode":
            n = moe_attn_decode_workspace_size(B, Hq, Hkv, D)
        elif op == "prefill":
            n = moe_attn_prefill_workspace_size(B, rows, Hq, Hkv, D)
        elif op == "tree":
            n = _moe.moe_attn_tree_workspace_size(B, rows, Hq, Hkv, D)
        elif op == "pages":
            n = _moe.moe_page_plan_workspace_size(B)
        else:
            raise ValueError(f"AttnWorkspace: unknown op {op!r}")
        if n == 0:
            raise _moe.MoeError(_moe.MOE_ERR_INVALID_ARG, "AttnWorkspace")
        self.nbytes = n
        self.buf = _moe._empty_bytes(n, device)
        self._ptr, self._gpu = self.buf.data_ptr(), self.buf.get_device()


def _wrong(t, name, what, dev):
    return ValueError(f"{name}: {what} on cuda:{dev} expected, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _gpu(t, name):
    """The GPU of a call's first tensor, which has to be the current one (the
    library launches there) and to hold all the other tensors."""
    dev = t.get_device()   # (-1: not on a GPU)
    if dev != _this_gpu():
        raise _wrong(t, name, "a tensor", _this_gpu())
    return dev


def _bf16(t, name, n, dev):
    if t.dtype is not _BF16 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != dev:
        raise _wrong(t, name, f"contiguous bfloat16 {(n,)}", dev)


def _rows(t, name, T, H, D, dev):
    """Checks rows [T][H][D] with contiguous heads; the stride between tokens."""
    if t.dtype is not _BF16 or t.shape != (T, H, D) or t.get_device() != dev:
        raise _wrong(t, name, f"bfloat16 {(T, H, D)}", dev)
    st = t.stride()
    if T and (st[2] != 1 or (H > 1 and st[1] != D)):
        raise ValueError(f"{name}: the heads of a token have to be contiguous")
    return st[0] if T > 1 else H * D


def _i32(t, name, shape, dev):
    if t.dtype is not _I32 or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise _wrong(t, name, f"contiguous int32 {shape}", dev)


def _p(t):
    return None if t is None else t.data_ptr()


def _on(stream, dev):
    """The stream handle of a call on GPU dev: its current stream unless
    ``stream`` (a torch stream or a handle) is given."""
    return _raw_stream(dev) if stream is None else getattr(stream, "cuda_stream", stream)


def _pool_of(stream):
    """A context in which torch takes memory from the pool of the call's
    stream.  A block of the current stream's pool may still be read or written
    by kernels queued there, which a call on another stream does not wait for."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream))
    return torch.cuda.stream(stream)


def _result(shape, dtype, device, stream):
    """A new buffer for what a call returns.  On a stream of the call's own it
    is marked as used by the current stream too, where the caller reads it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _pool_of(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _rows_out(T, H, D, device, stream):
    return _result((T, H, D), torch.bfloat16, device, stream)


def _workspace(ws, stream, dev, *size):
    """A new workspace, if the caller has none."""
    if ws is not None:
        raise _wrong(ws.buf, "workspace", "a buffer", dev)
    if stream is None:
        return AttnWorkspace(f"cuda:{dev}", *size)
    with _pool_of(stream):
        return AttnWorkspace(f"cuda:{dev}", *size)


def qk_rope_append(q, k, v, cos_sin, positions, cache, slots, q_norm=None, k_norm=None, eps=1e-6,
                   interleaved=False, q_out=None, k_out=None, workspace=None, stream=None):
    """Norm, rotation and cache write of T new tokens: q [T][Hq][D], k and v
    [T][Hkv][D], cos_sin [max_pos][rot] (None: no rotation), positions and
    slots [T] int32, cache a KVCache or None.  Returns q_out; ``k_out`` True
    or a tensor also returns the rotated keys, as (q_out, k_out)."""
    if torch is None:
        _need_torch()
    T, Hq, D = q.shape
    Hkv, dev = k.shape[1], _gpu(q, "q")
    sq = _rows(q, "q", T, Hq, D, dev)
    sk, sv = _rows(k, "k", T, Hkv, D, dev), _rows(v, "v", T, Hkv, D, dev)
    max_pos, rot = cos_sin.shape if cos_sin is not None else (0, 0)
    if rot:
        if cos_sin.dtype is not _F32 or not cos_sin.is_contiguous() or cos_sin.get_device() != dev:
            raise _wrong(cos_sin, "cos_sin", "contiguous float32 [max_pos][rot]", dev)
        _i32(positions, "positions", (T,), dev)
    if q_norm is not None:
        _bf16(q_norm, "q_norm", D, dev)
    if k_norm is not None:
        _bf16(k_norm, "k_norm", D, dev)
    if cache is not None:
        _i32(slots, "slots", (T,), dev)
        if cache._gpu != dev:
            raise _wrong(cache.data, "cache", "data", dev)
    if q_out is None:
        q_out = _rows_out(T, Hq, D, q.device, stream)
    if k_out is True:
        k_out = _rows_out(T, Hkv, D, q.device, stream)
    elif k_out is False:
        k_out = None
    sqo = _rows(q_out, "q_out", T, Hq, D, dev)
    sko = _rows(k_out, "k_out", T, Hkv, D, dev) if k_out is not None else 0
    ws = workspace
    if ws is None or ws._gpu != dev:
        ws = _workspace(ws, stream, dev)
    _moe._check((_moe._lib or _moe.load()).moe_qk_rope_append(
        q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, _p(q_norm), _p(k_norm), eps, _p(cos_sin),
        max_pos, rot, int(interleaved), positions.data_ptr() if rot else None,
        slots.data_ptr() if cache is not None else None, q_out.data_ptr(), sqo, _p(k_out), sko,
        cache._ref if cache is not None else None, T, Hq, Hkv, D, ws._ptr, ws.nbytes, _on(stream, dev)),
        "moe_qk_rope_append")
    return q_out if k_out is None else (q_out, k_out)


def kv_gather(cache, page_table, cu_k, total, k_out=None, v_out=None, workspace=None, stream=None):
    """The cached tokens of B sequences as packed bf16 (k, v)
    [total][Hkv][D]; page_table [B][n] and cu_k [B+1] int32."""
    if torch is None:
        _need_torch()
    (B, n), dev = page_table.shape, _gpu(page_table, "page_table")
    _i32(page_table, "page_table", (B, n), dev)
    _i32(cu_k, "cu_k", (B + 1,), dev)
    if cache._gpu != dev:
        raise _wrong(cache.data, "cache", "data", dev)
    shape = (total, cache.Hkv, cache.D)
    if k_out is None:
        k_out = _rows_out(*shape, page_table.device, stream)
    if v_out is None:
        v_out = _rows_out(*shape, page_table.device, stream)
    ws = workspace
    if ws is None or ws._gpu != dev:
        ws = _workspace(ws, stream, dev)
    _moe._check((_moe._lib or _moe.load()).moe_kv_gather(
        cache._ref, page_table.data_ptr(), n, cu_k.data_ptr(), B, total, k_out.data_ptr(),
        _rows(k_out, "k_out", *shape, dev), v_out.data_ptr(), _rows(v_out, "v_out", *shape, dev), ws._ptr,
        ws.nbytes, _on(stream, dev)), "moe_kv_gather")
    return k_out, v_out


def attn_decode(q, cache, page_table, seq_lens, scale=None, out=None, lse=None, workspace=None,
                stream=None, window=None, sinks=0):
    """Attention of one token of each of B sequences over its cached tokens:
    q [B][Hq][D], page_table [B][n] and seq_lens [B] int32; scale defaults to
    D^-1/2.  With a ``window`` the token sees the last ``window`` tokens (itself
    among them) and the first ``sinks``; table entries of pages that hold none of
    those are not read.  Returns out [B][Hq][D]; ``lse`` True or a float32
    [B][Hq] tensor also returns the logsumexp, as (out, lse)."""
    if torch is None:
        _need_torch()
    B, Hq, D = q.shape
    if D != cache.D:
        raise ValueError(f"q has heads of {D}, the cache of {cache.D}")
    n, dev = page_table.shape[1], _gpu(q, "q")
    if cache._gpu != dev:
        raise _wrong(cache.data, "cache", "data", dev)
    _i32(page_table, "page_table", (B, n), dev)
    _i32(seq_lens, "seq_lens", (B,), dev)
    sq = _rows(q, "q", B, Hq, D, dev)
    if out is None:
        out = _rows_out(B, Hq, D, q.device, stream)
    so = _rows(out, "out", B, Hq, D, dev)
    lse = _lse(lse, B, Hq, q.device, dev, stream)
    ws = workspace
    if ws is None or ws._gpu != dev:
        ws = _workspace(ws, stream, dev, "decode", B, B, Hq, cache.Hkv, D)
    lib = _moe._lib or _moe.load()
    rest = (D ** -0.5 if scale is None else scale, out.data_ptr(), so, _p(lse), B, Hq, ws._ptr, ws.nbytes,
            _on(stream, dev))
    args = (q.data_ptr(), sq, cache._ref, page_table.data_ptr(), n, seq_lens.data_ptr())
    if window is None:
        _no_sinks(sinks)
        _moe._check(lib.moe_attn_decode(*args, *rest), "moe_attn_decode")
    else:
        _moe._check(lib.moe_attn_decode_window(*args, *_window(window, sinks), *rest), "moe_attn_decode_window")
    return out if lse is None else (out, lse)


def _no_sinks(sinks):
    if sinks:
        raise ValueError("sinks: only with a window")


def _window(window, sinks):
    """The two as the C calls take them (which refuse what is out of range):
    more than 2^31 - 1 is all there is."""
    most = 2 ** 31 - 1
    return max(min(int(window), most), -1), max(min(int(sinks), most), -1)


def attn_prefill(q, k, v, cu_q, cu_k, causal=True, scale=None, out=None, lse=None, workspace=None,
                 stream=None, window=None, sinks=0):
    """Attention over packed sequences: q [Tq][Hq][D], k and v [Tk][Hkv][D],
    cu_q and cu_k [B+1] int32; the last query of a sequence stands at its last
    key.  With a ``window`` (causal only) a query sees the last ``window`` keys
    up to its own and the first ``sinks`` of its sequence.  Returns out
    [Tq][Hq][D]; ``lse`` True or a float32 [Tq][Hq] tensor also returns the
    logsumexp, as (out, lse)."""
    if torch is None:
        _need_torch()
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    B, dev = cu_q.shape[0] - 1, _gpu(q, "q")
    _i32(cu_q, "cu_q", (B + 1,), dev)
    _i32(cu_k, "cu_k", (B + 1,), dev)
    sq = _rows(q, "q", Tq, Hq, D, dev)
    sk, sv = _rows(k, "k", Tk, Hkv, D, dev), _rows(v, "v", Tk, Hkv, D, dev)
    if out is None:
        out = _rows_out(Tq, Hq, D, q.device, stream)
    so = _rows(out, "out", Tq, Hq, D, dev)
    lse = _lse(lse, Tq, Hq, q.device, dev, stream)
    ws = workspace
    if ws is None or ws._gpu != dev:
        ws = _workspace(ws, stream, dev, "prefill", B, Tq, Hq, Hkv, D)
    lib = _moe._lib or _moe.load()
    args = (q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, cu_q.data_ptr(), cu_k.data_ptr(), B, Tq, Tk,
            Hq, Hkv, D)
    rest = (D ** -0.5 if scale is None else scale, out.data_ptr(), so, _p(lse), ws._ptr, ws.nbytes,
            _on(stream, dev))
    if window is None:
        _no_sinks(sinks)
        _moe._check(lib.moe_attn_prefill(*args, int(causal), *rest), "moe_attn_prefill")
    else:
        if not causal:
            raise ValueError("window: only causal attention has one")
        _moe._check(lib.moe_attn_prefill_window(*args, *_window(window, sinks), *rest),
                    "moe_attn_prefill_window")
    return out if lse is None else (out, lse)


def _lse(lse, T, Hq, device, dev, stream):
    if lse is True:
        return _result((T, Hq), torch.float32, device, stream)
    if lse is False:
        return None
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, Hq) or
                            not lse.is_contiguous() or lse.get_device() != dev):
        raise _wrong(lse, "lse", f"contiguous float32 {(T, Hq)}", dev)
    return lse
