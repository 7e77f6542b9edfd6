"""The attention half's Python layer without a GPU: where its buffers come
from and what it hands to the C entry points.

The tensors, torch and the library are stand-ins that record their use."""
import contextlib

import pytest

import quantized_moe_expert_align_gb300 as moe
from quantized_moe_expert_align_gb300 import attention

BF16, I32, F32, U8 = "bf16", "i32", "f32", "u8"


class Stream:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


class ExternalStream(Stream):
    pass


class Tensor:
    def __init__(self, shape, dtype, device=0, pool=None):
        self.shape, self.dtype, self.index, self.pool = tuple(shape), dtype, device, pool
        self.is_cuda, self.device, self.recorded = True, f"cuda:{device}", []

    def stride(self):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st)

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.recorded.append(stream)


class Torch:
    """Allocations with the stream that was current when they were made."""
    bfloat16, int32, float32, uint8 = BF16, I32, F32, U8

    def __init__(self):
        self.home = self.now = Stream(7)
        self.made = []
        c = self.cuda = type("cuda", (), dict(Stream=Stream, ExternalStream=ExternalStream))

        @contextlib.contextmanager
        def stream(s):
            before, self.now = self.now, s
            try:
                yield
            finally:
                self.now = before
        c.stream, c.current_stream = staticmethod(stream), staticmethod(lambda device=None: self.now)

    def empty(self, shape, dtype=None, device=None):
        t = Tensor(shape if isinstance(shape, tuple) else (shape,), dtype, int(device.split(":")[1]), self.now)
        self.made.append(t)
        return t


class Lib:
    """Every entry point succeeds; `calls` holds its name and arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 65536 if name.endswith("workspace_size") else 0
        return call


class Cache:
    D, Hkv, page_size, num_pages, _ref, _gpu = 64, 2, 16, 8, None, 0
    data = Tensor((8, 2, 2, 16, 64), BF16)


@pytest.fixture
def fake(monkeypatch):
    t, lib = Torch(), Lib()
    monkeypatch.setattr(attention, "torch", t)
    monkeypatch.setattr(attention, "_BF16", BF16)
    monkeypatch.setattr(attention, "_I32", I32)
    monkeypatch.setattr(attention, "_F32", F32)
    monkeypatch.setattr(attention, "_raw_stream", lambda device: t.now.cuda_stream)
    monkeypatch.setattr(attention, "_this_gpu", lambda: 0)
    monkeypatch.setattr(moe, "_lib", lib)
    monkeypatch.setattr(moe, "_empty_bytes", lambda n, device: t.empty(n, U8, device))
    return t, lib


def _calls():
    """Each entry point with nothing but its inputs given."""
    q, k = Tensor((5, 4, 64), BF16), Tensor((5, 2, 64), BF16)
    cu, n, table = Tensor((4,), I32), Tensor((5,), I32), Tensor((5, 3), I32)
    return {
        "append": lambda **kw: moe.qk_rope_append(q, k, k, Tensor((9, 64), F32), n, Cache(), n,
                                                  k_out=True, **kw),
        "gather": lambda **kw: moe.kv_gather(Cache(), table, Tensor((6,), I32), 5, **kw),
        "decode": lambda **kw: moe.attn_decode(q, Cache(), table, n, lse=True, **kw),
        "prefill": lambda **kw: moe.attn_prefill(q, k, k, cu, cu, lse=True, **kw),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op", ["append", "gather", "decode", "prefill"])
def test_buffers_made_for_a_call_come_from_its_stream(fake, op, raw):
    """A block from another stream's pool may still be read or written by that
    stream's earlier kernels, which the call does not wait for.  What is
    returned is also marked as used by the caller's stream."""
    t, lib = fake
    side = Stream(99)
    out = _calls()[op](stream=99 if raw else side)
    assert lib.calls[-1][1][-1] == 99
    assert len(t.made) == 3   # two results and the workspace
    assert all(b.pool.cuda_stream == 99 for b in t.made)
    assert all(isinstance(b.pool, ExternalStream) == raw for b in t.made)
    assert all(t.home in o.recorded for o in out)
    assert t.now is t.home


@pytest.mark.parametrize("op", ["append", "gather", "decode", "prefill"])
def test_buffers_made_on_the_current_stream(fake, op):
    t, lib = fake
    _calls()[op]()
    assert lib.calls[-1][1][-1] == 7
    assert len(t.made) == 3 and all(b.pool is t.home and not b.recorded for b in t.made)


def test_no_logsumexp_and_no_keys(fake):
    """False is the same as None: only the first result is returned."""
    t, lib = fake
    q, k = Tensor((5, 4, 64), BF16), Tensor((5, 2, 64), BF16)
    cu, n, table = Tensor((4,), I32), Tensor((5,), I32), Tensor((5, 3), I32)
    for no in (None, False):
        t.made.clear()
        outs = [moe.qk_rope_append(q, k, k, None, None, None, None, k_out=no),
                moe.attn_decode(q, Cache(), table, n, lse=no), moe.attn_prefill(q, k, k, cu, cu, lse=no)]
        assert all(isinstance(o, Tensor) and o.shape == (5, 4, 64) for o in outs)
        assert len(t.made) == 6   # a result and a workspace each
        names = [c[0] for c in lib.calls if not c[0].endswith("_size")]
        assert names[-3:] == ["moe_qk_rope_append", "moe_attn_decode", "moe_attn_prefill"]
        append, decode, prefill = [c[1] for c in lib.calls if not c[0].endswith("_size")][-3:]
        assert append[17] is None and decode[9] is None and prefill[18] is None


def _another(t):
    return Tensor(t.shape, t.dtype, 1)


@pytest.mark.parametrize("op", ["append", "gather", "decode", "prefill"])
def test_tensors_of_another_gpu_are_refused(fake, op):
    """A kernel on one GPU must not be given another's memory: each tensor
    argument in turn, outputs, caches and workspaces among them."""
    t, lib = fake
    q, k = Tensor((5, 4, 64), BF16), Tensor((5, 2, 64), BF16)
    w, cs, i5, i6 = Tensor((64,), BF16), Tensor((9, 64), F32), Tensor((5,), I32), Tensor((6,), I32)
    table, lse = Tensor((5, 3), I32), Tensor((5, 4), F32)
    ws = attention.AttnWorkspace("cuda:0")
    cache, far = Cache(), Cache()
    far.data, far._gpu = _another(Cache.data), 1
    f, args = {
        "append": (moe.qk_rope_append, dict(q=q, k=k, v=k, cos_sin=cs, positions=i5, cache=cache, slots=i5,
                                            q_norm=w, k_norm=w, q_out=q, k_out=k, workspace=ws)),
        "gather": (moe.kv_gather, dict(cache=cache, page_table=table, cu_k=i6, total=5, k_out=k, v_out=k,
                                       workspace=ws)),
        "decode": (moe.attn_decode, dict(q=q, cache=cache, page_table=table, seq_lens=i5, out=q, lse=lse,
                                         workspace=ws)),
        "prefill": (moe.attn_prefill, dict(q=q, k=k, v=k, cu_q=i6, cu_k=i6, out=q, lse=lse, workspace=ws)),
    }[op]
    f(**args)
    n = len(lib.calls)
    for name, a in args.items():
        if isinstance(a, Tensor):
            bad = _another(a)
        elif a is cache:
            bad = far
        elif a is ws:
            bad = attention.AttnWorkspace("cuda:1")
        else:
            continue
        with pytest.raises(ValueError):
            f(**dict(args, **{name: bad}))
    assert all(c[0].endswith("_size") for c in lib.calls[n:])   # nothing was launched


@pytest.mark.parametrize("op", ["append", "gather", "decode", "prefill"])
def test_tensors_off_the_current_gpu_are_refused(fake, monkeypatch, op):
    """The library launches on the current device."""
    t, lib = fake
    monkeypatch.setattr(attention, "_this_gpu", lambda: 1)
    for kw in (dict(), dict(stream=Stream(99))):
        with pytest.raises(ValueError):
            _calls()[op](**kw)
    assert all(c[0].endswith("_size") for c in lib.calls)
