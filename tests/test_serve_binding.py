"""The Python layer of serving over the paged cache without a GPU: where its
buffers come from, what it hands to the C entry points and what it refuses.
The tensors, torch and the library are the stand-ins of test_attn_binding."""
import pytest

import quantized_moe_expert_align_gb300 as moe
from quantized_moe_expert_align_gb300 import attention, serving
from tests.test_attn_binding import BF16, I32, U8, Cache, ExternalStream, Lib, Stream, Torch
from tests.test_attn_binding import Tensor as _Tensor

I64 = "i64"


class Tensor(_Tensor):
    def numel(self):
        n = 1
        for v in self.shape:
            n *= v
        return n


class MoreTorch(Torch):
    int64 = I64

    def empty(self, shape, dtype=None, device=None):
        t = Tensor(shape if isinstance(shape, tuple) else (shape,), dtype, int(device.split(":")[1]), self.now)
        self.made.append(t)
        return t


@pytest.fixture
def fake(monkeypatch):
    t, lib = MoreTorch(), Lib()
    monkeypatch.setattr(attention, "torch", t)
    monkeypatch.setattr(attention, "_BF16", BF16)
    monkeypatch.setattr(attention, "_I32", I32)
    monkeypatch.setattr(attention, "_raw_stream", lambda device: t.now.cuda_stream)
    monkeypatch.setattr(attention, "_this_gpu", lambda: 0)
    monkeypatch.setattr(serving, "_need_torch", lambda: None)
    monkeypatch.setattr(moe, "_lib", lib)
    monkeypatch.setattr(moe, "_empty_bytes", lambda n, device: t.empty(n, U8, device))
    return t, lib


def _i(*shape, dev=0):
    return Tensor(shape, I32, dev)


def _args(dev=0):
    """Each entry point's arguments, all of them given."""
    far = Cache()
    far.data, far._gpu = Tensor((8, 2, 2, 16, 64), BF16, dev), dev
    q, f32 = Tensor((5, 4, 64), BF16, dev), Tensor((5, 4), "f32", dev)
    ws = attention.AttnWorkspace(f"cuda:{dev}")
    return {
        "pages": (moe.page_plan, dict(pool=moe.PagePool(_i(9, dev=dev), _i(2, dev=dev)), page_table=_i(5, 3, dev=dev),
                                      seq_lens=_i(5, dev=dev), new_lens=_i(5, dev=dev), page_size=16, rows=7,
                                      window=4, sinks=1, kept=_i(5, dev=dev), offsets=_i(7, dev=dev),
                                      dropped=_i(5, dev=dev),
                                      out=moe.PagePlan(_i(5, dev=dev), _i(6, dev=dev), _i(6, dev=dev), _i(7, dev=dev),
                                                       _i(7, dev=dev), _i(5, dev=dev), _i(2, dev=dev)),
                                      workspace=ws)),
        "tree": (moe.attn_tree, dict(q=q, cache=far, page_table=_i(3, 4, dev=dev), seq_lens=_i(3, dev=dev),
                                     cu_q=_i(4, dev=dev), tree=Tensor((5,), I64, dev), out=q, lse=f32, workspace=ws)),
        "accept": (moe.kv_accept, dict(cache=far, page_table=_i(3, 4, dev=dev), base=_i(3, dev=dev),
                                       accept=_i(3, 8, dev=dev), workspace=ws)),
        "wdecode": (moe.attn_decode, dict(q=q, cache=far, page_table=_i(5, 4, dev=dev), seq_lens=_i(5, dev=dev),
                                          out=q, lse=f32, workspace=ws, window=9, sinks=2)),
    }


OPS = ["pages", "tree", "accept", "wdecode"]


@pytest.mark.parametrize("op", OPS)
def test_arguments_reach_the_library(fake, op):
    t, lib = fake
    f, args = _args()[op]
    f(**args)
    name, sent = lib.calls[-1]
    assert name == {"pages": "moe_page_plan", "tree": "moe_attn_tree", "accept": "moe_kv_accept",
                    "wdecode": "moe_attn_decode_window"}[op]
    assert len(sent) == len(moe._serve_signatures()[name][1]) and sent[-1] == 7


@pytest.mark.parametrize("op", OPS)
def test_tensors_of_another_gpu_are_refused(fake, op):
    t, lib = fake
    f, args = _args()[op]
    _, far = _args(1)[op]
    n = len(lib.calls)
    for name, a in args.items():
        if isinstance(a, (int, float)):
            continue
        with pytest.raises(ValueError):
            f(**dict(args, **{name: far[name]}))
    assert all(c[0].endswith("_size") for c in lib.calls[n:])


@pytest.mark.parametrize("op,change", [
    ("pages", dict(seq_lens=_i(4))), ("pages", dict(new_lens=Tensor((5,), I64))), ("pages", dict(kept=None)),
    ("pages", dict(kept=_i(6))), ("pages", dict(offsets=_i(6))), ("pages", dict(dropped=_i(7))),
    ("pages", dict(rows=8)), ("pages", dict(window=0)),
    ("tree", dict(tree=Tensor((5,), I32))), ("tree", dict(tree=Tensor((4,), I64))), ("tree", dict(cu_q=_i(3))),
    ("tree", dict(seq_lens=_i(5))), ("tree", dict(q=Tensor((5, 4, 128), BF16))),
    ("accept", dict(base=_i(4))), ("accept", dict(accept=_i(4, 8))),
    ("wdecode", dict(window=None)), ("wdecode", dict(seq_lens=_i(4)))])
def test_refusals(fake, op, change):
    t, lib = fake
    f, args = _args()[op]
    n = len(lib.calls)
    with pytest.raises(ValueError):
        f(**dict(args, **change))
    assert all(c[0].endswith("_size") for c in lib.calls[n:])


def test_window_needs_causal_and_sinks_need_a_window(fake):
    q, k, cu = Tensor((5, 4, 64), BF16), Tensor((5, 2, 64), BF16), _i(4)
    with pytest.raises(ValueError):
        moe.attn_prefill(q, k, k, cu, cu, causal=False, window=5)
    with pytest.raises(ValueError):
        moe.attn_prefill(q, k, k, cu, cu, sinks=5)
    moe.attn_prefill(q, k, k, cu, cu, window=1 << 50, sinks=3)
    name, sent = fake[1].calls[-1]
    assert name == "moe_attn_prefill_window" and sent[14:16] == (2 ** 31 - 1, 3)


def test_a_plan_looks_at_its_tensors(fake):
    with pytest.raises(ValueError):
        moe.PagePlan(_i(5), _i(5), None, _i(7), _i(7))
    with pytest.raises(ValueError):
        moe.PagePlan(_i(5), _i(6), None, _i(7), _i(7, dev=1))
    plan = moe.PagePlan(_i(5), _i(6), None, _i(7), _i(7))
    with pytest.raises(ValueError):
        plan.state = _i(3)
    with pytest.raises(ValueError):
        moe.PagePool(_i(9), _i(3))
    with pytest.raises(ValueError):   # no place for the kept pages
        f, args = _args()["pages"]
        f(**dict(args, out=plan))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op,made", [("pages", 7), ("tree", 3), ("accept", 1)])
def test_buffers_made_for_a_call_come_from_its_stream(fake, op, made, raw):
    t, lib = fake
    f, args = _args()[op]
    t.made.clear()
    args = {k: v for k, v in args.items() if k not in ("out", "workspace")}
    if op == "tree":
        args["lse"] = True
    f(stream=99 if raw else Stream(99), **args)
    assert lib.calls[-1][1][-1] == 99
    assert len(t.made) == made and all(b.pool.cuda_stream == 99 for b in t.made)
    assert all(isinstance(b.pool, ExternalStream) == raw for b in t.made)
    assert t.now is t.home
