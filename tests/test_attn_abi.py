"""The attention half's C ABI without a GPU: exported symbols, sizes, and the
arguments that are refused on the host before anything is launched."""
import ctypes
import os
import re

import pytest

import quantized_moe_expert_align_gb300 as moe
from quantized_moe_expert_align_gb300 import build

HEADER = os.path.join(build.INCLUDE, "moe_attn.h")
P = 4096


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load()


def _cache(**kw):
    f = dict(data=P, scales=None, type=moe.MOE_KV_BF16, num_pages=8, page_size=16, Hkv=2, D=128)
    f.update(kw)
    return ctypes.byref(moe.moe_kv_cache_t(*[f[n] for n, _ in moe.moe_kv_cache_t._fields_]))


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_\w+)\s*\(", text)))
    assert len(names) == 7
    for n in names:
        assert hasattr(lib, n)


def test_status_string(lib):
    assert moe.moe_status_string(moe.MOE_ERR_DEVICE_BAD_INDEX).startswith("MOE_ERR_DEVICE_BAD_INDEX")


def test_cache_sizes(lib):
    assert moe.moe_kv_cache_size(moe.MOE_KV_BF16, 10, 16, 8, 128) == (moe.MOE_OK, 10 * 16 * 8 * 512, 0)
    assert moe.moe_kv_cache_size(moe.MOE_KV_FP8, 10, 64, 3, 64) == \
        (moe.MOE_OK, 10 * 64 * 3 * 128, 10 * 64 * 3 * 8)
    for bad in [(2, 10, 16, 8, 128), (0, 0, 16, 8, 128), (0, 10, 24, 8, 128), (0, 10, 8, 8, 128),
                (0, 10, 512, 8, 128), (0, 10, 16, 0, 128), (0, 10, 16, 8, 96),
                (0, 1 << 24, 64, 1, 128)]:
        assert moe.moe_kv_cache_size(*bad) == (moe.MOE_ERR_INVALID_ARG, 0, 0)


def test_workspace_sizes(lib):
    assert moe.moe_attn_decode_workspace_size(1, 64, 8, 128) >= 256
    assert moe.moe_attn_prefill_workspace_size(1, 1000, 64, 8, 128) >= 256
    for bad in [(-1, 8, 8, 128), (70000, 8, 8, 128), (1, 9, 8, 128), (1, 8, 0, 128), (1, 8, 8, 80),
                (1, 2048, 8, 128)]:
        assert moe.moe_attn_decode_workspace_size(*bad) == 0
    assert moe.moe_attn_prefill_workspace_size(1, -1, 8, 8, 128) == 0
    assert moe.moe_attn_prefill_workspace_size(1, 1 << 30, 8, 8, 128) == 0


def _refuses(fn, names, good, cases):
    for change, want in cases:
        a = dict(zip(names, good))
        assert set(change) <= set(a)
        a.update(change)
        assert fn(*[a[n] for n in names]) == want, change


def test_append_refusals(lib):
    names = ("q qs k ks v vs qw kw eps cs max_pos rot inter pos slots qo qos ko kos cache T Hq Hkv D "
             "ws wsb stream").split()
    good = [P, 1024, P, 256, P, 256, P, P, 1e-6, P, 100, 128, 0, P, P, P, 1024, P, 256, _cache(), 4, 8,
            2, 128, P, 256, None]
    inv, mis = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_MISALIGNED
    _refuses(lib.moe_qk_rope_append, names, good, [
        (dict(q=None), inv), (dict(k=None), inv), (dict(v=None), inv), (dict(qo=None), inv),
        (dict(cs=None), inv), (dict(pos=None), inv), (dict(slots=None), inv), (dict(ws=None), inv),
        (dict(rot=136), inv), (dict(rot=24), inv), (dict(rot=-16), inv), (dict(max_pos=0), inv),
        (dict(T=-1), inv), (dict(T=1 << 30), inv), (dict(Hq=7), inv), (dict(Hkv=0), inv),
        (dict(D=96), inv), (dict(D=64), inv), (dict(eps=-1.0), inv), (dict(eps=float("nan")), inv),
        (dict(qs=1016), inv), (dict(qs=1028), inv), (dict(ks=128), inv), (dict(kos=0), inv),
        (dict(cache=_cache(Hkv=4)), inv), (dict(cache=_cache(data=None)), inv),
        (dict(cache=_cache(type=moe.MOE_KV_FP8)), inv), (dict(cache=_cache(scales=P)), inv),
        (dict(cache=_cache(page_size=20)), inv), (dict(cache=_cache(data=P + 8)), mis),
        (dict(q=P + 2), mis), (dict(qw=P + 8), mis), (dict(cs=P + 4), mis), (dict(pos=P + 2), mis),
        (dict(ko=P + 8), mis), (dict(ws=P + 128), mis),
        (dict(wsb=255), moe.MOE_ERR_WORKSPACE_TOO_SMALL)])


def test_gather_refusals(lib):
    names = "cache table tstride cu B Tk ko kos vo vos ws wsb stream".split()
    good = [_cache(), P, 4, P, 2, 100, P, 256, P, 256, P, 256, None]
    inv, mis = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_MISALIGNED
    _refuses(lib.moe_kv_gather, names, good, [
        (dict(cache=None), inv), (dict(table=None), inv), (dict(tstride=0), inv), (dict(cu=None), inv),
        (dict(B=0), inv), (dict(B=70000), inv), (dict(Tk=-1), inv), (dict(ko=None), inv),
        (dict(vos=248), inv), (dict(kos=260), inv), (dict(vo=P + 8), mis), (dict(cu=P + 2), mis),
        (dict(wsb=0), moe.MOE_ERR_WORKSPACE_TOO_SMALL)])


def test_decode_refusals(lib):
    names = "q qs cache table tstride lens scale out os lse B Hq ws wsb stream".split()
    good = [P, 1024, _cache(), P, 4, P, 0.1, P, 1024, P, 2, 8, P, 1 << 30, None]
    inv, mis = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_MISALIGNED
    _refuses(lib.moe_attn_decode, names, good, [
        (dict(q=None), inv), (dict(cache=None), inv), (dict(table=None), inv), (dict(lens=None), inv),
        (dict(out=None), inv), (dict(ws=None), inv), (dict(tstride=0), inv), (dict(B=-1), inv),
        (dict(Hq=9), inv), (dict(scale=0.0), inv), (dict(scale=-1.0), inv),
        (dict(scale=float("inf")), inv), (dict(scale=float("nan")), inv), (dict(qs=1000), inv),
        (dict(os=1020), inv), (dict(q=P + 8), mis), (dict(out=P + 2), mis), (dict(lse=P + 2), mis),
        (dict(lens=P + 1), mis), (dict(wsb=16), moe.MOE_ERR_WORKSPACE_TOO_SMALL)])


def test_prefill_refusals(lib):
    names = "q qs k ks v vs cuq cuk B Tq Tk Hq Hkv D causal scale out os lse ws wsb stream".split()
    good = [P, 1024, P, 256, P, 256, P, P, 2, 50, 60, 8, 2, 128, 1, 0.1, P, 1024, None, P, 1 << 30, None]
    inv, mis = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_MISALIGNED
    _refuses(lib.moe_attn_prefill, names, good, [
        (dict(q=None), inv), (dict(k=None), inv), (dict(v=None), inv), (dict(cuq=None), inv),
        (dict(cuk=None), inv), (dict(out=None), inv), (dict(ws=None), inv), (dict(B=-1), inv),
        (dict(Tq=-1), inv), (dict(Tk=-1), inv), (dict(Hq=9), inv), (dict(D=32), inv),
        (dict(scale=-0.1), inv), (dict(qs=512), inv), (dict(ks=252), inv), (dict(os=1028), inv),
        (dict(k=P + 8), mis), (dict(v=P + 2), mis), (dict(cuk=P + 2), mis), (dict(ws=P + 16), mis),
        (dict(wsb=16), moe.MOE_ERR_WORKSPACE_TOO_SMALL)])


def test_no_gpu_reports_unsupported_device(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lib.moe_attn_decode(P, 1024, _cache(), P, 4, P, 0.1, P, 1024, None, 2, 8, P, 1 << 30,
                               None) == moe.MOE_ERR_UNSUPPORTED_DEVICE
