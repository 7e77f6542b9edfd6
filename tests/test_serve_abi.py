"""The C ABI of serving over the paged cache without a GPU: exported symbols,
sizes, and the arguments that are refused before anything is launched."""
import ctypes
import os
import re

import pytest

import quantized_moe_expert_align_gb300 as moe
from quantized_moe_expert_align_gb300 import build

HEADER = os.path.join(build.INCLUDE, "moe_attn_serve.h")
P = 4096
INV, MIS, SMALL = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_MISALIGNED, moe.MOE_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load()


def _cache(**kw):
    f = dict(data=P, scales=None, type=moe.MOE_KV_BF16, num_pages=8, page_size=16, Hkv=2, D=128)
    f.update(kw)
    return ctypes.byref(moe.moe_kv_cache_t(*[f[n] for n, _ in moe.moe_kv_cache_t._fields_]))


def _refuses(fn, names, good, cases):
    for change, want in cases:
        a = dict(zip(names.split(), good))
        assert set(change) <= set(a)
        a.update(change)
        assert fn(*a.values()) == want, change


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_\w+)\s*\(", text)))
    assert len(names) == 7
    for n in names:
        assert hasattr(lib, n)


def test_workspace_sizes(lib):
    assert moe.moe_page_plan_workspace_size(0) >= 256
    assert moe.moe_page_plan_workspace_size(-1) == moe.moe_page_plan_workspace_size(65536) == 0
    assert moe.moe_attn_tree_workspace_size(1, 7, 64, 8, 128) >= 256
    for bad in [(-1, 8, 8, 8, 128), (70000, 8, 8, 8, 128), (1, -1, 8, 8, 128), (1, 8, 9, 8, 128),
                (1, 8, 8, 8, 96), (1, 1 << 30, 8, 8, 128), (1, 8, 2048, 8, 128)]:
        assert moe.moe_attn_tree_workspace_size(*bad) == 0


def test_page_plan_refusals(lib):
    names = ("ring cap state state_out table tstride page lens new dropped kept offsets window sinks B rows lens_out "
             "kept_out cu_q cu_k pos slots ws wsb stream")
    good = [P, 100, P, P, P, 8, 16, P, P, None, P, P, 100, 4, 2, 10, P, P, P, P, P, P, P, 1 << 20, None]
    _refuses(lib.moe_page_plan, names, good, [
        (dict(ring=None), INV), (dict(cap=0), INV), (dict(cap=1 << 30), INV), (dict(state=None), INV),
        (dict(state_out=None), INV), (dict(table=None), INV), (dict(tstride=0), INV), (dict(page=24), INV),
        (dict(page=8), INV), (dict(lens=None), INV), (dict(new=None), INV), (dict(kept=None), INV),
        (dict(kept_out=None), INV), (dict(window=-1), INV), (dict(sinks=-1), INV), (dict(B=-1), INV),
        (dict(B=65536), INV), (dict(rows=-1), INV), (dict(rows=(1 << 31) - 1), INV), (dict(lens_out=None), INV),
        (dict(cu_q=None), INV), (dict(pos=None), INV), (dict(slots=None), INV), (dict(ws=None), INV),
        (dict(ring=P + 2), MIS), (dict(offsets=P + 1), MIS), (dict(dropped=P + 3), MIS), (dict(slots=P + 2), MIS), (dict(ws=P + 128), MIS),
        (dict(wsb=256), SMALL)])


def test_decode_window_refusals(lib):
    names = "q qs cache table tstride lens window sinks scale out os lse B Hq ws wsb stream"
    good = [P, 1024, _cache(), P, 4, P, 100, 4, 0.1, P, 1024, P, 2, 8, P, 1 << 30, None]
    _refuses(lib.moe_attn_decode_window, names, good, [
        (dict(window=0), INV), (dict(window=-1), INV), (dict(sinks=-1), INV), (dict(q=None), INV),
        (dict(cache=None), INV), (dict(table=None), INV), (dict(lens=None), INV), (dict(scale=0.0), INV),
        (dict(qs=1000), INV), (dict(Hq=9), INV), (dict(out=P + 2), MIS), (dict(wsb=16), SMALL)])


def test_prefill_window_refusals(lib):
    names = "q qs k ks v vs cuq cuk B Tq Tk Hq Hkv D window sinks scale out os lse ws wsb stream"
    good = [P, 1024, P, 256, P, 256, P, P, 2, 50, 60, 8, 2, 128, 100, 4, 0.1, P, 1024, None, P, 1 << 30, None]
    _refuses(lib.moe_attn_prefill_window, names, good, [
        (dict(window=0), INV), (dict(sinks=-1), INV), (dict(q=None), INV), (dict(cuk=None), INV),
        (dict(Tk=-1), INV), (dict(D=32), INV), (dict(os=1028), INV), (dict(k=P + 8), MIS), (dict(wsb=16), SMALL)])


def test_tree_refusals(lib):
    names = "q qs cache table tstride lens cu tree scale out os lse B T Hq ws wsb stream"
    good = [P, 1024, _cache(), P, 4, P, P, P, 0.1, P, 1024, P, 2, 10, 8, P, 1 << 30, None]
    _refuses(lib.moe_attn_tree, names, good, [
        (dict(q=None), INV), (dict(cache=None), INV), (dict(cache=_cache(Hkv=3)), INV), (dict(table=None), INV),
        (dict(tstride=0), INV), (dict(lens=None), INV), (dict(cu=None), INV), (dict(tree=None), INV),
        (dict(scale=float("nan")), INV), (dict(out=None), INV), (dict(qs=1020), INV), (dict(os=512), INV),
        (dict(B=-1), INV), (dict(T=-1), INV), (dict(T=1 << 29), INV), (dict(Hq=9), INV), (dict(ws=None), INV),
        (dict(q=P + 8), MIS), (dict(tree=P + 4), MIS), (dict(cu=P + 2), MIS), (dict(lse=P + 2), MIS),
        (dict(wsb=16), SMALL)])


def test_accept_refusals(lib):
    names = "cache table tstride base accept B P ws wsb stream"
    good = [_cache(), P, 4, P, P, 2, 8, P, 256, None]
    _refuses(lib.moe_kv_accept, names, good, [
        (dict(cache=None), INV), (dict(table=None), INV), (dict(tstride=0), INV), (dict(base=None), INV),
        (dict(accept=None), INV), (dict(B=-1), INV), (dict(B=65536), INV), (dict(P=-1), INV), (dict(P=65), INV),
        (dict(ws=None), INV), (dict(base=P + 2), MIS), (dict(ws=P + 64), MIS), (dict(wsb=255), SMALL)])


def test_no_gpu_reports_unsupported_device(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lib.moe_kv_accept(_cache(), P, 4, P, P, 2, 8, P, 256, None) == moe.MOE_ERR_UNSUPPORTED_DEVICE
    assert lib.moe_attn_tree(P, 1024, _cache(), P, 4, P, P, P, 0.1, P, 1024, P, 2, 10, 8, P, 1 << 30,
                             None) == moe.MOE_ERR_UNSUPPORTED_DEVICE
