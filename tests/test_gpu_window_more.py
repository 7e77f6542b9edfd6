"""Windowed decode in copies of either size; windowed prompts: batches of more
sequences than a warp has lanes, planned and not cut, planned and cut; how far a
NaN in v can reach."""
import pytest

from tests import attn_util as au, serve_util as su
from tests.test_gpu_window import _decode, _prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,window,sinks", [(8, 2, 64, 4), (4, 4, 100, 0), (16, 1, 1, 1), (6, 2, 200, 130)])
def test_many_sequences_and_a_short_window(gpu, Hq, Hkv, window, sinks, D):
    """A plan, but no key range is cut: a block's rows see fewer than 1024 keys."""
    nq = [(i * 37) % 150 for i in range(70)]
    _prefill(nq, [n + (i * 53) % 400 for i, n in enumerate(nq)], window, sinks, Hq, Hkv, D, seed=21, lead=13)


@pytest.mark.parametrize("D", [64, 128])
def test_many_sequences_and_a_long_window(gpu, D):
    """A plan, with key ranges that may be cut."""
    nq = [(i * 37) % 40 for i in range(45)]
    nk = [n + (i * 211) % 900 for i, n in enumerate(nq)]
    nq[7], nk[7] = 33, 12000
    _prefill(nq, nk, 2500, 20, 8, 2, D, seed=22)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [1, 2])
@pytest.mark.parametrize("sinks,at", [(4, 7), (131, 134), (131, 143), (0, 0), (4, 600), (100, 1500), (17, 2047)])
def test_a_nan_in_v_reaches_no_further_than_stated(gpu, sinks, at, H, D):
    """255 rows before the first that sees it, 270 after the last."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    n, window = 3500 + 71, 200
    q, k, v = (au.randn(30 + i, n, H, D) for i in range(3))
    cu = su.i32([0, n])
    v[at] = 1.0
    ref = moe.attn_prefill(q, k, v, cu, cu, window=window, sinks=sinks)
    v[at] = float("nan")
    out = moe.attn_prefill(q, k, v, cu, cu, window=window, sinks=sinks)
    bad = torch.isnan(out).any(-1).any(-1)
    assert bad[at:at + window].all()
    lo, hi = max(0, at - 255), at + window - 1 + 270
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[lo:hi + 1] = False
    assert not bad[rest].any() and torch.equal(out[rest], ref[rest])
    # beside the NaN nothing else changes
    assert torch.equal(out[~bad], ref[~bad])


@pytest.mark.parametrize("D,page", [(64, 64), (64, 128), (64, 256), (128, 64), (128, 256)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (32, 2)])
@pytest.mark.parametrize("window,sinks", [(499, 4), (500, 4), (501, 70), (2299, 0), (2300, 5), (2301, 64)])
def test_decode_with_copies_of_32_and_64_rows(gpu, window, sinks, Hq, Hkv, D, page):
    """Both sides of the windows from which on copies over fp8 have 64 rows."""
    _decode([0, 1, 63, 64, 65, 570, 2400, 3000, 2305], window, sinks, Hq, Hkv, D, True, page, seed=window)
