"""moe_attn_decode over an fp8 cache: a NaN code is NaN."""
import pytest

from tests import attn_util as au

pytestmark = pytest.mark.gpu


def _at(table, page, b, j):
    return int(table[b, j // page]), j % page


def _case(seed, lens, Hq, Hkv, D, fp8, page):
    import torch
    pages = sum(-(-n // page) for n in lens) + 2
    cache = au.make_cache(seed, pages, Hkv, page, D, fp8)
    table = au.make_table(seed + 1, lens, page, pages, 0)
    q = au.randn(seed + 2, len(lens), Hq, D)
    return cache, table, q, torch.tensor(lens, dtype=torch.int32, device="cuda")


HEADS = [(8, 1), (32, 2), (5, 1), (40, 1), (4, 4)]


@pytest.mark.parametrize("code", [0x7f, 0xff])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_nan_codes_in_values(gpu, Hq, Hkv, D, code):
    """A NaN code with a finite scale makes its column of its head NaN (and
    nothing else), wherever its key stands; past the end it does nothing."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    page = 32
    lens = [1, 40, 127, 700, 6001, 333, 16, 50]
    cache, table, q, n = _case(D + Hq, lens, Hq, Hkv, D, True, page)
    spots = [(0, 0, 3), (1, 39, D - 1), (2, 64, 0), (3, 17, 20), (3, 555, 33), (4, 5999, 47), (4, 0, 48)]
    raw = cache.data.view(torch.uint8)
    want = torch.zeros(len(lens), Hq, D, dtype=torch.bool, device="cuda")
    for i, (b, j, c) in enumerate(spots):
        pg, off = _at(table, page, b, j)
        h = i % Hkv
        raw[pg, h, 1, off, c] = code
        want[b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv), c] = True
    for b, j in ((6, 16), (7, 50)):   # the first key that is not there
        pg, off = _at(table, page, b, j)
        raw[pg, :, 1, off:] = code
    ws = moe.AttnWorkspace("cuda", "decode", len(lens), len(lens), Hq, Hkv, D)
    out, lse = moe.attn_decode(q, cache, table, n, lse=True, workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)
    assert torch.equal(out.isnan(), want)
    for b, m in enumerate(lens):
        k, v = au.cached_rows(cache, table, b, m)
        ref, rl, tol, tl = au.attention(q[b:b + 1], k, v, D ** -0.5, torch.full((1,), m, device="cuda"))
        assert torch.equal(ref.isnan()[0], want[b])
        fine = ~want[b]
        au.check(out[b][fine], ref[0][fine], tol[0][fine], f"out {b}")
        au.check(lse[b], rl[0], tl[0], f"lse {b}")


@pytest.mark.parametrize("D", [64, 128])
def test_nan_codes_in_keys(gpu, D):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    cache, table, q, n = _case(7, [50, 300], 16, 2, D, True, 16)
    pg, off = _at(table, 16, 1, 299)
    cache.data.view(torch.uint8)[pg, 1, 0, off, 9] = 0x7f
    out = moe.attn_decode(q, cache, table, n)
    assert out[1, 8:].isnan().all()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, :8]).all()
