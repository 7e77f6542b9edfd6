"""attn_decode and attn_prefill through a window with first tokens that stay
visible, against a plain 64-bit form; serve_util.seen_attention derives the
bounds."""
import pytest

from tests import attn_util as au, serve_util as su

pytestmark = pytest.mark.gpu

LENS = [0, 1, 5, 16, 17, 64, 100, 129, 300, 777, 2000]


def _decode(lens, window, sinks, Hq, Hkv, D, fp8, page, seed=0):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    B = len(lens)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = au.make_cache(seed, pages, Hkv, page, D, fp8)
    table = au.make_table(seed + 1, lens, page, pages, 0x7fffffff)
    t, keep, rows = table.cpu(), [], []
    for b, n in enumerate(lens):
        seen = [j for j in range(n) if j >= n - window or j < sinks]
        slots = [int(t[b, j // page]) * page + j % page for j in seen]
        rows.append(([j // page for j in seen], [j % page for j in seen]))
        keep += slots
        for p in range(-(-n // page)):  # pages that hold no seen key have gone
            if p not in {j // page for j in seen}:
                t[b, p] = -1 if p % 2 else 0x7ffffff0
    su.poison(cache, torch.tensor(keep, dtype=torch.long, device="cuda"))
    table = t.cuda()
    q = au.randn(seed + 2, B, Hq + 1, D)[:, :Hq]
    ws = moe.AttnWorkspace("cuda", "decode", B, B, Hq, Hkv, D)
    outs = []
    for _ in range(2):
        ws.buf.random_(0, 255)
        hold = torch.full((B, Hq + 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
        outs.append(moe.attn_decode(q, cache, table, su.i32(lens), out=hold[:, :Hq], lse=True, workspace=ws,
                                    window=window, sinks=sinks))
        assert au.status(ws) == (moe.MOE_OK, 0)
        assert (hold[:, Hq:] == 9.0).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for b, n in enumerate(lens):
        pg, off = (torch.tensor(x, dtype=torch.long, device="cuda") for x in rows[b])
        x = cache.data.view(torch.uint8 if fp8 else torch.int16)[table[b].long()[pg], :, :, off]
        x = x.view(cache.data.dtype).double()
        if fp8:
            x = x * cache.scales[table[b].long()[pg], :, :, off].double()[..., None]
        k, v = x[:, :, 0], x[:, :, 1]
        ref, rl, tol, tl = su.seen_attention(q[b:b + 1], k, v, D ** -0.5,
                                             torch.ones(1, len(pg), dtype=torch.bool, device="cuda"))
        au.check(outs[0][0][b:b + 1], ref, tol, f"out {b}")
        au.check(outs[0][1][b:b + 1], rl, tl, f"lse {b}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 8, 1, 16), (128, 16, 2, 64), (128, 15, 1, 256), (64, 40, 2, 32)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (16, 0), (100, 4), (128, 70), (1000, 1), (5000, 9000)])
def test_decode_window(gpu, window, sinks, D, Hq, Hkv, page, fp8):
    _decode(LENS, window, sinks, Hq, Hkv, D, fp8, page, seed=window + sinks)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_window_one_long_sequence(gpu, fp8):
    """The window's keys are spread over all of the GPU and joined."""
    _decode([30011], 8191, 5, 16, 2, 128, fp8, 64, seed=1)
    _decode([30011, 0, 9000], 4000, 0, 8, 8, 64, fp8, 16, seed=2)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_window_many_sequences(gpu, fp8):
    _decode([(37 * i * i) % 911 for i in range(200)], 130, 4, 8, 4, 128, fp8, 16, seed=3)


def test_decode_window_without_end_is_plain_decode(gpu):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    lens = [700, 3, 64]
    cache = au.make_cache(1, 60, 2, 16, 128, True)
    table, q = au.make_table(2, lens, 16, 60, 0), au.randn(3, 3, 16, 128)
    a = moe.attn_decode(q, cache, table, su.i32(lens))
    b = moe.attn_decode(q, cache, table, su.i32(lens), window=1 << 40, sinks=1 << 40)
    assert (a.float() - b.float()).abs().max() <= 2 * au.U_BF16 * a.float().abs().max()


# ---------------------------------------------------------------- prompts
def _prefill(nq, nk, window, sinks, Hq, Hkv, D, seed=0, lead=0):
    """lead: rows before the first sequence and behind the last that belong to none."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    B, Tq, Tk = len(nq), sum(nq) + 2 * lead, sum(nk) + 2 * lead
    qkv = au.randn(seed, max(Tq, Tk), Hq + 2 * Hkv, D)
    q, k, v = qkv[:Tq, :Hq], qkv[:Tk, Hq:Hq + Hkv], qkv[:Tk, Hq + Hkv:]
    if lead:
        for x in (k, v):
            x[:lead] = x[Tk - lead:] = float("nan")
    cu_q, cu_k = [n + lead for n in su.prefix(nq)], [n + lead for n in su.prefix(nk)]
    ws = moe.AttnWorkspace("cuda", "prefill", B, Tq, Hq, Hkv, D)
    outs = []
    for _ in range(2):
        ws.buf.random_(0, 255)
        hold = torch.full((Tq, Hq + 1, D), 9.0, dtype=torch.bfloat16, device="cuda")
        outs.append(moe.attn_prefill(q, k, v, su.i32(cu_q), su.i32(cu_k), out=hold[:, :Hq], lse=True,
                                     workspace=ws, window=window, sinks=sinks))
        assert au.status(ws) == (moe.MOE_OK, 0)
        assert (hold[:, Hq:] == 9.0).all()
        assert lead == 0 or ((hold[:lead] == 9.0).all() and (hold[Tq - lead:] == 9.0).all())
    own = slice(lead, Tq - lead)  # (what torch.empty holds in the others' lse stays)
    assert torch.equal(outs[0][0][own], outs[1][0][own]) and torch.equal(outs[0][1][own], outs[1][1][own])
    for b in range(B):
        i = slice(cu_q[b], cu_q[b + 1])
        j = slice(cu_k[b], cu_k[b + 1])
        pos = torch.arange(nq[b], device="cuda") + nk[b] - nq[b]
        ref, rl, tol, tl = su.seen_attention(q[i], k[j], v[j], D ** -0.5,
                                             su.window_seen(pos, nk[b], window, sinks))
        au.check(outs[0][0][i], ref, tol, f"out {b}")
        au.check(outs[0][1][i], rl, tl, f"lse {b}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (16, 2), (5, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (128, 4), (128, 0), (200, 130), (900, 128)])
def test_prefill_window(gpu, window, sinks, Hq, Hkv, D):
    _prefill([1, 0, 300, 129, 40], [1, 7, 300, 1000, 20], window, sinks, Hq, Hkv, D, seed=window)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_window_without_a_plan(gpu, D):
    """So few keys that every block finds its own items."""
    _prefill([3, 500], [200, 600], 100, 4, 8, 2, D, seed=1)
    _prefill([1000], [1000], 64, 3, 8, 1, D, seed=2)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_window_in_parts(gpu, D):
    """Few rows over long windows: key ranges are cut and joined."""
    _prefill([40], [9000], 5000, 4, 8, 2, D, seed=3)
    _prefill([100, 3], [12000, 7000], 6001, 300, 16, 2, D, seed=4)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_window_other_rows(gpu, D):
    """NaN in rows of no sequence, before and behind; their outputs stay."""
    _prefill([200, 77], [333, 77], 90, 4, 4, 2, D, seed=5, lead=50)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sinks", [4, 131])
def test_prefill_window_values_behind_the_first(gpu, D, sinks):
    """A NaN in v behind the first tokens stays with the rows about its
    window, although later rows copy the tile that holds it."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    n, window, H = 3000 + 71, 200, 2
    q, k, v = (au.randn(6 + i, n, H, D) for i in range(3))
    at = sinks + 3
    v[at] = float("nan")
    out = moe.attn_prefill(q, k, v, su.i32([0, n]), su.i32([0, n]), window=window, sinks=sinks)
    bad = torch.isnan(out).any(-1).any(-1).nonzero()[:, 0]
    assert bad.min() >= at - 255 and bad.max() <= at + window - 1 + 383
    assert torch.isnan(out[at:at + window]).all()
    v[at] = 1.0
    ref = moe.attn_prefill(q, k, v, su.i32([0, n]), su.i32([0, n]), window=window, sinks=sinks)
    assert torch.equal(out[at + window + 383:], ref[at + window + 383:])
