"""moe_attn_decode and moe_attn_prefill against a plain 64-bit attention;
attn_util.attention derives the bounds."""
import pytest

from tests import attn_util as au

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- decode
def _decode(lens, Hq, Hkv, D, fp8, page, seed=0, scale=None, poison=True, q_scale=1.0):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    B = len(lens)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = au.make_cache(seed, pages, Hkv, page, D, fp8)
    table = au.make_table(seed + 1, lens, page, pages, 0x7fffffff)
    if poison:   # what no sequence holds is NaN, infinite scales too
        used = torch.zeros(pages, page, dtype=torch.bool)
        t = table.cpu()
        for b, n in enumerate(lens):
            for j in range(-(-n // page)):
                used[t[b, j], :min(page, n - j * page)] = True
        free = ~used.cuda()[:, None, None, :].expand(pages, Hkv, 2, page)
        bits = cache.data.view(torch.uint8 if fp8 else torch.int16)
        bits[free] = 0x7f if fp8 else 0x7fc0
        if fp8:
            cache.scales[free] = float("inf")
    wide = au.randn(seed + 2, B, Hq + 1, D, scale=q_scale)
    q = wide[:, :Hq]
    scale = D ** -0.5 if scale is None else scale
    ws = moe.AttnWorkspace("cuda", "decode", B, B, Hq, Hkv, D)
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = []
    for _ in range(2):
        ws.buf.random_(0, 255)      # a workspace need not be initialised
        hold = torch.full((B, Hq + 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
        out, lse = moe.attn_decode(q, cache, table, lens_d, scale=scale, out=hold[:, :Hq], lse=True,
                                   workspace=ws)
        assert au.status(ws) == (moe.MOE_OK, 0)
        assert (hold[:, Hq:] == 9.0).all()
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for b, n in enumerate(lens):
        k, v = au.cached_rows(cache, table, b, n)
        ref, rl, tol, tl = au.attention(q[b:b + 1], k, v, scale,
                                        torch.full((1,), n, device="cuda"))
        au.check(outs[0][0][b:b + 1], ref, tol, f"out {b}")
        au.check(outs[0][1][b:b + 1], rl, tl, f"lse {b}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ([1], 1, 1, 64, 16), ([0], 8, 1, 128, 16), ([0, 1, 2, 0, 15, 16, 17], 8, 2, 128, 16),
    ([31, 32, 33, 63, 64, 65, 127, 128, 129, 0], 6, 2, 64, 32),
    ([517], 64, 8, 128, 16), ([700, 1, 300], 15, 3, 128, 256), ([255, 256, 257], 32, 1, 64, 64),
    ([40, 900], 20, 1, 128, 128), ([333], 96, 2, 128, 16), ([20011], 16, 2, 128, 64),
    ([3000 + 7 * i for i in range(9)], 8, 8, 64, 16)])
def test_decode(gpu, lens, Hq, Hkv, D, page, fp8):
    _decode(lens, Hq, Hkv, D, fp8, page)


@pytest.mark.parametrize("D", [64, 128])
def test_groups_of_more_heads_than_a_tile(gpu, D):
    """150 query heads over one: several head tiles, the last one partly filled."""
    _decode([700, 0, 33], 150, 1, D, False, 16, seed=11)
    _decode([700, 0, 33], 150, 1, D, True, 64, seed=12)
    _prefill([3, 40], [300, 40], 150, 1, D, True, seed=13)
    _prefill([2], [3000], 150, 1, D, False, seed=14)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_many_sequences(gpu, fp8):
    _decode([(37 * i * i) % 411 for i in range(200)], 8, 4, 128, fp8, 16, seed=3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_few_long_sequences(gpu, D, fp8):
    """Few pairs over all of the GPU, empty sequences between them."""
    _decode([0, 9001, 0, 20037, 1], 16, 1, D, fp8, 64, seed=21)
    _decode([4111, 0], 5, 1, D, fp8, 32, seed=22)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_score_ranges(gpu, fp8):
    """Scores from one dominating key to all but equal, wide and tiny q."""
    _decode([600, 77], 8, 2, 128, fp8, 16, seed=4, scale=3.0)
    _decode([600, 77], 8, 2, 128, fp8, 16, seed=5, q_scale=1e-20)
    _decode([600, 77], 8, 2, 128, fp8, 16, seed=6, q_scale=1e6, scale=1e-7)


def test_decode_uneven_value_scales(gpu):
    """fp8 values whose scales differ by many orders, with the largest first,
    last or in between, and zero rows."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    n, H, D, page = 400, 2, 128, 16
    for seed in range(3):
        cache = au.make_cache(seed, 26, H, page, D, True)
        g = torch.Generator(device="cuda").manual_seed(seed)
        e = torch.randint(-30, 1, cache.scales[:, :, 1].shape, generator=g, device="cuda").float()
        cache.scales[:, :, 1] *= torch.exp2(e)
        cache.scales[3, :, 1, 5] = 0
        table = au.make_table(seed, [n], page, 26, 0)
        q = au.randn(seed + 9, 1, 4, D)
        out, lse = moe.attn_decode(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                                   lse=True)
        k, v = au.cached_rows(cache, table, 0, n)
        ref, rl, tol, tl = au.attention(q, k, v, D ** -0.5, torch.full((1,), n, device="cuda"))
        au.check(out, ref, tol, "out")
        au.check(lse, rl, tl, "lse")


def test_decode_offsets_beyond_32_bits(gpu):
    """A cache of more than 2^32 bytes, the sequence in its last pages."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    pages, H, D, page = 140000, 1, 128, 64
    data = torch.empty(pages, H, 2, page, D, dtype=torch.bfloat16, device="cuda")
    assert data.numel() * 2 > 2 ** 32
    cache = moe.KVCache(data)
    use = torch.tensor([pages - 1, pages - 3, 2], dtype=torch.int32, device="cuda")
    data[use.long()] = au.randn(1, 3, H, 2, page, D)
    q = au.randn(2, 1, 4, D)
    n = 150
    out, lse = moe.attn_decode(q, cache, use[None].contiguous(),
                               torch.tensor([n], dtype=torch.int32, device="cuda"), lse=True)
    k, v = au.cached_rows(cache, use[None], 0, n)
    ref, rl, tol, tl = au.attention(q, k, v, D ** -0.5, torch.full((1,), n, device="cuda"))
    au.check(out, ref, tol, "out")
    au.check(lse, rl, tl, "lse")


def test_decode_bad_tables(gpu):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    cache = au.make_cache(5, 6, 2, 16, 64, False)
    q = au.randn(6, 3, 4, 64)
    ws = moe.AttnWorkspace("cuda", "decode", 3, 3, 4, 2, 64)
    good = [[0, 1], [2, 3], [4, 5]]
    ref = None
    for table, lens, want in [(good, [20, 32, 7], None), ([[0, 1], [2, 6], [4, 5]], [20, 32, 7], 1),
                              ([[0, 1], [-1, 3], [4, 5]], [20, 32, 7], 1),
                              (good, [20, 33, 7], 1), (good, [20, -1, 7], 1), (good, [20, 32, 7], None)]:
        out = moe.attn_decode(q, cache, torch.tensor(table, dtype=torch.int32, device="cuda"),
                              torch.tensor(lens, dtype=torch.int32, device="cuda"), workspace=ws)
        st = au.status(ws)
        assert st == ((moe.MOE_OK, 0) if want is None else (moe.MOE_ERR_DEVICE_BAD_INDEX, want))
        if ref is None:
            ref = out
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    assert torch.equal(out, ref)


def test_decode_on_another_stream_and_in_a_graph(gpu):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    lens = [100, 0, 2000]
    cache = au.make_cache(5, 140, 2, 16, 128, True)
    table = au.make_table(6, lens, 16, 140, 0)
    q = au.randn(7, 3, 16, 128)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref = moe.attn_decode(q, cache, table, n)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = moe.attn_decode(q, cache, table, n, stream=st)
    st.synchronize()
    assert torch.equal(out, ref)
    ws = moe.AttnWorkspace("cuda", "decode", 3, 3, 16, 2, 128)
    hold = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.attn_decode(q, cache, table, n, out=hold, workspace=ws)
    for lens in ([100, 0, 2000], [1, 900, 0]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        table.copy_(_pad(au.make_table(8, lens, 16, 140, 0), table.shape[1]))
        hold.fill_(5.0)
        graph.replay()
        assert torch.equal(hold, moe.attn_decode(q, cache, table, n))


def _pad(t, n):
    import torch
    out = torch.zeros(t.shape[0], n, dtype=t.dtype, device=t.device)
    out[:, :t.shape[1]] = t
    return out


# ---------------------------------------------------------------- prefill
def _prefill(nq, nk, Hq, Hkv, D, causal, seed=0, scale=None, fused=True, edit=None):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    B, Tq, Tk = len(nq), sum(nq), sum(nk)
    pre = lambda x: torch.tensor([0] + list(torch.tensor(x).cumsum(0)), dtype=torch.int32, device="cuda")
    cu_q, cu_k = pre(nq), pre(nk)
    q = au.randn(seed, Tq, Hq + 1, D)[:, :Hq]
    kv = au.randn(seed + 1, Tk, 2 * Hkv + 1, D)
    k, v = kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if edit:
        edit(q, k, v)
    scale = D ** -0.5 if scale is None else scale
    ws = moe.AttnWorkspace("cuda", "prefill", B, Tq, Hq, Hkv, D)
    outs = []
    for _ in range(2):
        ws.buf.random_(0, 255)
        hold = torch.full((Tq, Hq + 1, D), 9.0, dtype=torch.bfloat16, device="cuda")
        out, lse = moe.attn_prefill(q, k, v, cu_q, cu_k, causal=causal, scale=scale,
                                    out=hold[:, :Hq], lse=True, workspace=ws)
        assert au.status(ws) == (moe.MOE_OK, 0)
        assert (hold[:, Hq:] == 9.0).all()
        outs.append((out, lse))
    assert torch.equal(outs[0][0].view(torch.int16), outs[1][0].view(torch.int16))
    a = c = 0
    for b in range(B):
        limit = (torch.arange(nq[b], device="cuda") + nk[b] - nq[b] + 1 if causal else
                 torch.full((nq[b],), nk[b], device="cuda"))
        ref, rl, tol, tl = au.attention(q[a:a + nq[b]], k[c:c + nk[b]], v[c:c + nk[b]], scale, limit)
        if not (edit and b in edit.poisoned):
            au.check(outs[0][0][a:a + nq[b]], ref, tol, f"out {b}")
            au.check(outs[0][1][a:a + nq[b]], rl, tl, f"lse {b}")
        a, c = a + nq[b], c + nk[b]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D", [
    ([1], [1], 1, 1, 64), ([1, 1, 1], [1, 200, 129], 4, 2, 128),
    ([127, 128, 129], [127, 128, 129], 4, 1, 128), ([255, 1, 256, 257], [255, 1, 256, 257], 2, 2, 64),
    ([300, 0, 40], [300, 0, 40], 6, 2, 128), ([64, 5], [1000, 777], 5, 5, 64),
    ([200, 150], [70, 0], 3, 1, 128), ([0, 90], [50, 90], 8, 1, 64),
    ([600, 33, 7], [900, 33, 500], 4, 4, 128), ([1024], [1024], 8, 2, 128),
    ([513], [2100], 16, 1, 64)])
def test_prefill(gpu, nq, nk, Hq, Hkv, D, causal):
    _prefill(nq, nk, Hq, Hkv, D, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,Hq,Hkv,D", [
    ([16], [15016], 16, 2, 128), ([1, 40, 3], [9000, 1030, 20011], 8, 2, 64),
    ([3000], [2500], 2, 1, 64), ([700, 5], [700, 7003], 5, 1, 128), ([1], [30000], 1, 1, 128)])
def test_prefill_few_rows_over_many_keys(gpu, nq, nk, Hq, Hkv, D, causal):
    """Key ranges that are cut into parts and joined."""
    _prefill(nq, nk, Hq, Hkv, D, causal, seed=8)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_ranges_in_two_to_eight_parts(gpu, D):
    _prefill([90, 0, 41], [3000, 100, 2500], 16, 2, D, True, seed=31)
    _prefill([130], [4000], 9, 3, D, False, seed=32)
    _prefill([33, 5], [8000, 6500], 16, 4, D, True, seed=33)


def test_prefill_contiguous_rows_and_scales(gpu):
    _prefill([300, 17], [300, 400], 4, 2, 128, True, seed=2, scale=2.0, fused=False)
    _prefill([300, 17], [300, 400], 4, 2, 64, False, seed=3, scale=1e-6, fused=False)


def test_prefill_many_sequences(gpu):
    nq = [(13 * i * i) % 61 for i in range(150)]
    _prefill(nq, [n + (i % 7) * 9 for i, n in enumerate(nq)], 2, 1, 128, True, seed=4)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_other_sequences_do_not_matter(gpu, D):
    """NaN and infinities in one sequence reach no other one."""
    def edit(q, k, v):
        for t, n0, n1 in ((q, 100, 150), (k, 100, 150), (v, 100, 150)):
            t[n0:n1] = float("nan")
            t[n0 + 3, :, ::3] = float("inf")
    edit.poisoned = {1}
    _prefill([100, 50, 77], [100, 50, 77], 4, 2, D, True, seed=5, edit=edit)
    _prefill([100, 50, 77], [100, 50, 77], 4, 2, D, False, seed=5, edit=edit)
    # (key ranges in parts)
    _prefill([100, 50, 7], [100, 50, 5007], 4, 2, D, True, seed=5, edit=edit)


def test_prefill_extreme_scores(gpu):
    """Rows whose scores are far below zero, and far above, and equal."""
    def edit(q, k, v):
        q[:40] = 30.0
        k[:200] = -30.0
        q[40:80] = 0
        k[100:120] = 30.0
    edit.poisoned = set()
    _prefill([260], [260], 2, 1, 128, True, seed=6, edit=edit)


def test_prefill_bad_sequences(gpu):
    """A bad sequence is reported and not written; the others are as before."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    q, k, v = au.randn(1, 100, 4, 64), au.randn(2, 100, 2, 64), au.randn(3, 100, 2, 64)
    ws = moe.AttnWorkspace("cuda", "prefill", 3, 100, 4, 2, 64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    good = i32([0, 30, 60, 100])
    ref = moe.attn_prefill(q, k, v, good, good, workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)
    for cu_q, cu_k, bad, fine in [
            ([0, 30, 60, 101], [0, 30, 60, 100], 2, (0, 60)),
            ([0, 30, 60, 100], [0, 30, 60, 2 ** 31 - 1], 2, (0, 60)),
            ([-5, 30, 60, 100], [0, 30, 60, 100], 0, (30, 100)),
            ([0, 30, 60, 100], [0, 30, 20, 100], 1, (0, 30))]:
        out = torch.full_like(q, 3.0)
        moe.attn_prefill(q, k, v, i32(cu_q), i32(cu_k), out=out, workspace=ws)
        assert au.status(ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, bad)
        assert torch.equal(out[fine[0]:fine[1]], ref[fine[0]:fine[1]])
        if bad == 2:
            assert (out[60:] == 3.0).all()
    moe.attn_prefill(q, k, v, good, good, workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)


def test_prefill_over_a_read_back_context(gpu):
    """A chunk of a prompt over its cached context (bf16 cache) is the same as
    the whole prompt's last rows."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    n, ctx, Hq, Hkv, D, page = 500, 350, 8, 2, 128, 16
    q, k, v = au.randn(1, n, Hq, D), au.randn(2, n, Hkv, D), au.randn(3, n, Hkv, D)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    whole = moe.attn_prefill(q, k, v, i32([0, n]), i32([0, n]))
    cache = moe.KVCache.empty(40, Hkv, D, page, fp8=False)
    table = au.make_table(4, [n], page, 40, 0)
    t = torch.arange(n, device="cuda")
    slots = (table[0].long()[t // page] * page + t % page).to(torch.int32)
    moe.qk_rope_append(q, k, v, None, None, cache, slots)
    kc, vc = moe.kv_gather(cache, table, i32([0, n]), n)
    assert torch.equal(kc, k) and torch.equal(vc, v)
    part = moe.attn_prefill(q[ctx:], kc, vc, i32([0, n - ctx]), i32([0, n]))
    ref, _, tol, _ = au.attention(q[ctx:], k, v, D ** -0.5, torch.arange(ctx, n, device="cuda") + 1)
    au.check(part, ref, tol, "chunk")
    au.check(whole[ctx:], ref, tol, "whole")
    # and one decode step is the last row
    one = moe.attn_decode(q[-1:], cache, table, i32([n]))
    au.check(one, ref[-1:], tol[-1:], "decode")


def test_python_refusals(gpu):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    cache = au.make_cache(5, 4, 2, 16, 64, False)
    q = au.randn(1, 2, 4, 64)
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    for bad in [dict(q=q.float()), dict(q=q.cpu()), dict(q=au.randn(1, 2, 4, 128)),
                dict(table=table.long()), dict(lens=lens[:1]), dict(lens=lens.cpu()),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))]:
        a = dict(q=q, table=table, lens=lens, **{})
        a.update(bad)
        with pytest.raises(ValueError):
            moe.attn_decode(a["q"], cache, a["table"], a["lens"])
    with pytest.raises(moe.MoeError) as e:
        moe.attn_decode(au.randn(1, 2, 3, 64), cache, table, lens)   # 3 heads over 2
    assert e.value.status == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(moe.MoeError) as e:
        moe.attn_decode(q, cache, table, lens, scale=0.0)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG
    small = moe.AttnWorkspace("cuda")
    with pytest.raises((ValueError, moe.MoeError)):
        moe.attn_prefill(q, q[:, :3], q[:, :3], lens, lens, workspace=small)
    with pytest.raises(ValueError):
        moe.KVCache(torch.zeros(2, 2, 2, 16, 64, device="cuda"))


# ---------------------------------------------------------------- bounded waits
_STALL_CHILD = r"""
import json, sys, time
sys.path.insert(0, sys.argv[1])
import torch
import quantized_moe_expert_align_gb300 as moe
from tests import attn_util as au
res = []
for D in (64, 128):
    for fp8 in (False, True):
        cache = au.make_cache(1, 40, 2, 16, D, fp8)
        ws = moe.AttnWorkspace("cuda", "decode", 2, 2, 8, 2, D)
        table = au.make_table(2, [300, 40], 16, 40, 0)
        t0 = time.time()
        moe.attn_decode(au.randn(3, 2, 8, D), cache, table,
                        torch.tensor([300, 40], dtype=torch.int32, device="cuda"), workspace=ws)
        res.append([*au.status(ws), time.time() - t0])
    ws = moe.AttnWorkspace("cuda", "prefill", 2, 700, 8, 2, D)
    q, k = au.randn(4, 700, 8, D), au.randn(5, 700, 2, D)
    cu = torch.tensor([0, 650, 700], dtype=torch.int32, device="cuda")
    t0 = time.time()
    moe.attn_prefill(q, k, k, cu, cu, workspace=ws)
    res.append([*au.status(ws), time.time() - t0])
# the context is still usable afterwards
y = (torch.arange(1024, device="cuda", dtype=torch.float32) * 2).sum().item()
print(json.dumps({"res": res, "y": y}))
"""


def test_bounded_waits_run_out(gpu):
    """With the failure-path switch the kernels issue no copies: their waits
    give up after about a second, the status word says so, the kernels wind
    down and the context stays usable.  The switch is read once per process,
    so in a child."""
    import json
    import os
    import subprocess
    import sys

    import quantized_moe_expert_align_gb300 as moe
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _STALL_CHILD, root],
                       env=dict(os.environ, MOE_ATTN_TEST_NO_COPIES="1"), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["y"] == float(sum(2 * i for i in range(1024)))
    for st, detail, secs in out["res"]:
        assert st == moe.MOE_ERR_DEVICE_TIMEOUT and detail >= 1 and secs < 30
