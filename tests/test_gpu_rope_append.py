"""moe_qk_rope_append and moe_kv_gather against plain 64-bit forms.

Tolerances: the norm, the rotation and the scale are a handful of 32-bit
operations (2^-20 of the rotated pair's size covers them), then one rounding:
bf16 2^-8 relative, e4m3 half a step, 2^-4 relative or 2^-10 of the scale."""
import pytest

from tests import attn_util as au

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _rows64(x, w, cs, pos, inter):
    import torch
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()
    size = x.abs()
    rot = cs.shape[1] if cs is not None else 0
    if rot:
        h = rot // 2
        c, s = cs.double()[pos.long(), None, :h], cs.double()[pos.long(), None, h:]
        i = torch.arange(h, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + h)
        y, size = x.clone(), size.clone()
        y[..., ia] = x[..., ia] * c - x[..., ib] * s
        y[..., ib] = x[..., ib] * c + x[..., ia] * s
        size[..., ia] = size[..., ib] = x[..., ia].abs() + x[..., ib].abs()
        x = y
    return x, size


def _call(T, Hq, Hkv, D, rot, inter, norm, fp8, page, k_out, seed=0, x_scale=1.0, fused=True,
          in_place=False):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    qkv = au.randn(seed, T, Hq + 2 * Hkv, D, scale=x_scale)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw = (1 + 0.1 * au.randn(seed + 1, D, dtype=torch.float32)).bfloat16() if norm else None
    kw = (1 + 0.1 * au.randn(seed + 2, D, dtype=torch.float32)).bfloat16() if norm else None
    max_pos = 5000
    cs = moe.rope_table(max_pos, rot) if rot else None
    g = torch.Generator(device="cuda").manual_seed(seed + 3)
    pos = torch.randint(0, max_pos, (T,), generator=g, device="cuda", dtype=torch.int32)
    pages = T // page + 2
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 2:
        slots[1] = -1
    cache = au.make_cache(seed + 4, pages, Hkv, page, D, fp8)
    before = cache.data.view(torch.uint8).clone(), None if cache.scales is None else cache.scales.clone()
    ref_q, size_q = _rows64(q, qw, cs, pos, inter)
    ref_k, size_k = _rows64(k, kw, cs, pos, inter)
    ref_v = v.double()
    ws = moe.AttnWorkspace("cuda")
    out = moe.qk_rope_append(q, k, v, cs, pos, cache, slots, q_norm=qw, k_norm=kw, eps=EPS,
                             interleaved=inter, q_out=q if in_place else None,
                             k_out=(k if in_place else True) if k_out else None, workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)
    q_out, k_got = out if k_out else (out, None)
    au.check(q_out, ref_q, au.U_BF16 * ref_q.abs() + 2.0 ** -20 * size_q + 1e-30, "q")
    if k_out:
        au.check(k_got, ref_k, au.U_BF16 * ref_k.abs() + 2.0 ** -20 * size_k + 1e-30, "k_out")
    # the cache: what was written, and that nothing else was
    rows = torch.stack([ref_k, ref_v], 2)
    size = torch.stack([size_k, ref_v.abs()], 2)
    put = slots >= 0
    sl = slots[put].long()
    pg, off = sl // page, sl % page
    raw = cache.data.view(torch.uint8)
    got = raw[pg, :, :, off].view(cache.data.dtype).double()
    if fp8:
        sc = cache.scales[pg, :, :, off].double()
        amax = rows[put].abs().amax(-1)
        au.check(sc, amax / 448, 2.0 ** -19 * size[put].amax(-1) / 448 + 1e-40, "scales")
        au.check(got * sc[..., None], rows[put],
                 2.0 ** -4 * rows[put].abs() + 2.0 ** -10 * sc[..., None] + 2.0 ** -18 * size[put],
                 "cached values")
        rest = cache.scales.clone()
        rest[pg, :, :, off] = before[1][pg, :, :, off]
        assert torch.equal(rest, before[1])
    else:
        au.check(got, rows[put], au.U_BF16 * rows[put].abs() + 2.0 ** -20 * size[put] + 1e-30, "cached")
    raw = raw.clone()
    raw[pg, :, :, off] = before[0][pg, :, :, off]
    assert torch.equal(raw, before[0])


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm,fp8,page,k_out", [
    (1, 64, 8, 128, 128, False, True, True, 16, False),
    (1, 1, 1, 64, 64, True, True, False, 16, True),
    (90, 32, 4, 128, 64, True, True, False, 16, True),
    (33, 15, 5, 64, 32, False, True, True, 32, True),
    (33, 7, 7, 64, 16, True, False, True, 256, False),
    (17, 48, 3, 128, 0, False, True, True, 64, True),
    (5, 8, 2, 128, 32, False, False, False, 128, True),
    (1500, 10, 2, 128, 128, True, True, True, 64, True),
    (2048, 32, 4, 64, 64, False, True, False, 16, False),
])
def test_append(gpu, T, Hq, Hkv, D, rot, inter, norm, fp8, page, k_out):
    _call(T, Hq, Hkv, D, rot, inter, norm, fp8, page, k_out)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_in_place_and_wide_values(gpu, fp8):
    _call(70, 12, 4, 128, 128, False, True, fp8, 16, True, seed=7, in_place=True)
    _call(70, 12, 4, 128, 64, True, False, fp8, 16, True, seed=8, x_scale=1e15, fused=False)
    _call(70, 12, 4, 64, 64, False, False, fp8, 16, True, seed=9, x_scale=1e-12, fused=False)


def test_append_special_rows(gpu):
    """A zero row has scale 0 and codes 0; a row with an infinity or a NaN a
    NaN scale; neither touches its neighbours."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    T, H, D = 4, 2, 128
    x = au.randn(1, T, H, D)
    x[0, 0] = 0
    x[1, 0, 5] = float("inf")
    x[2, 1, 127] = float("nan")
    cache = au.make_cache(2, 2, H, 16, D, True)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    moe.qk_rope_append(x, x, x, None, None, cache, slots)
    sc = cache.scales[0, :, :, :T].permute(2, 0, 1)      # [T][H][2]
    codes = cache.data[0, :, :, :T].float().permute(2, 0, 1, 3)
    assert (sc[0, 0] == 0).all() and (codes[0, 0] == 0).all()
    assert sc[1, 0].isnan().all() and sc[2, 1].isnan().all()
    fine = torch.ones(T, H, dtype=torch.bool, device="cuda")
    fine[1, 0] = fine[2, 1] = False
    back = codes * sc[..., None]
    assert torch.isfinite(back[fine]).all()
    assert ((back[fine] - x[fine][:, None].float()).abs() <=
            2.0 ** -4 * x[fine][:, None].float().abs() + 2.0 ** -9 * sc[fine][..., None]).all()


def test_append_tiny_rows(gpu):
    """Rows whose largest magnitude is near or below 2^-128, with zeros among
    them: codes stay numbers, values stay within half a step."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    H, D = 2, 64
    sizes = [2.0 ** -110, 2.0 ** -118, 2.0 ** -121, 2.0 ** -127, 2.0 ** -133]
    x = torch.zeros(len(sizes), H, D, dtype=torch.float64, device="cuda")
    for t, size in enumerate(sizes):
        x[t, :, 3] = size
        x[t, :, 40] = -size
        x[t, 0, 8] = size / 4
    x = x.bfloat16()
    cache = au.make_cache(3, 1, H, 16, D, True)
    slots = torch.arange(len(sizes), dtype=torch.int32, device="cuda")
    moe.qk_rope_append(x, x, x, None, None, cache, slots)
    sc = cache.scales[0, :, :, :len(sizes)].permute(2, 0, 1).double()
    codes = cache.data[0, :, :, :len(sizes)].float().permute(2, 0, 1, 3).double()
    want = x.double()[:, :, None].expand(-1, -1, 2, -1)
    au.check(codes * sc[..., None], want,
             (2.0 ** -4 + 2.0 ** -20) * want.abs() + 2.0 ** -10 * sc[..., None], "values")
    assert (codes[want == 0] == 0).all()


def test_append_without_a_cache_and_without_tokens(gpu):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    x = au.randn(1, 3, 4, 64)
    cs = moe.rope_table(16, 64)
    pos = torch.tensor([0, 15, 3], dtype=torch.int32, device="cuda")
    q, k = moe.qk_rope_append(x, x, x, cs, pos, None, None, k_out=True)
    assert torch.equal(q, k)
    ref, size = _rows64(x, None, cs, pos, False)
    au.check(q, ref, au.U_BF16 * ref.abs() + 2.0 ** -20 * size, "q")
    none = moe.qk_rope_append(x[:0], x[:0], x[:0], cs, pos[:0], None, None)
    assert none.shape == (0, 4, 64)
    torch.cuda.synchronize()


def test_append_bad_indexes(gpu):
    """A bad position or slot leaves its token out and is reported; the next
    call reports anew."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    T, H, D = 6, 2, 128
    x = au.randn(3, T, H, D)
    cs = moe.rope_table(32, 128)
    cache = au.make_cache(4, 1, H, 16, D, False)
    before = cache.data.clone()
    pos = torch.tensor([0, 1, 32, 3, -1, 5], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 16, 2, -2, 4, 5], dtype=torch.int32, device="cuda")
    q = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = moe.AttnWorkspace("cuda")
    moe.qk_rope_append(x, x, x, cs, pos, cache, slots, q_out=q, workspace=ws)
    assert au.status(ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, 1)
    assert (q[1:5] == 7.0).all() and not (q[0] == 7.0).all() and not (q[5] == 7.0).all()
    same = (cache.data == before).all(-1).all(0).all(0).all(0)   # [page]
    assert [i for i in range(16) if not same[i]] == [0, 5]
    pos.zero_()
    slots.copy_(torch.arange(T, dtype=torch.int32))
    moe.qk_rope_append(x, x, x, cs, pos, cache, slots, q_out=q, workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)


def test_rope_table(gpu):
    import math
    import torch
    import quantized_moe_expert_align_gb300 as moe
    rot, base = 64, 10000.0
    plain = moe.rope_table(100, rot)
    for p, i in [(0, 0), (99, 0), (57, 13), (99, 31)]:
        a = p * base ** (-2 * i / rot)
        assert abs(plain[p, i].item() - math.cos(a)) < 1e-7
        assert abs(plain[p, rot // 2 + i].item() - math.sin(a)) < 1e-7
    # linear interpolation: position 4 p of the scaled table is position p
    assert torch.allclose(moe.rope_table(400, rot, factor=4.0)[::4], plain, atol=1e-6)
    # by parts: the fastest pair keeps its frequency, the slowest is divided
    m = 0.1 * math.log(4.0) + 1.0
    parts = moe.rope_table(100, rot, factor=4.0, original_max=4096) / m
    assert torch.allclose(parts[:, 0], plain[:, 0], atol=1e-6)
    slow = base ** (-2 * 31 / rot) / 4.0
    assert abs(parts[99, 31].item() - math.cos(99 * slow)) < 1e-6


@pytest.mark.parametrize("lens,Hkv,D,fp8,page", [
    ([1], 1, 64, False, 16), ([0, 1, 15, 16, 17, 0], 4, 128, True, 16),
    ([1000, 3, 257], 3, 128, False, 64), ([130, 64, 2000], 8, 64, True, 32),
    ([700], 2, 128, True, 256)])
def test_gather(gpu, lens, Hkv, D, fp8, page):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    pages = sum(-(-n // page) for n in lens) + 3
    cache = au.make_cache(5, pages, Hkv, page, D, fp8)
    table = au.make_table(6, lens, page, pages, 0x7fffffff)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    total = sum(lens)
    wide = torch.full((total, 2 * Hkv + 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = moe.AttnWorkspace("cuda")
    k, v = moe.kv_gather(cache, table, cu, total, k_out=wide[:, :Hkv], v_out=wide[:, Hkv:2 * Hkv],
                         workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)
    ref = [au.cached_rows(cache, table, b, n) for b, n in enumerate(lens)]
    # code * scale in 32 bits, rounded to bf16: the same two roundings
    assert torch.equal(k, torch.cat([r[0] for r in ref]).float().bfloat16())
    assert torch.equal(v, torch.cat([r[1] for r in ref]).float().bfloat16())
    assert (wide[:, 2 * Hkv] == 3.0).all()


def test_gather_bad_tables(gpu):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    cache = au.make_cache(5, 4, 2, 16, 64, False)
    ws = moe.AttnWorkspace("cuda")
    cu = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device="cuda")
    k, _ = moe.kv_gather(cache, table, cu, 40, workspace=ws)
    assert au.status(ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, 1)
    assert (k[36:] == 0).all() and torch.equal(k[20:36], cache.data[2, :, 0].transpose(0, 1))
    for bad, detail in [([0, 33, 40], 0), ([0, 25, 20], 1), ([0, 20, 39], 2), ([1, 20, 40], 2)]:
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        table[1, 1] = 3
        moe.kv_gather(cache, table, cu, 40, workspace=ws)
        assert au.status(ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, detail)
