"""moe_attn_tree against a plain 64-bit attention, and moe_kv_accept."""
import random

import pytest

from tests import attn_util as au, serve_util as su

pytestmark = pytest.mark.gpu


def _masks(rng, n, kind):
    out = []
    for i in range(n):
        if kind == "chain":
            m = (2 << i) - 1
        elif kind == "tree":
            m = (out[rng.randrange(max(0, i - 4), i)] if i else 0) | 1 << i
        else:  # anything, also nothing and tokens that come later or do not exist
            m = rng.choice([0, rng.getrandbits(64), 1 << i, (1 << 64) - 1])
        out.append(m)
    return out


def _tree(lens, nodes, Hq, Hkv, D, fp8, page, kind="tree", seed=0, lead=0):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    rng = random.Random(seed)
    B, T = len(lens), sum(nodes) + 2 * lead
    pages = sum(-(-n // page) for n in lens) + 2
    cache = au.make_cache(seed, pages, Hkv, page, D, fp8)
    table = au.make_table(seed + 1, lens, page, pages, 0x7fffffff)
    t = table.cpu()
    keep = [int(t[b, j // page]) * page + j % page for b, n in enumerate(lens) for j in range(n)]
    su.poison(cache, torch.tensor(keep, dtype=torch.long, device="cuda"))
    masks = [_masks(rng, n, kind) for n in nodes]
    flat = [0] * lead + [m for ms in masks for m in ms] + [0] * lead
    tree = torch.tensor([m - (1 << 64) if m >> 63 else m for m in flat], dtype=torch.int64, device="cuda")
    cu = [n + lead for n in su.prefix(nodes)]
    q = au.randn(seed + 2, T, Hq + 1, D)[:, :Hq]
    ws = moe.AttnWorkspace("cuda", "tree", B, T, Hq, Hkv, D)
    outs = []
    for _ in range(2):
        ws.buf.random_(0, 255)
        hold = torch.full((T, Hq + 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
        outs.append(moe.attn_tree(q, cache, table, su.i32(lens), su.i32(cu), tree, out=hold[:, :Hq], lse=True,
                                  workspace=ws))
        assert au.status(ws) == (moe.MOE_OK, 0)
        assert (hold[:, Hq:] == 9.0).all()
        assert lead == 0 or ((hold[:lead] == 9.0).all() and (hold[T - lead:] == 9.0).all())
    assert torch.equal(outs[0][0][lead:T - lead], outs[1][0][lead:T - lead])
    assert torch.equal(outs[0][1][lead:T - lead], outs[1][1][lead:T - lead])
    for b, n in enumerate(lens):
        k, v = au.cached_rows(cache, table, b, n)
        seen = torch.ones(nodes[b], n, dtype=torch.bool, device="cuda")
        for i, m in enumerate(masks[b]):
            seen[i, n - nodes[b]:] = torch.tensor([m >> x & 1 > 0 for x in range(nodes[b])], device="cuda")
        i = slice(cu[b], cu[b + 1])
        ref, rl, tol, tl = su.seen_attention(q[i], k, v, D ** -0.5, seen)
        au.check(outs[0][0][i], ref, tol, f"out {b}")
        au.check(outs[0][1][i], rl, tl, f"lse {b}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["chain", "tree", "any"])
@pytest.mark.parametrize("lens,nodes,Hq,Hkv,D,page", [
    ([1], [1], 1, 1, 64, 16), ([1, 0, 2, 64], [1, 0, 2, 64], 8, 2, 128, 16),
    ([517], [7], 64, 8, 128, 16), ([300, 65, 20, 1000], [5, 64, 0, 33], 6, 2, 64, 32),
    ([700, 129, 128, 127], [16, 1, 9, 2], 15, 3, 128, 256), ([255, 256, 257], [64, 3, 17], 16, 1, 64, 64),
    ([40, 900], [40, 11], 20, 1, 128, 128), ([6000], [50], 16, 2, 128, 64), ([9000, 10], [2, 3], 4, 4, 64, 16)])
def test_tree(gpu, lens, nodes, Hq, Hkv, D, page, kind, fp8):
    _tree(lens, nodes, Hq, Hkv, D, fp8, page, kind, seed=len(lens) + nodes[0])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_many_sequences(gpu, D, fp8):
    lens = [(37 * i * i) % 811 for i in range(100)]
    _tree(lens, [min(n, (i * 7) % 20) for i, n in enumerate(lens)], 8, 2, D, fp8, 16, seed=3)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_of_no_sequence(gpu, fp8):
    _tree([100, 300], [10, 64], 8, 2, 128, fp8, 16, seed=4, lead=9)


@pytest.mark.parametrize("fp8", [False, True])
def test_groups_of_many_heads(gpu, fp8):
    _tree([200, 33], [12, 33], 150, 1, 64, fp8, 16, seed=5)


def test_single_token_is_decode(gpu):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    lens = [700, 3, 64]
    cache = au.make_cache(1, 60, 2, 16, 128, False)
    table, q = au.make_table(2, lens, 16, 60, 0), au.randn(3, 3, 16, 128)
    a = moe.attn_decode(q, cache, table, su.i32(lens))
    one = torch.ones(3, dtype=torch.int64, device="cuda")
    b = moe.attn_tree(q, cache, table, su.i32(lens), su.i32([0, 1, 2, 3]), one)
    assert (a.float() - b.float()).abs().max() <= 2 * au.U_BF16 * a.float().abs().max()


@pytest.mark.parametrize("change,first", [
    (dict(cu=[0, 70, 72]), 0), (dict(cu=[0, 5, 4]), 1), (dict(cu=[0, 5, 90]), 1), (dict(cu=[-1, 5, 7]), 0),
    (dict(lens=[4, 50]), 0), (dict(lens=[100, -1]), 1), (dict(lens=[100, 1 << 20]), 1), (dict(page=99), 0)])
def test_bad_calls_are_reported(gpu, change, first):
    """Nothing is read or written outside the tensors; the first bad sequence is named."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    cache = au.make_cache(1, 20, 2, 16, 128, True)
    table = au.make_table(2, [100, 50], 16, 20, 0)
    if "page" in change:
        table[0, 2] = change["page"]
    T = 80
    tree = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    ws = moe.AttnWorkspace("cuda", "tree", 2, T, 8, 2, 128)
    moe.attn_tree(au.randn(3, T, 8, 128), cache, table, su.i32(change.get("lens", [100, 50])),
                  su.i32(change.get("cu", [0, 5, 7])), tree, workspace=ws)
    assert au.status(ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, first)


# ---------------------------------------------------------------- accepted tokens
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv,D,page", [(1, 64, 16), (8, 128, 64), (3, 128, 256), (40, 64, 32)])
def test_accept(gpu, Hkv, D, page, fp8):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    rng = random.Random(Hkv)
    base = [0, 1, 15, 16, 100, 255, 300]
    paths = [[], [0], [63], list(range(64)), [0, 2, 3, 5, 60], sorted(rng.sample(range(64), 40)), [1, 2, 3]]
    lens = [n + 64 for n in base]
    pages = sum(-(-n // page) for n in lens) + 2
    cache = au.make_cache(1, pages, Hkv, page, D, fp8)
    table = au.make_table(2, lens, page, pages, -1)
    bits = cache.data.view(torch.uint8 if fp8 else torch.int16)
    want, scales = bits.clone(), cache.scales.clone() if fp8 else None
    t = table.cpu()
    for b, path in enumerate(paths):
        for i, a in enumerate(path):
            s, d = base[b] + a, base[b] + i
            s, d = (int(t[b, s // page]), s % page), (int(t[b, d // page]), d % page)
            want[d[0], :, :, d[1]] = bits[s[0], :, :, s[1]]
            if fp8:
                scales[d[0], :, :, d[1]] = cache.scales[s[0], :, :, s[1]]
    accept = su.i32([p + [-1] * (64 - len(p)) for p in paths])
    ws = moe.AttnWorkspace("cuda")
    moe.kv_accept(cache, table, su.i32(base), accept, workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)
    assert torch.equal(bits, want) and (not fp8 or torch.equal(cache.scales, scales))


@pytest.mark.parametrize("bad", [dict(base=-1), dict(path=[1, 1]), dict(path=[3, 2]), dict(path=[-2, 4]),
                                 dict(base=1 << 30), dict(path=[0, 400]), dict(page=77), dict(page=-1)])
def test_accept_refuses(gpu, bad):
    """A bad sequence moves nothing, the others move."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    cache = au.make_cache(1, 20, 2, 16, 64, True)
    table = au.make_table(2, [64, 64, 64], 16, 20, -1)
    bits = cache.data.view(torch.uint8)
    t = table.cpu().tolist()
    if "page" in bad:
        table[1, 1] = bad["page"]
    want, scales = bits.clone(), cache.scales.clone()
    for b in (0, 2):
        want[t[b][0], :, :, 11] = bits[t[b][1], :, :, 4]
        scales[t[b][0], :, :, 11] = cache.scales[t[b][1], :, :, 4]
    path = bad.get("path", [0, 10])
    accept = su.i32([[0, 10], path, [0, 10]])
    ws = moe.AttnWorkspace("cuda")
    moe.kv_accept(cache, table, su.i32([10, bad.get("base", 10), 10]), accept, workspace=ws)
    assert au.status(ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, 1)
    assert torch.equal(bits, want) and torch.equal(cache.scales, scales)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_sequences_of_few_and_many_rows_in_turns(gpu, D, fp8):
    """Blocks that go from one row tile to two and back, several times."""
    lens = [200 + (53 * i * i) % 700 for i in range(120)]
    nodes = [(33, 5, 16, 20, 64, 1)[i % 6] for i in range(120)]
    _tree(lens, nodes, 16, 2, D, fp8, 64, seed=11)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_but_for_one_sequence(gpu, D, fp8):
    """Tiles of 16 rows, and a sequence that has many of them."""
    lens = [50 + 3 * i for i in range(40)]
    _tree(lens, [64 if i == 17 else 1 for i in range(40)], 8, 4, D, fp8, 16, seed=12)
