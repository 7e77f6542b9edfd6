"""moe_attn_tree over an fp8 cache whose scales and codes are not those of
normal values: scales of all sizes in one sequence, zero rows, NaN codes, and
queries with outliers.  Both ways of computing it: tiles of up to 16 rows (2
tokens), and of 128 (9, 40).

Bounds beside those of serve_util.seen_attention, from the header's rounding
notes: a value of q is off by up to 2^-17 of its head's largest; a value of v
by up to 2^-24 of the sequence's largest scale's power of two above."""
import math

import pytest

from tests import attn_util as au, serve_util as su

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE = 16, 2, 128, 16


def _setup(n, seed=0, hkv=HKV):
    import torch
    cache = au.make_cache(seed, -(-n // PAGE) + 1, hkv, PAGE, D, True)
    table = torch.randperm(-(-n // PAGE), generator=torch.Generator().manual_seed(seed)).int()[None].cuda()
    t = torch.arange(n, device="cuda")
    return cache, table, table[0].long()[t // PAGE], t % PAGE


def _run(cache, table, n, nodes, q, lse=True):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    tree = torch.tensor([(2 << i) - 1 for i in range(nodes)], dtype=torch.int64, device="cuda")
    ws = moe.AttnWorkspace("cuda", "tree", 1, nodes, HQ, cache.Hkv, D)
    out = moe.attn_tree(q, cache, table, su.i32([n]), su.i32([0, nodes]), tree, lse=lse, workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)
    return out


def _check(cache, table, n, nodes, q):
    import torch
    out, lse = _run(cache, table, n, nodes, q)
    k, v = au.cached_rows(cache, table, 0, n)
    seen = torch.arange(n, device="cuda")[None] <= torch.arange(n - nodes, n, device="cuda")[:, None]
    ref, rl, tol, tl = su.seen_attention(q, k, v, D ** -0.5, seen)
    G = HQ // cache.Hkv
    t = torch.arange(n, device="cuda")
    scales = cache.scales[table[0].long()[t // PAGE], :, 1, t % PAGE].double()   # [n][Hkv]
    for h in range(HQ):
        # what q's floor may move a score by, twice that relatively for a weight
        e = 2.0 ** -17 * q[:, h].double().abs().amax(-1) * k[:, h // G].abs().sum(-1).max() * D ** -0.5
        p_v = seen.double() @ v[:, h // G].abs()                   # a bound on sum p |v| of a moved weight
        most = v[:, h // G].abs().amax()
        tol[:, h] += 2 * (torch.exp(2 * e) - 1)[:, None].clamp_max(1e3) * torch.minimum(p_v, most)
        tol[:, h] += 2.0 ** -24 * 2.0 ** (math.floor(math.log2(max(float(scales[:, h // G].max()), 1e-38))) + 1)
        tl[:, h] += e
    au.check(out, ref, tol, "out")
    au.check(lse, rl, tl, "lse")


NODES = [2, 9, 40]


@pytest.mark.parametrize("nodes", NODES)
@pytest.mark.parametrize("how", ["rising", "falling", "random", "one large", "one small"])
def test_scales_of_all_sizes(gpu, how, nodes):
    import torch
    n = 1500
    cache, table, pg, off = _setup(n, 1)
    t = torch.arange(n, device="cuda", dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(2)
    f = {"rising": torch.exp2(torch.floor(t / 100) - 7), "falling": torch.exp2(7 - torch.floor(t / 100)),
         "random": torch.exp2(torch.randint(-6, 7, (n,), generator=g, device="cuda").float()),
         "one large": torch.where(t == 700, 4096.0, 1.0), "one small": torch.where(t == 700, 1e-20, 1.0)}[how]
    cache.scales[pg, :, 1, off] *= f[:, None]
    _check(cache, table, n, nodes, au.randn(3, nodes, HQ, D))


@pytest.mark.parametrize("nodes", NODES)
@pytest.mark.parametrize("factor", [1e-30, 1e-37, 1e30])
def test_values_all_small_or_large(gpu, factor, nodes):
    n = 300
    cache, table, pg, off = _setup(n, 4)
    cache.scales[pg, :, 1, off] *= factor
    _check(cache, table, n, nodes, au.randn(5, nodes, HQ, D))


@pytest.mark.parametrize("nodes", NODES)
def test_zero_rows(gpu, nodes):
    """Tokens whose values, or keys and values, are zero; then all of them."""
    import torch
    n = 400
    cache, table, pg, off = _setup(n, 6)
    cache.scales[pg[::3], :, 1, off[::3]] = 0.0
    cache.scales[pg[::5], :, :, off[::5]] = 0.0
    q = au.randn(7, nodes, HQ, D)
    _check(cache, table, n, nodes, q)
    cache.scales[pg, :, 1, off] = 0.0
    out, _ = _run(cache, table, n, nodes, q)
    assert (out == 0).all()


@pytest.mark.parametrize("nodes", NODES)
def test_queries_with_outliers(gpu, nodes):
    """One value of each head far larger than the others, or all of a head
    tiny, or zero."""
    import torch
    n = 700
    cache, table, pg, off = _setup(n, 8)
    q = au.randn(9, nodes, HQ, D)
    q[:, 0, 3] *= 64
    q[:, 1, 100] *= 1000
    q[:, 2] *= 1e-20
    q[:, 3] = 0
    q[:, 4] *= 2.0 ** -120
    _check(cache, table, n, nodes, q)


@pytest.mark.parametrize("nodes", NODES)
def test_nan_codes(gpu, nodes):
    """A NaN code of a key is NaN in all of its head's rows, of a value in its
    column; behind the last token it is nothing."""
    import torch
    n = 333
    cache, table, pg, off = _setup(n, 10)
    q = au.randn(11, nodes, HQ, D)
    ref, _ = _run(cache, table, n, nodes, q)
    bits = cache.data.view(torch.uint8)
    bits[pg[50], 0, 1, off[50], 7] = 0x7F
    bits[pg[60], 1, 1, off[60], 100] = 0xFF
    last = int(pg[n - 1])
    bits[last, :, :, n % PAGE:] = 0x7F
    cache.scales[last, :, :, n % PAGE:] = float("inf")
    out, _ = _run(cache, table, n, nodes, q)
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[:, :8, 7] = want[:, 8:, 100] = True
    assert torch.equal(bad, want) and torch.equal(out[~bad], ref[~bad])
    bits[pg[70], 1, 0, off[70], 0] = 0x7F
    out, lse = _run(cache, table, n, nodes, q)
    assert torch.isnan(out[:, 8:]).all() and torch.isnan(lse[:, 8:]).all()
    assert torch.equal(torch.isnan(out[:, :8]), want[:, :8])


@pytest.mark.parametrize("nodes", NODES)
def test_queries_that_are_not_finite(gpu, nodes):
    """A row of q with an infinity or NaN is NaN; the others are as they were."""
    import torch
    n = 500
    cache, table, pg, off = _setup(n, 12)
    q = au.randn(13, nodes, HQ, D)
    ref, _ = _run(cache, table, n, nodes, q)
    q[0, 2, 5], q[1, 9, 0] = float("inf"), float("nan")
    out, _ = _run(cache, table, n, nodes, q)
    keep = torch.ones(nodes, HQ, dtype=torch.bool, device="cuda")
    keep[0, 2] = keep[1, 9] = False
    assert torch.isnan(out[0, 2]).all() and torch.isnan(out[1, 9]).all()
    assert torch.equal(out[keep], ref[keep])
