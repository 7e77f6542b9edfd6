"""moe_attn_decode: what its roundings may add to the result's own.  Few keys,
or one that outweighs the others, show the rounding of the weights.

Scores are off by e (attn_util.attention), a weight so by 2 e.  32-bit sums: a
product of 16 keys is added with an error of at most 2^-21 of what was added up
so far, a few joins on top.  Weights enter the product with v
* over a bf16 cache as sums of two bf16, off by 2^-16 of the weight,
* over an fp8 cache with v's scale in them as one bf16, off by 2^-8.
Then the result is rounded once."""
import pytest

from tests import attn_util as au

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (32, 2), (5, 1), (40, 1), (4, 4)])
@pytest.mark.parametrize("fp8", [False, True])
def test_roundings(gpu, fp8, Hq, Hkv, D):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    lens, page, scale, G = [1, 2, 3, 17, 1, 130, 900, 1, 4, 2100], 16, 1.0, Hq // Hkv
    seed = 3 * D + Hq
    pages = sum(-(-n // page) for n in lens) + 2
    cache = au.make_cache(seed, pages, Hkv, page, D, fp8)
    table = au.make_table(seed + 1, lens, page, pages, 0)
    q = au.randn(seed + 2, len(lens), Hq, D)
    out = moe.attn_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=scale)
    for b, m in enumerate(lens):
        k, v = au.cached_rows(cache, table, b, m)
        for h in range(Hq):
            kh, vh, qh = k[:, h // G], v[:, h // G], q[b, h].double()
            p = torch.softmax(kh @ qh * scale, 0)
            ref, mags = p @ vh, p @ vh.abs()
            e = 2 * D * 2.0 ** -24 * (kh.abs() @ qh.abs()).max() * scale + 2.0 ** -20
            weight = 2.0 ** -8 if fp8 else 2.0 ** -16
            tol = au.U_BF16 * ref.abs() + (weight + 2 * e + (m / 16 + 16) * 2.0 ** -21) * mags
            au.check(out[b, h], ref, tol, f"sequence {b} head {h}")
