"""moe_attn_tree with scales so small that, times a tiny row of q, they leave
fp32's range: rows that are masked in part stay numbers."""
import pytest

from tests import attn_util as au, serve_util as su

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,nodes", [(128, 16, 2, 2), (128, 16, 2, 9), (128, 16, 2, 40), (64, 16, 2, 9),
                                            (64, 16, 2, 40)])
@pytest.mark.parametrize("scale", [1e-7, 1e-10, 1e-38])
def test_tiny_scales(gpu, scale, D, Hq, Hkv, nodes, fp8):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    n, page = 300, 16
    cache = au.make_cache(1, 20, Hkv, page, D, fp8)
    table = au.make_table(2, [n], page, 20, 0)
    q = au.randn(3, nodes, Hq, D)
    q[:, 0] = 0
    q[:, 1] *= 2.0 ** -120
    q[:, 2] *= 2.0 ** -60
    tree = torch.tensor([(2 << i) - 1 for i in range(nodes)], dtype=torch.int64, device="cuda")
    ws = moe.AttnWorkspace("cuda", "tree", 1, nodes, Hq, Hkv, D)
    out, lse = moe.attn_tree(q, cache, table, su.i32([n]), su.i32([0, nodes]), tree, scale=scale, lse=True,
                             workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)
    k, v = au.cached_rows(cache, table, 0, n)
    seen = torch.arange(n, device="cuda")[None] <= torch.arange(n - nodes, n, device="cuda")[:, None]
    ref, rl, tol, tl = su.seen_attention(q, k, v, scale, seen)
    au.check(out, ref, tol, "out")
    au.check(lse, rl, tl, "lse")
