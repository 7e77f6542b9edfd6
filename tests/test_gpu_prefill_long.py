"""moe_attn_prefill's plan over key ranges of more than a thousand key tiles:
a few rows over them are still shared out over the whole GPU."""
import pytest

from tests import attn_util as au

pytestmark = pytest.mark.gpu

HEAD = 256   # the plan's head in the workspace: items, taken, blocks in parts, parts


def _call(nq, nk, Hq, Hkv, D, seed=0):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    pre = lambda x: torch.tensor([0] + list(torch.tensor(x).cumsum(0)), dtype=torch.int32, device="cuda")  # noqa: E731
    q = au.randn(seed, sum(nq), Hq, D)
    k, v = au.randn(seed + 1, sum(nk), Hkv, D), au.randn(seed + 2, sum(nk), Hkv, D)
    ws = moe.AttnWorkspace("cuda", "prefill", len(nq), sum(nq), Hq, Hkv, D)
    out, lse = moe.attn_prefill(q, k, v, pre(nq), pre(nk), lse=True, workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)
    head = ws.buf[HEAD:HEAD + 16].view(torch.int32).tolist()
    return q, k, v, out, lse, dict(items=head[0], joins=head[2], parts=head[3])


@pytest.mark.parametrize("keys", [100000, 130900, 131100, 200000, 261700, 262144, 300000, 524288, 1048576])
def test_parts_of_one_long_range(gpu, keys):
    """16 rows, 8 heads over one: one block, so that the whole GPU's share of
    it is one part an SM.  Counted in rounds of a part, the busiest SM has at
    most twice the even share."""
    import torch
    q, k, v, out, lse, plan = _call([16], [keys], 8, 1, 64)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = -(-keys // 128)
    assert plan["joins"] == 1
    part = -(-tiles // plan["parts"])
    busiest = part * -(-plan["parts"] // sms)
    assert busiest <= 2 * -(-tiles // sms), plan
    if keys in (131100, 262144):
        limit = torch.arange(16, device="cuda") + keys - 15
        for h in (0, 7):
            ref, rl, tol, tl = au.attention(q[:, h:h + 1], k, v, 64 ** -0.5, limit)
            au.check(out[:, h:h + 1], ref, tol, "out")
            au.check(lse[:, h:h + 1], rl, tl, "lse")


def test_long_ranges_among_shorter_ones(gpu):
    """One range far longer than the others, all beyond a thousand key tiles,
    and short ones: it is still cut."""
    import torch
    nk = [600000, 140000, 150000, 500, 135000]
    _, _, _, _, _, plan = _call([8, 8, 8, 300, 8], nk, 8, 1, 64, seed=4)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = [-(-n // 128) for n in nk]
    share = -(-sum(tiles) // sms)
    # the longest alone in parts of at most two even shares
    assert plan["parts"] >= tiles[0] / (2 * share), plan
