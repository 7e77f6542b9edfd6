"""Prompts in chunks through a window: pages behind it go back at every step and
are somebody else's (here NaN); the context comes back by kv_gather, and the
attention of the new tokens sees nothing of what those pages hold."""
import pytest

from tests import attn_util as au, serve_util as su
from tests.test_gpu_serving_run import Server

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 4, 4), (128, 16, 1)])
@pytest.mark.parametrize("window,sinks", [(50, 4), (50, 0), (7, 20), (130, 33), (200, 64)])
def test_chunks(gpu, window, sinks, D, Hq, Hkv, page, fp8):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    B, width = 3, 2400 // page
    s = Server(B, B * width, page, Hkv, D, width, fp8, window, sinks)
    bits = s.cache.data.view(torch.uint8 if fp8 else torch.int16)
    for chunk in ([300, 1, 90], [100, 257, 0], [64, 100, 300], [1, 33, 128], [260, 3, 300]):
        q, _, _, plan = s.step(chunk, sum(chunk) + 5, Hq)
        head, count = s.pool.state.tolist()
        n = s.pool.ring.numel()
        free = s.pool.ring[(torch.arange(count, device="cuda") + head) % n].long()
        bits[free] = 0x7f if fp8 else 0x7fc1
        if fp8:
            s.cache.scales[free] = float("nan")
        lens = plan.seq_lens.tolist()
        ws = moe.AttnWorkspace("cuda")
        k, v = moe.kv_gather(s.cache, s.table, plan.cu_k, sum(lens), workspace=ws)
        assert au.status(ws) == (moe.MOE_OK, 0)
        T = sum(chunk)
        ws = moe.AttnWorkspace("cuda", "prefill", B, T, Hq, Hkv, D)
        out, lse = moe.attn_prefill(q[:T], k, v, plan.cu_q, plan.cu_k, lse=True, window=window, sinks=sinks,
                                    workspace=ws)
        assert au.status(ws) == (moe.MOE_OK, 0)
        at, ctx = 0, 0
        for b, (m, total) in enumerate(zip(chunk, lens)):
            i, j = slice(at, at + m), slice(ctx, ctx + total)
            at, ctx = at + m, ctx + total
            pos = torch.arange(total - m, total, device="cuda")
            ref, rl, tol, tl = su.seen_attention(q[i], k[j], v[j], D ** -0.5,
                                                 su.window_seen(pos, total, window, sinks))
            au.check(out[i], ref, tol, f"out {b}")
            au.check(lse[i], rl, tl, f"lse {b}")
    assert min(s.kept.tolist()) >= 0 and max(s.kept.tolist()) > 0
