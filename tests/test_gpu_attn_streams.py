"""The attention half's calls on a stream that is not the current one, and in
a captured graph: the same results as on the current stream."""
import pytest

from tests import attn_util as au

pytestmark = pytest.mark.gpu


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _calls():
    """Each call on fixed inputs: f(outputs or None, **kw) -> its outputs, and
    the outputs' and the workspace's sizes."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    lens, page, Hkv, D = [100, 0, 2000], 16, 2, 128
    total = sum(lens)
    cache = au.make_cache(5, 140, Hkv, page, D, True)
    into = au.make_cache(5, 140, Hkv, page, D, True)
    table = au.make_table(6, lens, page, 140, 0)
    q1, k1 = au.randn(7, 3, 16, D), au.randn(8, 3, Hkv, D)
    q, k, v = au.randn(9, total, 16, D), au.randn(10, total, Hkv, D), au.randn(11, total, Hkv, D)
    cs, pos, slots = moe.rope_table(100, D), _i32([3, 99, 0]), _i32([5, 300, 17])
    n, cu = _i32(lens), _i32([0, 100, 100, 2100])
    o = lambda outs, i: None if outs is None else outs[i]  # noqa: E731

    def append(outs=None, **kw):
        return moe.qk_rope_append(q1, k1, k1, cs, pos, into, slots, q_out=o(outs, 0),
                                  k_out=True if outs is None else outs[1], **kw)

    def gather(outs=None, **kw):
        return moe.kv_gather(cache, table, cu, total, k_out=o(outs, 0), v_out=o(outs, 1), **kw)

    def decode(outs=None, **kw):
        return moe.attn_decode(q1, cache, table, n, out=o(outs, 0),
                               lse=True if outs is None else outs[1], **kw)

    def prefill(outs=None, **kw):
        return moe.attn_prefill(q, k, v, cu, cu, out=o(outs, 0),
                                lse=True if outs is None else outs[1], **kw)
    torch.cuda.synchronize()
    return dict(append=(append, ()), gather=(gather, ()), decode=(decode, ("decode", 3, 3, 16, Hkv, D)),
                prefill=(prefill, ("prefill", 3, total, 16, Hkv, D)))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op", ["append", "gather", "decode", "prefill"])
def test_memory_freed_on_the_current_stream(gpu, op, raw):
    """The current stream still has to write blocks that were freed on it; a
    call on another stream must not be given them."""
    import torch
    f, _ = _calls()[op]
    ref = f()
    sizes = [(t.shape, t.dtype) for t in ref]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    blocks = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes]
    blocks += [torch.empty(64 << 20, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda._sleep(20_000_000)   # about 10 ms
    for b in blocks:
        b.zero_()
    del b, blocks
    got = f(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


@pytest.mark.parametrize("op", ["append", "gather", "prefill"])
def test_in_a_graph(gpu, op):
    """Captured with buffers that the caller keeps, and with ones made in the
    capture; replayed over wiped outputs."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    f, size = _calls()[op]
    ref = f()
    hold = [torch.empty_like(t) for t in ref]
    ws = moe.AttnWorkspace("cuda", *size)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(hold, workspace=ws)
        made = f()
    for _ in range(2):
        for t in (*hold, *made):
            t.zero_()
        graph.replay()
        for got in (hold, made):
            for a, b in zip(got, ref):
                assert torch.equal(a, b)
    assert au.status(ws) == (moe.MOE_OK, 0)
