"""Serving over the paged cache on a stream that is not the current one, with
memory that was freed on the current one, and in a captured graph: the same
results as on the current stream."""
import pytest

from tests import attn_util as au, serve_util as su

pytestmark = pytest.mark.gpu

OPS = ["pages", "wdecode", "wprefill", "tree", "accept"]


def _calls():
    """Each call on fixed inputs: f(outputs or None, **kw) -> its outputs; its
    workspace's sizes; what puts back the inputs that it changes."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    lens, page, Hkv, D = [100, 7, 2000], 16, 2, 128
    total = sum(lens)
    cache = au.make_cache(5, 140, Hkv, page, D, True)
    table = au.make_table(6, lens, page, 140, 0)
    data, scales = cache.data.view(torch.uint8).clone(), cache.scales.clone()
    q1, q = au.randn(7, 3, 16, D), au.randn(9, total, 16, D)
    k, v = au.randn(10, total, Hkv, D), au.randn(11, total, Hkv, D)
    n, cu = su.i32(lens), su.i32(su.prefix(lens))
    nodes, cu_t = 40 + 7 + 33, su.i32([0, 40, 47, 80])
    qt, tree = au.randn(12, nodes, 16, D), torch.full((nodes,), -1, dtype=torch.int64, device="cuda")
    accept = su.i32([[0, 3, 7], [1, -1, -1], [2, 5, 63]])
    pool = moe.PagePool(su.i32(list(range(500))), su.i32([490, 500]))
    plan_table = su.i32([[-1] * 200] * 3)
    first_state = su.i32([490, 500])
    o = lambda outs, i: None if outs is None else outs[i]  # noqa: E731

    lens0 = su.i32([0, 0, 0])

    def pages(outs=None, **kw):
        plan = None if outs is None else moe.PagePlan(*outs[:5], state=outs[5])
        p = moe.page_plan(pool, plan_table, lens0, n, page, total + 5, out=plan, **kw)
        return [p.seq_lens, p.cu_q, p.cu_k, p.positions, p.slots, p.state if outs else pool.state]

    def wdecode(outs=None, **kw):
        return moe.attn_decode(q1, cache, table, n, out=o(outs, 0), lse=True if outs is None else outs[1],
                               window=300, sinks=4, **kw)

    def wprefill(outs=None, **kw):
        return moe.attn_prefill(q, k, v, cu, cu, out=o(outs, 0), lse=True if outs is None else outs[1],
                                window=200, sinks=3, **kw)

    def trees(outs=None, **kw):
        return moe.attn_tree(qt, cache, table, n, cu_t, tree, out=o(outs, 0),
                             lse=True if outs is None else outs[1], **kw)

    def accepted(outs=None, **kw):
        moe.kv_accept(cache, table, base, accept, **kw)
        return [cache.data.view(torch.uint8), cache.scales]

    base = su.i32([30, 2, 1900])

    def put_back():
        cache.data.view(torch.uint8).copy_(data)
        cache.scales.copy_(scales)
        pool.state.copy_(first_state)
    torch.cuda.synchronize()
    return dict(pages=(pages, ("pages", 3), put_back), wdecode=(wdecode, ("decode", 3, 3, 16, Hkv, D), put_back),
                wprefill=(wprefill, ("prefill", 3, total, 16, Hkv, D), put_back),
                tree=(trees, ("tree", 3, nodes, 16, Hkv, D), put_back), accept=(accepted, (), put_back))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op", OPS)
def test_memory_freed_on_the_current_stream(gpu, op, raw):
    """The current stream still has to write blocks that were freed on it; a
    call on another stream must not be given them."""
    import torch
    f, size, put_back = _calls()[op]
    ref = [t.clone() for t in f()]
    put_back()
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


@pytest.mark.parametrize("op", OPS)
def test_in_a_graph(gpu, op):
    """Captured with buffers that the caller keeps, and with ones made in the
    capture; replayed over wiped outputs."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    f, size, put_back = _calls()[op]
    ref = [t.clone() for t in f()]
    hold = [torch.empty_like(t) for t in ref] if op != "accept" else f()
    ws = moe.AttnWorkspace("cuda", *size)
    put_back()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(hold, workspace=ws)
        put_back()
        made = f()
    for _ in range(2):
        put_back()
        for t in (*hold, *made):
            if op != "accept":
                t.zero_()
        put_back()
        graph.replay()
        for got in (hold, made):
            for a, b in zip(got, ref):
                assert torch.equal(a, b)
    assert au.status(ws) == (moe.MOE_OK, 0)


def test_two_calls_at_once(gpu):
    """Trees and windows on two streams with workspaces of their own."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    calls = _calls()
    (f, sf, _), (g, sg, _) = calls["tree"], calls["wdecode"]
    ref_f, ref_g = [t.clone() for t in f()], [t.clone() for t in g()]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    wf, wg = moe.AttnWorkspace("cuda", *sf), moe.AttnWorkspace("cuda", *sg)
    for _ in range(20):
        got_f, got_g = f(stream=a, workspace=wf), g(stream=b, workspace=wg)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got_f, ref_f))
    assert all(torch.equal(x, y) for x, y in zip(got_g, ref_g))
