"""Runs of the serving calls together, as a server makes them, against plain
64-bit attention over the tokens' own rows: a layer with windows whose pages go
back, and drafted trees that are verified and partly accepted."""
import random

import pytest

from tests import attn_util as au, serve_util as su

pytestmark = pytest.mark.gpu


class Server:
    """Requests over one cache; the tokens' keys and values are kept aside."""

    def __init__(self, B, pages, page, Hkv, D, width, fp8, window=0, sinks=0):
        import torch
        import quantized_moe_expert_align_gb300 as moe
        self.moe, self.page, self.window, self.sinks = moe, page, window, sinks
        self.cache = moe.KVCache.empty(pages, Hkv, D, page, fp8=fp8)
        self.pool = moe.PagePool.full(pages)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.lens = su.i32([0] * B)
        self.kept = su.i32([0] * B)
        self.cos_sin = moe.rope_table(4096, D)
        self.rows = [[] for _ in range(B)]   # of each request: (position, its k, its v), rotated
        self.seed = 100
        self.dropped = None

    def step(self, new, rows, Hq, offsets=None):
        """Plans and appends `new` tokens; the rotated queries, the plan, k and v as given."""
        moe, c = self.moe, self.cache
        ws = moe.AttnWorkspace("cuda", "pages", len(new))
        kw = dict(window=self.window, sinks=self.sinks, kept=self.kept) if self.window else {}
        plan = moe.page_plan(self.pool, self.table, self.lens, su.i32(new), self.page, rows, workspace=ws,
                             offsets=offsets, dropped=self.dropped, **kw)
        assert au.status(ws) == (moe.MOE_OK, 0)
        self.dropped = None
        qkv = au.randn(self.seed, rows, Hq + 2 * c.Hkv, c.D)
        self.seed += 1
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + c.Hkv], qkv[:, Hq + c.Hkv:]
        wa = moe.AttnWorkspace("cuda")
        q, k = moe.qk_rope_append(q, k, v, self.cos_sin, plan.positions, c, plan.slots, k_out=True, workspace=wa)
        assert au.status(wa) == (moe.MOE_OK, 0)
        at = 0
        for b, n in enumerate(new):
            if n < 0:
                self.rows[b] = []
            for i in range(max(n, 0)):
                self.rows[b].append((k[at], v[at]))
                at += 1
        self.lens = plan.seq_lens
        if self.window:
            self.kept = plan.kept
        return q, k, v, plan

    def cached(self, b, idx):
        """K and V of tokens idx as the cache holds them (codes times scales)."""
        return au.cached_rows(self.cache, self.table, b, max(idx) + 1)

    def tol_of_storage(self):
        """What a cached value may be off from its bf16 row, relative to the row's largest."""
        return 0.0 if self.cache.scales is None else 2.0 ** -4

    def same_rows(self, b, idx):
        """The cache holds the rows that were appended."""
        import torch
        if not idx:
            return
        k, v = self.cached(b, idx)
        for got, which in ((k[idx], 0), (v[idx], 1)):
            want = torch.stack([self.rows[b][i][which] for i in idx]).double()
            most = want.abs().amax(-1, keepdim=True)
            assert ((got - want).abs() <= self.tol_of_storage() * most).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_windows(gpu, fp8):
    """Prompts, then tokens one by one; a request finishes and another takes its
    place; at the end every page is back."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    B, Hq, Hkv, D, page, window, sinks, pages = 3, 8, 2, 64, 16, 50, 4, 34
    s = Server(B, pages, page, Hkv, D, 40, fp8, window, sinks)
    prompts = [150, 17, 70]
    q, k, v, plan = s.step(prompts, 250, Hq)
    out = moe.attn_prefill(q, k, v, plan.cu_q, plan.cu_q, window=window, sinks=sinks)
    at = 0
    for b, n in enumerate(prompts):
        i = slice(at, at + n)
        ref, _, tol, _ = su.seen_attention(q[i], k[i], v[i], D ** -0.5,
                                           su.window_seen(torch.arange(n, device="cuda"), n, window, sinks))
        au.check(out[i], ref, tol, f"prompt {b}")
        at += n
    for step in range(60):
        new = [1, 1, 1]
        if step == 30:   # (a step of its own for who comes and goes)
            s.step([-1, 0, 0], 0, Hq)
            q, k, v, plan = s.step([33, 0, 0], 40, Hq)
        q, k, v, plan = s.step(new, B, Hq)
        lens = plan.seq_lens.tolist()
        ws = moe.AttnWorkspace("cuda", "decode", B, B, Hq, Hkv, D)
        out, lse = moe.attn_decode(q, s.cache, s.table, plan.seq_lens, lse=True, window=window, sinks=sinks,
                                   workspace=ws)
        assert au.status(ws) == (moe.MOE_OK, 0)
        if step % 7 and step < 28:
            continue
        for b, n in enumerate(lens):
            idx = [j for j in range(n) if j >= n - window or j < sinks]
            s.same_rows(b, idx)
            kk, vv = s.cached(b, idx)
            ref, rl, tol, tl = su.seen_attention(q[b:b + 1], kk[idx], vv[idx], D ** -0.5,
                                                 torch.ones(1, len(idx), dtype=torch.bool, device="cuda"))
            au.check(out[b:b + 1], ref, tol, f"step {step} request {b}")
            au.check(lse[b:b + 1], rl, tl, f"lse {step} {b}")
        assert all(int(x) > 0 for b, x in enumerate(s.kept.tolist()) if lens[b] > window + 2 * page)
    s.step([-1] * B, 0, Hq)
    assert s.pool.state.tolist()[1] == pages
    assert sorted(s.pool.ring.tolist()) == list(range(pages))


@pytest.mark.parametrize("fp8", [False, True])
def test_drafts(gpu, fp8):
    """Trees are drafted, appended, verified and partly accepted, step after step."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    rng = random.Random(1)
    B, Hq, Hkv, D, page, pages = 3, 16, 2, 128, 16, 60
    s = Server(B, pages, page, Hkv, D, 20, fp8)
    s.step([37, 5, 100], 150, Hq)
    for step in range(8):
        nodes = [rng.choice([1, 3, 12, 30]) for _ in range(B)]
        masks, depth, accept = [], [], []
        for n in nodes:
            parents = [rng.randrange(max(0, i - 4), i) if i else -1 for i in range(n)]
            own, d = [], []
            for i, p in enumerate(parents):
                own.append((own[p] if p >= 0 else 0) | 1 << i)
                d.append(d[p] + 1 if p >= 0 else 0)
            leaf = rng.randrange(n)
            path = [i for i in range(n) if own[leaf] >> i & 1]
            accept.append(path[:rng.randint(1, len(path))])
            masks.append(own)
            depth.append(d)
        rows = sum(nodes) + 3
        flat = [x for d in depth for x in d] + [0] * 3
        before = s.lens.tolist()
        q, k, v, plan = s.step(nodes, rows, Hq, offsets=su.i32(flat))
        assert plan.positions.tolist() == [before[b] + x for b, d in enumerate(depth) for x in d] + [0] * 3
        tree = torch.tensor([m for o in masks for m in o] + [0] * 3, dtype=torch.int64, device="cuda")
        ws = moe.AttnWorkspace("cuda", "tree", B, rows, Hq, Hkv, D)
        out = moe.attn_tree(q, s.cache, s.table, plan.seq_lens, plan.cu_q, tree, workspace=ws)
        assert au.status(ws) == (moe.MOE_OK, 0)
        at = 0
        for b, n in enumerate(nodes):
            total = before[b] + n
            s.same_rows(b, list(range(total)))
            kk, vv = s.cached(b, [total - 1])
            seen = torch.ones(n, total, dtype=torch.bool, device="cuda")
            for i, m in enumerate(masks[b]):
                seen[i, before[b]:] = torch.tensor([m >> x & 1 > 0 for x in range(n)], device="cuda")
            ref, _, tol, _ = su.seen_attention(q[at:at + n], kk, vv, D ** -0.5, seen)
            au.check(out[at:at + n], ref, tol, f"step {step} request {b}")
            at += n
        most = max(len(p) for p in accept)
        base = su.i32(before)
        moe.kv_accept(s.cache, s.table, base, su.i32([p + [-1] * (most - len(p)) for p in accept]), workspace=ws)
        assert au.status(ws) == (moe.MOE_OK, 0)
        kept = su.i32([len(p) for p in accept])
        s.dropped = s.lens - base - kept
        s.lens = base + kept
        for b, p in enumerate(accept):
            new = [s.rows[b][before[b] + i] for i in p]
            s.rows[b] = s.rows[b][:before[b]] + new
            s.same_rows(b, list(range(len(s.rows[b]))))
    s.step([-1] * B, 0, Hq)
    assert sorted(s.pool.ring.tolist()) == list(range(pages)) and s.pool.state.tolist()[1] == pages
