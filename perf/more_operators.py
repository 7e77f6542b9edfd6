"""The operators of serving with a paged cache beyond plain attention, as cases to be measured.

Each case is one call that a server makes for a batch: the page tables and slot maps of a step from the
requests' lengths (``pages``), attention of single tokens through a sliding window with a few first tokens
that stay visible (``wdecode``), the same over packed prompts (``wprefill``), attention of a tree of drafted
tokens over the paged cache (``tree``), and the move of a tree's accepted tokens to their places in the cache
(``accept``).  ``run`` computes a case in plain torch operations (``own`` false) or through the framework's
entry points (``own`` true) on the same prepared inputs.

Cache layout (both sides): data [num_pages][Hkv][2 (K, V)][page][D] bf16 or fp8 e4m3, fp8 with fp32
scales [num_pages][Hkv][2][page], one per token and head; value = code * scale.
"""
import math
import random

import numpy as np
import torch

own = False

FP8_MAX = 448.0
NODES = 64         # drafted tokens of a tree at most


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 90 requests with windows: a token each, some finish, pages behind the
        # windows go back
        dict(name="pages_90", op="pages", mode="step", B=90, max_len=8192, page=16, window=1000, sinks=4),
        # admission of 256 prompts of ragged lengths in one call
        dict(name="pages_256", op="pages", mode="admit", B=256, max_len=8192, page=64, window=0, sinks=0),
        # one request with a short window: latency of a step
        dict(name="wdecode_1", op="wdecode", B=1, max_len=2000, window=128, sinks=4, Hq=64, Hkv=8, D=64,
             kv="bf16", page=16, lse=False),
        # 90 requests, a window that is no multiple of a page, bf16 cache in small pages
        dict(name="wdecode_90", op="wdecode", B=90, max_len=8192, window=1000, sinks=4, Hq=32, Hkv=4,
             D=128, kv="bf16", page=16, lse=True),
        # a full server of long requests, fp8 cache
        dict(name="wdecode_256", op="wdecode", B=256, max_len=32768, window=4096, sinks=4, Hq=64, Hkv=8,
             D=128, kv="fp8", page=64, lse=False),
        # chunks of up to 1000 tokens of four requests after long contexts, short window, heads of 64
        dict(name="wprefill_chunks", op="wprefill", B=4, max_q=1000, ctx=15000, window=128, sinks=4,
             Hq=32, Hkv=4, D=64, lse=True),
        # one long prompt
        dict(name="wprefill_16384", op="wprefill", B=1, max_q=16384, ctx=0, window=4096, sinks=4, Hq=64,
             Hkv=8, D=128, lse=False),
        # one request's seven drafted tokens after a short context: latency of a verification
        dict(name="tree_1x7", op="tree", B=1, nodes=7, max_len=517, Hq=64, Hkv=8, D=128, kv="bf16",
             page=16, lse=False),
        # 64 requests with trees of up to 16 tokens, fp8 cache
        dict(name="tree_64x16", op="tree", B=64, nodes=16, max_len=8192, Hq=64, Hkv=8, D=128, kv="fp8",
             page=64, lse=False),
        # 32 requests with trees of up to 64 tokens, bf16 cache in small pages
        dict(name="tree_32x64", op="tree", B=32, nodes=64, max_len=8192, Hq=32, Hkv=4, D=128, kv="bf16",
             page=16, lse=True),
        # one request's accepted tokens
        dict(name="accept_1", op="accept", B=1, nodes=7, path=3, max_len=517, Hkv=8, D=128, kv="fp8",
             page=16),
        # the accepted tokens of 256 requests
        dict(name="accept_256", op="accept", B=256, nodes=64, path=8, max_len=517, Hkv=8, D=128,
             kv="bf16", page=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(["pages", "wdecode", "wdecode", "wprefill", "wprefill", "tree", "tree", "tree",
                     "accept"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8, 8, 16])
    D = rng.choice([64, 128, 128])
    kv = rng.choice(["bf16", "fp8"])
    page = rng.choice([16, 32, 64, 128, 256])
    window, sinks = _log_int(rng, 1, 4096), rng.choice([0, 1, 4, 4, 16, 100])
    if op == "pages":
        some = rng.random() < 0.5
        return dict(op=op, mode=rng.choice(["step", "admit", "draft"]), B=_log_int(rng, 1, 2000),
                    max_len=_log_int(rng, NODES + 1, 32768), page=page, window=window if some else 0,
                    sinks=sinks if some else 0)
    if op == "wdecode":
        return dict(op=op, B=_log_int(rng, 1, 256), max_len=_log_int(rng, 1, 32768), window=window,
                    sinks=sinks, Hq=Hkv * G, Hkv=Hkv, D=D, kv=kv, page=page, lse=rng.random() < 0.5)
    if op == "wprefill":
        ctx = 0 if rng.random() < 0.5 else _log_int(rng, 1, 15000)
        return dict(op=op, B=_log_int(rng, 1, 8), max_q=_log_int(rng, 1, 16384), ctx=ctx,
                    window=window, sinks=sinks, Hq=Hkv * G, Hkv=Hkv, D=D, lse=rng.random() < 0.5)
    if op == "tree":
        nodes = _log_int(rng, 1, NODES)
        return dict(op=op, B=_log_int(rng, 1, 256), nodes=nodes, max_len=_log_int(rng, nodes, 32768),
                    Hq=Hkv * G, Hkv=Hkv, D=D, kv=kv, page=page, lse=rng.random() < 0.5)
    path = _log_int(rng, 1, 16)
    return dict(op=op, B=_log_int(rng, 1, 256), nodes=rng.randint(2 * path, NODES), path=path,
                max_len=_log_int(rng, NODES + 1, 2000), Hkv=Hkv, D=D, kv=kv, page=page)


def _cost(case):
    """Seconds that the case's plain form roughly takes, from what it holds in 32 bits."""
    op, B = case["op"], case["B"]
    if op == "pages":
        return B * case["max_len"] * 1e-11
    if op == "wdecode":
        return B * min(case["max_len"], case["window"] + case["sinks"]) * case["Hkv"] * case["D"] * 1e-11
    if op == "wprefill":
        reach = min(case["window"] + 512 + case["sinks"], case["max_q"] + case["ctx"])
        return B * case["max_q"] * reach * case["Hq"] * 1e-11 + B * case["max_q"] * 1e-6
    if op == "tree":
        return B * case["max_len"] * (case["Hkv"] * case["D"] + case["nodes"] * case["Hq"]) * 1e-11
    return B * case["max_len"] * case["Hkv"] * case["D"] * 1e-11


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = {k: max(most.get(c["op"], {}).get(k, 0), v) for k, v in
                         dict(work(c), cost=_cost(c)).items()}
    while True:
        c = _draw(rng)
        m = most[c["op"]]
        if all(v <= m[k] for k, v in dict(work(c), cost=_cost(c)).items()):
            return c


def _ragged(n, longest, salt, shortest=None):
    """n lengths in [longest/8, longest], the first the longest: a fixed function of its arguments."""
    r = random.Random(n * 1000003 + longest * 101 + salt)
    lo = max(1, longest // 8) if shortest is None else shortest
    return [longest] + [_log_int(r, lo, longest) for _ in range(n - 1)]


def _nodes(case):
    """Drafted tokens of each sequence of a tree case: from half of the most, never beyond the length."""
    n = _ragged(case["B"], case["nodes"], 4, max(1, case["nodes"] // 2))
    return [min(a, b) for a, b in zip(n, _key_lens(case))]


def _key_lens(case):
    """Cached tokens of each sequence (all that were ever cached: windows see the last of them)."""
    if case["op"] == "accept":  # contexts that the drafted tokens follow
        return [a - 1 for a in _ragged(case["B"], case["max_len"], 3)]
    return _ragged(case["B"], case["max_len"], 3)


def _prompt_lens(case):
    """(query lengths, key lengths) of the case's sequences."""
    nq = _ragged(case["B"], case["max_q"], 1)
    ctx = _ragged(case["B"], case["ctx"], 2) if case["ctx"] else [0] * case["B"]
    return nq, [a + b for a, b in zip(nq, ctx)]


def _paths(case):
    """Accepted tokens of each sequence."""
    return _ragged(case["B"], case["path"], 5, 1)


def _steps(case):
    """(lengths before, new tokens (-1: finished), first page held behind the sinks' after what went
    back) of a pages case."""
    B, page, window = case["B"], case["page"], case["window"]
    r = random.Random(B * 1009 + case["max_len"])
    if case["mode"] == "admit":
        return [0] * B, _ragged(B, case["max_len"], 6), [0] * B
    most = 1 if case["mode"] == "step" else NODES
    before = _ragged(B, case["max_len"] - most, 6)
    new = [-1 if r.random() < 0.05 else r.randint(1, most) for _ in range(B)]
    # (the last step looked at a window one to `most` tokens further back)
    kept = [max(0, (n - r.randint(1, most) + 1 - window) // page) if window else 0 for n in before]
    return before, new, kept


def work(case):
    op, B = case["op"], case["B"]
    if op == "pages":
        before, new, _ = _steps(case)
        grow = [max(n, 0) for n in new]
        page = case["page"]
        pages = sum(-(-(a + n) // page) - -(-a // page) for a, n in zip(before, grow))
        gone = sum(-(-a // page) for a, n in zip(before, new) if n < 0 and not case["window"])
        return {"bytes": 4 * (3 * B + 2 * (B + 1) + 2 * sum(grow) + 2 * pages + 2 * gone) +
                (8 * B if case["window"] else 0), "flops": 0}
    D, Hkv = case["D"], case["Hkv"]
    row = (D + 4) if case.get("kv") == "fp8" else 2 * D      # one cached K or V row of one head
    if op == "accept":
        paths = _paths(case)
        return {"bytes": sum(p - 1 for p in paths) * 2 * Hkv * row * 2 + 4 * sum(paths) + 4 * B, "flops": 0}
    Hq = case["Hq"]
    if op == "wdecode":
        seen = sum(min(n, case["window"] + case["sinks"]) for n in _key_lens(case))
        return {"bytes": seen * 2 * Hkv * row + B * Hq * D * 4 + (4 * Hq * B if case["lse"] else 0),
                "flops": 4 * Hq * D * seen}
    if op == "tree":
        nodes, nk = _nodes(case), _key_lens(case)
        T = sum(nodes)
        # (each drafted token sees the context and itself, and some of its elders)
        pairs = sum(n * (k - n + 1) for n, k in zip(nodes, nk))
        return {"bytes": sum(nk) * 2 * Hkv * row + T * (Hq * D * 4 + 8) + (4 * Hq * T if case["lse"] else 0),
                "flops": 4 * Hq * D * pairs}
    nq, nk = _prompt_lens(case)
    pairs, used = 0, 0
    for q, k in zip(nq, nk):
        pos = np.arange(k - q, k)
        pairs += int(np.minimum(pos + 1, case["window"] + np.minimum(case["sinks"], pos + 1)).sum())
        used += min(k, q + case["window"] - 1 + case["sinks"])
    return {"bytes": 4 * D * (sum(nq) * Hq + used * Hkv) + (4 * Hq * sum(nq) if case["lse"] else 0),
            "flops": 4 * Hq * D * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _quantise(x):
    """(codes as float8 values, scales) of rows of D values."""
    amax = x.abs().amax(-1)
    inv = torch.where(amax > 0, FP8_MAX / amax, torch.zeros_like(amax))
    return (x * inv[..., None]).to(torch.float8_e4m3fn), amax / FP8_MAX


def _filled_cache(g, pages, Hkv, page, D, kv):
    """A cache that earlier tokens filled: rows of normal values."""
    x = _randn(g, pages, Hkv, 2, page, D)
    if kv == "bf16":
        return x, None
    data, scales = _quantise(x.float())
    return data, scales


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prefix(lens):
    return _i32([0] + list(np.cumsum(lens)))


def _paged(g, lens, page, spare, dead=None):
    """Page table [B][most] over shuffled pages and the number of pages; entries past a sequence's end
    are 0, those of the pages in dead[b] (a range), which went back, -1."""
    need = [-(-n // page) for n in lens]
    live = [[p for p in range(n) if dead is None or p not in dead[b]] for b, n in enumerate(need)]
    total = sum(len(p) for p in live) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    table = np.zeros((len(lens), max(max(need), 1)), dtype=np.int32)
    at = 0
    for b, p in enumerate(live):
        table[b, :need[b]] = -1
        table[b, p] = order[at:at + len(p)]
        at += len(p)
    return torch.from_numpy(table).cuda(), total


def _trees(case, seed):
    """One mask a drafted token: the tokens of its tree that it sees, itself among them."""
    r = random.Random(int(seed) * 7919 + 11)
    masks = []
    for n in _nodes(case):
        own_masks = []
        for i in range(n):
            # (most are near the tree's end: deeper than they are wide)
            parent = r.randint(max(0, i - 4), i - 1) if i else -1
            own_masks.append((own_masks[parent] if i else 0) | 1 << i)
        masks += own_masks
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device="cuda")


def _prepare_pages(case, seed, s):
    before, new, kept = _steps(case)
    B, page = case["B"], case["page"]
    first = -(-case["sinks"] // page)
    grow = [max(n, 0) for n in new]
    width = max(max(-(-(a + n) // page) for a, n in zip(before, grow)), 1)
    held = [[p for p in range(-(-a // page)) if p < first or p >= max(k, first)] for a, k in zip(before, kept)]
    need = sum(-(-(a + n) // page) - -(-a // page) for a, n in zip(before, grow))
    used = sum(len(h) for h in held)
    pages = used + need + 5 + B // 8
    order = np.random.RandomState(int(seed) % (1 << 31)).permutation(pages).astype(np.int32)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, h] = order[at:at + len(h)]
        at += len(h)
    head, count = int(seed) % pages, pages - used
    ring = np.full(pages, -1, dtype=np.int32)
    ring[(head + np.arange(count)) % pages] = order[used:]
    s["table"], s["ring"] = torch.from_numpy(table).cuda(), torch.from_numpy(ring).cuda()
    s["state"] = _i32([head, count])
    s["before"], s["new"] = _i32(before), _i32(new)
    s["kept"] = _i32(kept) if case["window"] else None
    # a step's buffers have room for one row (or one tree) a request
    s["rows"] = {"step": B, "draft": B * NODES, "admit": sum(grow)}[case["mode"]]
    s["offsets"] = None
    if case["mode"] == "draft":  # a drafted token's depth in its tree
        s["offsets"] = (torch.arange(s["rows"], device="cuda") % 7).to(torch.int32)
    return s


def prepare(case, seed):
    s = {"case": dict(case)}
    op = case["op"]
    if op == "pages":
        return _prepare_pages(case, seed, s)
    g, D, Hkv = _gen(seed), case["D"], case["Hkv"]
    if op == "wprefill":
        nq, nk = _prompt_lens(case)
        s["nq"], s["nk"] = nq, nk
        s["cu_q"], s["cu_k"] = _prefix(nq), _prefix(nk)
        s["q"] = _randn(g, sum(nq), case["Hq"], D)
        kv = _randn(g, sum(nk), 2 * Hkv, D)
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        return s
    nk, page = _key_lens(case), case["page"]
    if op == "accept":
        s["base"] = _i32(nk)
        s["table"], pages = _paged(g, [n + case["nodes"] for n in nk], page, 8)
        # the root first, then ever later tokens of the tree
        r = random.Random(int(seed) * 31 + 7)
        accept = np.full((case["B"], case["path"]), -1, dtype=np.int32)
        for b, p in enumerate(_paths(case)):
            accept[b, :p] = [0] + sorted(r.sample(range(p, case["nodes"]), p - 1))
        s["accept"] = torch.from_numpy(accept).cuda()
    else:
        s["nk"] = _i32(nk)
        s["max_k"] = max(nk)
    if op == "wdecode":
        first = -(-case["sinks"] // page)
        dead = [range(first, max(first, (n - case["window"]) // page)) for n in nk]
        s["table"], pages = _paged(g, nk, page, 8, dead)
        s["q"] = _randn(g, case["B"], case["Hq"], D)
    if op == "tree":
        s["table"], pages = _paged(g, nk, page, 8)
        nodes = _nodes(case)
        s["n"], s["cu_q"], s["max_n"] = _i32(nodes), _prefix(nodes), max(nodes)
        s["q"] = _randn(g, sum(nodes), case["Hq"], D)
        s["tree"] = _trees(case, seed)
    s["data"], s["scales"] = _filled_cache(g, pages, Hkv, page, D, case["kv"])
    return s


# ---------------------------------------------------------------------------
# the plain forms: elementary operations in 32 bits, rounded once
# ---------------------------------------------------------------------------
def _plain_pages(s):
    c, table, ring = s["case"], s["table"], s["ring"]
    page, rows, B = c["page"], s["rows"], c["B"]
    cap = ring.shape[0]
    head, count = s["state"][0].long(), s["state"][1].long()
    before, new = s["before"].long(), s["new"].long()
    done = new < 0
    grow = new.clamp_min(0)
    after = torch.where(done, torch.zeros_like(before), before + grow)
    p0 = (before + page - 1) // page
    p1 = torch.where(done, p0, (after + page - 1) // page)
    need = p1 - p0
    taken = need.cumsum(0)
    d = torch.arange(table.shape[1], device="cuda")[None]
    # pages that go back: all of a finished request, those behind a window
    first = -(-c["sinks"] // page)
    out = {}
    if c["window"]:
        kept = s["kept"].long()
        behind = (before + 1 - c["window"]).clamp_min(0) // page
        lo = kept.clamp_min(first)
        gone = (d >= lo[:, None]) & (d < torch.where(done, p0, behind)[:, None])
        gone |= done[:, None] & (d < p0.clamp_max(first)[:, None])
        out["kept"] = torch.where(done, torch.zeros_like(kept), torch.maximum(kept, behind)).int()
    else:
        gone = done[:, None] & (d < p0[:, None])
    ring[(head + count + torch.arange(int(gone.sum()), device="cuda")) % cap] = table[gone]
    # pages that are taken
    fresh = (d >= p0[:, None]) & (d < p1[:, None])
    at = (head + (taken - need)[:, None] + d - p0[:, None]) % cap
    table.copy_(torch.where(fresh, ring[at], table))
    total = taken[-1]
    out["state"] = torch.stack([(head + total) % cap, count - total + gone.sum()]).int()
    # rows of the step
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    cu_q = torch.cat([zero, grow.cumsum(0)])
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(cu_q[1:], t, right=True).clamp_max(B - 1)
    there = t < cu_q[-1]
    j = before[b] + t - cu_q[b]
    pos = j if s["offsets"] is None else before[b] + s["offsets"].long()
    j = torch.where(there, j, torch.zeros_like(j))
    slot = table[b, j // page].long() * page + j % page
    out.update(seq_lens=after.int(), cu_q=cu_q.int(), cu_k=torch.cat([zero, after.cumsum(0)]).int(),
               positions=torch.where(there, pos, torch.zeros_like(pos)).int(),
               slots=torch.where(there, slot, torch.full_like(slot, -1)).int(), table=table, ring=ring)
    return out


def _rows_at(s, idx):
    """K and V [B][Hkv][n][D] fp32 of the tokens idx [B][n] (all of them in pages that are there)."""
    page = s["case"]["page"]
    pg = s["table"].long().gather(1, idx // page)
    off = idx % page
    data = s["data"]
    if data.dtype == torch.bfloat16:
        x = data[pg, :, :, off].float()                                   # [B][n][Hkv][2][D]
    else:
        x = data.view(torch.uint8)[pg, :, :, off].view(torch.float8_e4m3fn).float()
        x *= s["scales"][pg, :, :, off][..., None]
    x = x.permute(3, 0, 2, 1, 4)
    return x[0], x[1]


def _softmax_product(x, seen, v):
    """Rows of scores x (in place) over the keys `seen`, times v: (output, logsumexp)."""
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, m + total.log(), torch.full_like(total, -math.inf))
    return out, lse[..., 0]


def _plain_wdecode(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    w, sinks = min(c["window"], s["max_k"]), min(c["sinks"], s["max_k"])
    n = s["nk"].long()[:, None]
    i = torch.arange(sinks + w, device="cuda")[None]
    start = torch.maximum(n - c["window"], n.clamp_max(sinks))
    idx = torch.where(i < sinks, i, start + i - sinks)
    seen = idx < n
    k, v = _rows_at(s, torch.where(seen, idx, n - 1))
    x = torch.matmul(s["q"].float().view(B, Hkv, Hq // Hkv, D) * D ** -0.5, k.transpose(2, 3))
    out, lse = _softmax_product(x, seen[:, None, None], v)
    return {"out": out.reshape(B, Hq, D).bfloat16(), "lse": lse.reshape(B, Hq) if c["lse"] else None}


def _plain_wprefill(s):
    c = s["case"]
    Hq, Hkv, D, w, sinks = c["Hq"], c["Hkv"], c["D"], c["window"], c["sinks"]
    G = Hq // Hkv
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda") if c["lse"] else None
    q0 = k0 = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        k, v = s["k"][k0:k0 + nk], s["v"][k0:k0 + nk]
        for a in range(0, nq, 512):  # 512 rows and the keys that one of them sees
            b = min(a + 512, nq)
            first, last = a + nk - nq, b - 1 + nk - nq
            lo = max(0, first - w + 1)
            lead = min(sinks, lo)
            rows = lambda x: torch.cat([x[:lead], x[lo:last + 1]]).float().permute(1, 0, 2)[:, None]  # noqa: E731
            j = torch.cat([torch.arange(lead, device="cuda"), torch.arange(lo, last + 1, device="cuda")])
            pos = torch.arange(first, last + 1, device="cuda")[:, None]
            seen = (j[None] <= pos) & ((j[None] > pos - w) | (j[None] < sinks))
            q = s["q"][q0 + a:q0 + b].float().view(b - a, Hkv, G, D).permute(1, 2, 0, 3) * D ** -0.5
            o, l = _softmax_product(torch.matmul(q, rows(k).transpose(2, 3)), seen, rows(v))
            out[q0 + a:q0 + b] = o.permute(2, 0, 1, 3).reshape(b - a, Hq, D).bfloat16()
            if lse is not None:
                lse[q0 + a:q0 + b] = l.permute(2, 0, 1).reshape(b - a, Hq)
        q0, k0 = q0 + nq, k0 + nk
    return {"out": out, "lse": lse}


def _plain_tree(s):
    c = s["case"]
    B, Hq, Hkv, D, m, n = c["B"], c["Hq"], c["Hkv"], c["D"], s["max_k"], s["max_n"]
    j = torch.arange(m, device="cuda")[None]
    nk, nodes = s["nk"].long()[:, None], s["n"].long()[:, None]
    key = j < nk
    k, v = _rows_at(s, torch.where(key, j, nk - 1))
    i = torch.arange(n, device="cuda")[None]
    there = i < nodes
    iq = torch.where(there, s["cu_q"][:-1, None].long() + i, torch.zeros_like(i))
    q = s["q"][iq].float().view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4) * D ** -0.5
    node = (j - (nk - nodes))[:, None]                                   # [B][1][m]
    bit = (s["tree"][iq][..., None] >> node.clamp(0, 63)) & 1
    seen = key[:, None] & ((node < 0) | (bit != 0))
    out, lse = _softmax_product(torch.matmul(q, k[:, :, None].transpose(3, 4)), seen[:, None, None], v[:, :, None])
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[there].bfloat16()
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, Hq)[there]
    return {"out": out, "lse": lse if c["lse"] else None}


def _plain_accept(s):
    page = s["case"]["page"]
    accept, base = s["accept"].long(), s["base"].long()[:, None]
    live = accept >= 0
    i = torch.arange(accept.shape[1], device="cuda")[None].expand_as(accept)
    b = torch.arange(accept.shape[0], device="cuda")[:, None].expand_as(accept)
    b, src, dst = b[live], (base + accept)[live], (base + i)[live]
    table = s["table"].long()
    from_pg, to_pg = table[b, src // page], table[b, dst // page]
    data = s["data"].view(torch.uint8) if s["scales"] is not None else s["data"]
    data[to_pg, :, :, dst % page] = data[from_pg, :, :, src % page]
    if s["scales"] is not None:
        s["scales"][to_pg, :, :, dst % page] = s["scales"][from_pg, :, :, src % page]
    return {"data": s["data"], "scales": s["scales"]}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _kept(s):
    """What a serving loop makes once and keeps: the cache handle, workspaces and output buffers."""
    import quantized_moe_expert_align_gb300 as moe
    c, op = s["case"], s["case"]["op"]
    h = {"moe": moe}
    if op == "pages":
        h["pool"] = moe.PagePool(s["ring"], s["state"])
        h["plan"] = moe.PagePlan.empty(c["B"], s["rows"], windows=c["window"] > 0)
        h["plan"].state = torch.empty_like(s["state"])
        h["ws"] = moe.AttnWorkspace("cuda", "pages", c["B"])
        return h
    if op != "wprefill":
        h["cache"] = moe.KVCache(s["data"], s["scales"])
    if op == "accept":
        h["ws"] = moe.AttnWorkspace("cuda")
        return h
    rows = s["q"].shape[0]
    kind = {"wdecode": "decode", "wprefill": "prefill", "tree": "tree"}[op]
    h["ws"] = moe.AttnWorkspace("cuda", kind, c["B"], rows, c["Hq"], c["Hkv"], c["D"])
    h["out"] = torch.empty_like(s["q"])
    h["lse"] = torch.empty(rows, c["Hq"], dtype=torch.float32, device="cuda") if c["lse"] else None
    return h


def _own(s):
    if "handles" not in s:
        s["handles"] = _kept(s)
    h, c = s["handles"], s["case"]
    moe, op = h["moe"], c["op"]
    if op == "pages":
        p = moe.page_plan(h["pool"], s["table"], s["before"], s["new"], c["page"], s["rows"],
                          window=c["window"], sinks=c["sinks"], kept=s["kept"], offsets=s["offsets"],
                          out=h["plan"], workspace=h["ws"])
        out = dict(state=p.state, seq_lens=p.seq_lens, cu_q=p.cu_q, cu_k=p.cu_k, positions=p.positions,
                   slots=p.slots, table=s["table"], ring=s["ring"])
        if c["window"]:
            out["kept"] = p.kept
        return out
    if op == "accept":
        moe.kv_accept(h["cache"], s["table"], s["base"], s["accept"], workspace=h["ws"])
        return {"data": s["data"], "scales": s["scales"]}
    if op == "wdecode":
        moe.attn_decode(s["q"], h["cache"], s["table"], s["nk"], window=c["window"], sinks=c["sinks"],
                        out=h["out"], lse=h["lse"], workspace=h["ws"])
    elif op == "wprefill":
        moe.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], window=c["window"],
                         sinks=c["sinks"], out=h["out"], lse=h["lse"], workspace=h["ws"])
    else:
        moe.attn_tree(s["q"], h["cache"], s["table"], s["nk"], s["cu_q"], s["tree"], out=h["out"],
                      lse=h["lse"], workspace=h["ws"])
    return {"out": h["out"], "lse": h["lse"]}


_PLAIN = {"pages": _plain_pages, "wdecode": _plain_wdecode, "wprefill": _plain_wprefill,
          "tree": _plain_tree, "accept": _plain_accept}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits and sequence by sequence
# ---------------------------------------------------------------------------
def _exact_pages(s):
    c = s["case"]
    page, first, window = c["page"], -(-c["sinks"] // c["page"]), c["window"]
    table, ring = s["table"].cpu().numpy(), s["ring"].cpu().numpy()
    head, count = (int(v) for v in s["state"].cpu())
    cap = len(ring)
    before, new = s["before"].tolist(), s["new"].tolist()
    kept = s["kept"].tolist() if window else None
    offsets = s["offsets"].cpu().numpy() if s["offsets"] is not None else None
    pos, slots = np.zeros(s["rows"], np.int32), np.full(s["rows"], -1, np.int32)
    cu_q, lens, take, back = [0], [], 0, []
    for b in range(c["B"]):
        n, held = new[b], -(-before[b] // page)
        gone = list(range(held)) if n < 0 else []
        if window:
            behind = max(0, before[b] + 1 - window) // page
            gone = [p for p in gone if p < first or p >= kept[b]] if n < 0 else \
                list(range(max(first, kept[b]), behind))
            kept[b] = 0 if n < 0 else max(kept[b], behind)
        back += [table[b, p] for p in gone]
        n = max(n, 0)
        at, to = cu_q[-1], before[b] + n
        for p in range(held, -(-to // page)):
            table[b, p] = ring[(head + take) % cap]
            take += 1
        j = np.arange(before[b], to)
        slots[at:at + n] = table[b, j // page] * page + j % page
        pos[at:at + n] = j if offsets is None else before[b] + offsets[at:at + n]
        cu_q.append(at + n)
        lens.append(0 if new[b] < 0 else to)
    for i, p in enumerate(back):
        ring[(head + count + i) % cap] = p
    out = dict(state=_i32([(head + take) % cap, count - take + len(back)]), seq_lens=_i32(lens),
               cu_q=_i32(cu_q), cu_k=_prefix(lens), positions=_i32(pos), slots=_i32(slots),
               table=_i32(table), ring=_i32(ring))
    if window:
        out["kept"] = _i32(kept)
    return out


def _exact_cached(s, b, idx):
    """K and V [n][Hkv][D] of sequence b's tokens idx."""
    page = s["case"]["page"]
    pg, off = s["table"][b].long()[idx // page], idx % page
    d = s["data"]
    if d.dtype == torch.bfloat16:
        x = d[pg, :, :, off].double()
    else:
        x = d.view(torch.uint8)[pg, :, :, off].view(torch.float8_e4m3fn).double()
        x = x * s["scales"][pg, :, :, off].double()[..., None]
    return x[:, :, 0], x[:, :, 1]


def _exact_attention(q, k, v, seen):
    """q [n][Hq][D], k / v [m][Hkv][D], seen [n][m] (a key each at least): (out, lse)."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    out = torch.empty(n, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(n, Hq, dtype=torch.float64, device="cuda")
    for h in range(Hq):
        kh, vh = k[:, h * Hkv // Hq].double(), v[:, h * Hkv // Hq].double()
        x = (q[:, h].double() @ kh.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
        lse[:, h] = torch.logsumexp(x, -1)
        out[:, h] = torch.exp(x - lse[:, h:h + 1]) @ vh
    return out, lse


def _exact_accept(s):
    page, table = s["case"]["page"], s["table"].tolist()
    old, old_scales = s["data"].clone(), s["scales"].clone() if s["scales"] is not None else None
    for b, (base, path) in enumerate(zip(s["base"].tolist(), s["accept"].tolist())):
        for i, a in enumerate(path):
            if a < 0:
                break
            f, t = base + a, base + i
            to, fr = (table[b][t // page], t % page), (table[b][f // page], f % page)
            s["data"][to[0], :, :, to[1]] = old[fr[0], :, :, fr[1]]
            if old_scales is not None:
                s["scales"][to[0], :, :, to[1]] = old_scales[fr[0], :, :, fr[1]]
    return {"data": s["data"], "scales": s["scales"]}


def exact(case, seed):
    op = case["op"]
    if work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    if op == "pages":
        return _exact_pages(s)
    if op == "accept":
        return _exact_accept(s)
    outs, lses = [], []
    if op == "wprefill":
        q0 = k0 = 0
        for nq, nk in zip(s["nq"], s["nk"]):
            for a in range(0, nq, 2048):
                b = min(nq, a + 2048)
                pos = torch.arange(a, b, device="cuda") + nk - nq
                lo = max(0, a + nk - nq - case["window"] - case["sinks"])
                idx = torch.arange(lo, b + nk - nq, device="cuda")
                idx = torch.cat([torch.arange(min(case["sinks"], lo), device="cuda"), idx])
                seen = (idx[None] <= pos[:, None]) & ((pos[:, None] - idx[None] < case["window"]) |
                                                      (idx[None] < case["sinks"]))
                o, l = _exact_attention(s["q"][q0 + a:q0 + b], s["k"][k0 + idx], s["v"][k0 + idx], seen)
                outs.append(o)
                lses.append(l)
            q0, k0 = q0 + nq, k0 + nk
    else:
        at = 0
        for b, nk in enumerate(s["nk"].tolist()):
            idx = torch.arange(nk, device="cuda")
            if op == "wdecode":
                idx = idx[(idx >= nk - case["window"]) | (idx < case["sinks"])]
                n, seen = 1, torch.ones(1, len(idx), dtype=torch.bool, device="cuda")
            else:
                n = int(s["n"][b])
                seen = torch.ones(n, nk, dtype=torch.bool, device="cuda")
                for i, mask in enumerate(s["tree"][at:at + n].tolist()):
                    seen[i, nk - n:] = torch.tensor([mask >> x & 1 for x in range(n)], device="cuda") > 0
            o, l = _exact_attention(s["q"][at:at + n], *_exact_cached(s, b, idx), seen)
            outs.append(o)
            lses.append(l)
            at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses) if case["lse"] else None}
