"""The operators of a decoder layer's attention half, as cases to be measured.

Each case is one call (or one small chain of calls) that a server makes for a batch: per-head norms of
queries and keys with the rotation and the cache write (``append``), the read-back of cached tokens
(``gather``), attention of single tokens over the paged cache (``decode``) and attention over packed
prompts (``prefill``).  ``run`` computes a case in plain torch operations (``own`` false) or through the
framework's entry points (``own`` true) on the same prepared inputs.

Cache layout (both sides): data [num_pages][Hkv][2 (K, V)][page][D] bf16 or fp8 e4m3, fp8 with fp32
scales [num_pages][Hkv][2][page], one per token and head; value = code * scale.
"""
import math
import random

import torch

own = False

FP8_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token of one request: latency of the step's first kernel
        dict(name="append_token", op="append", T=1, Hq=64, Hkv=8, D=128, rot=128, inter=False,
             norm=True, kv="fp8", page=16, k_out=False),
        # a decode batch of 90 requests, interleaved rotation of half of each head, bf16 cache
        dict(name="append_90", op="append", T=90, Hq=32, Hkv=4, D=128, rot=64, inter=True,
             norm=True, kv="bf16", page=16, k_out=False),
        # prompts of 16384 tokens: rotated keys also go to the prompt attention
        dict(name="append_16384", op="append", T=16384, Hq=64, Hkv=8, D=128, rot=128, inter=False,
             norm=True, kv="fp8", page=64, k_out=True),
        # the context of one chunk of one request, read back for its prompt attention
        dict(name="gather_2000", op="gather", B=1, max_len=2000, Hkv=4, D=64, kv="bf16", page=16),
        # the contexts of eight long requests
        dict(name="gather_8x32768", op="gather", B=8, max_len=32768, Hkv=8, D=128, kv="fp8",
             page=64),
        # one request with a short context: latency of a decode step
        dict(name="decode_1x517", op="decode", B=1, max_len=517, Hq=64, Hkv=8, D=128, kv="bf16",
             page=16, lse=False),
        # one request with a long context: the keys have to be split over the whole card
        dict(name="decode_1x131072", op="decode", B=1, max_len=131072, Hq=64, Hkv=8, D=128,
             kv="fp8", page=64, lse=False),
        # 90 requests of ragged lengths, bf16 cache in small pages
        dict(name="decode_90x8192", op="decode", B=90, max_len=8192, Hq=32, Hkv=4, D=128,
             kv="bf16", page=16, lse=True),
        # a full server: 256 requests of ragged lengths, fp8 cache
        dict(name="decode_256x8192", op="decode", B=256, max_len=8192, Hq=64, Hkv=8, D=128,
             kv="fp8", page=64, lse=False),
        # one prompt of 1024 tokens: time to the first token
        dict(name="prefill_1024", op="prefill", B=1, max_q=1024, ctx=0, Hq=32, Hkv=4, D=128,
             causal=True, lse=False),
        # six prompts of ragged lengths up to 4096 in one call
        dict(name="prefill_6x4096", op="prefill", B=6, max_q=4096, ctx=0, Hq=64, Hkv=8, D=128,
             causal=True, lse=False),
        # chunks of up to 1000 tokens of four requests, each after a long context; heads of 64
        dict(name="prefill_chunks", op="prefill", B=4, max_q=1000, ctx=15000, Hq=32, Hkv=4, D=64,
             causal=True, lse=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(["append", "append", "gather", "decode", "decode", "decode", "prefill",
                     "prefill", "prefill"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8, 8, 16])
    D = rng.choice([64, 128, 128])
    kv = rng.choice(["bf16", "fp8"])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        rot = rng.choice([D, D, D // 2, D // 4, 0])
        return dict(op=op, T=_log_int(rng, 1, 16384), Hq=Hkv * G, Hkv=Hkv, D=D, rot=rot,
                    inter=rng.random() < 0.5, norm=rng.random() < 0.7, kv=kv, page=page,
                    k_out=rng.random() < 0.5)
    if op == "gather":
        return dict(op=op, B=_log_int(rng, 1, 64), max_len=_log_int(rng, 1, 32768), Hkv=Hkv, D=D,
                    kv=kv, page=page)
    if op == "decode":
        return dict(op=op, B=_log_int(rng, 1, 256), max_len=_log_int(rng, 1, 131072), Hq=Hkv * G,
                    Hkv=Hkv, D=D, kv=kv, page=page, lse=rng.random() < 0.5)
    ctx = 0 if rng.random() < 0.5 else _log_int(rng, 1, 15000)
    return dict(op=op, B=_log_int(rng, 1, 16), max_q=_log_int(rng, 1, 4096), ctx=ctx, Hq=Hkv * G,
                Hkv=Hkv, D=D, causal=rng.random() < 0.75, lse=rng.random() < 0.5)


def _cost(case):
    """Seconds that the case's plain form roughly takes, from what it holds in 32 bits."""
    op = case["op"]
    if op == "append":
        return case["T"] * (case["Hq"] + 2 * case["Hkv"]) * case["D"] * 1e-11
    if op in ("gather", "decode"):
        return case["B"] * case["max_len"] * case["Hkv"] * case["D"] * 1e-11
    return case["B"] * case["max_q"] * (case["max_q"] + case["ctx"]) * case["Hq"] * 1e-11


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


def _ragged(n, longest, salt):
    """n lengths in [longest/8, longest], the first the longest: a fixed function of its arguments."""
    r = random.Random(n * 1000003 + longest * 101 + salt)
    lo = max(1, longest // 8)
    return [longest] + [_log_int(r, lo, longest) for _ in range(n - 1)]


def _lens(case):
    """(query lengths, key lengths) of the case's sequences."""
    if case["op"] == "prefill":
        nq = _ragged(case["B"], case["max_q"], 1)
        ctx = _ragged(case["B"], case["ctx"], 2) if case["ctx"] else [0] * case["B"]
        return nq, [a + b for a, b in zip(nq, ctx)]
    return [1] * case["B"], _ragged(case["B"], case["max_len"], 3)


def work(case):
    D, Hkv, op = case["D"], case["Hkv"], case["op"]
    Hq = case.get("Hq", 0)
    row = (D + 4) if case.get("kv") == "fp8" else 2 * D      # one cached K or V row of one head
    if op == "append":
        T = case["T"]
        n = T * ((Hq + 2 * Hkv) * D * 2 + case["rot"] * 4 + 8 + Hq * D * 2 + 2 * Hkv * row)
        return {"bytes": n + (T * Hkv * D * 2 if case["k_out"] else 0),
                "flops": T * (Hq + Hkv) * D * 8}
    nq, nk = _lens(case)
    if op == "gather":
        return {"bytes": sum(nk) * 2 * Hkv * (row + 2 * D), "flops": sum(nk) * 2 * Hkv * D}
    if op == "decode":
        return {"bytes": sum(nk) * 2 * Hkv * row + case["B"] * Hq * D * 4,
                "flops": 4 * Hq * D * sum(nk)}
    pairs = sum((q * k - q * (q - 1) // 2) if case["causal"] else q * k for q, k in zip(nq, nk))
    return {"bytes": 4 * D * (sum(nq) * Hq + sum(nk) * Hkv) + (4 * Hq * sum(nq) if case["lse"] else 0),
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


def _rope_table(max_pos, rot):
    """[max_pos][rot] fp32: the rot/2 cosines, then the rot/2 sines, of pos * 10000^(-2i/rot)."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


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


def _paged(g, nk, page, spare):
    """Page table [B][most] (unused entries 0) over shuffled pages, and the number of pages."""
    need = [-(-n // page) for n in nk]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(nk), max(max(need), 1), dtype=torch.int32)
    at = 0
    order = order.cpu()
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda(), total


def _prefix(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g, op, D, Hkv = _gen(seed), case["op"], case["D"], case["Hkv"]
    s = {"case": dict(case)}
    if op == "append":
        T, Hq, page = case["T"], case["Hq"], case["page"]
        # the rows of one fused projection: queries, keys, values
        qkv = _randn(g, T, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q_norm"] = (1 + 0.1 * _randn(g, D, dtype=torch.float32)).bfloat16() if case["norm"] else None
        s["k_norm"] = (1 + 0.1 * _randn(g, D, dtype=torch.float32)).bfloat16() if case["norm"] else None
        max_pos = max(32768, T)
        s["cos_sin"] = _rope_table(max_pos, case["rot"])
        s["positions"] = torch.randint(0, max_pos, (T,), generator=g, device="cuda",
                                       dtype=torch.int32)
        pages = -(-T // page) + 8
        s["data"], s["scales"] = _filled_cache(g, pages, Hkv, page, D, case["kv"])
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
        return s
    nq, nk = _lens(case)
    s["nk"] = torch.tensor(nk, dtype=torch.int32, device="cuda")
    s["cu_k"] = _prefix(nk)
    s["total_k"] = sum(nk)
    if op in ("gather", "decode"):
        s["table"], pages = _paged(g, nk, case["page"], 8)
        s["data"], s["scales"] = _filled_cache(g, pages, Hkv, case["page"], D, case["kv"])
        if op == "decode":
            s["q"] = _randn(g, case["B"], case["Hq"], D)
        return s
    Hq = case["Hq"]
    s["nq"] = torch.tensor(nq, dtype=torch.int32, device="cuda")
    s["cu_q"] = _prefix(nq)
    s["q"] = _randn(g, sum(nq), Hq, D)
    kv = _randn(g, sum(nk), 2 * Hkv, D)
    s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
    s["max_q"], s["max_k"] = max(nq), max(nk)
    return s


# ---------------------------------------------------------------------------
# the plain forms: elementary operations in 32 bits, rounded once
# ---------------------------------------------------------------------------
def _norm_rotate(x, w, s):
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    h = c["rot"] // 2
    if h == 0:
        return x
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :h], cs[..., h:]
    y = x.clone()
    if c["inter"]:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_append(s):
    c = s["case"]
    q = _norm_rotate(s["q"], s["q_norm"], s).bfloat16()
    k = _norm_rotate(s["k"], s["k_norm"], s)
    rows = torch.stack([k, s["v"].float()], 2)                  # [T][Hkv][2][D]
    slot = s["slots"].long()
    page, off = slot // c["page"], slot % c["page"]
    if c["kv"] == "fp8":
        codes, scales = _quantise(rows)
        s["data"].view(torch.uint8)[page, :, :, off] = codes.view(torch.uint8)
        s["scales"][page, :, :, off] = scales
    else:
        s["data"][page, :, :, off] = rows.bfloat16()
    return {"q": q, "k": k.bfloat16() if c["k_out"] else None, "data": s["data"],
            "scales": s["scales"]}


def _cached(s):
    """Dequantised pages of every sequence: K and V, each [B][Hkv][pages * page][D] fp32."""
    t = s["table"].long()
    data = s["data"]
    if data.dtype == torch.bfloat16:
        x = data[t].float()
    else:
        x = data.view(torch.uint8)[t].view(torch.float8_e4m3fn).float()
        x *= s["scales"][t][..., None]
    B, n, Hkv, _, page, D = x.shape
    x = x.permute(3, 0, 2, 1, 4, 5).reshape(2, B, Hkv, n * page, D)
    return x[0], x[1]


def _packed_index(cu, lens, most):
    """For padded rows [B][most]: the packed row of each (0 where there is none) and which exist."""
    i = torch.arange(most, device="cuda")
    there = i[None] < lens[:, None]
    return torch.where(there, cu[:-1, None] + i[None], torch.zeros_like(i)[None]).long(), there


def _plain_gather(s):
    k, v = _cached(s)
    _, there = _packed_index(s["cu_k"], s["nk"], k.shape[2])
    return {"k": k.transpose(1, 2)[there].bfloat16(), "v": v.transpose(1, 2)[there].bfloat16()}


def _softmax_product(x, seen, v):
    """Rows of scores x (in place) over the keys `seen`, times v: (output, logsumexp)."""
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.where(total > 0, m + total.log(), torch.full_like(total, -math.inf))
    return out, lse[..., 0]


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    k, v = _cached(s)
    x = torch.matmul(s["q"].float().view(B, Hkv, Hq // Hkv, D) * D ** -0.5, k.transpose(2, 3))
    seen = torch.arange(k.shape[2], device="cuda")[None] < s["nk"][:, None]
    out, lse = _softmax_product(x, seen[:, None, None], v)
    return {"out": out.reshape(B, Hq, D).bfloat16(), "lse": lse.reshape(B, Hq) if c["lse"] else None}


def _plain_prefill(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    G, n, m = Hq // Hkv, s["max_q"], s["max_k"]
    iq, there = _packed_index(s["cu_q"], s["nq"], n)
    ik, key = _packed_index(s["cu_k"], s["nk"], m)
    q = s["q"][iq].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4) * D ** -0.5
    k = s["k"][ik].float().permute(0, 2, 3, 1)[:, :, None]
    v = s["v"][ik].float().permute(0, 2, 1, 3)[:, :, None]
    seen = key[:, None].expand(B, n, m)
    if c["causal"]:
        last = torch.arange(n, device="cuda")[None] + (s["nk"] - s["nq"])[:, None]
        seen = seen & (torch.arange(m, device="cuda")[None, None] <= last[..., None])
    out, lse = _softmax_product(torch.matmul(q, k), seen[:, None, None], v)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[there].bfloat16()
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, Hq)[there]
    return {"out": out, "lse": lse if c["lse"] else None}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _kept(s):
    """What a serving loop makes once and keeps: the cache handle, workspace and output buffers."""
    import quantized_moe_expert_align_gb300 as moe
    c, op, D = s["case"], s["case"]["op"], s["case"]["D"]
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    h = {"moe": moe}
    if op != "prefill":
        h["cache"] = moe.KVCache(s["data"], s["scales"])
    if op == "append":
        h["ws"] = moe.AttnWorkspace("cuda")
        h["q_out"] = new(c["T"], c["Hq"], D)
        h["k_out"] = new(c["T"], c["Hkv"], D) if c["k_out"] else None
    elif op == "gather":
        h["ws"] = moe.AttnWorkspace("cuda")
        h["k_out"], h["v_out"] = new(s["total_k"], c["Hkv"], D), new(s["total_k"], c["Hkv"], D)
    else:
        rows = c["B"] if op == "decode" else s["q"].shape[0]
        h["ws"] = moe.AttnWorkspace("cuda", op, c["B"], rows, c["Hq"], c["Hkv"], D)
        h["out"] = new(rows, c["Hq"], D)
        h["lse"] = new(rows, c["Hq"], dtype=torch.float32) if c["lse"] else None
    return h


def _own(s):
    if "kept" not in s:
        s["kept"] = _kept(s)
    h, c = s["kept"], s["case"]
    moe = h["moe"]
    if c["op"] == "append":
        moe.qk_rope_append(s["q"], s["k"], s["v"], s["cos_sin"], s["positions"], h["cache"],
                           s["slots"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                           interleaved=c["inter"], q_out=h["q_out"], k_out=h["k_out"],
                           workspace=h["ws"])
        return {"q": h["q_out"], "k": h["k_out"], "data": s["data"], "scales": s["scales"]}
    if c["op"] == "gather":
        moe.kv_gather(h["cache"], s["table"], s["cu_k"], s["total_k"], k_out=h["k_out"],
                      v_out=h["v_out"], workspace=h["ws"])
        return {"k": h["k_out"], "v": h["v_out"]}
    if c["op"] == "decode":
        moe.attn_decode(s["q"], h["cache"], s["table"], s["nk"], out=h["out"], lse=h["lse"],
                        workspace=h["ws"])
    else:
        moe.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"],
                         out=h["out"], lse=h["lse"], workspace=h["ws"])
    return {"out": h["out"], "lse": h["lse"]}


_PLAIN = {"append": _plain_append, "gather": _plain_gather, "decode": _plain_decode,
          "prefill": _plain_prefill}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _exact_rows(x, w, s):
    """Per-head norm and rotation as complex numbers."""
    c = s["case"]
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS) * w.double()
    rot = c["rot"]
    if rot == 0:
        return x
    turn = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(turn[:, :rot // 2], turn[:, rot // 2:])[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    if c["inter"]:
        z = torch.view_as_complex(head.unflatten(-1, (rot // 2, 2)).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(*head.chunk(2, -1)) * turn
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, rest], -1)


def _exact_append(s):
    c = s["case"]
    q, k = _exact_rows(s["q"], s["q_norm"], s), _exact_rows(s["k"], s["k_norm"], s)
    rows = torch.stack([k, s["v"].double()], 2)
    data = s["data"].float().double()
    scales = s["scales"].double() if s["scales"] is not None else None
    slot = s["slots"].long()
    page, off = slot // c["page"], slot % c["page"]
    if scales is not None:
        most = rows.abs().amax(-1)
        scales[page, :, :, off] = most / FP8_MAX
        # (the codes before their rounding to 8 bits)
        rows = torch.where(most[..., None] > 0, rows / most[..., None] * FP8_MAX, rows)
    data[page, :, :, off] = rows
    return {"q": q, "k": k if c["k_out"] else None, "data": data, "scales": scales}


def _exact_cached(s, b, n):
    """K and V [n][Hkv][D] of sequence b."""
    page = s["case"]["page"]
    t = torch.arange(n, device="cuda")
    pg, off = s["table"][b].long()[t // page], t % page
    d = s["data"]
    if d.dtype == torch.bfloat16:
        x = d[pg, :, :, off].double()
    else:
        x = d.view(torch.uint8)[pg, :, :, off].view(torch.float8_e4m3fn).double()
        x = x * s["scales"][pg, :, :, off].double()[..., None]
    return x[:, :, 0], x[:, :, 1]


def _exact_attention(q, k, v, limit):
    """q [n][Hq][D], k / v [m][Hkv][D]; row i sees its first limit[i] keys: (out, lse)."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    seen = torch.arange(m, device="cuda")[None] < limit[:, None]
    out, lse = torch.empty_like(q, dtype=torch.float64), torch.empty(n, Hq, dtype=torch.float64, device="cuda")
    for h in range(Hq):
        kh, vh = k[:, h * Hkv // Hq].double(), v[:, h * Hkv // Hq].double()
        x = (q[:, h].double() @ kh.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
        lse[:, h] = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[:, h:h + 1])
        out[:, h] = torch.where(seen.any(-1, keepdim=True), p, torch.zeros_like(p)) @ vh
    return out, lse


def exact(case, seed):
    nq, nk = _lens(case) if case["op"] != "append" else ([], [])
    if case["op"] in ("decode", "prefill") and work(case)["flops"] > 5e12:
        return None
    if case["op"] == "decode" and sum(nk) * case["Hq"] > 2e8:
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "gather":
        parts = [_exact_cached(s, b, n) for b, n in enumerate(nk)]
        return {"k": torch.cat([p[0] for p in parts]), "v": torch.cat([p[1] for p in parts])}
    outs, lses, at_q, at_k = [], [], 0, 0
    for b in range(case["B"]):
        q = s["q"][at_q:at_q + nq[b]]
        limit = torch.full((nq[b],), nk[b], device="cuda")
        if case["op"] == "decode":
            k, v = _exact_cached(s, b, nk[b])
        else:
            k, v = s["k"][at_k:at_k + nk[b]], s["v"][at_k:at_k + nk[b]]
            if case["causal"]:
                limit = torch.arange(nq[b], device="cuda") + nk[b] - nq[b] + 1
        o, l = _exact_attention(q, k, v, limit)
        outs.append(o)
        lses.append(l)
        at_q, at_k = at_q + nq[b], at_k + nk[b]
    return {"out": torch.cat(outs), "lse": torch.cat(lses) if case["lse"] else None}
