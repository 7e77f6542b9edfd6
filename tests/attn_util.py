"""Plain 64-bit forms of the attention half, and bounds on what 32-bit sums
with one rounding of weights and results may be off by."""
import math

import torch

U_BF16 = 2.0 ** -8     # half a unit in the last place of bf16, relative
FP8_MAX = 448.0


def randn(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def make_cache(seed, pages, Hkv, page, D, fp8):
    """A KVCache whose every token holds normal values."""
    import quantized_moe_expert_align_gb300 as moe
    x = randn(seed, pages, Hkv, 2, page, D)
    if not fp8:
        return moe.KVCache(x)
    x = x.float()
    amax = x.abs().amax(-1)
    return moe.KVCache((x * (FP8_MAX / amax)[..., None]).to(torch.float8_e4m3fn), amax / FP8_MAX)


def make_table(seed, lens, page, pages, spare_entry):
    """Shuffled pages; entries that no token needs hold `spare_entry`."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    need = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(need + [1]) + 1), spare_entry, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    assert at <= pages
    return table.cuda()


def cached_rows(cache, table, b, n):
    """K and V [n][Hkv][D] in 64 bits: code * scale."""
    t = torch.arange(n, device="cuda")
    pg, off = table[b].long()[t // cache.page_size], t % cache.page_size
    x = cache.data.view(torch.uint8 if cache.scales is not None else torch.int16)[pg, :, :, off]
    x = x.view(cache.data.dtype).double()
    if cache.scales is not None:
        x = x * cache.scales[pg, :, :, off].double()[..., None]
    return x[:, :, 0], x[:, :, 1]


def attention(q, k, v, scale, limit):
    """Row i of q [n][Hq][D] over its first limit[i] keys.  Returns the
    output and logsumexp in 64 bits and their bounds.

    Scores are fp32 sums of exact products: off by at most e = 2 D 2^-24
    max_j sum_d |q_d k_jd| scale plus 2^-20 for the exponent's own steps.
    A weight is then off by 2e relatively and rounded once to bf16, and the
    result is rounded to bf16."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    out = torch.zeros(n, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.full_like(lse, 1e-30)
    if m == 0 or n == 0:
        return out, lse, tol, tol_lse
    seen = torch.arange(m, device="cuda")[None] < limit[:, None]
    some = seen.any(-1)
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // Hkv)].double(), v[:, h // (Hq // Hkv)].double()
        x = (q[:, h].double() @ kh.T * scale).masked_fill(~seen, -math.inf)
        lse[:, h] = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[:, h:h + 1]).masked_fill(~seen, 0.0)
        # (a masked infinity or NaN takes no part)
        vh = torch.where(seen.any(0)[:, None], vh, torch.zeros_like(vh))
        out[:, h] = p @ vh
        mags = (q[:, h].double().abs() @ torch.where(seen.any(0)[:, None], kh, 0.0).abs().T) * scale
        e = 2 * D * 2.0 ** -24 * mags.masked_fill(~seen, 0.0).amax(-1) + 2.0 ** -20
        tol[:, h] = U_BF16 * out[:, h].abs() + (U_BF16 + 2 * e)[:, None] * (p @ vh.abs()) + 1e-30
        tol_lse[:, h] = e + 2.0 ** -22 * lse[:, h].abs()
    out[~some] = 0.0
    tol[~some] = 0.0
    tol_lse[~some] = 0.0
    return out, lse, tol, tol_lse


def check(got, ref, tol, what):
    got = got.double()
    same_inf = torch.isinf(ref) & (got == ref)
    d = torch.where(same_inf, torch.zeros_like(ref), (got - ref).abs())
    assert torch.isfinite(d).all(), f"{what}: not finite"
    bad = d > tol
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond tolerance, first at "
                             f"{i}: {got[i].item()} for {ref[i].item()}, tolerance {tol[i].item()}")


def status(ws):
    import quantized_moe_expert_align_gb300 as moe
    return moe.moe_w4a16_get_device_status(ws.buf)
