"""Plain forms of serving over the paged cache: attention by a matrix of which
key is seen, in 64 bits with bounds, and page plans token by token."""
import math

import torch

from tests import attn_util as au


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prefix(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def seen_attention(q, k, v, scale, seen):
    """q [n][Hq][D] over k, v [m][Hkv][D] where seen [n][m]: (out, lse) in 64
    bits and their bounds, those of attn_util.attention."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    out = torch.zeros(n, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    if m == 0 or n == 0:
        return out, lse, tol, tol_lse
    some, used = seen.any(1), seen.any(0)[:, None]
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // Hkv)].double(), v[:, h // (Hq // Hkv)].double()
        # (a masked infinity or NaN takes no part)
        kh, vh = torch.where(used, kh, 0.0), torch.where(used, vh, 0.0)
        x = (q[:, h].double() @ kh.T * scale).masked_fill(~seen, -math.inf)
        lse[:, h] = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[:, h:h + 1]).masked_fill(~seen, 0.0)
        out[:, h] = p @ vh
        mags = (q[:, h].double().abs() @ kh.abs().T) * scale
        e = 2 * D * 2.0 ** -24 * mags.masked_fill(~seen, 0.0).amax(-1) + 2.0 ** -20
        tol[:, h] = au.U_BF16 * out[:, h].abs() + (au.U_BF16 + 2 * e)[:, None] * (p @ vh.abs()) + 1e-30
        tol_lse[:, h] = e + 2.0 ** -22 * lse[:, h].abs()
    out[~some], lse[~some], tol[~some], tol_lse[~some] = 0.0, -math.inf, 0.0, 0.0
    return out, lse, tol, tol_lse


def window_seen(pos, m, window, sinks):
    """Which of m keys a row at each of the places pos sees."""
    j = torch.arange(m, device="cuda")[None]
    pos = pos[:, None]
    return (j <= pos) & ((j > pos - window) | (j < sinks))


def poison(cache, keep):
    """Everything of the cache but the slots in keep becomes NaN (scales too)."""
    free = torch.ones(cache.num_pages * cache.page_size, dtype=torch.bool, device="cuda")
    free[keep] = False
    free = free.view(cache.num_pages, 1, 1, cache.page_size).expand(-1, cache.Hkv, 2, -1)
    if cache.scales is not None:
        cache.data.view(torch.uint8)[free] = 0x7f
        cache.scales[free] = float("nan")
    else:
        cache.data[free] = float("nan")


def plan(ring, state, table, page, lens, new, kept, offsets, window, sinks, rows, dropped=None):
    """One step on the host (lists; ring and table change): state, lens, kept,
    cu_q, cu_k, positions, slots, or None if the step cannot be made."""
    cap, (head, count) = len(ring), state
    first = -(-sinks // page)
    lens2, kept2, cu, pos, slots, taken, back = [], [], [0], [], [], 0, []
    entries = {}
    for b, (n0, n) in enumerate(zip(lens, new)):
        held = -(-(n0 + (dropped[b] if dropped else 0)) // page)
        if n < 0:
            back += [table[b][p] for p in range(held) if not window or p < first or p >= kept[b]]
            lens2.append(0)
            kept2.append(0)
            cu.append(cu[-1])
            continue
        behind = max(0, n0 + 1 - window) // page if window else 0
        if window:
            back += [table[b][p] for p in range(max(first, kept[b]), behind)]
        kept2.append(max(kept[b], behind) if window else 0)
        back += [table[b][p] for p in range(-(-(n0 + n) // page), held)]
        for i in range(n):
            j = n0 + i
            p = j // page
            if p >= len(table[b]):
                return None
            if p >= held and (b, p) not in entries:
                if taken == count:
                    return None
                entries[b, p] = ring[(head + taken) % cap]
                taken += 1
            at = entries.get((b, p), table[b][p])
            pos.append(n0 + offsets[cu[-1] + i] if offsets is not None else j)
            slots.append(at * page + j % page)
        lens2.append(n0 + n)
        cu.append(cu[-1] + n)
    if cu[-1] > rows:
        return None
    for (b, p), v in entries.items():
        table[b][p] = v
    for i, v in enumerate(back):
        ring[(head + count + i) % cap] = v
    pos += [0] * (rows - len(pos))
    slots += [-1] * (rows - len(slots))
    return [(head + taken) % cap, count - taken + len(back)], lens2, kept2, cu, prefix(lens2), pos, slots
