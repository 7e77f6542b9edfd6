"""moe_attn_tree over an fp8 cache with unusual scales, codes and queries: heads
of 64 and of 128, pages of 64 and 256, several sequences in a call; in small
tiles, in one row tile of 128 and in two.

Bounds, from the header's rounding notes: a score is off by e, fp32's steps
(serve_util.seen_attention derives them) and 2^-17 of its head's largest value
of q times sum |k| scale; a weight then by exp(2 e) - 1 of itself.  Its rounding
(and that of v) is at most 2^-8 of sum p |v| in small tiles, 2^-9 in those of
128, where a value of v may be off by 2^-24 of the largest scale's power of two
above, and a weight by 2^-31 of the largest one's (fp16 with 2^6: 2^-25 / 2^6)."""
import math

import pytest

from tests import attn_util as au, serve_util as su

pytestmark = pytest.mark.gpu

HQ, HKV = 16, 2
LENS = [1500, 64, 333, 700]
# drafted tokens, what weights and values are rounded by
KINDS = {"small": ([1, 2, 1, 1], 2.0 ** -8), "one": ([9, 16, 3, 10], 2.0 ** -9),
         "two": ([40, 64, 5, 33], 2.0 ** -9)}
both = pytest.mark.parametrize("D,page", [(64, 64), (64, 256), (128, 64), (128, 256)])
kinds = pytest.mark.parametrize("kind", list(KINDS))


class Batch:
    def __init__(self, D, page, kind, seed):
        import torch
        self.D, self.page = D, page
        self.nodes, self.unit = KINDS[kind]
        pages = sum(-(-n // page) for n in LENS) + 1
        self.cache = au.make_cache(seed, pages, HKV, page, D, True)
        self.table = au.make_table(seed + 1, LENS, page, pages, 0)
        self.q = au.randn(seed + 2, sum(self.nodes), HQ, D)
        self.cu = su.prefix(self.nodes)
        self.tree = torch.tensor([(2 << i) - 1 if i < 63 else -1 for n in self.nodes for i in range(n)],
                                 dtype=torch.int64, device="cuda")

    def at(self, b):
        """Pages and places of sequence b's tokens."""
        import torch
        t = torch.arange(LENS[b], device="cuda")
        return self.table[b].long()[t // self.page], t % self.page

    def run(self):
        import quantized_moe_expert_align_gb300 as moe
        ws = moe.AttnWorkspace("cuda", "tree", len(LENS), sum(self.nodes), HQ, HKV, self.D)
        got = moe.attn_tree(self.q, self.cache, self.table, su.i32(LENS), su.i32(self.cu), self.tree, lse=True,
                            workspace=ws)
        assert au.status(ws) == (moe.MOE_OK, 0)
        return got

    def check(self):
        import torch
        out, lse = self.run()
        D, G, scale = self.D, HQ // HKV, self.D ** -0.5
        for b, n in enumerate(LENS):
            m, rows = self.nodes[b], slice(self.cu[b], self.cu[b + 1])
            pg, off = self.at(b)
            s = self.cache.scales[pg, :, :, off].double()
            x = self.cache.data.view(torch.uint8)[pg, :, :, off].view(self.cache.data.dtype).double() * s[..., None]
            seen = torch.arange(n, device="cuda")[None] <= torch.arange(n - m, n, device="cuda")[:, None]
            for h in range(HQ):
                k, v = x[:, h // G, 0], x[:, h // G, 1]
                q = self.q[rows, h].double()
                y = (q @ k.T * scale).masked_fill(~seen, -math.inf)
                ref_l = torch.logsumexp(y, -1)
                p = torch.exp(y - ref_l[:, None])
                ref = p @ v
                mags = (q.abs() @ k.abs().T * scale).amax(-1)
                e = 2 * D * 2.0 ** -24 * mags + 2.0 ** -20
                e = e + 2.0 ** -17 * q.abs().amax(-1) * k.abs().sum(-1).max() * scale
                pv = p @ v.abs()
                # (a moved weight, whatever the exponent, takes at most the largest |v| instead)
                moved = torch.minimum((torch.exp(2 * e) - 1)[:, None] * pv, 2 * v.abs().amax())
                tol = self.unit * pv + moved + n * 2.0 ** -31 * v.abs().amax()
                if self.unit < 2.0 ** -8:
                    tol = tol + 2.0 ** -24 * 2.0 ** (math.floor(math.log2(max(float(s[:, h // G, 1].max()), 1e-38))) + 1)
                tol = (1 + 2.0 ** -8) * tol + 2.0 ** -8 * ref.abs() + 1e-30
                au.check(out[rows, h], ref, tol, f"out {b} {h}")
                au.check(lse[rows, h], ref_l, e + 2.0 ** -22 * ref_l.abs(), f"lse {b} {h}")


@both
@kinds
def test_normal_values(gpu, kind, D, page):
    Batch(D, page, kind, 1).check()


@both
@kinds
@pytest.mark.parametrize("how", ["rising", "falling", "random", "one large", "one small"])
def test_scales_of_all_sizes(gpu, how, kind, D, page):
    import torch
    x = Batch(D, page, kind, 4)
    g = torch.Generator(device="cuda").manual_seed(7)
    for b, n in enumerate(LENS):
        t = torch.arange(n, device="cuda", dtype=torch.float32)
        f = {"rising": torch.exp2(torch.floor(t * 15 / n) - 7), "falling": torch.exp2(7 - torch.floor(t * 15 / n)),
             "random": torch.exp2(torch.randint(-6, 7, (n,), generator=g, device="cuda").float()),
             "one large": torch.where(t == n // 2, 4096.0, 1.0),
             "one small": torch.where(t == n // 2, 1e-20, 1.0)}[how]
        pg, off = x.at(b)
        x.cache.scales[pg, :, 1, off] *= f[:, None]
    x.check()


@both
@kinds
def test_zero_rows(gpu, kind, D, page):
    x = Batch(D, page, kind, 8)
    for b in range(len(LENS)):
        pg, off = x.at(b)
        x.cache.scales[pg[::3], :, 1, off[::3]] = 0.0
        x.cache.scales[pg[::5], :, :, off[::5]] = 0.0
    x.check()


@both
@kinds
def test_queries_with_outliers(gpu, kind, D, page):
    x = Batch(D, page, kind, 12)
    x.q[:, 0, 3] *= 64
    x.q[:, 1, D - 3] *= 1000
    x.q[:, 2] *= 1e-20
    x.q[:, 3] = 0
    x.q[:, 4] *= 2.0 ** -120
    x.check()


@both
@kinds
def test_nan_codes_and_infinite_queries(gpu, kind, D, page):
    """They stay with their column, or their row, of their own sequence."""
    import torch
    x = Batch(D, page, kind, 16)
    ref, ref_l = x.run()
    bits = x.cache.data.view(torch.uint8)
    pg, off = x.at(2)
    bits[pg[50], 0, 1, off[50], 7] = 0x7F
    bits[pg[60], 1, 1, off[60], D - 28] = 0xFF
    last, end = int(pg[-1]), LENS[2] % page
    if end:  # behind the last token it is nothing
        bits[last, :, :, end:] = 0x7F
        x.cache.scales[last, :, :, end:] = float("inf")
    a, z = x.cu[2], x.cu[3]
    want = torch.zeros_like(ref, dtype=torch.bool)
    want[a:z, :8, 7] = want[a:z, 8:, D - 28] = True
    out, lse = x.run()
    assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], ref[~want]) and torch.equal(lse, ref_l)
    bits[pg[70], 1, 0, off[70], 0] = 0x7F
    x.q[0, 3, D - 1], x.q[x.cu[3], 9, 0] = float("inf"), float("nan")
    want[a:z, 8:] = want[0, 3] = want[x.cu[3], 9] = True
    out, lse = x.run()
    assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], ref[~want])
    assert torch.equal(torch.isnan(lse), want.all(-1))
