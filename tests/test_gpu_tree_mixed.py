"""moe_attn_tree over batches whose sequences have few rows on average but for
some, with page tables so wide that small tiles do not have them all: over fp8
sequences of up to 16 rows a key/value head in small tiles and the others in
large ones, in two launches; over bf16 all in large ones."""
import json
import os
import random
import subprocess
import sys

import pytest

from tests import attn_util as au, serve_util as su
from tests.test_gpu_tree import _masks

pytestmark = pytest.mark.gpu


def _width(T, Hq, Hkv, D, fp8, page):
    """Table columns from which on small tiles do not have all (twice as many)."""
    rows = -(-T * (Hq // Hkv) // 8) * Hkv * (2 * D + 8 if fp8 else 4 * D)
    return 2 * (256 << 20) // (rows * page) + 1


def _batch(lens, nodes, Hq, Hkv, D, fp8, page, kind="tree", seed=0):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    rng = random.Random(seed)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = au.make_cache(seed, pages, Hkv, page, D, fp8)
    narrow = au.make_table(seed + 1, lens, page, pages, 0x7fffffff)
    T = sum(nodes)
    assert T * (Hq // Hkv) <= 8 * len(lens)
    table = torch.full((len(lens), _width(T, Hq, Hkv, D, fp8, page)), 0x7fffffff, dtype=torch.int32, device="cuda")
    table[:, :narrow.shape[1]] = narrow
    t = narrow.cpu()
    keep = [int(t[b, j // page]) * page + j % page for b, n in enumerate(lens) for j in range(n)]
    su.poison(cache, torch.tensor(keep, dtype=torch.long, device="cuda"))
    masks = [_masks(rng, n, kind) for n in nodes]
    tree = torch.tensor([m - (1 << 64) if m >> 63 else m for ms in masks for m in ms], dtype=torch.int64,
                        device="cuda")
    ws = moe.AttnWorkspace("cuda", "tree", len(lens), T, Hq, Hkv, D)
    return dict(cache=cache, table=table, narrow=narrow, lens=su.i32(lens), cu=su.i32(su.prefix(nodes)), tree=tree,
                masks=masks, q=au.randn(seed + 2, T, Hq, D), ws=ws)


def _call(x, out=None, lse=True, **change):
    import quantized_moe_expert_align_gb300 as moe
    x = dict(x, **change)
    return moe.attn_tree(x["q"], x["cache"], x["table"], x["lens"], x["cu"], x["tree"], out=out, lse=lse,
                         workspace=x["ws"])


def _check(x, out, lse, lens, nodes, skip=()):
    import torch
    at, D = 0, x["cache"].D
    for b, n in enumerate(lens):
        m, i = nodes[b], slice(at, at + nodes[b])
        at += m
        if m == 0 or b in skip:
            continue
        k, v = au.cached_rows(x["cache"], x["narrow"], b, n)
        seen = torch.ones(m, n, dtype=torch.bool, device="cuda")
        seen[:, n - m:] = torch.tensor([[w >> j & 1 > 0 for j in range(m)] for w in x["masks"][b]], device="cuda")
        ref, rl, tol, tl = su.seen_attention(x["q"][i], k, v, D ** -0.5, seen)
        au.check(out[i], ref, tol, f"out {b}")
        au.check(lse[i], rl, tl, f"lse {b}")


# (lengths, drafted tokens, heads): few rows on average
IDLE = [0] * 35 + [300] + [0] * 34, [0] * 35 + [64] + [0] * 34, 16, 2
MANY = {7: 20, 27: 40, 47: 20}
SOME = [100 + 7 * i for i in range(60)], [MANY.get(i, i % 2) for i in range(60)], 8, 2
BORDER = [60 + i for i in range(40)], [(4, 5, 0, 0, 0, 1, 0, 0)[i % 8] for i in range(40)], 16, 4
THIRDS = [90 + 5 * i for i in range(50)], [(5, 6, 0, 1, 0)[i % 5] for i in range(50)], 6, 2
FIFTHS = [200 - i for i in range(50)], [(3, 4, 0, 0, 1)[i % 5] for i in range(50)], 5, 1
WIDE = [400 if i % 9 == 2 else 0 for i in range(64)], [2 if i % 9 == 2 else 0 for i in range(64)], 20, 1
ONES = [1 + i for i in range(70)], [1] * 70, 8, 1


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 64)])
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("batch", [IDLE, SOME, BORDER, THIRDS, FIFTHS, WIDE, ONES])
def test_few_and_many_rows(gpu, batch, kind, D, page, fp8):
    import torch
    import quantized_moe_expert_align_gb300 as moe
    lens, nodes, Hq, Hkv = batch
    x = _batch(lens, nodes, Hq, Hkv, D, fp8, page, kind, seed=len(lens))
    got = []
    for _ in range(2):
        x["ws"].buf.random_(0, 255)
        got.append(_call(x))
        assert au.status(x["ws"]) == (moe.MOE_OK, 0)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    _check(x, *got[0], lens, nodes)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_behind_the_last_sequence(gpu, fp8):
    """Their outputs stay as they were."""
    import torch
    lens, nodes, Hq, Hkv = SOME
    x = _batch(lens, nodes, Hq, Hkv, 128, fp8, 16)
    T = sum(nodes)
    hold = torch.full((T + 12, Hq, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 12, Hq), 9.0, device="cuda")
    more = torch.nn.functional.pad
    _call(x, out=hold, lse=lse, q=more(x["q"], (0, 0, 0, 0, 0, 12)), tree=more(x["tree"], (0, 12)))
    assert (hold[T:] == 9.0).all() and (lse[T:] == 9.0).all()
    _check(x, hold[:T], lse[:T], lens, nodes)


@pytest.mark.parametrize("page_of,length_of,first", [
    ([3], [], 3), ([7], [], 7), ([7, 3], [], 3), ([3, 7], [50], 3), ([27], [9], 9), ([47], [50], 47), ([], [47], 47)])
def test_the_first_bad_sequence_of_both_launches(gpu, page_of, length_of, first):
    """Of few rows (3, 9, 50) or many (7, 27, 47): the first one is named, the others are right."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    lens, nodes, Hq, Hkv = SOME
    nodes = [max(n, 1) if i in (3, 9, 50) else n for i, n in enumerate(nodes)]
    x = _batch(lens, nodes, Hq, Hkv, 128, True, 16)
    table, d_lens = x["table"].clone(), x["lens"].clone()
    for b in page_of:
        table[b, 1] = -5
    for b in length_of:
        d_lens[b] = -1
    out, lse = _call(x, table=table, lens=d_lens)
    assert au.status(x["ws"]) == (moe.MOE_ERR_DEVICE_BAD_INDEX, first)
    _check(x, out, lse, lens, nodes, skip=page_of + length_of)
    out, lse = _call(x)
    assert au.status(x["ws"]) == (moe.MOE_OK, 0)
    _check(x, out, lse, lens, nodes)


@pytest.mark.parametrize("fp8", [False, True])
def test_captured(gpu, fp8):
    """One graph, other numbers of drafted tokens at every replay."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    lens, Hq, Hkv, D = [150 + 3 * i for i in range(60)], 8, 2, 128
    plans = [SOME[1], [2] * 60, [0] * 58 + [64, 56]]
    xs = [_batch(lens, n, Hq, Hkv, D, fp8, 16, seed=5) for n in plans]
    T = max(sum(n) for n in plans)
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    tree, cu = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros_like(xs[0]["cu"])
    out, lse = torch.zeros_like(q), torch.zeros(T, Hq, device="cuda")
    x = dict(xs[0], ws=moe.AttnWorkspace("cuda", "tree", 60, T, Hq, Hkv, D))

    def load(i):
        n = sum(plans[i])
        q[:n], tree[:n] = xs[i]["q"], xs[i]["tree"]
        cu.copy_(xs[i]["cu"])

    load(0)
    _call(x, out=out, lse=lse, q=q, tree=tree, cu=cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(x, out=out, lse=lse, q=q, tree=tree, cu=cu)
    for i in (0, 1, 2, 1, 0):
        load(i)
        out.fill_(9.0)
        graph.replay()
        assert au.status(x["ws"]) == (moe.MOE_OK, 0)
        n = sum(plans[i])
        _check(xs[i], out[:n], lse[:n], lens, plans[i])
        assert (out[n:] == 9.0).all()


_CHILD = """
import json, sys, time
sys.path.insert(0, sys.argv[1])
import torch
from tests import attn_util as au, test_gpu_tree_mixed as m
res = []
for fp8, D in ((False, 64), (True, 128)):
    # work for both launches, for the second alone, for the first alone
    for nodes in (m.SOME[1], [0] * 58 + [64, 50], [2] * 60):
        x = m._batch([100] * 60, nodes, 8, 2, D, fp8, 16)
        t0 = time.time()
        m._call(x)
        res.append([*au.status(x["ws"]), time.time() - t0])
y = (torch.arange(1024, device="cuda", dtype=torch.float32) * 2).sum().item()
print(json.dumps({"res": res, "y": y}))
"""


def test_bounded_waits_run_out(gpu):
    """The kernels issue no copies (a switch that is read once per process): the
    status says so, whichever launch's waits gave up."""
    import quantized_moe_expert_align_gb300 as moe
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _CHILD, root], env=dict(os.environ, MOE_ATTN_TEST_NO_COPIES="1"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    got = json.loads(r.stdout.strip().splitlines()[-1])
    assert got["y"] == float(sum(2 * i for i in range(1024))) and len(got["res"]) == 6
    for st, detail, secs in got["res"]:
        assert st == moe.MOE_ERR_DEVICE_TIMEOUT and detail >= 1 and secs < 30
