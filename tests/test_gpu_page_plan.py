"""moe_page_plan against plans made token by token."""
import random

import pytest

from tests import attn_util as au, serve_util as su

pytestmark = pytest.mark.gpu


class Both:
    """A pool, a table and lengths on both sides."""

    def __init__(self, B, width, pages, page, window=0, sinks=0, head=0):
        import quantized_moe_expert_align_gb300 as moe
        self.page, self.window, self.sinks = page, window, sinks
        order = list(range(pages))
        random.Random(pages).shuffle(order)
        self.ring = [order[(i - head) % pages] for i in range(pages)]
        self.state, self.table = [head, pages], [[-7] * width for _ in range(B)]
        self.lens, self.kept = [0] * B, [0] * B
        self.pool = moe.PagePool(su.i32(self.ring), su.i32(self.state))
        self.d_table, self.d_lens, self.d_kept = su.i32(self.table), su.i32(self.lens), su.i32(self.kept)
        self.ws = moe.AttnWorkspace("cuda", "pages", B)

    def step(self, new, rows, offsets=None, in_place=True, detail=None, own_state=False,
             dropped=None):
        import torch
        import quantized_moe_expert_align_gb300 as moe
        own = dict(seq_lens=self.d_lens, kept=self.d_kept if self.window else None) if in_place else {}
        out = moe.PagePlan.empty(len(new), rows, self.window > 0, **own)
        if own_state:
            out.state = torch.full_like(self.pool.state, -9)
        self.ws.buf.random_(0, 255)
        got = moe.page_plan(self.pool, self.d_table, self.d_lens, su.i32(new), self.page, rows,
                            window=self.window, sinks=self.sinks, kept=self.d_kept if self.window else None,
                            offsets=None if offsets is None else su.i32(offsets), out=out, workspace=self.ws,
                            dropped=None if dropped is None else su.i32(dropped))
        assert got is out
        want = su.plan(self.ring, self.state, self.table, self.page, self.lens, new, self.kept, offsets,
                       self.window, self.sinks, rows, dropped)
        status = au.status(self.ws)
        if want is None:
            assert detail is not None and status == (moe.MOE_ERR_DEVICE_BAD_INDEX, detail)
            B = len(new)
            want = self.state, self.lens, self.kept, [0] * (B + 1), [0] * (B + 1), [0] * rows, [-1] * rows
        else:
            assert detail is None and status == (moe.MOE_OK, 0)
        self.state, self.lens, self.kept = want[:3]
        names = ["state", "seq_lens", "kept", "cu_q", "cu_k", "positions", "slots"]
        for name, w in zip(names, want):
            if name != "state" and (name != "kept" or self.window):
                assert getattr(out, name).tolist() == list(w), name
        if own_state:
            assert out.state.tolist() == self.state
            self.pool.state.copy_(out.state)
        assert self.pool.state.tolist() == self.state
        assert torch.equal(self.d_table, su.i32(self.table))
        assert torch.equal(self.pool.ring, su.i32(self.ring))
        self.d_lens = out.seq_lens
        if self.window:
            self.d_kept = out.kept
        return out


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 4), (100, 40)])
@pytest.mark.parametrize("B,page,in_place", [(1, 16, True), (7, 16, False), (40, 64, True), (1500, 16, True)])
def test_steps(gpu, B, page, in_place, window, sinks):
    """Prompts, single tokens, drafts, finished requests and new ones in their places."""
    rng = random.Random(B + window)
    width = -(-700 // page)
    x = Both(B, width, B * width + 3, page, window, sinks, head=5 % (B * width + 3))
    x.step([rng.choice([0, 1, 5, 200]) for _ in range(B)], 200 * B + 9, in_place=in_place)
    for _ in range(6):
        new = [-1 if rng.random() < 0.1 else rng.choice([1, 1, 0, 3, 90]) for _ in range(B)]
        rows = sum(max(n, 0) for n in new) + rng.choice([0, 13])
        x.step(new, rows, in_place=in_place)
        new = [min(1, max(v, 0)) for v in new]
        n = sum(new)
        x.step(new, n, offsets=[rng.randrange(9) for _ in range(n)], in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows", [4096, 4097, 20000])
def test_one_prompt(gpu, rows, in_place):
    """Both sides of the size up to which one block fills the rows."""
    x = Both(1, 1000, 1100, 16)
    x.step([4000], rows, in_place=in_place)
    x.step([-1], rows, in_place=in_place)
    x.step([96], rows, in_place=in_place)


@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 20)])
@pytest.mark.parametrize("B", [3, 900, 1024, 1025])
def test_many_rows_with_new_outputs(gpu, B, window, sinks):
    """Every block makes the sums for itself, up to 1024 sequences; lengths, kept
    pages and the pool's state go to tensors of their own."""
    rng = random.Random(B)
    n = 9000 // B + 30
    width = -(-4 * n // 16) + 1
    x = Both(B, width, B * width, 16, window, sinks)
    for last in range(3):
        new = [rng.choice([n, n // 2, 0, 3, -1 if last else 1]) for _ in range(B)]
        x.step(new, max(5000, sum(max(v, 0) for v in new) + 7), in_place=False, own_state=True)


def test_empty_sequences_about_few_rows(gpu):
    B = 6000
    x = Both(B, 3, B, 16)
    x.step([1 if b in (0, 2999, B - 1) else 0 for b in range(B)], 40)
    x.step([1 if b in (1, 2999) else -1 if b == 0 else 0 for b in range(B)], 2)


def test_a_ring_as_large_as_the_pages(gpu):
    """All pages taken, all given back, time and again, past the ring's end."""
    x = Both(3, 4, 12, 16, head=11)
    for _ in range(5):
        x.step([64, 33, 64], 161)
        x.step([-1, 31, -1], 31)
        x.step([0, -1, 0], 0)


def test_nothing(gpu):
    import quantized_moe_expert_align_gb300 as moe
    x = Both(2, 4, 4, 16)
    x.step([0, 0], 0)
    out = moe.page_plan(x.pool, x.d_table[:0], x.d_lens[:0], x.d_lens[:0], 16, 3)
    assert out.cu_q.tolist() == [0] and out.slots.tolist() == [-1] * 3 and x.pool.state.tolist() == x.state


@pytest.mark.parametrize("new,rows,detail", [
    ([10, 100, 10], 200, 1),      # its table's end
    ([60, 60, 60], 200, 0),       # (21 + 60 of 80)
    ([50, 60, 50], 200, 2),       # more pages than there are free ones
    ([10, 10, 10], 29, 2),        # more rows than there are
    ([10, -2, 10], 200, 1)])
def test_all_or_nothing(gpu, new, rows, detail):
    x = Both(3, 5, 12, 16)
    x.step([20, 20, 0], 40)
    x.step([1, -1, 30], 31)
    want = [max(n, 0) for n in new]
    if -2 in new:
        import quantized_moe_expert_align_gb300 as moe
        out = moe.page_plan(x.pool, x.d_table, x.d_lens, su.i32(new), 16, rows, workspace=x.ws,
                            out=moe.PagePlan.empty(3, rows))
        assert au.status(x.ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, detail)
        assert out.seq_lens.tolist() == x.lens and out.slots.tolist() == [-1] * rows
        assert x.pool.state.tolist() == x.state
    else:
        x.step(want, rows, detail=detail)
    x.step([1, 1, 1], 3)


@pytest.mark.parametrize("lens,kept,state", [
    ([5, -1], [0, 0], [0, 8]), ([5, 100], [0, 0], [0, 8]), ([5, 5], [0, 2], [0, 8]), ([5, 5], [-1, 0], [0, 8]),
    ([5, 5], [0, 0], [8, 8]), ([5, 5], [0, 0], [-1, 3]), ([5, 5], [0, 0], [0, 9]), ([5, 5], [0, 0], [0, -1])])
def test_numbers_out_of_range(gpu, lens, kept, state):
    import quantized_moe_expert_align_gb300 as moe
    pool = moe.PagePool(su.i32(list(range(8))), su.i32(state))
    table, ws = su.i32([[0, 1, 2], [3, 4, 5]]), moe.AttnWorkspace("cuda", "pages", 2)
    out = moe.page_plan(pool, table, su.i32(lens), su.i32([1, 1]), 16, 2, window=8, kept=su.i32(kept),
                        workspace=ws)
    bad_state = state != [0, 8]
    assert au.status(ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, 2 if bad_state and state[1] >= 0 else
                             0 if bad_state or kept[0] < 0 else 1)
    assert out.seq_lens.tolist() == lens and out.kept.tolist() == kept and out.slots.tolist() == [-1, -1]
    assert pool.state.tolist() == state and table.tolist() == [[0, 1, 2], [3, 4, 5]]


def test_pages_given_back_twice(gpu):
    import quantized_moe_expert_align_gb300 as moe
    pool = moe.PagePool(su.i32(list(range(8))), su.i32([3, 8]))
    ws = moe.AttnWorkspace("cuda", "pages", 1)
    moe.page_plan(pool, su.i32([[0, 1]]), su.i32([20]), su.i32([-1]), 16, 0, workspace=ws)
    assert au.status(ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, 1)
    assert pool.ring.tolist() == list(range(8)) and pool.state.tolist() == [3, 8]


@pytest.mark.parametrize("B,in_place", [(5, True), (40, False), (1100, True)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
def test_drafts_that_are_dropped(gpu, B, in_place, window, sinks):
    """Pages of rejected tokens are used by the next ones, or go back; none is lost."""
    rng = random.Random(B)
    width = 30
    x = Both(B, width, B * width, 16, window, sinks)
    x.step([rng.choice([1, 15, 16, 100]) for _ in range(B)], 100 * B, in_place=in_place)
    for _ in range(6):
        drafts = [rng.choice([1, 16, 40, 64]) for _ in range(B)]
        x.step(drafts, 64 * B, in_place=in_place)
        gone = [rng.randrange(n) for n in drafts]
        x.lens = [a - b for a, b in zip(x.lens, gone)]
        x.d_lens = su.i32(x.lens)
        new = [rng.choice([0, 1, 1, 30, -1]) for _ in range(B)]
        x.step(new, 30 * B, in_place=in_place, dropped=gone)
    x.step([-1] * B, 0, in_place=in_place)
    assert x.state[1] == B * width and sorted(x.pool.ring.tolist()) == list(range(B * width))


@pytest.mark.parametrize("new", [0, 1, -1])
def test_dropped_tokens_that_a_window_has_left(gpu, new):
    """Pages 0 to 2 went back behind the window; the sequence cannot lose tokens of page 2."""
    import quantized_moe_expert_align_gb300 as moe
    pool = moe.PagePool(su.i32([7, 6, 5, 0, 1, 2, -1, -1]), su.i32([0, 6]))
    table, ws = su.i32([[0, 1, 2, 3]]), moe.AttnWorkspace("cuda", "pages", 1)
    for left, status in ((30, (moe.MOE_ERR_DEVICE_BAD_INDEX, 0)), (48, (moe.MOE_OK, 0))):
        before = pool.ring.tolist(), pool.state.tolist()
        out = moe.page_plan(pool, table, su.i32([left]), su.i32([new]), 16, 1, window=8, kept=su.i32([3]),
                            dropped=su.i32([60 - left]), workspace=ws)
        assert au.status(ws) == status
        if status[0]:
            assert (pool.ring.tolist(), pool.state.tolist(), out.kept.tolist()) == (*before, [3])
    # (48 tokens left: page 3 goes back too, unless a new token needs it)
    assert pool.ring.tolist() == [7, 6, 5, 0, 1, 2, -1 if new == 1 else 3, -1]
    assert pool.state.tolist() == [0, 6 if new == 1 else 7]
