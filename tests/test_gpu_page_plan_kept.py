"""moe_page_plan: tokens dropped into pages that went back behind a window.

Page 16, window 8: of 60 tokens, pages 0 to 2 (tokens 0 to 47) have gone back.
A sequence with fewer than 48 tokens left would put the next one into page 2,
which is in the free ring."""
import pytest

from tests import attn_util as au, serve_util as su

pytestmark = pytest.mark.gpu


def _step(left, new, kept, sinks=0, page=16, width=4, rows=8):
    import quantized_moe_expert_align_gb300 as moe
    pool = moe.PagePool(su.i32([7, 6, 5, 0, 1, 2, -1, -1]), su.i32([0, 6]))
    table, ws = su.i32([list(range(width))]), moe.AttnWorkspace("cuda", "pages", 1)
    out = moe.page_plan(pool, table, su.i32([left]), su.i32([new]), page, rows, window=8, sinks=sinks,
                        kept=su.i32([kept]), dropped=su.i32([60 - left]), workspace=ws)
    return au.status(ws), out, pool, table


@pytest.mark.parametrize("new", [0, 1, 5, -1])
@pytest.mark.parametrize("left", [0, 31, 32, 33, 40, 47])
def test_pages_that_went_back_are_not_written(gpu, left, new):
    import quantized_moe_expert_align_gb300 as moe
    status, out, pool, table = _step(left, new, 3)
    assert status == (moe.MOE_ERR_DEVICE_BAD_INDEX, 0)
    assert out.slots.tolist() == [-1] * 8 and out.cu_q.tolist() == [0, 0]
    assert out.seq_lens.tolist() == [left] and out.kept.tolist() == [3]
    assert pool.ring.tolist() == [7, 6, 5, 0, 1, 2, -1, -1] and pool.state.tolist() == [0, 6]
    assert table.tolist() == [[0, 1, 2, 3]]


@pytest.mark.parametrize("left", [48, 49, 59])
def test_tokens_behind_them_can_be_dropped(gpu, left):
    import quantized_moe_expert_align_gb300 as moe
    status, out, pool, _ = _step(left, 2, 3)
    assert status == (moe.MOE_OK, 0)
    assert out.slots.tolist()[:2] == [j if j < 64 else 7 * 16 + j - 64 for j in (left, left + 1)]
    assert out.seq_lens.tolist() == [left + 2] and out.kept.tolist() == [3]


@pytest.mark.parametrize("left", [30, 32, 40, 47, 48])
def test_pages_of_first_tokens_never_went_back(gpu, left):
    """Four pages hold first tokens: whatever `kept` counts up to there, they are the sequence's own."""
    import quantized_moe_expert_align_gb300 as moe
    status, out, pool, _ = _step(left, 1, 3, sinks=50)
    assert status == (moe.MOE_OK, 0)
    assert out.slots.tolist()[0] == left and out.seq_lens.tolist() == [left + 1]
    # pages that the new length does not need go back
    back = list(range(-(-(left + 1) // 16), 4))
    assert pool.state.tolist() == [0, 6 + len(back)]
    assert pool.ring.tolist()[6:] == (back + [-1, -1])[:2]


@pytest.mark.parametrize("page,left,kept,ok", [(64, 63, 1, False), (64, 64, 1, True), (256, 255, 1, False),
                                               (256, 256, 1, True), (32, 95, 3, False), (32, 96, 3, True)])
def test_other_pages(gpu, page, left, kept, ok):
    import quantized_moe_expert_align_gb300 as moe
    pool = moe.PagePool(su.i32([9, 8, -1, -1, -1, -1]), su.i32([0, 2]))
    ws = moe.AttnWorkspace("cuda", "pages", 1)
    moe.page_plan(pool, su.i32([[0, 1, 2, 3, 4, 5]]), su.i32([left]), su.i32([1]), page, 1, window=8,
                  kept=su.i32([kept]), dropped=su.i32([20]), workspace=ws)
    assert (au.status(ws)[0] == moe.MOE_OK) == ok


def test_many_sequences_one_of_them_short(gpu):
    """Where the second kernel finishes the step, the first such sequence is named and nothing moves."""
    import quantized_moe_expert_align_gb300 as moe
    B, width = 1100, 5
    n = B * width
    pool = moe.PagePool(su.i32([5000 + i for i in range(3 * B)] + [-1] * n), su.i32([0, 3 * B]))
    table = su.i32([[width * b + p for p in range(width)] for b in range(B)])
    lens = [47 if b in (700, 900) else 48 for b in range(B)]
    ws = moe.AttnWorkspace("cuda", "pages", B)
    before = pool.ring.clone()
    out = moe.page_plan(pool, table, su.i32(lens), su.i32([1] * B), 16, B, window=8, kept=su.i32([3] * B),
                        workspace=ws)
    assert au.status(ws) == (moe.MOE_ERR_DEVICE_BAD_INDEX, 700)
    assert out.slots.tolist() == [-1] * B and pool.state.tolist() == [0, 3 * B]
    assert (pool.ring == before).all()
