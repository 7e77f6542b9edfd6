"""moe_qk_rope_append where values are not rotated: an infinity or NaN there
stays in its own place, and without a norm the values come out as they are."""
import pytest

from tests import attn_util as au

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _run(D, rot, inter, norm, fp8, spots):
    """Rows of normal values with spots[token] = {column: value} in head 0 of
    q, k and v; returns q_out, k_out, the cached K rows (codes as they stand,
    scales or None) and the inputs."""
    import torch
    import quantized_moe_expert_align_gb300 as moe
    T, H, page = len(spots), 2, 16
    x = au.randn(3 + D + rot, T, H, D)
    for t, spot in enumerate(spots):
        for c, value in spot.items():
            x[t, 0, c] = value
    w = (1 + 0.1 * au.randn(4, D, dtype=torch.float32)).bfloat16() if norm else None
    cs = moe.rope_table(64, rot) if rot else None
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 5 % 64
    cache = au.make_cache(5, 2, H, page, D, fp8)
    slots = torch.arange(T, dtype=torch.int32, device="cuda") + 3
    ws = moe.AttnWorkspace("cuda")
    q, k = moe.qk_rope_append(x, x, x, cs, pos, cache, slots, q_norm=w, k_norm=w, eps=EPS,
                              interleaved=inter, k_out=True, workspace=ws)
    assert au.status(ws) == (moe.MOE_OK, 0)
    at = slots.long()
    rows = cache.data.view(torch.uint8 if fp8 else torch.int16)[at // page, :, 0, at % page]
    sc = cache.scales[at // page, :, 0, at % page] if fp8 else None
    return x, w, cs, pos, q, k, rows.view(cache.data.dtype), sc


def _spots(D, rot):
    inf, nan = float("inf"), float("nan")
    out = [{}, {rot: inf}, {D - 1: nan}, {rot + 5: -inf, rot + 6: nan}]
    out += [{c: inf} for c in range(rot, min(D, rot + 8))]
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 0), (128, 0), (64, 32), (128, 64), (128, 16), (64, 48)])
def test_unrotated_values_come_out_as_they_are(gpu, D, rot, inter, fp8):
    import torch
    x, _, _, _, q, k, rows, sc = _run(D, rot, inter, False, fp8, _spots(D, rot))
    same = lambda a, b: ((a == b) | (a.isnan() & b.isnan())).all()  # noqa: E731
    for got in (q, k):
        assert same(got[..., rot:], x[..., rot:])
        assert torch.isfinite(got[..., :rot]).all()
    if not fp8:
        assert torch.equal(rows.view(torch.int16), k.view(torch.int16))
    else:   # rows that hold an infinity or NaN have a NaN scale, the others none
        assert torch.equal(sc.isnan(), ~torch.isfinite(x).all(-1))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 0), (128, 64)])
def test_unrotated_values_under_a_norm(gpu, D, rot, inter):
    """A row with an infinity: rsqrt(infinity) = 0, so its finite values become
    0 and the infinity NaN, at its own place; a NaN makes the whole row NaN."""
    import torch
    inf, nan = float("inf"), float("nan")
    x, w, cs, pos, q, k, _, _ = _run(D, rot, inter, True, False, [{}, {rot + 3: inf}, {D - 2: -inf},
                                                                  {rot: nan}, {}])
    for got in (q, k):
        for t, c in ((1, rot + 3), (2, D - 2)):
            want = torch.zeros(D, device="cuda")
            want[c] = nan
            row = got[t, 0].float()
            assert torch.equal(row.isnan(), want.isnan()) and (row[~want.isnan()] == 0).all()
        assert got[3, 0].isnan().all()
        assert torch.isfinite(got[[0, 4]]).all() and torch.isfinite(got[:, 1]).all()
        # values without a rotation: three 32-bit operations and one rounding
        z = x[0].double()
        z = (z / torch.sqrt((z * z).mean(-1, keepdim=True) + EPS) * w.double())[..., rot:]
        au.check(got[0][..., rot:], z, (au.U_BF16 + 2.0 ** -20) * z.abs() + 1e-30, "row")
