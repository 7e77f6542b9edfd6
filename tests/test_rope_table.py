"""rope_table by parts against its definition, pair by pair (on the CPU)."""
import math

import pytest

torch = pytest.importorskip("torch")


def _frequency(i, rot, base, factor, original_max, fast, slow):
    """Of pair i: kept from `fast` turns within original_max positions on,
    divided by factor up to `slow` turns, blended linearly in the index in
    between, whose ends are whole indexes (within [0, rot - 1])."""
    def at(turns):   # the pair that makes that many turns
        return rot / 2 * math.log(original_max / (2 * math.pi * turns)) / math.log(base)
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    w = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
    f = base ** (-2.0 * i / rot)
    return f * (1 - w) + f / factor * w


@pytest.mark.parametrize("rot,base,factor,original_max,fast,slow", [
    (64, 1e4, 4.0, 4096, 32.0, 1.0), (128, 1e4, 40.0, 4096, 32.0, 1.0),
    # the blend ends past the last pair: none makes as few as `slow` turns
    (64, 1e4, 8.0, 65536, 32.0, 1.0), (128, 1e4, 4.0, 131072, 32.0, 1.0),
    (128, 1e4, 2.0, 131072, 32.0, 0.25), (64, 500.0, 3.0, 32768, 20.0, 2.0),
    # fast and slow within one pair
    (16, 1e6, 16.0, 8192, 2.0, 1.9)])
def test_by_parts(rot, base, factor, original_max, fast, slow):
    import quantized_moe_expert_align_gb300 as moe
    n = 3000
    got = moe.rope_table(n, rot, base=base, factor=factor, original_max=original_max, beta_fast=fast,
                         beta_slow=slow, magnitude=1.0, device="cpu").double()
    pos = torch.arange(n, dtype=torch.float64)
    for i in range(rot // 2):
        f = _frequency(i, rot, base, factor, original_max, fast, slow)
        turns = original_max * base ** (-2.0 * i / rot) / (2 * math.pi)
        if turns >= fast:
            assert f == base ** (-2.0 * i / rot)
        # cosines and sines are rounded once to 32 bits; the angle is good to
        # a few units in its last place of 64 bits
        assert (got[:, i] - torch.cos(pos * f)).abs().max() < 2.0 ** -24 + 1e-9
        assert (got[:, rot // 2 + i] - torch.sin(pos * f)).abs().max() < 2.0 ** -24 + 1e-9
    if original_max * base ** (-2.0 * (rot // 2 - 1) / rot) / (2 * math.pi) > slow:
        assert _frequency(rot // 2 - 1, rot, base, factor, original_max, fast, slow) > \
            base ** (-2.0 * (rot // 2 - 1) / rot) / factor
