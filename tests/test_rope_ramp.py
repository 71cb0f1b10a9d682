"""The ramp of fs_rope_make_plan where its upper end lies beyond the last pair (host only)."""
import math

import pytest

from long_context_lm_gb300 import fs


@pytest.mark.parametrize("rot,original,base,factor", [
    (128, 65536, 10000.0, 4.0), (128, 131072, 10000.0, 8.0), (64, 163840, 10000.0, 2.0),
    (64, 4096, 10000.0, 8.0),                  # ends before the last pair
    (32, 1 << 30, 100.0, 2.0),                 # both ends beyond the last pair; the upper one at r - 1
    (2, 4096, 10000.0, 2.0),
])
def test_the_ramp_may_end_beyond_the_last_pair(rot, original, base, factor):
    # pair i makes beta turns in `original` tokens where i = r ln(original / (2 pi beta)) / (2 ln base);
    # the ramp between beta_fast = 32 and beta_slow = 1, outwards to whole pairs, from 0 to r - 1
    ends = [rot * math.log(original / (2 * math.pi * beta)) / (2 * math.log(base)) for beta in (32.0, 1.0)]
    lo, hi = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rot - 1)
    plan = fs.fs_rope_plan(rot, scaling="ramp", factor=factor, original=original, base=base)
    for i in range(rot // 2):
        g = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        f = base ** (-2.0 * i / rot)
        f = f * (1 - g) + f / factor * g
        assert plan.turns[i] / 2.0 ** 64 == pytest.approx(f / (2 * math.pi), rel=1e-14)
