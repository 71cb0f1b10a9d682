"""The sines and cosines of fs_rope in fp32 (GPU only).

A pair (1, 0) turns into (cos, sin) without another rounding.  The angle, less the nearest quarter
turn, is cut to 2^-34 of a turn (2 pi 2^-34 radians) and converted to fp32: at most a quarter of a half
turn, off by half a step, 2^-27 of a half turn (pi 2^-27 radians); the sine and cosine of what is
left are within one step of a number below 1, 2^-24.  Together 2^-24 + pi 2^-27 + 2 pi 2^-34."""
import math

import pytest
import torch

from long_context_lm_gb300 import fs

pytestmark = pytest.mark.gpu
BOUND = 2.0 ** -24 + math.pi * 2.0 ** -27 + 2 * math.pi * 2.0 ** -34


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("first", [0, 1 << 20, 2 ** 31 - 70000, -70000])
def test_sines_and_cosines(first, inverse, layout):
    rot, n = 64, 65536
    plan = fs.fs_rope_plan(rot, layout=layout)
    x = torch.zeros((1, 1, n, rot), device="cuda")
    lanes = torch.arange(rot // 2, device="cuda")
    ia, ib = (lanes, lanes + rot // 2) if layout == "half" else (2 * lanes, 2 * lanes + 1)
    x[..., ia] = 1.0
    y, _ = fs.fs_rope(x, None, first, plan, inverse=inverse)
    # position times the plan's fraction of a turn, modulo one, in 64-bit whole numbers
    turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in plan.turns[:rot // 2]],
                         dtype=torch.int64, device="cuda")
    t = (first + torch.arange(n, device="cuda"))[:, None] * turns
    angle = t.double() * (2 * math.pi / 2.0 ** 64)
    sine = -torch.sin(angle) if inverse else torch.sin(angle)
    for got, want in ((y[0, 0][:, ia], torch.cos(angle)), (y[0, 0][:, ib], sine)):
        err = (got.double() - want).abs()
        assert err.max() <= BOUND + 2.0 ** -50, float(err.max() / BOUND)


def test_quarter_turns_are_exact():
    # a plan whose first pair turns by a quarter a position: a multiple of it is exact
    plan = fs.fs_rope_plan(2)
    plan.turns[0] = 1 << 62
    x = torch.tensor([3.0, -5.0], device="cuda").expand(1, 1, 9, 2).contiguous()
    y, _ = fs.fs_rope(x, None, -4, plan)
    want = [[3.0, -5.0], [5.0, 3.0], [-3.0, 5.0], [-5.0, -3.0]]
    assert y[0, 0].tolist() == [want[(p - 4) % 4] for p in range(9)]
