"""Workspaces of fs_linear_attn and fs_linear_attn_bwd, their alignment and sizes, and what else may lie off
its place.  Runs without a GPU: every
call here is refused."""
import pytest

from long_context_lm_gb300 import fs
from test_layer_args import INVALID, UNSUPPORTED, linear, linear_bwd


def test_gradients_of_shared_heads_want_a_workspace_on_32_bytes():
    # the kernels store their parts 32 bytes at a time
    assert linear_bwd(ws=272) == UNSUPPORTED
    assert linear_bwd(ws=272 + 8, Hkv=4) == UNSUPPORTED and linear(ws=272 + 8) == UNSUPPORTED
    assert linear_bwd(ws=272, n=16) == INVALID


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("H,Hkv,d", [(1, 1, 64), (16, 16, 64), (16, 4, 128), (24, 8, 64), (33, 11, 128), (100, 100, 64)])
def test_a_workspace_does_for_smaller_batches_and_lengths(H, Hkv, d, backward):
    n = fs.load().fs_linear_workspace_bytes
    # around the borders of one pass and two, of bands and of stretches
    lengths = sorted({1, 2, 16, 17, 128, 129, 1024, 1025, 1152, 2047, 2048, 2049, 8191, 65536, 81920, 81921, 82048, 163840,
                      163841, 262144, *(int(17 * 1.31 ** i) for i in range(40))})
    batches = [b for b in (1, 2, 3, 4, 5, 8, 9, 10, 14, 15, 18, 19, 20, 24, 32, 64) if b * H <= 2000]
    last = [0] * len(batches)
    for T in lengths:
        row = [n(b, H, Hkv, T, d, backward) for b in batches]
        assert all(x > 0 for x in row) and row == sorted(row), (T, row)
        assert all(x >= y for x, y in zip(row, last)), (T, row, last)
        last = row


@pytest.mark.parametrize("cycles", [0, -1, 4 * 10 ** 9 + 1])
def test_limits_of_waits_outside(cycles):
    L, none = fs.load(), [None] * 7
    assert L.fs_selftest_linear_wait(*none, 1, 1, 1, 32, 64, None, 1.0, None, None, None, None, None, 0, cycles,
                                     None) == INVALID
    assert L.fs_selftest_linear_wait_bwd(*none, 1, 1, 1, 32, 64, None, 1.0, *[None] * 12, 0, cycles, None) == INVALID


@pytest.mark.parametrize("kw", [dict(decay=258), dict(count=4097), dict(decay=257, T=4), dict(count=4098, T=4)])
@pytest.mark.parametrize("call", [linear, linear_bwd])
def test_numbers_off_their_size(call, kw):
    assert call(**kw) == INVALID
