"""Workspaces of fs_linear_attn and fs_linear_attn_bwd: alignment and sizes.  Runs without a GPU: every
call here is refused."""
import pytest

from test_layer_args import INVALID, UNSUPPORTED, linear, linear_bwd


def test_gradients_of_shared_heads_want_a_workspace_on_32_bytes():
    # the kernels store their parts 32 bytes at a time
    assert linear_bwd(ws=272) == UNSUPPORTED
    assert linear_bwd(ws=272 + 8, Hkv=4) == UNSUPPORTED and linear(ws=272 + 8) == UNSUPPORTED
    assert linear_bwd(ws=272, n=16) == INVALID
