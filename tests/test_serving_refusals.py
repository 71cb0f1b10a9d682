"""More refusals of the serving calls before anything is launched, and calls whose
bounds decide.  Runs without a GPU: no call here reaches CUDA's kernels."""
import ctypes

import pytest

from long_context_lm_gb300 import fs


def _desc(**kw):
    a = dict(codes=256, scales=256, table=256, status=None, pages=4, page=16, Hkv=2, d=64, format=2,
             batch=3, max_pages=2)
    a.update(kw)
    return fs.fs_cache_t(*[a[f] for f, _ in fs.fs_cache_t._fields_])


def _vp(x):
    return None if x is None else ctypes.c_void_p(x)


@pytest.mark.parametrize("cycles", [0, -1, 4 * 10 ** 9 + 1])
def test_wait_limits_outside_are_refused(cycles):
    rc = fs.load().fs_selftest_tree_wait(_vp(256), _desc(), _vp(256), None, None, 4, 8, 0, 0.125,
                                         _vp(1 << 30), _vp(256), 1 << 40, cycles, None)
    assert rc == fs.FS_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rot=2 ** 32 + 64), dict(rot=64, scaling="ramp", original=2 ** 32 + 4096),
                                dict(rot=64 - 2 ** 32)])
def test_plan_sizes_past_32_bits_are_refused(kw):
    with pytest.raises(ValueError):
        fs.fs_rope_plan(**kw)
