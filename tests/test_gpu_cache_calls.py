"""Calls of the cache and of fs_rope that their documentation allows at the ends of its
ranges (GPU only)."""
import pytest
import torch

from long_context_lm_gb300 import fs
import serving_ref as ref

pytestmark = pytest.mark.gpu


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(need, Hkv, page, d, fmt, seed=0):
    table, total = ref.random_table(need, seed=seed)
    return fs.fs_cache_alloc(total, Hkv, page, d, fmt, table.cuda())


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_append_of_a_batch_padded_to_many_tokens(fmt):
    # 2^24 token places of 8 heads of 128, nearly all of them past the count: one row of values
    # repeated with a stride of 0
    T, n = 1 << 24, 37
    a, b = (_cache([4], 8, 16, 128, fmt, seed=2) for _ in range(2))
    x, y = torch.randn((2, 1, 8, 1, 128), device="cuda").bfloat16().unbind(0)
    fs.fs_cache_append(a, x.expand(1, 8, T, 128), y.expand(1, 8, T, 128), _ints([3]), _ints([n]))
    fs.fs_cache_append(b, x.expand(1, 8, n, 128), y.expand(1, 8, n, 128), _ints([3]))
    assert torch.equal(a.codes, b.codes)
    assert a.scales is None or torch.equal(a.scales, b.scales)
    fs.fs_check_status(a.status)
