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


def test_strides_of_axes_of_one_do_not_matter():
    # one sequence, or one token, out of a buffer whose rows in between are of odd length
    H, T, d = 4, 21, 64
    flat = torch.randn(2 * H * T * d + 8, device="cuda").bfloat16()
    for size, strides in (((1, H, T, d), (3, T * d, d, 1)), ((1, H, 1, d), (12345, d, 7, 1)),
                          ((1, 1, T, d), (1, 5, d, 1))):
        x = torch.as_strided(flat, size, strides)
        y = x.clone(memory_format=torch.contiguous_format)
        a, b = (_cache([2], size[1], 16, d, "int8", seed=4) for _ in range(2))
        # (the binding passes no strides for what torch calls contiguous: the C call with them)
        start = _ints([3])
        args = (fs._Strides(*strides[:3]),) * 2 + (size[2], start.data_ptr(), None)
        fs._launch(a.device, None, fs.load().fs_cache_append, "fs_cache_append", a.desc, x.data_ptr(),
                   x.data_ptr(), *args)
        fs.fs_cache_append(b, y, y, start)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    x = torch.as_strided(flat, (1, H, T, d), (H * T * d + 3, d, H * d, 1))    # token-major
    a, b = (_cache([2], H, 16, d, "int8", seed=4) for _ in range(2))
    fs.fs_cache_append(a, x, x, _ints([3]))
    fs.fs_cache_append(b, x.contiguous(), x.contiguous(), _ints([3]))
    assert torch.equal(a.codes, b.codes)
    plan = fs.fs_rope_plan(d)
    assert torch.equal(fs.fs_rope(x, None, 5, plan)[0], fs.fs_rope(x.contiguous(), None, 5, plan)[0])


def test_workspaces_that_are_not_their_own_memory_are_refused():
    cache = _cache([4], 2, 16, 64, "int8")
    q = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    need = fs.fs_tree_workspace(cache, 1, 4, 2).numel()
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(need),
               torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            fs.fs_tree_attn(q, cache, _ints([3]), ws=ws)


def test_windows_past_32_bits():
    cache = _cache([40], 2, 16, 64, "int8")
    k, q = (torch.randn((1, 2, n, 64), device="cuda").bfloat16() for n in (600, 2))
    fs.fs_cache_append(cache, k, k, _ints([0]))
    want = fs.fs_tree_attn(q, cache, _ints([590]))
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 64, 2 ** 40):       # all of it
        assert torch.equal(fs.fs_tree_attn(q, cache, _ints([590]), window=window), want)
    with pytest.raises(fs.FSError):
        fs.fs_tree_attn(q, cache, _ints([590]), window=64 - 2 ** 32)
