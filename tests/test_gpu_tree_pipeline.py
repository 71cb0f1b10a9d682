"""The waits of the many-row kernel of fs_tree_attn (GPU only): stretches of short
segments, where few of its roles wait for one another."""
import pytest
import torch

from long_context_lm_gb300 import fs
import serving_ref as ref

pytestmark = pytest.mark.gpu


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bf16(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _short(fmt, d, past, Hkv, G, T, seed):
    """(cache, q, past) for one sequence of past[b] + T tokens per b."""
    n = max(past) + T
    table, total = ref.random_table([-(-(p + T) // 16) for p in past], seed=seed)
    cache = fs.fs_cache_alloc(total, Hkv, 16, d, fmt, table.cuda())
    fs.fs_cache_append(cache, _bf16((len(past), Hkv, n, d), seed), _bf16((len(past), Hkv, n, d), seed + 1),
                       _ints([0] * len(past)), _ints([p + T for p in past]))
    return cache, _bf16((len(past), Hkv * G, T, d), seed + 2), _ints(past)


def _check(cache, q, past, out):
    """Within 2^-8 of the value and 2^-9 of its terms' mean magnitude (a row's probabilities are off
    by 2^-11 each; scores below 64 by (d + 3) 2^-24 64 2.3 < 2^-10)."""
    B, H, T, d = q.shape
    G = H // cache.Hkv
    for b in range(B):
        n = past[b] + T
        k, v = (ref.values(*ref.gather(cache, b, n, part), cache.format).transpose(0, 1) for part in (0, 1))
        seen = torch.arange(n, device="cuda") <= past[b] + torch.arange(T, device="cuda")[:, None]
        s = q[b].double().reshape(cache.Hkv, G, T, d) @ k[:, None].transpose(2, 3) * d ** -0.5
        p = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
        want, mean = p @ v[:, None], p @ v[:, None].abs()
        err = (out[b].double().reshape(want.shape) - want).abs()
        assert torch.all(err <= 1.01 * 2.0 ** -8 * want.abs() + 2.0 ** -9 * mean), b


@pytest.mark.parametrize("fmt,d", [("bf16", 64), ("bf16", 128), ("int8", 64), ("int8", 128), ("int4", 64),
                                   ("e4m3", 128)])
@pytest.mark.parametrize("past", [[0] * 100, [0, 40, 70, 100, 130, 200] * 20])
def test_many_short_segments(past, fmt, d):
    # segments of one tile by the dozen in every block, or of one to four tiles in turn
    cache, q, at = _short(fmt, d, past, Hkv=16, G=2, T=40, seed=len(past) + d)
    out = fs.fs_tree_attn(q, cache, at)
    _check(cache, q, past, out)
    ws, again = fs.fs_tree_workspace(cache, len(past), 32, 40), torch.empty_like(out)
    for _ in range(20):
        fs.fs_tree_attn(q, cache, at, out=again, ws=ws)
        assert torch.equal(out, again)
    fs.fs_check_status(cache.status)


@pytest.mark.parametrize("fmt,d", [("bf16", 64), ("bf16", 128), ("int8", 64), ("e4m3", 128), ("int4", 64)])
def test_waits_that_give_up(fmt, d):
    # The limit runs out in other places each time, with copies and products under way; the call ends
    # with a status, and the next one is right.  64 x 4 rows: the many-row kernel.
    past = [5000, 300, 0, 1900]
    cache, q, at = _short(fmt, d, past, Hkv=4, G=4, T=64, seed=d)
    # values that are not finite, so that the rows, too, wait for products
    bad = torch.full((4, 4, 1, d), float("inf"), device="cuda").bfloat16()
    fs.fs_cache_append(cache, bad, bad, _ints([4990, 290, 0, 1950]))
    want = fs.fs_tree_attn(q, cache, at)
    fs.fs_check_status(cache.status)
    ws, gave_up = fs.fs_tree_workspace(cache, 4, 16, 64), 0
    for cycles in (1, 100, 300, 1000, 2000, 4000, 8000, 16000, 32000, 64000, 10 ** 9):
        out = torch.empty_like(q)
        fs.fs_selftest_tree_wait(q, cache, at, cycles, out=out, ws=ws)
        torch.cuda.synchronize()
        status = int(cache.status[0])
        assert status in (0, fs.FS_ERR_TIMEOUT)
        gave_up += status != 0
        if status == 0:
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        cache.status.zero_()
        again = fs.fs_tree_attn(q, cache, at, ws=ws)
        fs.fs_check_status(cache.status)
        assert torch.equal(again.view(torch.int16), want.view(torch.int16))
    assert gave_up > 0 and status == 0
