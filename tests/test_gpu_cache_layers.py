"""Which keys a paged cache holds for which reader (GPU only).

An FS-L layer rotates inside: fs_attention_fwd, fs_cell_summarize and the decode state take unrotated
keys, so a cache that feeds them holds unrotated ones.  fs_tree_attn takes scores from the cache as it
is: a cache for it holds rotated keys, and a reader that rotates itself gets them through the inverse
rotation.  Both ways against the fp64 oracle on the keys and values that were read."""
import dataclasses

import numpy as np
import pytest
import torch

from long_context_lm_gb300 import fs
from long_context_lm_gb300.inputs import make_inputs
from parity import compare_forward, to_device
import serving_ref as ref
from test_gpu_decode import PAGE, _decode, _init_state
from test_gpu_forward import run_fwd

pytestmark = pytest.mark.gpu


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _through_a_cache(k, v, fmt, page=32):
    B, H, N, d = k.shape
    table, total = ref.random_table([N // page] * B, seed=N)
    cache = fs.fs_cache_alloc(total, H, page, d, fmt, table.cuda())
    fs.fs_cache_append(cache, k, v, _ints([0] * B))
    k, v = fs.fs_cache_read(cache, _ints([0] * B), T=N)
    fs.fs_check_status(cache.status)
    return k, v


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_a_cache_of_unrotated_keys_feeds_an_fsl_layer(fmt):
    N, N0 = 1408, 1280
    inp = make_inputs(2, 2, N, seed=11, sigma_ln=0.8)
    k, v = _through_a_cache(inp.k.cuda(), inp.v.cuda(), fmt)
    inp = dataclasses.replace(inp, k=k.cpu(), v=v.cpu())
    out, sel, _ = run_fwd(inp, PAGE)
    compare_forward(inp, PAGE, np.arange(N), out, sel)
    # the bounded decode state from the cached prefix, and the next tokens
    d = to_device(inp)
    out, sel = _decode(d, _init_state(d, N, N0, PAGE), N0, N0 + 40, PAGE)
    compare_forward(inp, PAGE, np.arange(N0, N0 + 40), out, sel)


def test_a_cache_of_rotated_keys_feeds_it_through_the_inverse_rotation():
    N = 1024
    inp = make_inputs(1, 2, N, seed=12, sigma_ln=0.8)
    plan = fs.fs_rope_plan(64, base=PAGE["rope_base"])
    rotated, _ = fs.fs_rope(inp.k.cuda(), None, 0, plan)
    k, v = _through_a_cache(rotated, inp.v.cuda(), "bf16")
    assert torch.equal(k, rotated)
    k, _ = fs.fs_rope(k, None, 0, plan, inverse=True)
    # two roundings to bf16, the first of a pair's two elements: 2^-8 (|a| + |b|) of the pair before
    # and after the rotation, whose sum is at most 2^(1/2) times the unrotated pair's
    x = inp.k.cuda().double().abs()
    pair = (x[..., :32] + x[..., 32:]).repeat(1, 1, 1, 2)
    assert torch.all((k.double() - inp.k.cuda().double()).abs() <= 2.0 ** -8 * 3 * pair)
    inp = dataclasses.replace(inp, k=k.cpu(), v=v.cpu())
    out, sel, _ = run_fwd(inp, PAGE)
    compare_forward(inp, PAGE, np.arange(N), out, sel)
    # and the window branch, which rotates inside, agrees with fs_tree_attn over the rotated cache: the
    # last tokens as drafted ones, row i seeing the last w positions
    T, w = 16, PAGE["w"]
    table, total = ref.random_table([N // 32], seed=5)
    cache = fs.fs_cache_alloc(total, 2, 32, 64, "bf16", table.cuda())
    q = inp.q.cuda()
    qr, kr = fs.fs_rope(q, inp.k.cuda(), 0, plan)
    fs.fs_cache_append(cache, kr, inp.v.cuda(), _ints([0]))
    tree = fs.fs_tree_attn(qr[:, :, N - T:].contiguous(), cache, _ints([N - T]), window=w)
    win = fs.fs_window_attn(q, inp.k.cuda(), inp.v.cuda(), None, None, PAGE)[:, :, N - T:]
    # q and k are rounded to bf16 after the rotation, by 2^-9 each: a score is off by 2^-8 of the
    # magnitudes that it adds up, a probability by that relative; the outputs by 2^-8 and 2^-11
    past, count = [N - T], [T]
    _, mean, most = ref.tree_attention(qr[:, :, N - T:], cache, past, None, count, window=w)
    bound = (2 * 2.0 ** -8 * most + 2.0 ** -7) * mean
    err = (tree.double() - win.double()).abs()
    assert torch.all(err <= bound)
    # (over unrotated keys it does not)
    fs.fs_cache_append(cache, inp.k.cuda(), inp.v.cuda(), _ints([0]))
    tree = fs.fs_tree_attn(q[:, :, N - T:].contiguous(), cache, _ints(past), window=w)
    assert not torch.all((tree.double() - win.double()).abs() <= bound)
