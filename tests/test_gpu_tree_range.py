"""fs_tree_attn where values differ by many powers of two and where scores rise
within a sequence, against the 64-bit definition on the cache's own codes (GPU
only).

Error of one output element of a row that sees n keys, from the arithmetic.  P_k
are its probabilities, M = sum P_k |v_k| its mean magnitude, a_k the largest
magnitude of value row k.
  * A score is a sum of d products in fp32 with its factors: (d + 3) 2^-24 of
    the magnitudes that are added.  Those are at most |q|_1 times the key row's
    largest magnitude, 2.3 times that where integer codes go in with a bias of
    half their range (128 to 127, 8 to 7).  ds is the largest such error over the
    keys that the row sees: a probability is off by ds relative, 2^-21 for the
    exponential.
  * A quantised value's weight P_k s_k is held in fp16, half a step 2^-11; a bf16
    value's in 16 bits.  The row's largest weight is held as 2^7 or more, so a weight
    below fp16's normal range is off by 2^-32 of the largest, twice that where it is
    scaled down to a new reference: n 2^-31 max P_k a_k together.
  * Weights and probabilities are added in fp32: n 2^-24 of their sum each.
So the output is within
  (2 ds + 2^-11 + 2^-18 + n 2^-23) M + n 2^-31 max P_k a_k
and rounded to bf16, by 2^-8 relative.  What a row does not see has no part in
its bound."""
import math

import pytest
import torch

from long_context_lm_gb300 import fs
import serving_ref as ref

pytestmark = pytest.mark.gpu

# rows to a kv head of every kernel form: up to 8, 16 and 32 on mma.sync, 64 and 256 (tcgen05)
FORMS = [(2, 1), (16, 1), (32, 1), (64, 1), (64, 4)]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def _cache(k, v, fmt, page=16, seed=0):
    """A cache that holds the tokens k, v [B, Hkv, n, d]; the rest of it NaN."""
    B, Hkv, n, d = k.shape
    table, total = ref.random_table([-(-n // page)] * B, seed=seed)
    cache = fs.fs_cache_alloc(total, Hkv, page, d, fmt, table.cuda())
    cache.codes.fill_(0xff)
    if cache.scales is not None:
        cache.scales.fill_(float("nan"))
    fs.fs_cache_append(cache, k.bfloat16().contiguous(), v.bfloat16().contiguous(), _ints([0] * B))
    return cache


def _sight(past, T, tree, window):
    """[T, past + T] bool: what the rows of one sequence see."""
    seen = torch.zeros((T, past + T), dtype=torch.bool)
    for i in range(T):
        bits = ((1 << (i + 1)) - 1 if tree is None else int(tree[i])) & ((1 << T) - 1)
        seen[i, max(0, past + bin(bits).count("1") - window) if window else 0:past] = True
        seen[i, past:] = torch.tensor([bool(bits >> j & 1) for j in range(T)])
    return seen.cuda()


def _check(q, cache, past, out, tree=None, window=0, scale=None):
    """Every row of every sequence (``past`` tokens each) within the bound above."""
    B, H, T, d = q.shape
    G, scale = H // cache.Hkv, d ** -0.5 if scale is None else scale
    wide = 2.3 if cache.format in ("int8", "int4") else 1.0
    n = past + T
    for b in range(B):
        seen = _sight(past, T, None if tree is None else tree[b], window)
        rows = [ref.gather(cache, b, n, part) for part in (0, 1)]
        for h in range(cache.Hkv):
            k, v = (ref.values(c[:, h], None if s is None else s[:, h], cache.format) for c, s in rows)
            qq = q[b, h * G:(h + 1) * G].double()
            s = (scale * qq @ k.T).masked_fill(~seen, -math.inf)
            p = torch.softmax(s, -1).masked_fill(~seen, 0.0).nan_to_num(0.0)
            want, mean = p @ v, p @ v.abs()
            size = (qq.abs().sum(-1, keepdim=True) * k.abs().amax(-1)).masked_fill(~seen, 0.0).amax(-1)
            ds = ((d + 3) * 2.0 ** -24 * scale * wide * size)[..., None]
            assert ds.max() < 2.0 ** -8
            peak = (p * v.abs().amax(-1)).amax(-1, keepdim=True)
            bound = 1.01 * 2.0 ** -8 * want.abs() + n * 2.0 ** -31 * peak + \
                (2 * ds + 2.0 ** -11 + 2.0 ** -18 + n * 2.0 ** -23) * mean + 1e-38
            o = out[b, h * G:(h + 1) * G].double()
            assert torch.isfinite(o).all()
            err = (o - want).abs()
            assert torch.all(err <= bound), (b, h, float((err / bound).max()))


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,H", FORMS)
def test_large_values_that_a_row_does_not_see(T, H, d, fmt):
    # the first drafted token's values are 2^40 times the others', and only it sees itself
    for past in (5, 20, 700):
        n = past + T
        k, v = _randn((1, 1, n, d), 1), _randn((1, 1, n, d), 2)
        v[:, :, past] *= 2.0 ** 40
        cache = _cache(k, v, fmt)
        tree = torch.tensor([[1] + [1 << i if i < 63 else -(1 << 63) for i in range(1, T)]]).cuda()
        q = _randn((1, H, T, d), 3).bfloat16()
        out = fs.fs_tree_attn(q, cache, _ints([past]), tree=tree)
        _check(q, cache, past, out, tree)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("T,H", FORMS)
def test_large_values_that_leave_the_window(T, H, fmt):
    # row i sees the prefix from past + i + 1 - 64 on: only the first rows see the large values
    past, d = 300, 64
    k, v = _randn((1, 1, past + T, d), 1), _randn((1, 1, past + T, d), 2)
    v[:, :, past - 63] *= 2.0 ** 40
    v[:, :, past - 63 - 20:past - 63] *= 2.0 ** 60      # before every row's window
    cache = _cache(k, v, fmt)
    q = _randn((1, H, T, d), 3).bfloat16()
    _check(q, cache, past, fs.fs_tree_attn(q, cache, _ints([past]), window=64), window=64)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("T,H", FORMS)
def test_large_values_of_little_weight(T, H, fmt):
    # keys whose probability is about 2^-90, with values 2^50 times the others'
    past, d = 900, 64
    k, v = 0.1 * _randn((1, 1, past + T, d), 1), _randn((1, 1, past + T, d), 2)
    for at in (3, 70, 500):
        k[:, :, at] = -1.0
        v[:, :, at] *= 2.0 ** 50
    cache = _cache(k, v, fmt)
    q = torch.ones((1, H, T, d), device="cuda").bfloat16()
    _check(q, cache, past, fs.fs_tree_attn(q, cache, _ints([past]), scale=1.0), scale=1.0)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("size", [1e-20, 1.0, 1e20, 1e30, 1e36])
@pytest.mark.parametrize("T,H,Hkv,B,past", [(1, 16, 16, 4, 4096), (16, 16, 16, 4, 4096),
                                            (64, 4, 1, 16, 8192)])
def test_zero_values_keep_their_share_of_the_sum(T, H, Hkv, B, past, size, fmt):
    # equal scores; rows of zeros and rows of one size in turn, 256 at a time, and enough of them that
    # one warp (one stream) gets both, the zeros first
    d, n = 64, past + T
    k, v = _randn((B, Hkv, n, d), 1), size * (1.0 + _randn((B, Hkv, n, d), 2).abs())
    v[:, :, (torch.arange(n, device="cuda") // 256) % 2 == 0] = 0.0
    cache = _cache(k, v, fmt, page=64)
    q = torch.zeros((B, H, T, d), device="cuda").bfloat16()
    out = fs.fs_tree_attn(q, cache, _ints([past] * B))
    _check(q, cache, past, out)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [5.0, 9.0, 17.0])      # log2 from one raised key to the next
@pytest.mark.parametrize("T,H", FORMS)
def test_scores_that_rise(T, H, step, d, fmt):
    # raised keys in the first and second 32 keys of a tile, in the first and in later tiles of
    # either parity, at the border of the prefix and among the drafted tokens; ordinary keys
    # keep a share of the sum
    for past, places in ((1000, (5, 40, 100, 130, 200, 420, 800, 999, 1000)),
                         (1003, (33, 64, 127, 128, 600, 1002, 1003, 1004)),
                         (50, (2, 34, 49, 50)), (300, (255, 256, 257, 299))):
        n = past + T
        k, v = 0.02 * _randn((1, 1, n, d), 1), _randn((1, 1, n, d), 2)
        q = (1.0 + 0.02 * _randn((1, H, T, d), 3)).bfloat16()
        for i, at in enumerate(places):
            if at < n:
                k[:, :, at] += (i + 1) * step / d
                v[:, :, at] *= 2.0 ** (-step * (i % 3))
        cache = _cache(k, v, fmt)
        scale = math.log(2.0)
        _check(q, cache, past, fs.fs_tree_attn(q, cache, _ints([past]), scale=scale), scale=scale)
        tree = torch.full((1, T), (1 << min(T, 63)) - 1, dtype=torch.int64).cuda()   # all drafted
        _check(q, cache, past, fs.fs_tree_attn(q, cache, _ints([past]), tree=tree, scale=scale), tree,
               scale=scale)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("T,H", FORMS)
def test_tiny_queries_and_large_keys(T, H, fmt):
    # scores of 2^-12 64 scale, from numbers near both ends of bf16; values with the keys' signs, so that
    # an error of the scores shows in full
    past, d, scale = 900, 64, 0.01
    k = torch.ones((1, 1, past + T, d), device="cuda") * 2.0 ** 100
    k[:, :, ::2] *= -1.0
    v = k.sign() + 0.01 * _randn(k.shape, 2)
    cache = _cache(k, v, fmt)
    q = torch.full((1, H, T, d), 2.0 ** -112, device="cuda").bfloat16()
    _check(q, cache, past, fs.fs_tree_attn(q, cache, _ints([past]), scale=scale), scale=scale)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,H", FORMS)
def test_a_key_of_no_probability_whose_values_decide(T, H, d, fmt):
    # its probability is 2^-80 of the others', its values are 2^84 times theirs
    past = 300
    k, v = 0.01 * _randn((1, 1, past + T, d), 1), 2.0 ** -40 * _randn((1, 1, past + T, d), 2)
    k[:, :, 200] = -1.25 * 64 / d
    v[:, :, 200] *= 2.0 ** 84
    cache = _cache(k, v, fmt)
    q = torch.ones((1, H, T, d), device="cuda").bfloat16()
    scale = math.log(2.0)
    _check(q, cache, past, fs.fs_tree_attn(q, cache, _ints([past]), scale=scale), scale=scale)
