"""fs_tree_attn against the 64-bit definition on the cache's own codes (GPU
only).

Error of one output element, from the arithmetic.  A score is a sum of d
products in fp32 (at most (d + 3) 2^-24 of the sum of their magnitudes, the
scale factors included), so a probability is off by that much (ds) relative,
and by 2^-21 for the exponential and the running rescaling.  A probability is
held for the product with the values in no less than fp16: half a step is 2^-11
relative and, below 2^-14, 2^-25.  The largest probability of a row, and with it
their sum, is held as 2^7 at least (a reference follows the maximum to within a
factor of 2^8 below the 2^15 that the largest may reach), so 2^-25 is 2^-32 of
the sum, twice that where a probability is scaled down to a new reference and
rounded again; the value it multiplies is |v| at most: n 2^-31 max|v| together.
The values are exact, or scaled in fp32 (2^-24).  The sum of probabilities is off
by ds + 2^-20.  So the output is within
    (2 ds + 2^-11 + 2^-18) M + n 2^-31 max|v|,   M = sum p |v| / sum p,
and then rounded to bf16, by at most 2^-8 relative."""
import pytest
import torch

from long_context_lm_gb300 import fs
import serving_ref as ref

pytestmark = pytest.mark.gpu


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(shape, seed, spread=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))).bfloat16()


def _filled(past, T, Hkv, page, d, fmt, seed=0, spread=0.5):
    """A cache with past[b] + T tokens of every sequence; the rest of it NaN."""
    need = [max(1, -(-(p + T) // page)) for p in past]
    table, total = ref.random_table(need, seed=seed)
    cache = fs.fs_cache_alloc(total, Hkv, page, d, fmt, table.cuda())
    cache.codes.fill_(0xff)
    if cache.scales is not None:
        cache.scales.fill_(float("nan"))
    n = max(past) + T
    k, v = _rows((len(past), Hkv, n, d), seed + 1, spread), _rows((len(past), Hkv, n, d), seed + 2)
    fs.fs_cache_append(cache, k, v, _ints([0] * len(past)), _ints([p + T for p in past]))
    return cache


def _trees(B, T, seed):
    """Random trees: every token sees itself and its ancestors."""
    g = torch.Generator().manual_seed(seed)
    tree = torch.zeros((B, T), dtype=torch.int64)
    for b in range(B):
        for i in range(T):
            up = int(tree[b, max(0, i - int(torch.randint(1, 5, (), generator=g)))]) if i else 0
            x = (up & ((1 << 64) - 1)) | 1 << i
            tree[b, i] = x - (1 << 64) if x >> 63 else x
    return tree.cuda()


def _check(q, cache, past, out, tree=None, count=None, window=0, scale=None):
    T, d = q.shape[2:]
    count = [T] * len(past) if count is None else count
    want, mean, most = ref.tree_attention(q, cache, past, tree, count, window, scale)
    ds = (d + 3) * 2.0 ** -24 * most
    assert ds < 2.0 ** -9
    vmax = 0.0
    for b, p in enumerate(past):
        c, s = ref.gather(cache, b, p + count[b], 1)
        x = ref.values(c, s, cache.format)
        x = x[torch.isfinite(x)]
        vmax = max(vmax, float(x.abs().max()) if x.numel() else 0.0)
    bound = 1.01 * 2.0 ** -8 * want.abs() + (2 * ds + 2.0 ** -11 + 2.0 ** -18) * mean + \
        (max(past) + T) * 2.0 ** -31 * vmax
    for b, n in enumerate(count):
        w, o = want[b, :, :n], out[b, :, :n].double()
        fine = torch.isfinite(w)
        assert torch.equal(torch.isnan(w), torch.isnan(o))
        assert torch.equal(torch.isinf(w), torch.isinf(o))
        err = (o - w).abs()[fine]
        lim = bound[b, :, :n][fine]
        assert torch.all(err <= lim), (b, float((err / lim).max()))


CASES = [
    # past, T, count, H, Hkv, page, d
    ([0], 1, None, 1, 1, 16, 64),                          # one token sees itself alone
    ([5], 1, None, 4, 4, 16, 64),
    ([127, 128, 129], 1, None, 16, 2, 32, 64),             # grouped heads, around a tile
    ([0, 1, 15, 16, 17, 100], 8, [8, 0, 1, 7, 8, 3], 6, 3, 16, 64),
    ([1000, 333], 17, [17, 9], 4, 1, 64, 128),
    ([70, 2000], 64, [64, 50], 8, 1, 256, 64),             # 512 rows to a kv head
    ([640], 33, None, 5, 5, 128, 128),
    ([3, 900, 31], 64, [1, 64, 0], 4, 2, 16, 128),
    ([4095], 16, None, 32, 4, 16, 64),
    ([2500, 0], 3, [3, 2], 12, 4, 32, 128),
]


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("past,T,count,H,Hkv,page,d", CASES)
def test_tree_matches_the_definition(past, T, count, H, Hkv, page, d, fmt):
    B = len(past)
    cache = _filled(past, T, Hkv, page, d, fmt, seed=T + d)
    q = _rows((B, H, T, d), 7, 0.3)
    for tree, window in ((None, 0), (_trees(B, T, T), 0), (_trees(B, T, T + 1), 64), (None, 200)):
        out = torch.full_like(q, 9.0)
        fs.fs_tree_attn(q, cache, _ints(past), tree=tree, window=window, out=out,
                        count=None if count is None else _ints(count))
        _check(q, cache, past, out, tree, count, window)
        for b, n in enumerate(count or [T] * B):
            assert torch.all(out[b, :, n:] == 9.0)         # rows past the count: as they were
    fs.fs_check_status(cache.status)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("past,T,H,Hkv,d", [
    ([70001], 1, 8, 8, 64), ([70001], 5, 8, 1, 128), ([30000, 12345], 16, 4, 2, 64),
    ([20000], 64, 4, 1, 64), ([9000, 20001], 40, 6, 3, 128),
])
def test_long_caches(past, T, H, Hkv, d, fmt):
    cache = _filled(past, T, Hkv, 16, d, fmt, seed=3)
    q = _rows((len(past), H, T, d), 8, 0.3)
    tree = _trees(len(past), T, 3)
    out = fs.fs_tree_attn(q, cache, _ints(past), tree=tree)
    _check(q, cache, past, out, tree)
    out = fs.fs_tree_attn(q, cache, _ints(past), tree=tree, window=512)
    _check(q, cache, past, out, tree, window=512)


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_rows_that_see_nothing_and_single_bits(fmt):
    past, T = [0, 0, 300], 64
    cache = _filled(past, T, 2, 16, 64, fmt)
    tree = torch.zeros((3, T), dtype=torch.int64)
    for i in range(0, T, 2):                               # odd rows see no drafted token
        j = (i * 7 + 3) % T                                # one drafted token, not itself
        tree[:, i] = (1 << j) - (1 << 64) if j == 63 else 1 << j
    tree = tree.cuda()
    q = _rows((3, 4, T, 64), 7)
    out = fs.fs_tree_attn(q, cache, _ints(past), tree=tree)
    _check(q, cache, past, out, tree)
    assert torch.all(out[:2, :, 1::2] == 0)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("T,H,Hkv", [(8, 2, 1), (64, 4, 1), (8, 1, 1), (7, 2, 2), (24, 1, 1)])
def test_not_finite_rows_reach_only_the_rows_that_see_them(fmt, T, H, Hkv):
    past = [200, 7]
    cache = _filled(past, T, Hkv, 16, 64, fmt, seed=5)
    bad = _rows((2, Hkv, 3, 64), 1)
    bad[:, :, 0, 5], bad[:, :, 1, 6], bad[:, :, 2, 7] = float("nan"), float("inf"), float("-inf")
    fine = _rows((2, Hkv, 3, 64), 2)
    at = _ints([past[0] + 2, past[1] + 2])
    tree = _trees(2, T, 1)
    q = _rows((2, H, T, 64), 3)
    for k, v in ((fine, bad), (bad, fine)):
        fs.fs_cache_append(cache, k, v, at)
        out = fs.fs_tree_attn(q, cache, _ints(past), tree=tree)
        want, _, _ = ref.tree_attention(q, cache, past, tree, [T, T])
        assert torch.equal(torch.isfinite(want), torch.isfinite(out))
        unseen = ((tree >> 2) & 7) == 0
        assert unseen.any()
        for b in range(2):
            assert torch.all(torch.isfinite(out[b][:, unseen[b]]))


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("H", [2, 4])
def test_not_finite_rows_outside_the_window(fmt, H):
    # row i sees the last 64 positions: the poisoned ones leave the window row by row
    past, T = [500], 32
    cache = _filled(past, T, 2, 32, 64, fmt, seed=6)
    x = torch.full((1, 2, 8, 64), float("inf"), device="cuda").bfloat16()
    fs.fs_cache_append(cache, _rows((1, 2, 8, 64), 1), x, _ints([440]))
    fs.fs_cache_append(cache, x, x, _ints([100]))          # far outside for every row
    q = _rows((1, H, T, 64), 3)
    out = fs.fs_tree_attn(q, cache, _ints(past), window=64)
    want, _, _ = ref.tree_attention(q, cache, past, None, [T], window=64)
    assert torch.equal(torch.isfinite(want), torch.isfinite(out))
    assert torch.isfinite(want[0, :, 12:]).all() and not torch.isfinite(want[0, :, :11]).any()


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_not_finite_rows_outside_the_window_of_few_rows(fmt):
    past, T = [500], 8
    cache = _filled(past, T, 2, 32, 64, fmt, seed=6)
    x = torch.full((1, 2, 4, 64), float("nan"), device="cuda").bfloat16()
    fs.fs_cache_append(cache, _rows((1, 2, 4, 64), 1), x, _ints([437]))   # 437 .. 440
    q = _rows((1, 2, T, 64), 3)
    out = fs.fs_tree_attn(q, cache, _ints(past), window=64)                # row i from 437 + i on
    want, _, _ = ref.tree_attention(q, cache, past, None, [T], window=64)
    assert torch.equal(torch.isfinite(want), torch.isfinite(out))
    assert torch.isfinite(want[0, :, 4:]).all() and not torch.isfinite(want[0, :, :4]).any()


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("T,H", [(6, 1), (6, 2), (30, 1), (50, 1)])
def test_queries_that_are_not_finite_stay_in_their_row(fmt, T, H):
    cache = _filled([300], T, 1, 16, 64, fmt)
    q = _rows((1, H, T, 64), 3)
    fine = fs.fs_tree_attn(q, cache, _ints([300]))
    q[0, 0, 2, 7], q[0, H - 1, 4, 9] = float("nan"), float("inf")
    out = fs.fs_tree_attn(q, cache, _ints([300]))
    bad = torch.zeros((1, H, T), dtype=torch.bool, device="cuda")
    bad[0, 0, 2] = bad[0, H - 1, 4] = True
    assert torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], fine[~bad])


@pytest.mark.parametrize("fmt,d", [("bf16", 64), ("int8", 64), ("bf16", 128), ("int4", 128)])
@pytest.mark.parametrize("B,T", [(33, 2), (70, 40), (300, 1), (600, 3), (530, 34)])
def test_large_batches(B, T, fmt, d):
    # more sequences than a warp, than a block has threads; many of them empty
    g = torch.Generator().manual_seed(B)
    past = torch.randint(0, 90, (B,), generator=g).tolist()
    count = torch.randint(0, T + 1, (B,), generator=g).tolist()
    past[B // 2], count[-1] = 1500, T
    cache = _filled(past, T, 1, 16, d, fmt, seed=1)
    q = _rows((B, 1, T, d), 3)
    out = torch.full_like(q, 9.0)
    fs.fs_tree_attn(q, cache, _ints(past), out=out, count=_ints(count))
    _check(q, cache, past, out, None, count)
    fs.fs_check_status(cache.status)


def test_scales_scores_and_values_of_extreme_sizes():
    # one token far above all others, then tiny and huge values; the softmax neither overflows nor
    # loses the many small probabilities
    past, T = [5000], 2
    for fmt in ref.FORMATS:
        cache = _filled(past, T, 1, 16, 64, fmt)
        q = torch.ones((1, 1, T, 64), device="cuda").bfloat16()
        k = torch.zeros((1, 1, 1, 64), device="cuda").bfloat16()
        k[..., :] = 2.0
        for size in (1.0, 2.0 ** -60, 2.0 ** 60):
            v = _rows((1, 1, 5002, 64), 4) * size
            kk = _rows((1, 1, 5002, 64), 5, 0.1)
            kk[:, :, 77:78] = k
            fs.fs_cache_append(cache, kk, v, _ints([0]))
            out = fs.fs_tree_attn(q, cache, _ints(past), scale=0.13)
            _check(q, cache, past, out, scale=0.13)


def test_pages_outside_and_tables_that_end():
    past, T = [100, 40], 4
    cache = _filled(past, T, 1, 16, 64, "int8")
    q = _rows((2, 2, T, 64), 3)
    good = fs.fs_tree_attn(q, cache, _ints(past))
    cache.table[0, 2] = 1 << 20
    bad = fs.fs_tree_attn(q, cache, _ints(past))
    assert torch.equal(good[1], bad[1])
    with pytest.raises(fs.FSError) as e:
        fs.fs_check_status(cache.status)
    assert e.value.status == fs.FS_ERR_CACHE
    # what can be read is: the same as with tokens 32 .. 47 left out
    lo, hi = (fs.fs_cache_read(cache, _ints([0, 0]), _ints([n, 0]), T=104, dtype=torch.float32)
              for n in (32, 104))
    k = torch.cat((hi[0][0, 0, :32], hi[0][0, 0, 48:]))
    v = torch.cat((hi[1][0, 0, :32], hi[1][0, 0, 48:]))
    seen = torch.ones((4, 88), dtype=torch.bool, device="cuda")
    seen[:, 84:] = torch.tril(torch.ones((4, 4), device="cuda")).bool()
    x = (q[0].double() @ k.double().T / 8).masked_fill(~seen, float("-inf"))
    want = torch.softmax(x, -1) @ v.double()
    assert torch.all((bad[0].double() - want).abs() <= 2.0 ** -7 * (want.abs() + v.abs().max()))
    cache.status.zero_()
    fs.fs_tree_attn(q, cache, _ints([10 ** 6, -5]))        # past the table; before it
    with pytest.raises(fs.FSError):
        fs.fs_check_status(cache.status)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("page,d,H", [(16, 64, 2), (32, 128, 2), (64, 64, 4), (128, 128, 1)])
def test_pages_outside_with_many_rows(page, d, H, fmt):
    # 64 to 256 rows to a kv head; a page of the prefix and the last one cannot be read
    past, T = [1000, 700], 64
    cache = _filled(past, T, 1, page, d, fmt, seed=2)
    q = _rows((2, H, T, d), 3, 0.3)
    good = fs.fs_tree_attn(q, cache, _ints(past))
    gone = 256 // page
    cache.table[0, gone] = cache.codes.shape[0]    # one past the last
    cache.table[0, (past[0] + T - 1) // page] = -1
    bad = fs.fs_tree_attn(q, cache, _ints(past))
    assert torch.equal(good[1], bad[1])
    with pytest.raises(fs.FSError) as e:
        fs.fs_check_status(cache.status)
    assert e.value.status == fs.FS_ERR_CACHE
    keys = torch.arange(past[0] + T, device="cuda")
    there = (keys // page != gone) & (keys // page != (past[0] + T - 1) // page)
    cache.table[0, gone] = cache.table[0, 0]
    cache.table[0, (past[0] + T - 1) // page] = cache.table[0, 0]
    kv = [ref.values(*ref.gather(cache, 0, past[0] + T, x), cache.format)[there, 0] for x in (0, 1)]
    rows = torch.arange(T, device="cuda")
    seen = (keys[None] <= past[0] + rows[:, None])[:, there]
    s = (q[0].double() @ kv[0].T * d ** -0.5).masked_fill(~seen, float("-inf"))
    p = torch.softmax(s, -1)
    want, mean = p @ kv[1], p @ kv[1].abs()
    ds = (d + 3) * 2.0 ** -24 * d ** -0.5 * float((q[0].double().abs() @ kv[0].abs().T).max())
    bound = 1.01 * 2.0 ** -8 * want.abs() + (2 * ds + 2.0 ** -11 + 2.0 ** -18) * mean + \
        len(keys) * 2.0 ** -31 * float(kv[1].abs().max())
    assert torch.all((bad[0].double() - want).abs() <= bound)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("page,d,H,window", [(16, 64, 2, 64), (128, 128, 1, 100), (64, 64, 3, 0)])
def test_not_finite_values_and_many_rows(page, d, H, window, fmt):
    # values that are not finite in the last tile of the prefix, among the drafted tokens and
    # where the window of some rows begins, with and without earlier tiles
    for past in (20, 2000):
        T = 64
        cache = _filled([past], T, 1, page, d, fmt, seed=6)
        q, tree = _rows((1, H, T, d), 3, 0.3), _trees(1, T, 5)
        x = _rows((1, 1, 3, d), 1)
        x[:, :, 0, 3], x[:, :, 1, 40], x[:, :, 2, d - 1] = float("inf"), float("nan"), float("-inf")
        for at in (past + 1, past + 40, max(past - window + 5, 0) if window else past + 20):
            fs.fs_cache_append(cache, _rows((1, 1, 3, d), 2), x, _ints([at]))
        out = fs.fs_tree_attn(q, cache, _ints([past]), tree=tree, window=window)
        want, _, _ = ref.tree_attention(q, cache, [past], tree, [T], window=window)
        assert torch.equal(torch.isfinite(want), torch.isfinite(out))
        assert not torch.isfinite(want).all()


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_long_sequences_with_many_rows(fmt):
    # many tiles to a block, so that every ring goes round often; several segments to a block
    for B, Hkv, past, d in ((1, 1, 40000, 64), (1, 1, 40000, 128), (70, 3, 700, 64), (5, 1, 30000, 128)):
        cache = _filled([past] * B, 64, Hkv, 64, d, fmt, seed=4)
        q, tree = _rows((B, 2 * Hkv, 64, d), 8, 0.3), _trees(B, 64, 3)
        at = _ints([past] * B)
        out = fs.fs_tree_attn(q, cache, at, tree=tree)
        _check(q[:2], cache, [past] * min(B, 2), out[:2], tree[:2])
        for _ in range(3):
            assert torch.equal(out, fs.fs_tree_attn(q, cache, at, tree=tree))
        fs.fs_check_status(cache.status)


def test_sequences_that_share_pages_and_repeat():
    cache = _filled([64, 64, 64], 4, 2, 16, 64, "e4m3", seed=8)
    cache.table[1, :4] = cache.table[0, :4]                # a shared prefix
    cache.table[2] = cache.table[0]
    q = _rows((3, 4, 4, 64), 3)
    q[2] = q[0]
    past = [64, 64, 64]
    out = fs.fs_tree_attn(q, cache, _ints(past))
    _check(q, cache, past, out)
    assert torch.equal(out[0], out[2])
    for _ in range(3):                                     # the same bits every time
        assert torch.equal(out, fs.fs_tree_attn(q, cache, _ints(past)))


@pytest.mark.parametrize("T,past", [(1, 3000), (16, 20000), (64, 4000)])
def test_streams_graphs_and_workspaces(T, past):
    cache = _filled([past], T, 2, 32, 64, "int8")
    tree = _trees(1, T, 2)
    q, q2 = _rows((1, 8, T, 64), 3), _rows((1, 8, T, 64), 4)
    at = _ints([past])
    want, want2 = fs.fs_tree_attn(q, cache, at, tree=tree), fs.fs_tree_attn(q2, cache, at, tree=tree)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, out2 = torch.zeros_like(q), torch.zeros_like(q)
    ws, ws2 = fs.fs_tree_workspace(cache, 1, 8, T), fs.fs_tree_workspace(cache, 1, 8, T)
    ws.fill_(0xff)                                         # nothing in a workspace need be zero
    ws2.fill_(0x7f)
    torch.cuda.synchronize()
    # two calls at once, each with its own workspace
    fs.fs_tree_attn(q, cache, at, tree=tree, out=out, ws=ws, stream=s)
    fs.fs_tree_attn(q2, cache, at, tree=tree, out=out2, ws=ws2)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(out2, want2)
    # two graphs that share a workspace, replayed one after the other
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        fs.fs_tree_attn(q, cache, at, tree=tree, out=out, ws=ws)
    with torch.cuda.graph(g2):
        fs.fs_tree_attn(q2, cache, at, tree=tree, out=out2, ws=ws)
    for _ in range(2):
        out.zero_(), out2.zero_()
        g1.replay(), g2.replay(), g1.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, want2)


def test_binding_refusals():
    cache = _filled([32], 2, 2, 16, 64, "int8")
    q = _rows((1, 4, 2, 64), 3)
    ok = dict(past=_ints([32]))
    with pytest.raises(ValueError):
        fs.fs_tree_attn(q.float(), cache, **ok)
    with pytest.raises(ValueError):
        fs.fs_tree_attn(q.transpose(1, 2), cache, **ok)
    with pytest.raises(ValueError):
        fs.fs_tree_attn(q, cache, past=torch.tensor([32], device="cuda"))     # int64
    with pytest.raises(ValueError):
        fs.fs_tree_attn(q, cache, tree=_ints([[1, 3]]), **ok)
    with pytest.raises(ValueError):
        fs.fs_tree_attn(q, cache, ws=torch.empty(1 << 20, dtype=torch.uint8), **ok)
    with pytest.raises(fs.FSError):
        fs.fs_tree_attn(q, cache, window=10, **ok)
    with pytest.raises(fs.FSError):
        fs.fs_tree_attn(q, cache, ws=torch.empty(16, dtype=torch.uint8, device="cuda"), **ok)
    with pytest.raises(fs.FSError):
        fs.fs_tree_attn(_rows((1, 3, 2, 64), 3), cache, **ok)
    with pytest.raises(fs.FSError):
        fs.fs_tree_attn(q, cache, out=q, **ok)             # rows of q are read later on


def test_a_verification_step_end_to_end():
    """Prefill into the cache, draft a tree, verify, keep a path, go on; then the framework's own
    attention and bounded decode state over what the cache gives back."""
    B, H, N, d, T = 2, 4, 256, 64, 8
    plan = fs.fs_rope_plan(d)
    for fmt in ref.FORMATS:
        table, total = ref.random_table([32] * B, seed=1)
        cache = fs.fs_cache_alloc(total, H, 16, d, fmt, table.cuda())
        k, v = _rows((B, H, N, d), 1), _rows((B, H, N, d), 2)
        _, kr = fs.fs_rope(k, k, 0, plan)
        fs.fs_cache_append(cache, kr, v, _ints([0] * B))
        past = _ints([N] * B)
        # a tree of two branches under token 0: 0-1-3-5-7 and 0-2-4-6
        parent = [-1, 0, 0, 1, 2, 3, 4, 5]
        bits, depth = [], []
        for i, p in enumerate(parent):
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        tree = torch.tensor([bits] * B, device="cuda")
        pos = _ints([[N + x for x in depth]] * B)
        q, kn, vn = _rows((B, H, T, d), 3), _rows((B, H, T, d), 4), _rows((B, H, T, d), 5)
        qr, knr = fs.fs_rope(q, kn, pos, plan)
        fs.fs_cache_append(cache, knr, vn, past)
        out = fs.fs_tree_attn(qr, cache, past, tree=tree)
        _check(qr, cache, [N] * B, out, tree)
        # the branch 0-1-3-5-7 is accepted in sequence 0, token 0 alone in sequence 1
        path, keep = _ints([[0, 1, 3, 5, 7], [0, 0, 0, 0, 0]]), _ints([5, 1])
        fs.fs_cache_accept(cache, past, path, keep)
        now = past + keep
        # decoding the last accepted token again from the compacted cache gives its row of the tree
        again = fs.fs_tree_attn(qr[:, :, [7]].contiguous(), cache, now - 1)
        assert torch.equal(again[0], out[0, :, [7]]) or \
            torch.all((again[0].double() - out[0, :, [7]].double()).abs() <= 2.0 ** -6 * (
                out[0, :, [7]].double().abs() + vn.abs().max().double()))
        _check(qr[:, :, [7]].contiguous(), cache, (now - 1).tolist(), again)
        # the cache back in bf16 feeds the forward and the bounded decode state
        kc, vc = fs.fs_cache_read(cache, _ints([0] * B), T=N)
        lam, sigma, mix = (torch.full((H,), x, device="cuda") for x in (1.0, 4.0, 0.5))
        o = fs.fs_attention_fwd(kc, kc, vc, lam, sigma, mix)
        kbar, amax = fs.fs_cell_summarize(kc)
        pool, n = fs.fs_prune_cells(amax, N)
        state = fs.fs_decode_state_init(B, H, k=kc, v=vc, kbar=kbar, amax=amax, pool=pool,
                                        pool_count=n, N0=N)
        ko, vo = fs.fs_cache_read(cache, _ints([N] * B), T=1)
        t = fs.fs_decode_step(ko[:, :, 0].contiguous(), ko[:, :, 0].contiguous(),
                              vo[:, :, 0].contiguous(), N, state, lam, sigma, mix)
        torch.cuda.synchronize()
        assert torch.isfinite(o).all() and torch.isfinite(t).all()
        fs.fs_check_status(state)
        fs.fs_check_status(cache.status)
