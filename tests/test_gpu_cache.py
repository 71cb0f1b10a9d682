"""The paged cache: fs_cache_append, fs_cache_read and fs_cache_accept (GPU
only).  Codes and scales are whole numbers and single roundings, so they are
compared bit for bit with the 64-bit statement; a row reads back as one fp32
product, rounded once more to bf16."""
import pytest
import torch

from long_context_lm_gb300 import fs
import serving_ref as ref

pytestmark = pytest.mark.gpu


def _cache(need, Hkv, page, d, fmt, seed=0, fill=0xff):
    """A cache whose free space holds ``fill`` bytes (NaN codes and scales)."""
    table, total = ref.random_table(need, seed=seed)
    cache = fs.fs_cache_alloc(total, Hkv, page, d, fmt, table.cuda())
    cache.codes.fill_(fill)
    if cache.scales is not None:
        cache.scales.fill_(float("nan"))
    return cache


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _keys(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp(torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))).bfloat16()


def _expected(before, cache, k, v, start, count):
    """The codes and scales that an append must leave."""
    codes, scales = before[0].clone(), None if before[1] is None else before[1].clone()
    for part, x in enumerate((k, v)):
        c, s = ref.quantise(x, cache.format)
        for b in range(cache.batch):
            for t in range(count[b]):
                at = start[b] + t
                page = int(cache.table[b, at // cache.page])
                codes[page, part, :, at % cache.page] = c[b, :, t]
                if scales is not None:
                    scales[page, part, :, at % cache.page] = s[b, :, t]
    return codes, scales


def _same(a, b):
    return (a is None and b is None) or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("Hkv,page,d,T,start,count", [
    (1, 16, 64, 1, [0], [1]),
    (3, 16, 128, 40, [5, 0, 31], [40, 0, 17]),     # ragged, an empty sequence, page borders
    (4, 64, 64, 129, [63, 64], [129, 1]),
    (2, 256, 64, 7, [255, 3, 250, 600], [7, 7, 7, 7]),
    (5, 32, 128, 33, [1], [33]),
])
def test_append_and_read(fmt, Hkv, page, d, T, start, count):
    need = [-(-(s + T) // page) for s in start]
    cache = _cache(need, Hkv, page, d, fmt, seed=T)
    before = cache.codes.clone(), None if cache.scales is None else cache.scales.clone()
    k, v = _keys((len(start), Hkv, T, d), T), _keys((len(start), Hkv, T, d), T + 1)
    fs.fs_cache_append(cache, k, v, _ints(start), _ints(count))
    codes, scales = _expected(before, cache, k, v, start, count)
    assert _same(cache.codes, codes) and _same(cache.scales, scales)
    for dtype in (torch.float32, torch.bfloat16):
        ko, vo = (torch.full((len(start), Hkv, T, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        fs.fs_cache_read(cache, _ints(start), _ints(count), ko, vo)
        for x, got in ((k, ko), (v, vo)):
            c, s = ref.quantise(x, fmt)
            want = ref.values(c, s, fmt, torch.float32).to(dtype)
            for b, n in enumerate(count):
                assert torch.equal(got[b, :, :n], want[b, :, :n])
                assert torch.all(got[b, :, n:] == 7.0)      # rows past the count: as they were
    fs.fs_check_status(cache.status)


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
def test_quotients_next_to_and_on_borders(fmt):
    # every bf16 magnitude under a largest one of 1.9921875 (255 / 128, no exact reciprocal), 1.0,
    # 1.1015625 and of the ends of bf16's range; each row starts with its largest value
    rows = []
    for top in (255 / 128, 1.0, 141 / 128, 2.0 ** 100, 3.3895313892515355e38, 2.0 ** -126, 2.0 ** -133,
                3 * 2.0 ** -133, 2.0 ** 64, 193 * 2.0 ** 58):
        bits = torch.tensor(top, dtype=torch.float32).bfloat16().view(torch.int16).item()
        x = torch.arange(max(bits - 1600, 0), bits + 1, dtype=torch.int16).view(torch.bfloat16).flip(0)
        x = x[:1 + (len(x) - 1) // 63 * 63][1:].reshape(-1, 63)
        x = torch.cat((torch.full((len(x), 1), top).bfloat16(), x), 1)
        rows += [x, -x]
    x = torch.cat([r for r in rows if len(r)])
    T = len(x)
    cache = _cache([-(-T // 256)], 1, 256, 64, fmt)
    x = x.cuda().reshape(1, 1, T, 64)
    fs.fs_cache_append(cache, x, -x, _ints([0]))
    for part, y in ((0, x), (1, -x)):
        c, s = ref.quantise(y, fmt)
        got_c, got_s = ref.gather(cache, 0, T, part)
        assert torch.equal(got_s[:, 0], s[0, 0])
        assert torch.equal(got_c[:, 0], c[0, 0])


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_zero_and_not_finite_rows(fmt):
    x = torch.randn((1, 1, 5, 64), device="cuda").bfloat16()
    x[0, 0, 0] = 0
    x[0, 0, 1, 9] = float("nan")
    x[0, 0, 2, 63] = float("inf")
    x[0, 0, 3, 0] = float("-inf")
    cache = _cache([1], 1, 16, 64, fmt)
    fs.fs_cache_append(cache, x, x, _ints([0]))
    k, _ = fs.fs_cache_read(cache, _ints([0]), T=5, dtype=torch.float32)
    if fmt == "bf16":
        assert torch.equal(k.nan_to_num(nan=99.0), x.float().nan_to_num(nan=99.0))
        return
    assert torch.all(k[0, 0, 0] == 0) and torch.all(torch.isfinite(k[0, 0, 4]))
    assert torch.all(torch.isnan(k[0, 0, 1:4]))
    codes, _ = ref.gather(cache, 0, 5, 0)
    assert torch.all(codes[1:4] == 0)


def test_strided_inputs_and_refusals():
    B, T, H, d = 2, 21, 4, 64
    big = torch.randn((B, T, 3, H, d), device="cuda").bfloat16()
    k, v = (big[:, :, i].transpose(1, 2) for i in (1, 2))
    a, b = (_cache([2, 2], H, 16, d, "int8", seed=4) for _ in range(2))
    fs.fs_cache_append(a, k, v, _ints([3, 0]))
    fs.fs_cache_append(b, k.contiguous(), v.contiguous(), _ints([3, 0]))
    assert _same(a.codes, b.codes) and _same(a.scales, b.scales)
    odd = torch.randn((B, H, T, d + 4), device="cuda").bfloat16()[..., :d]     # rows of 136 bytes
    with pytest.raises(fs.FSError):
        fs.fs_cache_append(a, odd, odd, _ints([0, 0]))
    with pytest.raises(ValueError):
        fs.fs_cache_append(a, k.float(), v, _ints([0, 0]))
    with pytest.raises(ValueError):
        fs.fs_cache_append(a, k, v, _ints([0]))
    with pytest.raises(ValueError):
        fs.fs_cache_append(a, k[:, :3], v[:, :3], _ints([0, 0]))
    with pytest.raises(ValueError):
        fs.fs_cache_read(a, _ints([0, 0]))


@pytest.mark.parametrize("fmt", ref.FORMATS)
def test_positions_and_pages_outside_are_skipped_and_reported(fmt):
    cache = _cache([2, 2, 2], 2, 16, 64, fmt)
    cache.table[1, 1] = cache.codes.shape[0]           # one past the last page
    cache.table[2, 0] = -7
    before = cache.codes.clone(), None if cache.scales is None else cache.scales.clone()
    x = _keys((3, 2, 8, 64), 1)
    start = [28, 12, 12]                               # past the table; into a bad page; out of one
    fs.fs_cache_append(cache, x, x, _ints(start))
    codes, scales = before[0].clone(), None if before[1] is None else before[1].clone()
    c, s = ref.quantise(x, fmt)
    for b, (t0, t1) in enumerate(((0, 4), (0, 4), (4, 8))):   # what has a place
        for t in range(t0, t1):
            at = start[b] + t
            page = int(cache.table[b, at // 16])
            codes[page, :, :, at % 16] = c[b, :, t]
            if scales is not None:
                scales[page, :, :, at % 16] = s[b, :, t]
    assert _same(cache.codes, codes) and _same(cache.scales, scales)
    with pytest.raises(fs.FSError) as e:
        fs.fs_check_status(cache.status)
    assert e.value.status == fs.FS_ERR_CACHE
    cache.status.zero_()
    k = torch.full((3, 2, 8, 64), 5.0, device="cuda")
    fs.fs_cache_read(cache, _ints([28, -3, 0]), None, k, torch.empty_like(k))
    assert torch.all(k[0, :, 4:] == 5.0) and torch.all(k[1, :, :3] == 5.0) and torch.all(k[2] == 5.0)
    assert not torch.any(k[0, :, :4] == 5.0)
    with pytest.raises(fs.FSError):
        fs.fs_check_status(cache.status)


@pytest.mark.parametrize("fmt", ref.FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_accept_moves_the_path(fmt, d):
    start = [13, 0, 40, 7]
    cache = _cache([5, 5, 7, 5], 3, 16, d, fmt, seed=9)
    x, y = _keys((4, 3, 64, d), 2), _keys((4, 3, 64, d), 3)
    fs.fs_cache_append(cache, x, y, _ints(start))
    before = cache.codes.clone(), None if cache.scales is None else cache.scales.clone()
    # ascending; nothing; any order with repeats (sources that are also targets); all of it
    path = torch.zeros((4, 64), dtype=torch.int32)
    path[0, :5] = torch.tensor([0, 2, 3, 40, 63])
    path[2, :9] = torch.tensor([8, 7, 6, 5, 4, 3, 2, 2, 0])
    path[3] = torch.arange(63, -1, -1)
    count = [5, 0, 9, 64]
    fs.fs_cache_accept(cache, _ints(start), path.cuda(), _ints(count))
    codes, scales = before[0].clone(), None if before[1] is None else before[1].clone()
    for b, n in enumerate(count):
        for i in range(n):
            src, dst = start[b] + int(path[b, i]), start[b] + i
            ps, pd = int(cache.table[b, src // 16]), int(cache.table[b, dst // 16])
            codes[pd, :, :, dst % 16] = before[0][ps, :, :, src % 16]
            if scales is not None:
                scales[pd, :, :, dst % 16] = before[1][ps, :, :, src % 16]
    assert _same(cache.codes, codes) and _same(cache.scales, scales)
    fs.fs_check_status(cache.status)


def test_accept_with_indices_outside():
    cache = _cache([5], 1, 16, 64, "int8")
    x = _keys((1, 1, 64, 64), 2)
    fs.fs_cache_append(cache, x, x, _ints([10]))
    before = cache.codes.clone()
    fs.fs_cache_accept(cache, _ints([10]), _ints([[64, -1, 3]]))
    want = before.clone()
    src, dst = 13, 12
    want[int(cache.table[0, 0]), :, :, dst] = before[int(cache.table[0, 0]), :, :, src]
    assert torch.equal(cache.codes, want)
    with pytest.raises(fs.FSError) as e:
        fs.fs_check_status(cache.status)
    assert e.value.status == fs.FS_ERR_CACHE


def test_cache_calls_in_a_graph_and_on_a_stream():
    cache, other = (_cache([4, 4], 2, 16, 64, "e4m3", seed=1) for _ in range(2))
    x, y = _keys((2, 2, 10, 64), 5), _keys((2, 2, 10, 64), 6)
    start, count, path = _ints([20, 0]), _ints([10, 4]), _ints([[1, 4], [0, 3]])
    ko, vo = (torch.zeros((2, 2, 10, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(c, **kw):
        fs.fs_cache_append(c, x, y, start, count, **kw)
        fs.fs_cache_accept(c, start, path, **kw)
        return fs.fs_cache_read(c, start, count, ko, vo, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(cache, stream=s)
    s.synchronize()
    want = ko.clone(), vo.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(other)
    ko.zero_(), vo.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ko, want[0]) and torch.equal(vo, want[1]) and torch.equal(cache.codes, other.codes)
