"""The serving operators around a growing key/value cache, as cases to measure.

Four kinds of pass, each in a plain form (elementary torch operations) and through the library's entry points:

``rope``    rotary positions of queries and keys, or of their gradients (the transposed rotation);
``cache``   new keys and values quantised into a paged cache, then read back as bf16 (what the prefill and the
            decode-state initialisation take);
``accept``  drafted rows written to the cache, the rows of the accepted path moved to the front, and read back;
``tree``    attention of drafted tokens (one token: plain decoding) over the paged cache.

Cache layout: ``codes`` [pages, 2 (k, v), Hkv, page, row bytes] uint8, ``scales`` [pages, 2, Hkv, page] fp32,
``table`` [batch, pages a sequence] int32.  A row is one token's d values of one head: bf16, e4m3, int8, or int4
(two a byte, the even one in the low half).  Its scale is amax / Q and its codes round(Q x / amax), ties to even,
with Q = 448, 127, 7.
"""
import math
import random

import torch

own = False

BITS = {"bf16": 16, "e4m3": 8, "int8": 8, "int4": 4}
TOP = {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}


# --- cases --------------------------------------------------------------------------------------------------------

def _rope(name, B, H, Hkv, N, d, rot, layout="half", scaling="none", factor=1.0, amplitude=1.0, far=0, dtype="bf16",
          token_major=False, grad=False):
    return dict(name=name, kind="rope", B=B, H=H, Hkv=Hkv, N=N, d=d, rot=rot, layout=layout, scaling=scaling,
                factor=factor, amplitude=amplitude, far=far, dtype=dtype, token_major=token_major, grad=grad)


def _cache(name, B, Hkv, T, d, fmt, page, past=0, ragged=True):
    return dict(name=name, kind="cache", B=B, Hkv=Hkv, T=T, d=d, fmt=fmt, page=page, past=past, ragged=ragged)


def _accept(name, B, Hkv, T, d, fmt, page, past, keep):
    return dict(name=name, kind="accept", B=B, Hkv=Hkv, T=T, d=d, fmt=fmt, page=page, past=past, keep=keep)


def _tree(name, B, H, Hkv, T, past, d, fmt, page, window=0, ragged=True):
    return dict(name=name, kind="tree", B=B, H=H, Hkv=Hkv, T=T, past=past, d=d, fmt=fmt, page=page, window=window,
                ragged=ragged)


def listed():
    return [
        # One decoding step of eight sequences at far positions: the queries and keys of 16 heads of 64.
        _rope("rope_step", 8, 16, 16, 1, 64, 64, far=200000),
        # The prefill of one sequence of 65536 tokens, 16 heads of 64.
        _rope("rope_prefill", 1, 16, 16, 65536, 64, 64),
        # The gradients of a training step (fp32, as the attention's backward gives them): adjacent pairs on half of
        # the head, frequencies stretched by parts for eight times the length, an odd number of tokens, stored token-major.
        _rope("rope_grad", 2, 16, 4, 16383, 64, 32, layout="pairs", scaling="ramp", factor=8.0, amplitude=1.2079,
              dtype="fp32", token_major=True, grad=True),
        # One decoding step of 16 sequences writes its keys and values.
        _cache("cache_step", 16, 16, 1, 64, "int8", 32, past=5000),
        # A prefill of 65536 tokens goes into an e4m3 cache and comes back for the prefill's attention.
        _cache("cache_prefill", 1, 16, 65536, 64, "e4m3", 128, ragged=False),
        # A ragged batch of prompts in four bits, grouped heads of 128, pages that end anywhere.
        _cache("cache_ragged", 5, 4, 8191, 128, "int4", 16, past=333),
        # Eight drafted tokens of one sequence verified, four kept.
        _accept("accept_small", 1, 16, 8, 64, "bf16", 64, past=1000, keep=4),
        # 64 drafted tokens of each of 48 sequences, up to 17 kept.
        _accept("accept_batch", 48, 16, 64, 64, "int8", 16, past=2047, keep=17),
        # One token of one sequence over 4096 cached ones: the smallest call, where latency counts.
        _tree("tree_step", 1, 16, 16, 1, 4096, 64, "bf16", 64),
        # 16 drafted tokens of four long sequences over an e4m3 cache, every head with its own keys.
        _tree("tree_long", 4, 16, 16, 16, 65536, 64, "e4m3", 128),
        # One token over 262144 cached ones in four bits, eight query heads to a key head.
        _tree("tree_far", 1, 32, 4, 1, 262144, 128, "int4", 32),
        # Full trees of 64 tokens, four query heads to a key head, a ragged batch over an int8 cache.
        _tree("tree_wide", 8, 32, 8, 64, 16384, 64, "int8", 16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "cache", "accept", "tree", "tree"])
    d = rng.choice([64, 64, 128])
    fmt, page = rng.choice(list(BITS)), rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    if kind == "rope":
        G, B = rng.choice([1, 1, 2, 4]), _log(rng, 1, 16)
        Hkv = min(Hkv, 16 // G)
        N = _log(rng, 1, max(1, 65536 * 16 * 64 * 2 // (2 * B * (G + 1) * Hkv * d)))
        scaling = rng.choice(["none", "linear", "base", "ramp"])
        c = _rope("", B, G * Hkv, Hkv, N, d, rng.choice([d, d, d // 2, d // 4]), rng.choice(["half", "pairs"]), scaling,
                  1.0 if scaling == "none" else rng.choice([2.0, 8.0, 40.0]), 1.1 if scaling == "ramp" else 1.0,
                  rng.randrange(250000), rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.5, rng.random() < 0.3)
    elif kind == "cache":
        B = _log(rng, 1, 32)
        c = _cache("", B, Hkv, _log(rng, 1, max(1, 65536 * 16 * 64 // (B * Hkv * d))), d, fmt, page, rng.randrange(2000))
    elif kind == "accept":
        T = rng.randint(2, 64)
        c = _accept("", _log(rng, 1, 48), Hkv, T, d, fmt, page, _log(rng, 1, 4000), rng.randint(1, min(T, 17)))
    else:
        T, G, B = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 2, 64)]), rng.choice([1, 1, 2, 4, 8]), _log(rng, 1, 16)
        most = min(65536 * 64 * 64 // (B * Hkv * d), 8 * 32 * 64 * 16384 * 64 // (B * Hkv * G * T * d))
        c = _tree("", B, Hkv * G, Hkv, T, _log(rng, 16, max(16, min(262144, most))), d, fmt, page,
                  rng.choice([0, 0, 0, 512]))
    c.pop("name")
    return c


def _lengths(case):
    """Cached tokens of each sequence and new tokens of each: from the case alone, so that the work is known."""
    r = random.Random(case["T"] * 7919 + case["past"] * 31 + case["B"])
    some = case.get("ragged", True)
    past = [case["past"] if b == 0 or not some else r.randint(case["past"] * 3 // 4, case["past"]) for b in range(case["B"])]
    new = [case["T"] if b == 0 or not some else r.randint((case["T"] + 1) // 2, case["T"]) for b in range(case["B"])]
    return past, new


def work(case):
    if case["kind"] == "rope":
        n = case["B"] * (case["H"] + case["Hkv"]) * case["N"]
        return {"bytes": 2 * n * case["d"] * (2 if case["dtype"] == "bf16" else 4) + 4 * case["B"] * case["N"],
                "flops": 3 * n * case["rot"]}
    past, new = _lengths(case)
    stored = case["d"] * BITS[case["fmt"]] // 8 + (0 if case["fmt"] == "bf16" else 4)
    rows = 2 * case["Hkv"]
    if case["kind"] == "cache":
        n = rows * sum(new)
        return {"bytes": n * (4 * case["d"] + stored), "flops": 4 * n * case["d"]}
    if case["kind"] == "accept":
        keep = rows * sum(min(case["keep"], t) for t in new)
        n = rows * sum(new)
        return {"bytes": n * (2 * case["d"] + stored) + keep * 2 * case["d"], "flops": 3 * n * case["d"] + keep * case["d"]}
    w = case["window"] or 1 << 30
    keys = [min(p, w + t) + t for p, t in zip(past, new)]
    seen = [(min(p, w) + (t + 1) / 2) * t for p, t in zip(past, new)]
    q = sum(new) * case["H"] * case["d"]
    return {"bytes": int(rows * sum(keys) * stored + 4 * q), "flops": int(4 * case["d"] * case["H"] * sum(seen))}


# --- inputs -------------------------------------------------------------------------------------------------------

def _keys(g, shape, spread=0.5):
    """Keys whose norms vary from token to token, as a trained model's do."""
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))).to(torch.bfloat16)


def _pages(case, g, past, room):
    """An empty cache with a shuffled table: pages of a sequence lie anywhere, entries past its last are -1."""
    page, d, fmt, Hkv = case["page"], case["d"], case["fmt"], case["Hkv"]
    need = [-(-(p + room) // page) for p in past]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(past), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    codes = torch.zeros((total, 2, Hkv, page, d * BITS[fmt] // 8), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((total, 2, Hkv, page), device="cuda")
    return codes, scales, table.cuda()


def _trees(r, T, new):
    """Visible drafted tokens of every drafted token: itself and its ancestors in a random tree, as bits."""
    rows = []
    for t in new:
        bits = []
        for i in range(T):
            up = bits[max(0, i - r.randint(1, 4))] if i else 0
            bits.append(up | 1 << i)
        rows.append([x - (1 << 64) if x >> 63 else x for x in bits])
    return torch.tensor(rows, dtype=torch.int64, device="cuda")


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7 + 1)
    r = random.Random(seed)
    s = dict(case)
    if case["kind"] == "rope":
        B, N, d = case["B"], case["N"], case["d"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        for name, heads in (("q", case["H"]), ("k", case["Hkv"])):
            shape = (B, N, heads, d) if case["token_major"] else (B, heads, N, d)
            x = torch.randn(shape, generator=g, device="cuda").to(dt)
            s[name] = x.transpose(1, 2) if case["token_major"] else x
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = (first + torch.arange(N, device="cuda")).to(torch.int32)
        if own:
            from long_context_lm_gb300 import fs
            s["plan"] = fs.fs_rope_plan(case["rot"], layout=case["layout"], scaling=case["scaling"], base=10000.0,
                                        factor=case["factor"], original=4096, amplitude=case["amplitude"])
        return s
    past, new = _lengths(case)
    B, Hkv, T, d = case["B"], case["Hkv"], case["T"], case["d"]
    s["past"], s["new"] = _int(past), _int(new)
    s["codes"], s["scales"], s["table"] = _pages(case, g, past, T)
    if case["kind"] == "tree":
        n = s["codes"].shape[0]
        step = max(1, (1 << 26) // (s["scales"][0].numel() * d))
        for a in range(0, n, step):
            rows = _keys(g, s["scales"][a:a + step].shape + (d,))
            s["codes"][a:a + step], s["scales"][a:a + step] = _quantise(rows, case["fmt"])
        s["q"] = torch.randn((B, case["H"], T, d), generator=g, device="cuda").to(torch.bfloat16)
        s["tree"] = _trees(r, T, new) if T > 1 else None
        s["out"] = torch.zeros_like(s["q"])
    else:
        s["k"], s["v"] = _keys(g, (B, Hkv, T, d)), _keys(g, (B, Hkv, T, d), 0.2)
        n = T
        if case["kind"] == "accept":
            keep = [min(case["keep"], t) for t in new]
            n = case["keep"]
            s["path"] = _int([sorted(r.sample(range(t), m)) + [0] * (n - m) for t, m in zip(new, keep)])
            s["keep"] = _int(keep)
        s["k_out"], s["v_out"] = (torch.zeros((B, Hkv, n, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if own:
        from long_context_lm_gb300 import fs
        s["cache"] = fs.fs_cache(s["codes"], s["scales"], s["table"], case["fmt"])
        if case["kind"] == "tree":
            s["ws"] = fs.fs_tree_workspace(s["cache"], B, case["H"], T)
    return s


# --- the plain form -----------------------------------------------------------------------------------------------

def _frequencies(case):
    """Radians a position of each pair, in 64 bits."""
    r, base, F = case["rot"], 10000.0, case["factor"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "base":
        base = base * F ** (r / (r - 2))
    f = base ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        f = f / F
    if case["scaling"] == "ramp":
        turn = [r * math.log(4096 / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        lo, hi = max(math.floor(turn[0]), 0), min(math.ceil(turn[1]), r // 2 - 1)
        part = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - part) + f / F * part
    return f


def _rotate(case, x, cos, sin):
    r = case["rot"]
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if case["layout"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])
    a, b = a.float(), b.float()
    y = torch.empty_like(x)
    u, v = a * cos - b * sin, b * cos + a * sin
    if case["layout"] == "half":
        y[..., :r // 2], y[..., r // 2:r] = u.to(x.dtype), v.to(x.dtype)
    else:
        y[..., 0:r:2], y[..., 1:r:2] = u.to(x.dtype), v.to(x.dtype)
    y[..., r:] = x[..., r:]
    return y


def _quantise(x, fmt):
    """Rows of bf16 values -> (codes as bytes, scales)."""
    if fmt == "bf16":
        return x.contiguous().view(torch.uint8), torch.zeros(x.shape[:-1], device=x.device)
    x = x.double()  # quotients next to a border between two codes
    amax = x.abs().amax(-1)
    y = x * TOP[fmt] / torch.where(amax > 0, amax, 1.0)[..., None]
    scale = amax.float() / TOP[fmt]
    if fmt == "e4m3":
        return y.float().to(torch.float8_e4m3fn).view(torch.uint8), scale
    y = torch.round(y).to(torch.int8)
    if fmt == "int4":
        y = (y[..., 0::2] & 15) | (y[..., 1::2] << 4)
    return y.view(torch.uint8), scale


def _values(codes, scales, fmt):
    if fmt == "bf16":
        return codes.view(torch.bfloat16).float()
    if fmt == "e4m3":
        x = codes.view(torch.float8_e4m3fn).float()
    elif fmt == "int8":
        x = codes.view(torch.int8).float()
    else:
        c = codes.view(torch.int8)
        x = torch.stack(((c << 4) >> 4, c >> 4), -1).flatten(-2).float()
    return x * scales[..., None]


def _place(s, at):
    """Page and row inside it of positions `at` [B, n]; positions that the table has no page for get page 0."""
    at = at.long()
    block = (at // s["page"]).clamp(max=s["table"].shape[1] - 1)
    return torch.gather(s["table"].long(), 1, block).clamp(min=0), at % s["page"]


def _fetch(s, at, part):
    """Values [B, Hkv, n, d] in 32 bits of the keys (part 0) or values (1) at positions `at`."""
    p, o = _place(s, at)
    return _values(s["codes"][p, part, :, o], s["scales"][p, part, :, o], s["fmt"]).transpose(1, 2)


def _store(s, at, have, x, part):
    codes, scales = _quantise(x.transpose(1, 2), s["fmt"])
    p, o = _place(s, at)
    s["codes"][p[have], part, :, o[have]] = codes[have]
    s["scales"][p[have], part, :, o[have]] = scales[have]


def _append(s):
    t = torch.arange(s["T"], device="cuda")
    at, have = s["past"][:, None] + t, t < s["new"][:, None]
    for part, x in enumerate((s["k"], s["v"])):
        _store(s, at, have, x, part)


def _read(s, count, n):
    t = torch.arange(n, device="cuda")
    have = (t < count[:, None])[:, None, :, None]
    return tuple(torch.where(have, _fetch(s, s["past"][:, None] + t, part), 0).to(torch.bfloat16) for part in (0, 1))


def _move(s):
    n = s["path"].shape[1]
    t = torch.arange(n, device="cuda")
    have = t < s["keep"][:, None]
    src, dst = _place(s, s["past"][:, None] + s["path"]), _place(s, (s["past"][:, None] + t).expand(-1, n))
    for x in (s["codes"], s["scales"]):
        for part in (0, 1):
            x[dst[0][have], part, :, dst[1][have]] = x[src[0], part, :, src[1]][have]


def _attend(s):
    B, H, T, d = s["q"].shape
    Hkv = s["Hkv"]
    S = s["table"].shape[1] * s["page"]
    at = torch.arange(S, device="cuda").expand(B, S)
    k, v = _fetch(s, at, 0), _fetch(s, at, 1)
    past, t = s["past"].long()[:, None, None], torch.arange(T, device="cuda")
    tree = s["tree"] if s["tree"] is not None else torch.ones((B, 1), dtype=torch.int64, device="cuda")
    j = at[:, None, :] - past
    drafted = (j >= 0) & (j < s["new"][:, None, None]) & (((tree[:, :, None] >> j.clamp(0, 63)) & 1) == 1)
    before = j < 0
    if s["window"]:
        own_bits = ((tree[:, :, None] >> torch.arange(64, device="cuda")) & 1).sum(-1)
        before = before & (j > (own_bits - 1 - s["window"])[:, :, None])
    q = s["q"].float().reshape(B, Hkv, -1, d)
    x = (q @ k.transpose(2, 3)).reshape(B, Hkv, H // Hkv, T, S) / math.sqrt(d)
    x = torch.where((drafted | before)[:, None, None], x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, -1, S) @ v).reshape(B, Hkv, H // Hkv, T, d) / torch.where(total > 0, total, 1.0)
    have = (t < s["new"][:, None])[:, None, :, None]
    return torch.where(have, o.reshape(B, H, T, d), 0).to(torch.bfloat16)


def _plain(s):
    if s["kind"] == "rope":
        angle = s["pos"].double()[:, None, :, None] * _frequencies(s)
        cos, sin = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
        sin = -sin if s["grad"] else sin
        return _rotate(s, s["q"], cos, sin), _rotate(s, s["k"], cos, sin)
    if s["kind"] == "tree":
        return _attend(s)
    _append(s)
    if s["kind"] == "cache":
        return _read(s, s["new"], s["T"])
    _move(s)
    return _read(s, s["keep"], s["path"].shape[1])


def run(s):
    if not own:
        return _plain(s)
    from long_context_lm_gb300 import fs
    if s["kind"] == "rope":
        return fs.fs_rope(s["q"], s["k"], s["pos"], s["plan"], inverse=s["grad"])
    if s["kind"] == "tree":
        return fs.fs_tree_attn(s["q"], s["cache"], s["past"], tree=s["tree"], count=s["new"], window=s["window"],
                               out=s["out"], ws=s["ws"])
    fs.fs_cache_append(s["cache"], s["k"], s["v"], s["past"], s["new"])
    if s["kind"] == "cache":
        return fs.fs_cache_read(s["cache"], s["past"], s["new"], s["k_out"], s["v_out"])
    fs.fs_cache_accept(s["cache"], s["past"], s["path"], s["keep"])
    return fs.fs_cache_read(s["cache"], s["past"], s["keep"], s["k_out"], s["v_out"])


# --- the definition in 64 bits ------------------------------------------------------------------------------------

def _exact_rows(x, fmt):
    """What rows of values read back as."""
    x = x.double()
    if fmt == "bf16":
        return x
    top = x.abs().max(-1, keepdim=True).values
    unit = torch.where(top > 0, top, 1.0) / TOP[fmt]
    y = x * TOP[fmt] / torch.where(top > 0, top, 1.0)
    if fmt == "e4m3":  # three fraction bits, the least exponent -6
        steps = torch.tensor([2.0 ** (e - 4) for e in range(-5, 10)], dtype=torch.float64, device="cuda")
        step = steps[torch.frexp(y).exponent.long().clamp(min=-5) + 5]
        return torch.round(y / step) * step * unit
    return torch.round(y) * unit


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        z, r = [], case["rot"]
        base = 10000.0 * (case["factor"] ** (r / (r - 2.0)) if case["scaling"] == "base" else 1.0)
        f = [math.pow(base, -i / r) for i in range(0, r, 2)]
        if case["scaling"] in ("linear", "ramp"):
            edge = [r / 2 * math.log(4096 / (2 * math.pi * b), base) for b in (32, 1)]
            lo, hi = max(0, math.floor(edge[0])), min(r // 2 - 1, math.ceil(edge[1]))
            slow = [1.0 if case["scaling"] == "linear" else min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo))) for i in range(r // 2)]
            f = [x * (1 - w + w / case["factor"]) for x, w in zip(f, slow)]
        f = torch.tensor(f, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full((), case["amplitude"], dtype=torch.float64, device="cuda").expand(case["B"], case["N"], len(f)),
                           s["pos"].double()[..., None] * f)
        turn = torch.conj(turn) if case["grad"] else turn
        for x in (s["q"], s["k"]):
            y = x.double()
            part = y[..., :r]
            c = torch.complex(*(part.unflatten(-1, (2, -1)).unbind(-2) if case["layout"] == "half" else part.unflatten(-1, (-1, 2)).unbind(-1)))
            c = torch.view_as_real(c * turn[:, None])
            c = c.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else c.flatten(-2)
            z.append(torch.cat((c, y[..., r:]), -1))
        return tuple(z)
    past, new = _lengths(case)
    if case["kind"] != "tree":
        outs = []
        for x in (s["k"], s["v"]):
            y = _exact_rows(x, case["fmt"])
            z = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
            for b, t in enumerate(new):
                at = list(range(t)) if case["kind"] == "cache" else s["path"][b, :int(s["keep"][b])].tolist()
                z[b, :, :len(at)] = y[b][:, at]
            outs.append(z)
        return tuple(outs)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    G = case["H"] // case["Hkv"]
    for b, (n, t) in enumerate(zip(past, new)):
        pages = s["table"][b, :-(-(n + t) // case["page"])].long()
        seen = torch.ones((t, n + t), dtype=torch.bool, device="cuda")
        for i in range(t):
            bits = 1 if s["tree"] is None else int(s["tree"][b, i]) & ((1 << 64) - 1)
            seen[i, n:] = torch.tensor([bool(bits >> j & 1) for j in range(t)], device="cuda")
            if case["window"]:
                seen[i, :max(0, n + bin(bits).count("1") - case["window"])] = False
        for h in range(case["Hkv"]):
            kv = []
            for part in (0, 1):
                c = s["codes"][pages, part, h].reshape(len(pages) * case["page"], -1)[:n + t]
                if case["fmt"] == "bf16":
                    kv.append(c.view(torch.bfloat16).double())
                    continue
                if case["fmt"] == "int4":
                    c = torch.stack((c % 16, c // 16), -1).flatten(-2).double()
                    c = torch.where(c > 7, c - 16, c)
                else:
                    c = c.view(torch.float8_e4m3fn if case["fmt"] == "e4m3" else torch.int8).to(torch.float32).double()
                kv.append(c * s["scales"][pages, part, h].reshape(-1)[:n + t, None].double())
            q = s["q"][b, h * G:(h + 1) * G, :t].double()
            x = torch.matmul(q, kv[0].T) * case["d"] ** -0.5
            p = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
            out[b, h * G:(h + 1) * G, :t] = torch.matmul(p, kv[1])
    return out
