"""Plain 64-bit statements of the rotary positions, the paged cache and the
attention over it, for the tests of fs_rope, fs_cache_* and fs_tree_attn.
They take and give torch tensors on any device and use none of the library."""
import math

import torch

TOP = {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}
BITS = {"bf16": 16, "e4m3": 8, "int8": 8, "int4": 4}
FORMATS = list(BITS)


def frequencies(rot, scaling="none", base=10000.0, factor=1.0, original=4096, beta_fast=32.0,
                beta_slow=1.0):
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "ramp":
        def pair(beta):
            return rot * math.log(original / (2 * math.pi * beta)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot // 2 - 1)
        g = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        f = [x * (1 - w) + x / factor * w for x, w in zip(f, g)]
    return f


def rope(x, pos, f, layout, amplitude=1.0, inverse=False):
    """x [B, H, N, d], pos [B, N] -> fp64."""
    y = x.double().clone()
    r = 2 * len(f)
    ang = pos.double()[:, None, :, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    c, s = amplitude * torch.cos(ang), amplitude * torch.sin(ang)
    s = -s if inverse else s
    ia = torch.arange(r // 2) if layout == "half" else 2 * torch.arange(r // 2)
    ib = ia + r // 2 if layout == "half" else ia + 1
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def _e4m3_values(device):
    """All finite e4m3 magnitudes, ascending (three fraction bits, bias 7)."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    return torch.tensor(v, dtype=torch.float64, device=device)


def quantise(x, fmt):
    """Rows of bf16 values [..., d] -> (codes uint8 [..., row bytes], scales fp32)."""
    if fmt == "bf16":
        return x.contiguous().view(torch.uint8), None
    z = x.double()
    bad = ~torch.isfinite(z).all(-1)
    amax = z.abs().amax(-1)
    scale = (amax / TOP[fmt]).float()
    y = z * TOP[fmt] / torch.where((amax > 0) & ~bad, amax, torch.inf)[..., None]
    y = torch.where(bad[..., None], 0.0, y)
    scale = torch.where(bad, torch.nan, scale)
    if fmt == "e4m3":
        vals = _e4m3_values(x.device)
        mid = (vals[1:] + vals[:-1]) / 2
        m = y.abs().contiguous()
        code = torch.searchsorted(mid, m)                 # ties (m == mid) give the lower
        tie = (code < len(mid)) & (m == mid[code.clamp(max=len(mid) - 1)])
        code = code + (tie & (code % 2 == 1))             # to the even code
        return (code + 128 * (torch.signbit(y)).long()).to(torch.uint8), scale
    code = torch.round(y).long()
    if fmt == "int8":
        return (code & 255).to(torch.uint8), scale
    return ((code[..., 0::2] & 15) | ((code[..., 1::2] & 15) << 4)).to(torch.uint8), scale


def values(codes, scales, fmt, dtype=torch.float64):
    """What rows stand for: code * scale in ``dtype``."""
    if fmt == "bf16":
        return codes.contiguous().view(torch.bfloat16).to(dtype)
    c = codes.long()
    if fmt == "e4m3":
        vals = _e4m3_values(codes.device)
        m = vals[(c & 127).clamp(max=126)]
        x = torch.where(c >= 128, -m, m)
        x = torch.where((c & 127) == 127, torch.nan, x)
    elif fmt == "int8":
        x = torch.where(c > 127, c - 256, c)
    else:
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2)
        x = torch.where(c > 7, c - 16, c)
    return x.to(dtype) * scales.to(dtype)[..., None]


def random_table(need, extra=3, seed=0):
    """A shuffled page table for sequences that need ``need`` pages; -1 past the last."""
    g = torch.Generator().manual_seed(seed)
    total = sum(need) + extra
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def gather(cache, b, n, part):
    """Rows 0 .. n-1 of sequence b: (codes [n, Hkv, row], scales [n, Hkv])."""
    t = torch.arange(n, device=cache.codes.device)
    page = cache.table[b].long()[t // cache.page]
    codes = cache.codes[page, part, :, t % cache.page]
    scales = None if cache.scales is None else cache.scales[page, part, :, t % cache.page]
    return codes, scales


def tree_attention(q, cache, past, tree, count, window=0, scale=None):
    """(out, weight) in fp64: the definition, and the mean of |v| under the same probabilities
    (what a relative error of every probability is multiplied by), with the largest sum of
    |scale q k|."""
    B, H, T, d = q.shape
    G = H // cache.Hkv
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros((B, H, T, d), dtype=torch.float64, device=q.device)
    mean = torch.zeros_like(out)
    most = 0.0
    for b in range(B):
        p0, n = int(past[b]), int(count[b])
        if n == 0:
            continue
        seen = torch.zeros((n, p0 + n), dtype=torch.bool, device=q.device)
        for i in range(n):
            bits = ((1 << (i + 1)) - 1 if tree is None else int(tree[b, i])) & ((1 << n) - 1)
            first = max(0, p0 + bin(bits).count("1") - window) if window else 0
            seen[i, first:p0] = True
            seen[i, p0:] = torch.tensor([bool(bits >> j & 1) for j in range(n)])
        kc, ks = gather(cache, b, p0 + n, 0)
        vc, vs = gather(cache, b, p0 + n, 1)
        k, v = values(kc, ks, cache.format), values(vc, vs, cache.format)
        for h in range(H):
            qq, kk, vv = q[b, h, :n].double(), k[:, h // G], v[:, h // G]
            s = (scale * qq @ kk.T).masked_fill(~seen, -math.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
            p = torch.where(seen, p, 0.0)
            total = p.sum(-1, keepdim=True)
            p = p / torch.where(total == 0, 1.0, total)
            # a masked key's NaN or infinity does not reach the row
            for i in range(n):
                keys = seen[i]
                out[b, h, i] = p[i, keys] @ vv[keys]
                mean[b, h, i] = p[i, keys] @ vv[keys].abs()
            if seen.any():
                big = scale * (qq.abs() @ kk.abs().T)
                big = torch.where(seen & torch.isfinite(big), big, 0.0)
                most = max(most, float(big.max()))
    return out, mean, most
