"""Plain 64-bit statements of linear attention with a decay for each head and of the norms
around a block, with their gradients, for the tests of fs_linear_attn* and fs_block_norm*.
Torch tensors on any device; none of the library is used."""
import torch


def heads(x, H):
    return x.repeat_interleave(H // x.shape[1], 1)


def linear(q, k, v, decay, S0=None, count=None, scale=None):
    """Token after token.  Returns (out [B, H, T, d], last state [B, H, d, d]), zeros past count."""
    B, H, T, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    q, k, v = q.double(), heads(k.double(), H), heads(v.double(), H)
    lam = torch.exp(decay.double())[None, :, None, None]
    S = torch.zeros((B, H, d, d), dtype=torch.float64, device=q.device) if S0 is None else S0.double()
    out = torch.zeros((B, H, T, d), dtype=torch.float64, device=q.device)
    n = torch.full((B,), T) if count is None else count.cpu()
    for t in range(T):
        have = (t < n).to(q.device)[:, None, None, None]
        new = torch.where(lam > 0, lam * S, 0) + k[:, :, t, :, None] * v[:, :, t, None, :]
        S = torch.where(have, new, S)
        out[:, :, t] = torch.where(have, scale * (q[:, :, t, :, None] * S).sum(2, keepdim=True), 0)[:, :, 0]
    return out, S


def linear_grads(q, k, v, decay, dout, S0=None, G=None, count=None, scale=None):
    """(dq, dk, dv, dS0), token after token."""
    B, H, T, d = q.shape
    Hkv = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    q, k, v, dout = q.double(), heads(k.double(), H), heads(v.double(), H), dout.double()
    lam = torch.exp(decay.double())[None, :, None, None]
    keep = lambda x: torch.where(lam > 0, lam * x, 0)  # noqa: E731
    zero = torch.zeros((B, H, d, d), dtype=torch.float64, device=q.device)
    S = zero if S0 is None else S0.double()
    n = torch.full((B,), T) if count is None else count.cpu()
    have = [(t < n).to(q.device)[:, None, None, None] for t in range(T)]
    dq, dk, dv = (torch.zeros((B, H, T, d), dtype=torch.float64, device=q.device) for _ in range(3))
    for t in range(T):
        S = torch.where(have[t], keep(S) + k[:, :, t, :, None] * v[:, :, t, None, :], S)
        dq[:, :, t] = torch.where(have[t][..., 0], scale * (S * dout[:, :, t, None, :]).sum(-1), 0)
    P = zero if G is None else G.double()                     # lam R of the token behind
    for t in reversed(range(T)):
        R = P + scale * q[:, :, t, :, None] * dout[:, :, t, None, :]
        dk[:, :, t] = torch.where(have[t][..., 0], (R * v[:, :, t, None, :]).sum(-1), 0)
        dv[:, :, t] = torch.where(have[t][..., 0], (R * k[:, :, t, :, None]).sum(-2), 0)
        P = torch.where(have[t], keep(R), P)
    dk, dv = (x.reshape(B, Hkv, H // Hkv, T, d).sum(2) for x in (dk, dv))
    return dq, dk, dv, P


def norm(x, gate=None, residual=None, groups=0, gain=None, next_gain=None, scale=1.0, eps=1e-6):
    """(z, y) in 64 bits of [M, D]; y is the second norm of z."""
    x = x.double()
    M, D = x.shape
    a = x
    if groups:
        a = a.reshape(M, groups, -1)
        a = (a / torch.sqrt((a * a).mean(-1, keepdim=True) + eps)).reshape(M, D)
    if gain is not None:
        a = a * gain.double()
    if gate is not None:
        a = a * gate.double() / (1 + torch.exp(-gate.double()))
    z = scale * a
    if residual is not None:
        z = z + residual.double()
    y = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
    return z, y if next_gain is None else y * next_gain.double()


def norm_grads(x, dz=None, dy=None, gate=None, residual=None, groups=0, gain=None, next_gain=None,
               scale=1.0, eps=1e-6):
    """The formulas of the gradients, and for each a bound of the terms that it is the sum of:
    dict name -> (gradient, magnitude)."""
    x = x.double()
    M, D = x.shape
    one = torch.ones(D, dtype=torch.float64, device=x.device)
    gain_, next_ = (one if g is None else g.double() for g in (gain, next_gain))
    split = lambda t: t.reshape(M, groups, -1)  # noqa: E731
    h, inv = x, torch.ones_like(x)
    if groups:
        inv = (1 / torch.sqrt((split(x) ** 2).mean(-1, keepdim=True) + eps)).expand(M, groups, D // groups).reshape(M, D)
        h = x * inv
    sig = silu = torch.ones_like(x)
    if gate is not None:
        sig = 1 / (1 + torch.exp(-gate.double()))
        silu = gate.double() * sig
    g = torch.zeros_like(x) if dz is None else dz.double()
    size, res = g.abs(), {}
    if dy is not None:
        z = scale * h * gain_ * silu + (0 if residual is None else residual.double())
        # z is itself a sum: what it loses goes by its two terms' sizes, also where they cancel
        sz = (scale * h * gain_ * silu).abs() + (0 if residual is None else residual.double().abs())
        r = 1 / torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
        w = dy.double() * next_
        g = g + r * (w - z * r * r * (w * z).mean(-1, keepdim=True))
        size = size + r * (w.abs() + sz * r * r * (w.abs() * sz).mean(-1, keepdim=True))
        t = dy.double() * r
        res["next_gain"] = ((t * z).sum(0), (t.abs() * sz).sum(0))
    res["residual"] = (g, size)
    if gate is not None:
        f = scale * h * gain_ * sig * (1 + gate.double() * (1 - sig))
        part = (scale * h * gain_).abs() * sig * (1 + gate.double().abs() * (1 - sig))
        res["gate"] = (g * f, size * part)
    t = scale * silu * h
    res["gain"] = ((g * t).sum(0), (size * t.abs()).sum(0))
    u, su = scale * g * silu * gain_, abs(scale) * size * (silu * gain_).abs()
    if groups:
        c = split(u * h).mean(-1, keepdim=True).expand(M, groups, D // groups).reshape(M, D)
        sc = split(su * h.abs()).mean(-1, keepdim=True).expand(M, groups, D // groups).reshape(M, D)
        u, su = inv * (u - h * c), inv * (su + h.abs() * sc)
    res["x"] = (u, su)
    return res
