"""The operators of a linear-attention layer, as cases to measure.

``prompt``     linear attention with a decay for each head over whole prompts, from and to a state;
``step``       the same for one new token of every sequence (the recurrent form);
``grad``       its gradients;
``norm``       the norms after and before a block with its gate and residual scale;
``norm_grad``  their gradients.

Each in a plain form (elementary torch operations) and through the library's entry points.

Linear attention, lam = exp(decay of the head), states [d (key), d (value)]:

    S_t = lam S_{t-1} + k_t v_t^T          out_t = scale q_t S_t

and, with the gradients dout_t of the outputs and G of the last state,

    R_t = scale q_t dout_t^T + lam R_{t+1},  lam R_T = G
    dq_t = scale S_t dout_t      dk_t = R_t v_t      dv_t = R_t^T k_t      dS_0 = lam R_0

Norms: a = x, normalised in groups, times a gain, times silu(gate); z = residual + scale a; y = z normalised, times
another gain.  Each of these parts can be missing.
"""
import math
import random

import torch

own = False

EPS = 1e-6
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --- cases --------------------------------------------------------------------------------------------------------

def _linear(name, kind, B, H, Hkv, T, d, ragged=False, state=True, token_major=False):
    return dict(name=name, kind=kind, B=B, H=H, Hkv=Hkv, T=T, d=d, ragged=ragged, state=state, token_major=token_major)


def _norm(name, kind, M, D, groups, gate, residual, next, scale, dtype="bf16", res_dtype="bf16"):
    return dict(name=name, kind=kind, M=M, D=D, groups=groups, gate=gate, residual=residual, next=next, scale=scale,
                dtype=dtype, res_dtype=res_dtype)


def listed():
    return [
        # One decoding step of one sequence, 16 heads of 64: the smallest call, where latency counts.
        _linear("step_one", "step", 1, 16, 16, 1, 64),
        # One decoding step of 128 sequences, heads of 128, four query heads to a key head.
        _linear("step_batch", "step", 128, 16, 4, 1, 128),
        # Short prompts of a ragged batch, stored token-major as a projection leaves them.
        _linear("prompt_short", "prompt", 8, 16, 16, 333, 64, ragged=True, token_major=True),
        # The prompt of one sequence of 65536 tokens, 16 heads of 64, from an empty state.
        _linear("prompt_long", "prompt", 1, 16, 16, 65536, 64, state=False),
        # Pieces of longer prompts, continued from the states of the pieces before; grouped heads of 128.
        _linear("prompt_piece", "prompt", 5, 16, 4, 8191, 128, ragged=True),
        # A training step on sequences of 4096 tokens.
        _linear("grad_train", "grad", 4, 16, 16, 4096, 64, state=False),
        # A long sequence in training, cut into pieces whose states carry gradients; grouped heads of 128.
        _linear("grad_piece", "grad", 1, 16, 4, 16383, 128),
        # Between two blocks of a decoding step of eight sequences: the residual and the next block's norm.
        _norm("norm_step", "norm", 8, 1024, 0, False, True, True, 1.0),
        # The heads' outputs of 65536 tokens, 16 heads of 64, normalised a head and gated.
        _norm("norm_heads", "norm", 65536, 1024, 16, True, False, False, 1.0),
        # Between two blocks of a wide model: the block's output normalised, scaled, added to an fp32 residual.
        _norm("norm_wide", "norm", 16384, 8192, 1, False, True, True, 0.25, res_dtype="fp32"),
        # The gradients of the gated heads of a training step.
        _norm("norm_grad_heads", "norm_grad", 16384, 1024, 16, True, False, False, 1.0),
        # The gradients between two blocks, odd sizes, everything in fp32.
        _norm("norm_grad_odd", "norm_grad", 8191, 2500, 1, True, True, True, 0.5, dtype="fp32", res_dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "step", "grad", "norm", "norm_grad"])
    if kind in ("norm", "norm_grad"):
        D = rng.choice([64, 1000, 1024, 2048, 4096, 5120, 8192, _log(rng, 1, 8192)])
        groups = rng.choice([0, 1, 1] + ([D // 64] if D % 64 == 0 else []))
        residual = rng.random() < 0.6
        res = rng.choice(["bf16", "fp32"])
        c = _norm("", kind, _log(rng, 1, min(131072, 16384 * 4096 // D)), D, groups, rng.random() < 0.5, residual,
                  rng.random() < 0.5, rng.choice([1.0, 0.5, 0.1]), "fp32" if residual and res == "fp32" and rng.random() < 0.3
                  else "bf16", res if residual else "bf16")
    else:
        d, Hkv, G = rng.choice([64, 64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 1, 2, 4])
        B = _log(rng, 1, 128 if kind == "step" else 16)
        most = 65536 * 16 * 64 // (B * G * Hkv * d) // (4 if kind == "grad" else 1)
        T = 1 if kind == "step" else _log(rng, 2, max(2, min(65536, most)))
        c = _linear("", kind, B, G * Hkv, Hkv, T, d, kind != "step" and rng.random() < 0.5, rng.random() < 0.7,
                    rng.random() < 0.5)
    c.pop("name")
    return c


def _lengths(case):
    """Tokens of each sequence: from the case alone, so that the work is known."""
    r = random.Random(case["T"] * 7919 + case["B"])
    return [case["T"] if b == 0 or not case["ragged"] else r.randint(case["T"] // 2, case["T"]) for b in range(case["B"])]


def work(case):
    if case["kind"] in ("norm", "norm_grad"):
        n, x, r = case["M"] * case["D"], 2 if case["dtype"] == "bf16" else 4, 2 if case["res_dtype"] == "bf16" else 4
        back = case["kind"] == "norm_grad"
        parts = x * (1 + case["gate"] + case["next"]) + r * (1 + case["residual"])   # x, gate, y or dy; z or dz, residual
        if back:  # dx, dgate; the residual's gradient; without a next norm the residual's values are not needed
            parts += x * (1 + case["gate"]) + r * case["residual"] - r * (case["residual"] and not case["next"])
        return {"bytes": n * parts, "flops": n * (20 if back else 10)}
    B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    n = sum(_lengths(case))
    states = 4 * B * H * d * d
    if case["kind"] == "grad":
        return {"bytes": 2 * n * d * (3 * H + 4 * Hkv) + states * (3 if case["state"] else 0), "flops": 10 * n * H * d * d}
    return {"bytes": 2 * n * d * 2 * (H + Hkv) + states * (2 if case["state"] else 1), "flops": 4 * n * H * d * d}


# --- inputs -------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 11 + 5)
    s = dict(case)

    def normal(shape, dtype=torch.float32, spread=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * spread).to(dtype)

    if case["kind"] in ("norm", "norm_grad"):
        M, D = case["M"], case["D"]
        dt, rdt = DTYPE[case["dtype"]], DTYPE[case["res_dtype"]]
        # rows of different sizes, as blocks put them out
        s["x"] = (normal((M, D)) * torch.exp(0.5 * normal((M, 1)))).to(dt)
        s["gate_in"] = normal((M, D), dt) if case["gate"] else None
        s["res_in"] = normal((M, D), rdt, 2.0) if case["residual"] else None
        s["gain"] = 1 + 0.2 * normal((D,))
        s["next_gain"] = 1 + 0.2 * normal((D,)) if case["next"] else None
        if case["kind"] == "norm_grad":
            s["dz"] = normal((M, D), rdt)
            s["dy"] = normal((M, D), dt) if case["next"] else None
        if own:
            from long_context_lm_gb300 import fs
            s["ws"] = fs.fs_block_norm_workspace(M, D, "cuda") if case["kind"] == "norm_grad" else None
        return s
    B, H, Hkv, T, d = (case[n] for n in ("B", "H", "Hkv", "T", "d"))

    def rows(heads):
        if case["token_major"]:
            return normal((B, T, heads, d), torch.bfloat16).transpose(1, 2)
        return normal((B, heads, T, d), torch.bfloat16)

    s["q"], s["k"], s["v"] = rows(H), rows(Hkv), rows(Hkv)
    # memories of about two tokens to several thousand, one to a head
    reach = 1 + 12 * torch.rand((H,), generator=g, device="cuda")
    s["decay"] = -torch.exp2(-reach)
    lengths = _lengths(case)
    s["count"] = torch.tensor(lengths, dtype=torch.int32, device="cuda") if case["ragged"] else None
    s["S0"] = normal((B, H, d, d), spread=4.0) if case["state"] else None
    if case["kind"] == "grad":
        s["dout"] = rows(H)
        s["G"] = normal((B, H, d, d), spread=0.5) if case["state"] else None
        s["dS0"] = torch.zeros((B, H, d, d), device="cuda") if case["state"] else None
        s["grads"] = tuple(torch.zeros_like(x) for x in (s["q"], s["k"], s["v"]))
    else:
        s["out"] = torch.zeros_like(s["q"])
        s["S1"] = torch.zeros((B, H, d, d), device="cuda")
    if own:
        from long_context_lm_gb300 import fs
        s["ws"] = fs.fs_linear_workspace(B, H, Hkv, T, d, "cuda", backward=case["kind"] == "grad")
    return s


# --- the plain form -----------------------------------------------------------------------------------------------

def _power(decay, n):
    """exp(decay)^n in 32 bits, from 64."""
    return torch.exp(decay.double() * n).float()


def _chunks(s, q, k, v, S, late, scale):
    """Linear attention in chunks of 64 tokens.  ``late`` 1: the state S goes into token 0 without a decay.
    k and v are zero past each sequence's tokens.  Returns the outputs and the last state."""
    B, H, T, d = q.shape
    L = 64
    n = -(-T // L)
    g = s["decay"]
    count = torch.full((B,), T, device="cuda") if s["count"] is None else s["count"].long()
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, n * L - T)).reshape(B, x.shape[1], n, L, d) for x in (q, k, v))
    k, v = (x.repeat_interleave(H // x.shape[1], 1) for x in (k, v))
    i = torch.arange(L, device="cuda")
    seen = _power(g[:, None, None], (i[:, None] - i).clamp(min=0)) * (i[:, None] >= i)
    out = ((q @ k.transpose(-1, -2)) * seen[None, :, None]) @ v
    size = (count[:, None] - torch.arange(n, device="cuda") * L).clamp(0, L)                 # tokens of each chunk
    left = (size[:, None, :, None] - 1 + late - i).clamp(min=0)
    U = (k * _power(g[None, :, None, None], left)[..., None]).transpose(-1, -2) @ v
    keep = torch.exp(g.double()[None, :, None] * size[:, None])
    S = torch.zeros((B, H, d, d), dtype=torch.float64, device="cuda") if S is None else S.double()
    before = torch.empty((B, H, n, d, d), device="cuda")
    for c in range(n):
        before[:, :, c] = S
        S = S * keep[:, :, c, None, None] + U[:, :, c]
    out = out + (q @ before) * _power(g[:, None], i + 1 - late)[None, :, None, :, None]
    return (out * scale).reshape(B, H, n * L, d)[:, :, :T], S


def _masked(s, x):
    x = x.float()
    if s["count"] is None:
        return x
    t = torch.arange(s["T"], device="cuda")
    return torch.where((t < s["count"][:, None])[:, None, :, None], x, 0)


def _backwards(s, x):
    """Tokens in reverse within each sequence."""
    if s["count"] is None:
        return x.flip(2)
    t = torch.arange(s["T"], device="cuda")
    at = s["count"].long()[:, None] - 1 - t
    return x.gather(2, torch.where(at < 0, t, at)[:, None, :, None].expand(x.shape))


def _plain_linear(s):
    scale = s["d"] ** -0.5
    q, k, v = (_masked(s, s[n]) for n in ("q", "k", "v"))
    if s["kind"] != "grad":
        out, S = _chunks(s, q, k, v, s["S0"], 0, scale)
        return _masked(s, out).to(torch.bfloat16), S.float()
    G = s["H"] // s["Hkv"]
    k, v = (x.repeat_interleave(G, 1) for x in (k, v))
    dout = _masked(s, s["dout"])
    S0, G1 = s["S0"], s["G"]
    dq, _ = _chunks(s, dout, v, k, None if S0 is None else S0.transpose(-1, -2), 0, scale)
    q, k, v, dout = (_backwards(s, x) for x in (q, k, v, dout))
    G1 = None if G1 is None else G1 / scale
    dk, _ = _chunks(s, v, dout, q, None if G1 is None else G1.transpose(-1, -2), 1, scale)
    dv, R = _chunks(s, k, q, dout, G1, 1, scale)
    dk, dv = (_backwards(s, x).unflatten(1, (-1, G)).sum(2) for x in (dk, dv))
    grads = [_masked(s, x).to(torch.bfloat16) for x in (dq, dk, dv)]
    return (*grads, (R * scale).float()) if S0 is not None else tuple(grads)


def _forward(s):
    """x and gate in 32 bits, the factors of x's groups, x normalised, the sigmoid of the gate, a and z."""
    x = s["x"].float()
    M, D = x.shape
    inv, h = None, x
    if s["groups"]:
        xg = x.reshape(M, s["groups"], -1)
        inv = torch.rsqrt((xg * xg).mean(-1, keepdim=True) + EPS)
        h = (xg * inv).reshape(M, D)
    a, gate, sig = h * s["gain"], None, None
    if s["gate"]:
        gate = s["gate_in"].float()
        sig = 1 / (1 + torch.exp(-gate))
        a = a * (gate * sig)
    z = s["scale"] * a
    if s["residual"]:
        z = z + s["res_in"].float()
    return gate, inv, h, sig, z


def _plain_norm(s):
    gate, inv, h, sig, z = _forward(s)
    dt, rdt = DTYPE[s["dtype"]], DTYPE[s["res_dtype"]]
    r = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) if s["next"] else None
    if s["kind"] == "norm":
        return (z.to(rdt), (z * r * s["next_gain"]).to(dt)) if s["next"] else (z.to(rdt),)
    dz, outs = s["dz"].float(), {}
    if s["next"]:
        dy, zn = s["dy"].float(), z * r
        outs["next_gain"] = (dy * zn).sum(0, dtype=torch.float64).float()
        w = dy * s["next_gain"]
        dz = dz + r * (w - zn * (w * zn).mean(-1, keepdim=True))
    if s["residual"]:
        outs["residual"] = dz.to(rdt)
    da = s["scale"] * dz
    if s["gate"]:
        outs["gate"] = (da * h * s["gain"] * sig * (1 + gate * (1 - sig))).to(dt)
        da = da * gate * sig
    outs["gain"] = (da * h).sum(0, dtype=torch.float64).float()
    dh = da * s["gain"]
    if s["groups"]:
        hg, dg = (t.reshape(t.shape[0], s["groups"], -1) for t in (h, dh))
        dh = (inv * (dg - hg * (dg * hg).mean(-1, keepdim=True))).reshape(h.shape)
    outs["x"] = dh.to(dt)
    return outs


def run(s):
    linear = s["kind"] in ("prompt", "step", "grad")
    if not own:
        return _plain_linear(s) if linear else _plain_norm(s)
    from long_context_lm_gb300 import fs
    if s["kind"] == "grad":
        dq, dk, dv = s["grads"]
        fs.fs_linear_attn_bwd(s["q"], s["k"], s["v"], s["decay"], s["dout"], state=s["S0"], dstate_out=s["G"],
                              count=s["count"], dq=dq, dk=dk, dv=dv, dstate=s["dS0"], ws=s["ws"])
        return (dq, dk, dv, s["dS0"]) if s["state"] else (dq, dk, dv)
    if linear:
        out = fs.fs_linear_attn(s["q"], s["k"], s["v"], s["decay"], state=s["S0"], state_out=s["S1"], count=s["count"],
                                out=s["out"], ws=s["ws"])
        return out, s["S1"]
    form = dict(gate=s["gate_in"], residual=s["res_in"], groups=s["groups"], gain=s["gain"], scale=s["scale"], eps=EPS)
    if s["kind"] == "norm":
        z, y = fs.fs_block_norm(s["x"], next_norm=s["next"], next_gain=s["next_gain"], **form)
        return (z, y) if s["next"] else (z,)
    grads = fs.fs_block_norm_bwd(s["x"], dz=s["dz"], dy=s["dy"], next_gain=s["next_gain"], ws=s["ws"], **form)
    return {n: grads[n] for n in ("next_gain", "residual", "gate", "gain", "x") if grads[n] is not None}


# --- the definition in 64 bits ------------------------------------------------------------------------------------

def _blocks(n, size=256):
    return [(a, min(n, a + size)) for a in range(0, n, size)]


def _exact_linear(case, s):
    B, H, Hkv, T, d = (case[n] for n in ("B", "H", "Hkv", "T", "d"))
    G, scale = H // Hkv, 1 / math.sqrt(d)
    g = s["decay"].double()[:, None]
    grad = case["kind"] == "grad"
    zeros = lambda heads: torch.zeros((B, heads, T, d), dtype=torch.float64, device="cuda")  # noqa: E731
    outs = [zeros(H), zeros(Hkv), zeros(Hkv)] if grad else [zeros(H)]
    last = torch.zeros((B, H, d, d), dtype=torch.float64, device="cuda")

    def weights(m):
        t = torch.arange(m, dtype=torch.float64, device="cuda")
        lag = t[:, None] - t
        return torch.where(lag >= 0, torch.exp(g[..., None] * lag.clamp(min=0)), 0.0), t

    for b, n in enumerate(_lengths(case)):
        q = s["q"][b].double()
        k, v = (s[x][b].double()[torch.arange(H, device="cuda") // G] for x in ("k", "v"))
        S = last[b].clone() if s["S0"] is None else s["S0"][b].double()
        do = s["dout"][b].double() if grad else None
        for lo, hi in _blocks(n):
            W, t = weights(hi - lo)
            qb, kb, vb = q[:, lo:hi], k[:, lo:hi], v[:, lo:hi]
            first = torch.exp(g * (t + 1))[..., None]
            if grad:
                A = torch.einsum("hte,hse->hts", do[:, lo:hi], vb) * W
                outs[0][b, :, lo:hi] = scale * (torch.einsum("hts,hsc->htc", A, kb)
                                                + torch.einsum("hce,hte->htc", S, do[:, lo:hi]) * first)
            else:
                A = torch.einsum("htc,hsc->hts", qb, kb) * W
                outs[0][b, :, lo:hi] = scale * (torch.einsum("hts,hse->hte", A, vb)
                                                + torch.einsum("htc,hce->hte", qb, S) * first)
            end = torch.exp(g * (hi - lo - 1 - t))[..., None]
            S = torch.exp(g * (hi - lo))[..., None] * S + torch.einsum("hsc,hse->hce", kb * end, vb)
        last[b] = S
        if grad:
            R = torch.zeros_like(S) if s["G"] is None else s["G"][b].double()        # lam R of the block after
            dk, dv = torch.zeros_like(k), torch.zeros_like(v)
            for lo, hi in reversed(_blocks(n)):
                W, t = weights(hi - lo)
                qb, kb, vb, db = q[:, lo:hi], k[:, lo:hi], v[:, lo:hi], do[:, lo:hi]
                left = torch.exp(g * (hi - lo - 1 - t))[..., None]
                dk[:, lo:hi] = scale * torch.einsum("hts,htc->hsc", W * torch.einsum("hte,hse->hts", db, vb), qb)
                dk[:, lo:hi] += left * torch.einsum("hce,hse->hsc", R, vb)
                dv[:, lo:hi] = scale * torch.einsum("hts,hte->hse", W * torch.einsum("htc,hsc->hts", qb, kb), db)
                dv[:, lo:hi] += left * torch.einsum("hce,hsc->hse", R, kb)
                R = torch.exp(g * (hi - lo))[..., None] * R \
                    + scale * torch.einsum("htc,hte->hce", qb * torch.exp(g * (t + 1))[..., None], db)
            last[b] = R
            outs[1][b], outs[2][b] = (x.reshape(Hkv, G, T, d).sum(1) for x in (dk, dv))
            for x in outs[1:]:
                x[b, :, n:] = 0
    return (*outs, last) if not grad or case["state"] else tuple(outs)


def _exact_norm(case, s):
    """The gradients by the chain rule over the whole graph of the definition."""
    grad = case["kind"] == "norm_grad"
    leaves = {"x": s["x"], "gate": s["gate_in"], "residual": s["res_in"], "gain": s["gain"], "next_gain": s["next_gain"]}
    leaves = {n: t.double().requires_grad_(grad) for n, t in leaves.items() if t is not None}
    a = leaves["x"]
    M, D = a.shape
    if case["groups"]:
        a = a.view(M, case["groups"], D // case["groups"])
        a = (a / (a.square().sum(2, keepdim=True) * (case["groups"] / D) + EPS).sqrt()).view(M, D)
    a = a * leaves["gain"]
    if case["gate"]:
        a = a * leaves["gate"] * torch.sigmoid(leaves["gate"])
    z = a * case["scale"] + leaves.get("residual", 0.0)
    y = z / (z.square().sum(1, keepdim=True) / D + EPS).sqrt() * leaves["next_gain"] if case["next"] else None
    if not grad:
        return (z, y) if case["next"] else (z,)
    total = (z * s["dz"].double()).sum()
    if case["next"]:
        total = total + (y * s["dy"].double()).sum()
    names = [n for n in ("next_gain", "residual", "gate", "gain", "x") if n in leaves]
    return dict(zip(names, torch.autograd.grad(total, [leaves[n] for n in names])))


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("norm", "norm_grad"):
        return _exact_norm(case, s)
    return _exact_linear(case, s)
