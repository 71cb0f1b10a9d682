"""fs_linear_attn and fs_linear_attn_bwd against a statement in 64 bits, token after token (GPU
only).

Tolerances.  M is the same sum with every factor's magnitude (the statement on |q|, |k|, |v|, |S|).
 * bf16 results: half a step, 2^-8 of the value, and what the sums lose: factors of products are bf16
   numbers or sums of bf16 parts good to 2^-16 of themselves, two such factors to a term
   (a score and none, or a state and none: 2^-16 each, the weights' own 2^-21 below that); fp32 sums of
   at most 128 + d terms in steps of 16, each step off by 2^-23 of the sum: (24 + 8) 2^-23 < 2^-18.
   Together below 2^-15 M.
 * states: three parts, 24 bits; a chunk's sum is 8 steps of three products, each 2^-23, the
   weights 2^-21 at most (an exponential and its argument), every chunk's update two roundings of
   2^-24, and the recurrent form two a token for up to 16 tokens:
   (24 + 4 + 32 + T / 64) 2^-23 M, taken as (64 + T / 16) 2^-23 M."""
import pytest
import torch

from long_context_lm_gb300 import fs
import layer_ref as ref

pytestmark = pytest.mark.gpu
DECAYS = [0.0, -1e-4, -0.01, -0.3, -2.0, -30.0, -200.0, float("-inf")]


def inputs(B, H, Hkv, T, d, seed=0, state=True, ragged=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = {n: torch.randn((B, h, T, d), generator=g, device="cuda").bfloat16()
         for n, h in (("q", H), ("k", Hkv), ("v", Hkv), ("dout", H))}
    decay = torch.tensor([DECAYS[(i * 3 + 2) % len(DECAYS)] for i in range(H)], device="cuda")
    S0, G = (torch.randn((B, H, d, d), generator=g, device="cuda") if state else None for _ in range(2))
    count = None
    if ragged:
        count = torch.randint(0, T + 1, (B,), generator=g, device="cuda").int()
        count[0] = T
        if B > 1:
            count[-1] = 0
        for t in x.values():   # what lies behind a sequence is nobody's
            for b in range(B):
                t[b, :, int(count[b]):] = float("nan")
    return x["q"], x["k"], x["v"], x["dout"], decay, S0, G, count


def clean(x, count):
    if count is None:
        return x
    t = torch.arange(x.shape[2], device=x.device)
    return torch.where((t < count[:, None])[:, None, :, None], x, 0)


def mag(x):
    return None if x is None else x.abs()


def near(got, want, tol):
    assert got.isfinite().all()
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), ((got.double() - want).abs() / tol.clamp(min=1e-300)).max().item())


def state_tol(M, T):
    return (64 + T / 16) * 2.0 ** -23 * M + 1e-30


def check_forward(q, k, v, decay, S0, count, **kw):
    S1 = torch.full((*q.shape[:2], q.shape[3], q.shape[3]), 7.0, device="cuda")
    out = torch.full_like(q, 3.0)
    got = fs.fs_linear_attn(q, k, v, decay, state=S0, state_out=S1, count=count, out=out, **kw)
    assert got is out
    a = [clean(t, count) for t in (q, k, v)]
    want, S = ref.linear(*a, decay, S0, count, kw.get("scale"))
    scale = abs(kw.get("scale") or q.shape[3] ** -0.5)
    M, MS = ref.linear(*(t.abs() for t in a), decay, mag(S0), count, scale)
    t = torch.arange(q.shape[2], device="cuda")
    have = torch.ones_like(want, dtype=torch.bool) if count is None else \
        (t < count[:, None])[:, None, :, None].expand(want.shape)
    assert (out[~have] == 3.0).all()
    near(torch.where(have, out, 0), want, 2.0 ** -8 * want.abs() + 2.0 ** -15 * M + 1e-30)
    near(S1, S, state_tol(MS, q.shape[2]))
    return out, S1


SHAPES = [(1, 1, 1, 1, 64), (2, 3, 1, 1, 128), (1, 2, 2, 2, 64), (3, 4, 2, 16, 64), (2, 2, 2, 17, 64),
          (1, 8, 8, 31, 128), (2, 8, 4, 63, 64), (2, 2, 1, 64, 128), (3, 2, 2, 65, 64), (2, 8, 2, 127, 128),
          (1, 8, 8, 128, 64), (4, 2, 2, 129, 64), (2, 4, 4, 129, 128), (3, 4, 1, 255, 64), (2, 8, 8, 300, 128),
          (5, 3, 3, 511, 64), (1, 2, 2, 1000, 64), (1, 2, 1, 1025, 128), (3, 2, 2, 1153, 64), (70, 2, 1, 1100, 64),
          (2, 3, 3, 2305, 128)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("state,ragged", [(True, False), (False, True), (True, True)])
def test_forward(shape, state, ragged):
    q, k, v, _, decay, S0, _, count = inputs(*shape, seed=shape[3], state=state, ragged=ragged)
    check_forward(q, k, v, decay, S0, count)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("state,ragged", [(True, False), (False, True), (True, True)])
def test_backward(shape, state, ragged):
    q, k, v, dout, decay, S0, G, count = inputs(*shape, seed=shape[3] + 1, state=state, ragged=ragged)
    grads = [torch.full_like(t, 3.0) for t in (q, k, v)]
    dS = torch.full((*q.shape[:2], q.shape[3], q.shape[3]), 7.0, device="cuda")
    got = fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G, count=count, dq=grads[0],
                                dk=grads[1], dv=grads[2], dstate=dS)
    a = [clean(t, count) for t in (q, k, v)]
    do = clean(dout, count)
    want = ref.linear_grads(*a, decay, do, S0, G, count)
    M = ref.linear_grads(*(t.abs() for t in a), decay, do.abs(), mag(S0), mag(G), count)
    T = q.shape[2]
    for x, w, m in zip(got, want, M):
        have = torch.ones_like(w, dtype=torch.bool) if count is None else \
            (torch.arange(T, device="cuda") < count[:, None])[:, None, :, None].expand(w.shape)
        assert (x[~have] == 3.0).all()
        near(torch.where(have, x, 0), w, 2.0 ** -8 * w.abs() + 2.0 ** -15 * m + 1e-30)
    near(dS, want[3], state_tol(M[3], T))


@pytest.mark.parametrize("B,H,Hkv,T,d", [(1, 2, 1, 5, 64), (2, 2, 2, 200, 64), (1, 4, 2, 333, 128)])
def test_gradients_are_the_forwards_differences(B, H, Hkv, T, d):
    # The outputs are linear in q, in v, in k and in the state (in the last two with the state, or k
    # and v, held at zero), so a difference along any direction x is the forward at x itself:
    #   <dq, x> = <dout, out(q = x)>,  <dv, x> = <dout, out> + <G, S> at v = x without a state, ...
    # Both sides round bf16 results (half a step, 2^-8, of each), so they agree to
    # 2^-8 (<|dq|, |x|> + <|dout|, |out|>) and 2^-15 of the magnitudes; errors of that many
    # numbers never line up, so an eighth of the bound is asked for.
    q, k, v, dout, decay, S0, G, _ = inputs(B, H, Hkv, T, d, seed=T)
    dS = torch.empty_like(S0)
    dq, dk, dv = fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G, dstate=dS)
    S1 = torch.empty_like(S0)
    dot = lambda a, b: ((a.double() * b.double()).sum().item(), (a.double() * b.double()).abs().sum().item())  # noqa: E731
    x = torch.randn((B, H, T, d), device="cuda").bfloat16()
    y = torch.randn((B, Hkv, T, d), device="cuda").bfloat16()
    Y = torch.randn_like(S0)
    zero = torch.zeros_like(k)
    for got, (args, state, states) in (
            (dot(dq, x), ((x, k, v), S0, False)), (dot(dk, y), ((q, y, v), None, True)),
            (dot(dv, y), ((q, k, y), None, True)), (dot(dS, Y), ((q, zero, v), Y, True))):
        out = fs.fs_linear_attn(*args, decay, state=state, state_out=S1)
        a, sa = dot(dout, out)
        b, sb = dot(G, S1) if states else (0.0, 0.0)
        assert abs(got[0] - a - b) <= 2.0 ** -11 * (got[1] + sa + sb), (got, a, b)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 7, 200])
def test_strides(d, T):
    # token-major rows, parts of one projection's output, and outputs that lie likewise
    B, H, Hkv = 2, 4, 2
    fused = torch.randn((B, T, H + 2 * Hkv, d), device="cuda").bfloat16()
    q, k, v = (t.transpose(1, 2) for t in fused.split([H, Hkv, Hkv], 2))
    decay = torch.tensor([-0.1, 0.0, -1.0, -0.01], device="cuda")
    out = torch.full((B, T, H + 3, d), 5.0, device="cuda", dtype=torch.bfloat16)
    S0, S1, S2 = (torch.randn((B, H, d, d), device="cuda") for _ in range(3))
    got = fs.fs_linear_attn(q, k, v, decay, state=S0, state_out=S1, out=out[:, :, 1:H + 1].transpose(1, 2))
    want = fs.fs_linear_attn(*(t.contiguous() for t in (q, k, v)), decay, state=S0, state_out=S2)
    assert torch.equal(got, want) and torch.equal(S1, S2)
    assert (out[:, :, 0] == 5).all() and (out[:, :, H + 1:] == 5).all()
    dout = torch.randn((B, T, H, d), device="cuda").bfloat16().transpose(1, 2)
    grads = torch.empty_like(fused)
    dq, dk, dv = (t.transpose(1, 2) for t in grads.split([H, Hkv, Hkv], 2))
    fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dq=dq, dk=dk, dv=dv)
    want = fs.fs_linear_attn_bwd(*(t.contiguous() for t in (q, k, v)), decay, dout.contiguous(), state=S0)
    for a, b in zip((dq, dk, dv), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [3, 150])
def test_inputs_repeated_by_strides_of_zero(T):
    # one sequence's keys and one head's values for all
    B, H, d = 3, 2, 64
    q = torch.randn((B, H, T, d), device="cuda").bfloat16()
    k = torch.randn((1, H, T, d), device="cuda").bfloat16().expand(B, H, T, d)
    v = torch.randn((B, 1, T, d), device="cuda").bfloat16().expand(B, H, T, d)
    decay = torch.tensor([-0.5, -0.02], device="cuda")
    assert torch.equal(fs.fs_linear_attn(q, k, v, decay), fs.fs_linear_attn(q, k.contiguous(), v.contiguous(), decay))
    a, b = (fs.fs_linear_attn_bwd(q, kk, vv, decay, q) for kk, vv in ((k, v), (k.contiguous(), v.contiguous())))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pieces", [[1] * 5, [130, 1, 1, 16, 17, 128], [129, 300, 2]])
def test_a_sequence_in_pieces(d, pieces):
    # prompts and single tokens on from the state of the piece before, in place
    B, H, T = 2, 3, sum(pieces)
    q, k, v, _, decay, S0, _, _ = inputs(B, H, H, T, d, seed=T)
    want, S = ref.linear(q, k, v, decay, S0)
    M, MS = ref.linear(q.abs(), k.abs(), v.abs(), decay, S0.abs())
    state, at, outs = S0.clone(), 0, []
    for n in pieces:
        cut = slice(at, at + n)
        outs.append(fs.fs_linear_attn(q[:, :, cut], k[:, :, cut], v[:, :, cut], decay, state=state, state_out=state))
        at += n
    near(torch.cat(outs, 2), want, 2.0 ** -8 * want.abs() + 2.0 ** -15 * M)
    near(state, S, len(pieces) * state_tol(MS, T))


def test_scale_of_either_sign():
    q, k, v, dout, decay, S0, G, _ = inputs(2, 4, 2, 150, 64, seed=9)
    check_forward(q, k, v, decay, S0, None, scale=-3.0)
    a = fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G, scale=-3.0)
    want = ref.linear_grads(q, k, v, decay, dout, S0, G, scale=-3.0)
    M = ref.linear_grads(q.abs(), k.abs(), v.abs(), decay, dout.abs(), S0.abs(), G.abs(), scale=3.0)
    for x, w, m in zip(a, want, M):
        near(x, w, 2.0 ** -8 * w.abs() + 2.0 ** -15 * m)


@pytest.mark.parametrize("d,T", [(64, 9), (64, 200), (128, 200), (64, 700)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_reach_later_tokens_only(d, T, value):
    q, k, v, _, decay, S0, _, _ = inputs(1, 3, 3, T, d, seed=4)
    decay[:] = -0.05
    want, S = fs.fs_linear_attn(q, k, v, decay, state=S0, state_out=(S1 := torch.empty_like(S0))), S1
    for at, col in ((T // 2, 5), (T - 1, d - 1), (0, 0)):
        w = v.clone()
        w[0, 1, at, col] = value
        out = fs.fs_linear_attn(q, k, w, decay, state=S0, state_out=(S2 := torch.empty_like(S0)))
        assert not out[0, 1, at:, col].isfinite().any() and not S2[0, 1, :, col].isfinite().any()
        out, S2 = out.clone(), S2.clone()
        out[0, 1, at:, col], S2[0, 1, :, col] = want[0, 1, at:, col], S[0, 1, :, col]
        assert torch.equal(out, want) and torch.equal(S2, S)


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("T", [9, 200])
def test_other_inputs_that_are_not_finite(which, T):
    q, k, v, _, decay, S0, _, _ = inputs(1, 2, 2, T, 64, seed=4)
    decay[:] = -0.05
    want = fs.fs_linear_attn(q, k, v, decay, state=S0)
    at = T // 2
    {"q": q, "k": k}[which][0, 0, at, 3] = float("nan")
    out = fs.fs_linear_attn(q, k, v, decay, state=S0)
    rows = slice(at, at + 1) if which == "q" else slice(at, T)
    assert out[0, 0, rows].isnan().all()
    out[0, 0, rows] = want[0, 0, rows]
    assert torch.equal(out, want)


def test_empty_sequences_keep_their_states():
    q, k, v, dout, decay, S0, G, _ = inputs(3, 2, 2, 140, 64)
    count = torch.zeros(3, dtype=torch.int32, device="cuda")
    S1, dS = torch.empty_like(S0), torch.empty_like(S0)
    out = torch.full_like(q, 2.0)
    fs.fs_linear_attn(q, k, v, decay, state=S0, state_out=S1, count=count, out=out)
    assert torch.equal(S1, S0) and (out == 2.0).all()
    grads = [torch.full_like(q, 2.0) for _ in range(3)]
    fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G, count=count, dstate=dS,
                          dq=grads[0], dk=grads[1], dv=grads[2], scale=0.25)
    assert torch.equal(dS, G) and all((g == 2.0).all() for g in grads)


def test_counts_outside_are_held_to_the_rows():
    q, k, v, _, decay, S0, _, _ = inputs(3, 2, 2, 140, 64)
    count = torch.tensor([-5, 2 ** 31 - 1, 140], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 140, 140], dtype=torch.int32, device="cuda")
    assert torch.equal(fs.fs_linear_attn(q, k, v, decay, count=count), fs.fs_linear_attn(q, k, v, decay, count=good))


@pytest.mark.parametrize("T", [1, 400])
def test_the_same_bits_every_time_and_in_graphs_and_on_other_streams(T):
    q, k, v, dout, decay, S0, G, _ = inputs(2, 4, 2, T, 64, seed=2)

    def both():
        S1, dS = torch.empty_like(S0), torch.empty_like(S0)
        out = fs.fs_linear_attn(q, k, v, decay, state=S0, state_out=S1)
        return (out, S1, *fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G, dstate=dS), dS)

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taken = both()
    for _ in range(2):
        for t in taken:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, taken))
    assert all(torch.equal(a, b) for a, b in zip(want, other))


def test_a_stream_argument_and_two_calls_at_once():
    q, k, v, _, decay, _, _, _ = inputs(2, 4, 4, 2000, 64, seed=2)
    want = fs.fs_linear_attn(q, k, v, decay)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[fs.fs_linear_attn(q, k, v, decay, stream=s) for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for pair in outs for o in pair)


@pytest.mark.parametrize("B,H,T,d", [(1, 2, 20000, 64), (1, 1, 12345, 128), (300, 2, 130, 64), (4, 32, 12000, 64)])
def test_long_sequences_and_large_batches(B, H, T, d):
    # against the same call in pieces of 1111 tokens, each of which the small tests cover: states
    # agree as pieces do with the statement, outputs to two roundings and both calls' sums
    q, k, v, _, _, S0, _, _ = inputs(B, H, H, T, d, seed=3)
    decay = -torch.exp2(-torch.arange(3, 3 + 5 * H, 5, device="cuda").float())
    S1, state = torch.empty_like(S0), S0.clone()
    out = fs.fs_linear_attn(q, k, v, decay, state=S0, state_out=S1)
    M, MS = (fs.fs_linear_attn(q.abs(), k.abs(), v.abs(), decay, state=S0.abs(), state_out=(t := torch.empty_like(S0))), t)
    for a in range(0, T, 1111):
        cut = slice(a, min(T, a + 1111))
        got = fs.fs_linear_attn(q[:, :, cut], k[:, :, cut], v[:, :, cut], decay, state=state, state_out=state)
        near(out[:, :, cut], got.double(), 2.0 ** -7 * got.double().abs() + 2.0 ** -14 * M[:, :, cut].double())
    near(S1, state.double(), 2 * state_tol(MS.double(), T))


@pytest.mark.parametrize("B,H,Hkv,T,d", [(2, 2, 1, 200, 64), (1, 2, 2, 2000, 64), (2, 4, 2, 2000, 128)])
def test_an_error_word_that_is_set_ends_the_waits(B, H, Hkv, T, d):
    """A call whose workspace holds an error gives its waits up early, wherever each one is, and ends;
    the status is reported; with the word cleared the next call is whole again."""
    q, k, v, dout, decay, S0, G, _ = inputs(B, H, Hkv, T, d, seed=7)
    ws = fs.fs_linear_workspace(B, H, Hkv, T, d, q.device)
    wb = fs.fs_linear_workspace(B, H, Hkv, T, d, q.device, backward=True)

    def run():
        return (fs.fs_linear_attn(q, k, v, decay, state=S0, ws=ws),
                *fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G, ws=wb))

    want = run()
    fs.fs_check_status(ws), fs.fs_check_status(wb)
    for w in (ws, wb):
        w[:4].view(torch.int32).fill_(fs.FS_ERR_TIMEOUT)
    run()
    for w in (ws, wb):
        with pytest.raises(fs.FSError):
            fs.fs_check_status(w)
        w[:256].zero_()
    for a, b in zip(run(), want):
        assert torch.equal(a, b)
    fs.fs_check_status(ws), fs.fs_check_status(wb)


@pytest.mark.parametrize("B,H,Hkv,T,d", [(2, 4, 2, 1300, 64), (3, 6, 1, 1999, 64), (2, 6, 3, 1300, 128)])
@pytest.mark.parametrize("state,ragged", [(True, False), (False, True), (True, True)])
def test_shared_heads_of_longer_prompts(B, H, Hkv, T, d, state, ragged):
    test_forward((B, H, Hkv, T, d), state, ragged)
    test_backward((B, H, Hkv, T, d), state, ragged)


@pytest.mark.parametrize("B,H,Hkv,T,d,counts", [(3, 33, 11, 7000, 64, (7000, 3000, 0)), (1, 100, 100, 7000, 64, None),
                                                (2, 40, 8, 9000, 64, (9000, 4000)), (1, 80, 80, 9000, 64, None),
                                                (2, 24, 8, 5000, 128, (4999, 1111))])
def test_gradients_of_long_sequences(B, H, Hkv, T, d, counts):
    # against the calls in pieces of 900 tokens, whose states and states' gradients chain them; tolerances
    # as in the forward's test
    q, k, v, dout, _, S0, G, _ = inputs(B, H, Hkv, T, d, seed=4)
    count = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    decay = -torch.exp2(-torch.arange(H, device="cuda").float() % 12 - 3)
    got = fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G, count=count,
                                dstate=(dS := torch.empty_like(S0)))
    M = fs.fs_linear_attn_bwd(*(t.abs() for t in (q, k, v)), decay, dout.abs(), state=S0.abs(), dstate_out=G.abs(),
                              count=count, dstate=(MS := torch.empty_like(S0)))
    cuts = [slice(a, min(T, a + 900)) for a in range(0, T, 900)]
    part = [None if count is None else (count - c.start).clamp(0, c.stop - c.start) for c in cuts]
    states = [S0]
    for c, n in zip(cuts[:-1], part):
        states.append(torch.empty_like(S0))
        fs.fs_linear_attn(q[:, :, c], k[:, :, c], v[:, :, c], decay, state=states[-2], state_out=states[-1], count=n)
    for c, n, S in reversed(list(zip(cuts, part, states))):
        want = fs.fs_linear_attn_bwd(q[:, :, c], k[:, :, c], v[:, :, c], decay, dout[:, :, c], state=S, dstate_out=G,
                                     count=n, dstate=(back := torch.empty_like(S0)))
        G = back
        for x, w, m in zip(got, want, M):
            near(x[:, :, c], w.double(), 2.0 ** -7 * w.double().abs() + 2.0 ** -14 * m[:, :, c].double())
    near(dS, G.double(), 2 * state_tol(MS.double(), T))


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,T,d", [(2, 9, 64), (2, 300, 64), (3, 1400, 64), (2, 1400, 128)])
def test_gradients_where_an_input_is_not_finite(which, value, H, T, d):
    # reach exactly the gradients that the definition's reach: of that token, of earlier and later ones
    a = list(inputs(1, H, H, T, d, seed=T + which)[:4])
    decay = torch.tensor([-0.01, -0.3, 0.0][:H], device="cuda")
    M = ref.linear_grads(*(t.abs() for t in a[:3]), decay, a[3].abs())
    a[which][0, 1, T // 2 + 1, 5] = value
    got = fs.fs_linear_attn_bwd(*a[:3], decay, a[3])
    want = ref.linear_grads(*a[:3], decay, a[3])
    for x, w, m in zip(got, want, M):
        fine = w.isfinite()
        assert torch.equal(x.isfinite(), fine)
        near(torch.where(fine, x, 0), torch.where(fine, w, 0), 2.0 ** -8 * w.abs().nan_to_num(0, 0, 0) + 2.0 ** -15 * m + 1e-30)
