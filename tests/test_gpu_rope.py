"""fs_rope against the 64-bit rotation (GPU only).

Error of one output y = m (a cos - b sin) computed in fp32: the sine and
cosine are within 2^-22 (sincospi's own error below 2^-23, the angle's 2^-30),
the amplitude's and the products' roundings 2^-24 each, so the sum is within
(|a| + |b|) m 2^-21; the result is rounded once, by at most half a step of its
type (bf16 2^-8 relative, fp32 2^-24)."""
import pytest
import torch

from long_context_lm_gb300 import fs
import serving_ref as ref

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _check(x, y, pos, layout, rot, amplitude=1.0, inverse=False, **scaling):
    f = ref.frequencies(rot, **scaling)
    want = ref.rope(x, pos, f, layout, amplitude, inverse)
    size = ref.rope(x.double().abs(), torch.zeros_like(pos), f, layout)  # |x|
    pair = size.clone()
    ia = torch.arange(rot // 2) if layout == "half" else 2 * torch.arange(rot // 2)
    ib = ia + rot // 2 if layout == "half" else ia + 1
    pair[..., ia] = pair[..., ib] = size[..., ia] + size[..., ib]
    bound = HALF[x.dtype] * 1.01 * want.abs() + pair * amplitude * 2.0 ** -21 + 1e-38
    err = (y.double() - want).abs()
    assert torch.all(err <= bound), float((err / bound).max())
    assert torch.equal(y[..., rot:], x[..., rot:])   # the rest passes through


def _positions(B, N, top, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, top, (B, N), generator=g).to(torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,kw", [
    (1, 1, 1, 1, 64, 64, {}),
    (2, 16, 16, 37, 64, 64, {}),
    (3, 5, 1, 130, 128, 96, dict(scaling="linear", factor=8.0)),
    (1, 8, 2, 257, 128, 128, dict(scaling="base", factor=4.0)),
    (2, 3, 3, 65, 64, 32, dict(scaling="ramp", factor=8.0)),
    (1, 2, 1, 33, 80, 20, {}),        # pieces of 16 bytes do not fit: element by element
    (1, 2, 2, 5, 6, 2, {}),
    (1, 1, 1, 3, 256, 256, {}),
    (1, 2, 1, 9000, 64, 64, {}),
])
def test_rope_matches_the_rotation(B, Hq, Hk, N, d, rot, kw, layout, dtype):
    g = torch.Generator(device="cuda").manual_seed(N + d)
    q = torch.randn((B, Hq, N, d), generator=g, device="cuda").to(dtype)
    k = torch.randn((B, Hk, N, d), generator=g, device="cuda").to(dtype)
    pos = _positions(B, N, 1 << 20, seed=N)
    for inverse, amplitude in ((False, 1.0), (True, 1.25)):
        plan = fs.fs_rope_plan(rot, layout=layout, amplitude=amplitude, **kw)
        yq, yk = fs.fs_rope(q, k, pos, plan, inverse=inverse)
        for x, y in ((q, yq), (k, yk)):
            _check(x, y, pos, layout, rot, amplitude, inverse, **kw)


def test_far_and_negative_positions():
    # the angle is exact at any 32-bit position
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -1, 0]], dtype=torch.int32).cuda()
    x = torch.randn((1, 2, 5, 64), device="cuda")
    y, none = fs.fs_rope(x, None, pos, fs.fs_rope_plan(64))
    assert none is None
    # the reference's own angle p f_i is a double: 2^31 * 2^-53 turns are 2^-20 off at most
    f = ref.frequencies(64)
    err = (y.double() - ref.rope(x, pos, f, "half")).abs()
    size = x.double().abs()
    size = (size[..., :32] + size[..., 32:]).repeat(1, 1, 1, 2)
    assert torch.all(err <= size * (2.0 ** -21 + 2.0 ** -19))


def test_shared_consecutive_and_strided_positions():
    x = torch.randn((3, 2, 50, 64), device="cuda").bfloat16()
    plan = fs.fs_rope_plan(64)
    at = torch.arange(7, 57, dtype=torch.int32, device="cuda")
    a, _ = fs.fs_rope(x, None, 7, plan)
    b, _ = fs.fs_rope(x, None, at, plan)
    c, _ = fs.fs_rope(x, None, at.expand(3, 50).contiguous(), plan)
    assert torch.equal(a, b) and torch.equal(a, c)
    with pytest.raises(ValueError):
        fs.fs_rope(x, None, at.expand(3, 50), plan)       # a table that is not contiguous
    with pytest.raises(ValueError):
        fs.fs_rope(x, None, at.long(), plan)


@pytest.mark.parametrize("offset", [0, 1, 8])
def test_strides_slices_and_in_place(offset):
    # q and k as slices of one token-major projection [B, N, 3, H, d + pad]
    B, N, H, d = 2, 19, 4, 64
    g = torch.Generator(device="cuda").manual_seed(offset)
    big = torch.randn((B, N, 3, H, d + 16), generator=g, device="cuda").bfloat16()
    q, k = (big[:, :, i, :, offset:offset + d].transpose(1, 2) for i in (0, 1))
    keep = big.clone()
    pos = _positions(B, N, 5000, seed=1)
    plan = fs.fs_rope_plan(64, layout="pairs")
    yq, yk = fs.fs_rope(q, k, pos, plan)
    assert torch.equal(big, keep)
    _check(q, yq, pos, "pairs", 64)
    _check(k, yk, pos, "pairs", 64)
    fs.fs_rope(q, k, pos, plan, q_out=q, k_out=k)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    rest = big.clone()
    for i, y in ((0, yq), (1, yk)):                       # nothing else in the buffer changed
        rest[:, :, i, :, offset:offset + d] = keep[:, :, i, :, offset:offset + d]
    assert torch.equal(rest, keep)
    with pytest.raises(ValueError):
        fs.fs_rope(big[:, :, 0].transpose(2, 3)[..., :d].transpose(1, 2), None, pos, plan)


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_the_inverse_is_the_gradient(layout):
    # against central differences of the rotation itself, in fp32 with steps that are exact
    x = torch.randint(-8, 8, (1, 1, 6, 16), device="cuda").float()
    g = torch.randn((1, 1, 6, 16), device="cuda")
    plan = fs.fs_rope_plan(12, layout=layout, amplitude=1.5, scaling="linear", factor=2.0)
    pos = _positions(1, 6, 3000, seed=2)
    dx, _ = fs.fs_rope(g, None, pos, plan, inverse=True)
    for e in range(16):
        step = torch.zeros_like(x)
        step[..., e] = 4.0
        up, _ = fs.fs_rope(x + step, None, pos, plan)
        down, _ = fs.fs_rope(x - step, None, pos, plan)
        diff = ((up.double() - down.double()) / 8.0 * g.double()).sum(-1)
        # each side is within (|a| + |b|) m 2^-21 <= 24 * 1.5 * 2^-21 of the rotation, 16 terms
        bound = 16 * g.abs().double().amax() * 2 * 36 * 2.0 ** -21 / 8 + 2.0 ** -19
        assert torch.all((diff - dx[..., e].double()).abs() <= bound)


def test_values_that_are_not_finite_stay_in_their_pair():
    x = torch.ones((1, 1, 2, 64), device="cuda")
    x[0, 0, 0, 3], x[0, 0, 1, 40] = float("nan"), float("inf")
    y, _ = fs.fs_rope(x, None, 5, fs.fs_rope_plan(64))
    bad = ~torch.isfinite(y[0, 0])
    assert bad.nonzero().tolist() == [[0, 3], [0, 35], [1, 8], [1, 40]]


def test_rope_refusals_on_the_gpu():
    x = torch.randn((2, 2, 4, 64), device="cuda")
    plan = fs.fs_rope_plan(64)
    with pytest.raises(fs.FSError):
        fs.fs_rope(x, None, 0, plan, q_out=x[:1].clone().expand(2, 2, 4, 64))
    with pytest.raises(fs.FSError):
        fs.fs_rope(x, None, 2 ** 31 - 3, plan)
    with pytest.raises(ValueError):
        fs.fs_rope(x, None, 2 ** 31, plan)
    with pytest.raises(ValueError):
        fs.fs_rope(x, x[:, :, :2], 0, plan)
    y, _ = fs.fs_rope(x[:1].expand(2, 2, 4, 64), None, 0, plan)      # an input may repeat
    z, _ = fs.fs_rope(x[:1], None, 0, plan)
    assert torch.equal(y, z.expand(2, 2, 4, 64))


def test_rope_streams_and_graphs():
    x = torch.randn((2, 4, 100, 64), device="cuda").bfloat16()
    pos = _positions(2, 100, 9999, seed=3)
    plan = fs.fs_rope_plan(64)
    want, _ = fs.fs_rope(x, None, pos, plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = fs.fs_rope(x, None, pos, plan, q_out=torch.empty_like(x), stream=s)
    s.synchronize()
    assert torch.equal(want, got)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fs_rope(x, None, pos, plan, q_out=out)
    x.copy_(torch.randn_like(x, dtype=torch.float32))
    graph.replay()
    again, _ = fs.fs_rope(x, None, pos, plan)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
