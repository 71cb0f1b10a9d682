"""fs_block_norm and fs_block_norm_bwd against a statement in 64 bits (GPU only).

Tolerances: half a step of the result's type (bf16 2^-8, fp32 2^-24 of the value), and what fp32
loses on the way.  A row's mean of squares is off by at most 2^-24 per addition of a thread's values
and of the team's tree, (32 + 10) 2^-24, halved by the root; a handful of products and the
root's, reciprocal's and exponential's own errors (2^-22; bf16 results take the
special-function unit's, 2^-20) come on top: 2^-18 of the terms' magnitudes for results in bf16,
2^-19 for those in fp32.  Two means, one inside the other, double that in the backward pass."""
import pytest
import torch

from long_context_lm_gb300 import fs
import layer_ref as ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -24}
TYPES = [(BF, BF), (BF, FP), (FP, FP)]


def make(M, D, dt, rdt, gate, residual, gains, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = (r(M, D) * torch.exp(r(M, 1))).to(dt)
    return dict(x=x, gate=(2 * r(M, D)).to(dt) if gate else None, residual=r(M, D).to(rdt) if residual else None,
                gain=1 + 0.3 * r(D) if gains else None), (1 + 0.3 * r(D) if gains else None), r(M, D).to(rdt), r(M, D).to(dt)


def near(got, want, size, loss):
    assert got.isfinite().all()
    tol = HALF[got.dtype] * want.abs() + loss * size + 1e-35
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), ((got.double() - want).abs() / tol).max().item())


def loss(dt):
    return 2.0 ** -18 if dt is BF else 2.0 ** -19


def check(M, D, groups, dt, rdt, gate, residual, next, gains=True, scale=0.7, eps=1e-6, seed=0):
    form, next_gain, dz, dy = make(M, D, dt, rdt, gate, residual, gains, seed)
    form.update(groups=groups, scale=scale, eps=eps)
    next_gain = next_gain if next else None
    z, y = fs.fs_block_norm(next_norm=next, next_gain=next_gain, z=torch.empty((M, D), dtype=rdt, device="cuda"), **form)
    wz, wy = ref.norm(next_gain=next_gain, **form)
    size = wz.abs() + (0 if not residual else 2 * form["residual"].double().abs())
    near(z, wz, size, loss(dt))
    assert (y is None) == (not next)
    if next:
        near(y, wy, wy.abs() * (size / wz.abs().clamp(min=1e-30)), loss(dt))
    got = fs.fs_block_norm_bwd(dz=dz, dy=dy if next else None, next_gain=next_gain, **form)
    want = ref.norm_grads(dz=dz, dy=dy if next else None, next_gain=next_gain, **form)
    for n in ("x", "gate", "residual", "gain", "next_gain"):
        have = {"x": True, "gate": gate, "residual": residual, "gain": gains, "next_gain": gains and next}[n]
        assert (got[n] is not None) == have
        if have:
            near(got[n], *want[n], 2 * loss(dt))


SIZES = [(1, 1, 1), (3, 7, 1), (2, 8, 0), (9, 64, 1), (5, 64, 8), (4, 65, 5), (33, 96, 3), (6, 100, 4), (7, 120, 10),
         (2, 128, 2), (3, 250, 2), (11, 256, 4), (5, 257, 0), (4, 512, 8), (3, 1000, 1), (2, 1000, 25),
         (13, 1024, 16), (5, 1024, 1024), (3, 1536, 12), (2, 2048, 32), (3, 2500, 1), (2, 4096, 1), (2, 5000, 2),
         (2, 8192, 64), (2, 8200, 1), (1, 16384, 128), (2, 16383, 3), (1, 16384, 0)]


@pytest.mark.parametrize("M,D,groups", SIZES)
@pytest.mark.parametrize("dt,rdt", TYPES)
def test_all_parts(M, D, groups, dt, rdt):
    check(M, D, groups, dt, rdt, True, True, True, seed=D)


@pytest.mark.parametrize("gate,residual,next,gains", [(False, True, True, True), (True, False, False, True),
                                                      (False, False, True, False), (True, True, False, False),
                                                      (False, False, False, True), (True, False, True, True)])
@pytest.mark.parametrize("M,D,groups", [(5, 64, 0), (300, 1024, 16), (700, 72, 1), (6, 1000, 0), (3, 4096, 1)])
@pytest.mark.parametrize("dt,rdt", TYPES)
def test_parts_missing(M, D, groups, dt, rdt, gate, residual, next, gains):
    check(M, D, groups, dt, rdt, gate, residual, next, gains, scale=1.0, seed=M)


@pytest.mark.parametrize("M,D", [(5000, 64), (20000, 40), (3001, 512), (2000, 1024), (1500, 2048), (700, 4096)])
def test_many_rows(M, D):
    # sums over rows: a block's rows in fp32 (at most M / (4 x 152) of them to a team, each addition
    # 2^-24 of the sum's magnitude), the blocks' with their errors carried
    check(M, D, 1, BF, BF, True, True, True, seed=5)


def test_gradients_against_differences():
    # central differences of the statement in 64 bits, step 1e-4: off by the third derivative
    # times 1e-8 / 6, below 1e-6 of the gradients' size here, and 1e-12 / 1e-4 of rounding
    M, D = 2, 24
    form, next_gain, dz, dy = make(M, D, FP, FP, True, True, True, seed=8)
    form.update(groups=3, scale=0.6, eps=1e-3)
    got = fs.fs_block_norm_bwd(dz=dz, dy=dy, next_gain=next_gain, **form)

    def value(**kw):
        z, y = ref.norm(**{**form, "next_gain": next_gain, **kw})
        return (z * dz.double()).sum() + (y * dy.double()).sum()

    for n in ("x", "gate", "residual", "gain", "next_gain"):
        t = (next_gain if n == "next_gain" else form[n]).double()
        flat = t.flatten()
        for i in range(0, flat.numel(), 5):
            a, b = flat.clone(), flat.clone()
            a[i] += 1e-4
            b[i] -= 1e-4
            diff = (value(**{n: a.view(t.shape)}) - value(**{n: b.view(t.shape)})) / 2e-4
            assert abs(diff.item() - got[n].flatten()[i].item()) < 2e-5 * max(1.0, abs(diff.item())), (n, i)


@pytest.mark.parametrize("D", [1024, 1001])
@pytest.mark.parametrize("dt,rdt", TYPES)
def test_strides_and_shapes(D, dt, rdt):
    # slices of a wider projection, outputs in wider buffers, and [batch, T, D] tensors
    B, T = 3, 5
    wide = torch.randn((B, T, 3 * D + 8), device="cuda").to(dt)
    x, gate = wide[..., :D], wide[..., D:2 * D]
    res = torch.randn((B, T, 2 * D), device="cuda").to(rdt)[..., D:]
    z, y = (torch.full((B, T, D + 24), 9.0, device="cuda", dtype=t) for t in (rdt, dt))
    form = dict(groups=1, gain=torch.rand(D, device="cuda"), next_gain=torch.rand(D, device="cuda"))
    a = fs.fs_block_norm(x, gate=gate, residual=res, z=z[..., :D], y=y[..., :D], **form)
    b = fs.fs_block_norm(x.contiguous(), gate=gate.contiguous(), residual=res.contiguous(), next_norm=True, **form)
    # (rows off sixteen bytes are added in another order: to one step of the type more)
    for p, q, t in zip(a, b, (rdt, dt)):
        near(p, q.double(), q.double().abs() + 1, 2 * HALF[t] + 2 * loss(dt))
    assert (z[..., D:] == 9).all() and (y[..., D:] == 9).all()
    grads = {n: torch.full((B, T, D + 16), 9.0, device="cuda", dtype=t) for n, t in
             (("dx", dt), ("dgate", dt), ("dresidual", rdt))}
    dz, dy = torch.randn((B, T, D), device="cuda").to(rdt), torch.randn((B, T, D), device="cuda").to(dt)
    a = fs.fs_block_norm_bwd(x, dz=dz, dy=dy, gate=gate, residual=res, **{n: t[..., :D] for n, t in grads.items()}, **form)
    b = fs.fs_block_norm_bwd(x.contiguous(), dz=dz, dy=dy, gate=gate.contiguous(), residual=res.contiguous(), **form)
    for n in a:
        near(a[n], b[n].double(), b[n].double().abs() + 4, 2 * HALF[b[n].dtype] + 4 * loss(dt))
    assert all((t[..., D:] == 9).all() for t in grads.values())


@pytest.mark.parametrize("M,D", [(37, 64), (50, 1000), (9, 1024), (3, 8192)])
@pytest.mark.parametrize("dt,rdt", TYPES)
def test_in_place(M, D, dt, rdt):
    form, next_gain, dz, dy = make(M, D, dt, rdt, True, True, True)
    want = fs.fs_block_norm(groups=1, next_norm=True, next_gain=next_gain, **form)
    grads = fs.fs_block_norm_bwd(dz=dz, dy=dy, groups=1, next_gain=next_gain, **form)
    c = {n: t.clone() for n, t in form.items()}
    z, y = fs.fs_block_norm(groups=1, next_gain=next_gain, z=c["residual"], y=c["x"], **c)
    assert z is c["residual"] and y is c["x"] and torch.equal(z, want[0]) and torch.equal(y, want[1])
    c = {n: t.clone() for n, t in form.items()}
    dz, dy = dz.clone(), dy.clone()
    got = fs.fs_block_norm_bwd(dz=dz, dy=dy, groups=1, next_gain=next_gain, dx=c["x"], dgate=c["gate"],
                               dresidual=dz, **c)
    assert all(torch.equal(got[n], grads[n]) for n in grads)


@pytest.mark.parametrize("D", [64, 1000, 1024, 4096])
def test_rows_of_zeros_and_values_that_are_not_finite(D):
    # a row's values stay in its row; eps 0 leaves rows that are not all zeros as they should be
    x = torch.randn((6, D), device="cuda").bfloat16()
    x[1] = 0
    want = fs.fs_block_norm(x, groups=1, next_norm=True)
    assert (want[0][1] == 0).all() and (want[1][1] == 0).all()
    x[2, D // 2], x[4, 0] = float("nan"), float("inf")
    z, y = fs.fs_block_norm(x, groups=1, next_norm=True)
    for r in (0, 1, 3, 5):
        assert torch.equal(z[r], want[0][r]) and torch.equal(y[r], want[1][r])
    assert z[2].isnan().all() and y[2].isnan().all() and z[4, 0].isnan() and y[4].isnan().all()
    z, y = fs.fs_block_norm(x[3:4, :D - 3], groups=1, eps=0.0, next_norm=True)
    assert z.isfinite().all() and y.isfinite().all()


def test_broadcast_rows_as_inputs():
    x = torch.randn((1, 1024), device="cuda").bfloat16()
    res = torch.randn((5, 1024), device="cuda").bfloat16()
    a = fs.fs_block_norm(x.expand(5, 1024), residual=res, groups=1, next_norm=True)
    b = fs.fs_block_norm(x.repeat(5, 1), residual=res, groups=1, next_norm=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_the_same_bits_every_time_and_in_graphs_and_on_other_streams():
    form, next_gain, dz, dy = make(3000, 1024, BF, FP, True, True, True)

    def both():
        f = fs.fs_block_norm(groups=16, next_norm=True, next_gain=next_gain, **form)
        return (*f, *fs.fs_block_norm_bwd(dz=dz, dy=dy, groups=16, next_gain=next_gain, **form).values())

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
