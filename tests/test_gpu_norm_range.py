"""fs_block_norm and fs_block_norm_bwd at the ends of their ranges, against a statement in 64 bits (GPU
only).  Tolerances as in test_gpu_norm.py: half a step of the result's type, and 2^-18 (bf16 x) or 2^-19
(fp32) of the terms' magnitudes, twice that in the backward pass."""
import pytest
import torch

from long_context_lm_gb300 import fs
import layer_ref as ref
from test_gpu_norm import BF, FP, TYPES, loss, make, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 33])
@pytest.mark.parametrize("D,groups", [(40, 5), (64, 1), (64, 8), (100, 1), (256, 4), (512, 1), (512, 16), (1024, 16)])
@pytest.mark.parametrize("dt,rdt", TYPES)
@pytest.mark.parametrize("next", [False, True])
def test_gradients_with_eps_0(M, D, groups, dt, rdt, next):
    # rows that are not zero have factors without eps, and a block's places without a row add nothing
    form, next_gain, dz, dy = make(M, D, dt, rdt, True, True, True, seed=D + M)
    form.update(groups=groups, scale=0.7, eps=0.0)
    dy, next_gain = (dy, next_gain) if next else (None, None)
    got = fs.fs_block_norm_bwd(dz=dz, dy=dy, next_gain=next_gain, **form)
    want = ref.norm_grads(dz=dz, dy=dy, next_gain=next_gain, **form)
    for n in ("x", "gate", "residual", "gain", "next_gain"):
        assert (got[n] is None) == (n == "next_gain" and not next)
        if got[n] is not None:
            near(got[n], *want[n], 2 * loss(dt))


# gates from next to nothing to the type's ends, both signs
GATES = [1e-30, 1e-6, 0.1, 1.0, 5.0, 10.0, 17.0, 20.0, 40.0, 80.0, 86.0, 88.0, 89.0, 95.0, 100.0, 104.0, 1e3, 1e5, 3e7, 1e8,
         1e20, 1e30, 1e37, 2.3e38, 2.5e38, 3.3e38]


def gates(M, D, dt, bound=float("inf")):
    g = torch.tensor([v for v in GATES if v <= bound], dtype=torch.float64)
    ends = torch.tensor([torch.finfo(dt).max], dtype=torch.float64) if bound > 3.4e38 else g[:0]
    g = torch.cat([g, -g, ends, -ends, torch.zeros(1, dtype=torch.float64)])
    return g[torch.arange(M * D) * 7 % len(g)].reshape(M, D).to(dt).cuda()


@pytest.mark.parametrize("D", [64, 1000, 1024, 4099])
@pytest.mark.parametrize("dt,rdt", TYPES)
@pytest.mark.parametrize("residual", [False, True])
def test_gates_of_any_size(D, dt, rdt, residual):
    # x within a half, so that the products with the type's largest numbers stay within it
    form, _, dz, _ = make(6, D, dt, rdt, True, residual, False, seed=D)
    form.update(x=(form["x"].float().sigmoid() - 0.5).to(dt), gate=gates(6, D, dt), scale=0.7)
    z, _ = fs.fs_block_norm(z=torch.empty((6, D), dtype=rdt, device="cuda"), **form)
    want, _ = ref.norm(**form)
    size = want.abs() + (2 * form["residual"].double().abs() if residual else 0)
    near(z, want, size, loss(dt))
    if dt is FP and not residual:
        # also where the sigmoid lies below fp32's normal range: steps of 2^-149 of it, times a gate
        # of 104 at most and |x| of a half
        assert ((z.double() - want).abs() <= 2.0 ** -19 * want.abs() + 104 * 2.0 ** -149).all()
    dz = (dz.float().sigmoid() - 0.5).to(rdt)
    got = fs.fs_block_norm_bwd(dz=dz, **form)
    want = ref.norm_grads(dz=dz, **form)
    near(got["x"], *want["x"], 2 * loss(dt))
    near(got["gate"], *want["gate"], 2 * loss(dt))   # (the slope past 17 is 1, not a difference of two gates)


@pytest.mark.parametrize("dt,rdt", TYPES)
def test_gates_of_any_size_before_a_second_norm(dt, rdt):
    # squares of z fit fp32 for gates up to 1e16
    form, next_gain, dz, dy = make(6, 1024, dt, rdt, True, True, True, seed=3)
    form.update(gate=gates(6, 1024, dt, 1e16), groups=16, scale=0.7, eps=1e-6)
    z, y = fs.fs_block_norm(next_norm=True, next_gain=next_gain, **form)
    wz, wy = ref.norm(next_gain=next_gain, **form)
    size = wz.abs() + 2 * form["residual"].double().abs()
    near(z, wz, size, loss(dt))
    near(y, wy, wy.abs() * (size / wz.abs().clamp(min=1e-30)), loss(dt))
    got = fs.fs_block_norm_bwd(dz=dz, dy=dy, next_gain=next_gain, **form)
    want = ref.norm_grads(dz=dz, dy=dy, next_gain=next_gain, **form)
    for n in want:
        near(got[n], *want[n], 2 * loss(dt))


@pytest.mark.parametrize("dt", [BF, FP])
def test_gates_that_are_not_finite(dt):
    # +inf opens without a bound; -inf is 0 times infinity, as the formula has it; both in their elements alone
    x = torch.randn((3, 256), device="cuda").to(dt)
    gate = torch.randn((3, 256), device="cuda").to(dt)
    want, _ = fs.fs_block_norm(x, gate=gate)
    gate[0, 5], gate[1, 7], gate[2, 9] = float("inf"), float("-inf"), float("nan")
    z, _ = fs.fs_block_norm(x, gate=gate)
    assert z[0, 5] == x[0, 5] * float("inf") and z[1, 7].isnan() and z[2, 9].isnan()
    z[0, 5], z[1, 7], z[2, 9] = want[0, 5], want[1, 7], want[2, 9]
    assert torch.equal(z, want)


@pytest.mark.parametrize("D", [64, 1024, 1001, 2500])
@pytest.mark.parametrize("dt", [BF, FP])
def test_gates_beside_an_fp32_residual_stream(D, dt):
    # z and the gains' gradients are fp32 numbers there, whatever x is: an exponential of 2^-22 and no more
    # than eight roundings of 2^-24 on the way to them
    g = torch.Generator(device="cuda").manual_seed(D)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    gate = (160 * torch.rand((1, D), generator=g, device="cuda") - 80).to(dt)
    form = dict(x=r(1, D).to(dt), gate=gate, gain=1 + 0.3 * r(D), scale=0.7)
    z, _ = fs.fs_block_norm(z=torch.empty((1, D), device="cuda"), **form)
    want, _ = ref.norm(**form)
    assert ((z.double() - want).abs() <= (2.0 ** -22 + 8 * 2.0 ** -24) * want.abs()).all()
    dz = r(1, D)
    got = fs.fs_block_norm_bwd(dz=dz, **form)["gain"]
    want = ref.norm_grads(dz=dz, **form)["gain"][0]
    assert ((got.double() - want).abs() <= (2.0 ** -22 + 8 * 2.0 ** -24) * want.abs()).all()


@pytest.mark.parametrize("M", [1, 40, 5000])
@pytest.mark.parametrize("D", [64, 1024])
def test_gains_gradients_that_are_not_finite(M, D):
    # an infinite sum is infinite, of its sign; infinities of both signs make NaN; other columns keep theirs
    g = torch.Generator(device="cuda").manual_seed(M)
    x, dz = (torch.randn((M, D), generator=g, device="cuda") for _ in range(2))
    x[:, 3:6] = x[:, 3:6].abs() + 0.1
    gain = torch.ones(D, device="cuda")
    want = fs.fs_block_norm_bwd(x, dz=dz, gain=gain)["gain"]
    dz[M // 2, 3], dz[0, 4], dz[M - 1, 5] = float("inf"), float("-inf"), float("nan")
    if M > 1:
        dz[0, 6], dz[M - 1, 6] = float("inf"), float("-inf")
        x[:, 6] = 1.0
        want[6] = float("nan")
    got = fs.fs_block_norm_bwd(x, dz=dz, gain=gain)["gain"]
    want[3], want[4], want[5] = float("inf"), float("-inf"), float("nan")
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0.5), want.nan_to_num(0.5))
