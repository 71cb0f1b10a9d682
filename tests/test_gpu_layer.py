"""A linear-attention layer of the library's calls, as a model runs it: projections, linear
attention, the heads' norm and gate, the residual and the next block's norm; its prompt against its
decoding, and its gradients against a statement in 64 bits (GPU only)."""
import pytest
import torch

from long_context_lm_gb300 import fs
import layer_ref as ref

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, H, d, D, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.H, self.d, self.D = H, d, D
        self.w_in = (r(4 * H * d, D) / D ** 0.5).bfloat16()       # q, k, v, gate
        self.w_out = (r(D, H * d) / (H * d) ** 0.5).bfloat16()
        self.gain, self.next_gain = 1 + 0.1 * r(H * d), 1 + 0.1 * r(D)
        self.decay = -torch.exp2(-torch.arange(1, H + 1, device="cuda").float())

    def project(self, x):
        B, T, _ = x.shape
        y = x @ self.w_in.T
        q, k, v, gate = y.split(self.H * self.d, 2)
        return (*(t.view(B, T, self.H, self.d).transpose(1, 2) for t in (q, k, v)), gate)

    def __call__(self, x, residual, state):
        """x normalised, the residual stream beside it.  Returns the same for the next block."""
        B, T, _ = x.shape
        q, k, v, gate = self.project(x)
        o = torch.empty((B, T, self.H, self.d), dtype=torch.bfloat16, device="cuda")
        fs.fs_linear_attn(q, k, v, self.decay, state=state, state_out=state, out=o.transpose(1, 2))
        o, _ = fs.fs_block_norm(o.view(B, T, -1), gate=gate, groups=self.H, gain=self.gain)
        residual, x = fs.fs_block_norm(o @ self.w_out.T, residual=residual, scale=0.5, next_norm=True,
                                       next_gain=self.next_gain)
        return x, residual


@pytest.mark.parametrize("H,d,D", [(4, 64, 256), (3, 128, 192)])
def test_a_prompt_and_its_decoding(H, d, D):
    layer = Layer(H, d, D)
    torch.manual_seed(6)
    B, T, more = 2, 150, 6
    x = torch.randn((B, T + more, D), device="cuda").bfloat16()
    res = torch.randn((B, T + more, D), device="cuda")
    full = torch.zeros((B, H, d, d), device="cuda")
    want = layer(x, res, full)
    state = torch.zeros_like(full)
    got = [layer(x[:, :T], res[:, :T].contiguous(), state)]
    for t in range(T, T + more):
        got.append(layer(x[:, t:t + 1], res[:, t:t + 1].contiguous(), state))
    # The calls differ in the last step of bf16 here and there (outputs of the two forms of the
    # attention, products of other sizes), each of the three roundings between the attention and the
    # residual 2^-8 of a value; w_out sums H d of them with weights of 1 / sqrt(H d): like the values.
    for a, b in zip((torch.cat([g[i] for g in got], 1) for i in (0, 1)), want):
        assert (a.float() - b.float()).abs().max() < 8 * 2.0 ** -8 * b.float().abs().max()
        assert (a.float() - b.float()).square().mean().sqrt() < 2.0 ** -8 * b.float().square().mean().sqrt()
    # the states are sums of the same products
    assert (state - full).abs().max() < 2.0 ** -12 * full.abs().max()


def test_a_training_step_of_the_layer():
    H, d, D, B, T = 2, 64, 128, 2, 140
    torch.manual_seed(5)
    layer = Layer(H, d, D, seed=1)
    x = torch.randn((B, T, D), device="cuda").bfloat16()
    res, dres, dy = (torch.randn((B, T, D), device="cuda") for _ in range(3))
    dy = dy.bfloat16()
    q, k, v, gate = layer.project(x)
    o = fs.fs_linear_attn(q, k, v, layer.decay, out=torch.empty((B, T, H, d), dtype=torch.bfloat16, device="cuda").transpose(1, 2))
    o = o.transpose(1, 2).reshape(B, T, -1)
    a, _ = fs.fs_block_norm(o, gate=gate, groups=H, gain=layer.gain)
    b = a @ layer.w_out.T
    form = dict(residual=res, scale=0.5, next_gain=layer.next_gain)
    g2 = fs.fs_block_norm_bwd(b, dz=dres, dy=dy, **form)
    da = g2["x"] @ layer.w_out
    g1 = fs.fs_block_norm_bwd(o, dz=da, gate=gate, groups=H, gain=layer.gain)
    do = g1["x"].view(B, T, H, d).transpose(1, 2)
    dq, dk, dv = fs.fs_linear_attn_bwd(q, k, v, layer.decay, do)
    dy_in = torch.cat([*(t.transpose(1, 2).reshape(B, T, -1) for t in (dq, dk, dv)), g1["gate"]], 2)
    grads = dict(x=dy_in @ layer.w_in, res=g2["residual"], gain=g1["gain"], next_gain=g2["next_gain"],
                 w_in=dy_in.flatten(0, 1).float().T @ x.flatten(0, 1).float())

    # The statement in 64 bits goes through the very numbers that the layer went through: at each
    # stage its value is replaced by the layer's, its derivative kept.  (Left to itself it would
    # differ without bound: the first token's output is (q . k) v, where q . k may be as near to 0 as
    # one likes, and the norm behind it divides by that, so that the rounding of q alone
    # moves the gradient by 2^-8 |q| |k| / |q . k| of itself.)
    leaves = dict(x=x, res=res, gain=layer.gain, next_gain=layer.next_gain, w_in=layer.w_in)
    leaves = {n: t.double().requires_grad_() for n, t in leaves.items()}
    through = lambda t, value: t + (value.double().reshape(t.shape) - t).detach()  # noqa: E731
    y = through(leaves["x"] @ leaves["w_in"].T, x @ layer.w_in.T)
    q, k, v, gate = y.split(H * d, 2)
    q, k, v = (t.view(B, T, H, d).transpose(1, 2) for t in (q, k, v))
    lag = torch.arange(T, device="cuda")[:, None] - torch.arange(T, device="cuda")
    W = torch.where(lag >= 0, torch.exp(layer.decay.double()[:, None, None] * lag.clamp(min=0)), 0.0)
    o64 = ((q @ k.transpose(2, 3)) * W) @ v * d ** -0.5
    o64 = through(o64.transpose(1, 2).reshape(B * T, -1), o)
    a64, _ = ref.norm(o64, gate=gate.reshape(B * T, -1), groups=H, gain=leaves["gain"])
    b64 = through(through(a64, a) @ layer.w_out.double().T, b)
    z, n = ref.norm(b64, residual=leaves["res"].view(B * T, D), scale=0.5, next_gain=leaves["next_gain"])
    loss = (z * dres.double().view(B * T, D)).sum() + (n * dy.double().view(B * T, D)).sum()
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    # a chain of up to ten roundings to bf16 (2^-8 at most, half of it on average at the most), each of
    # which carries through to the gradients like the values themselves
    for n, w in want.items():
        err = (grads[n].double() - w).square().mean().sqrt() / w.square().mean().sqrt()
        assert err < 10 * 2.0 ** -8 / 2, (n, err.item())
