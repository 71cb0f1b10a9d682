"""fs_linear_attn and fs_linear_attn_bwd in calls that the documentation allows and a first user would
not make (GPU only)."""
import pytest
import torch

from long_context_lm_gb300 import fs
from test_gpu_linear import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv,T,d,off", [(4, 2, 300, 64, 32), (4, 2, 300, 128, 32), (4, 2, 16, 64, 16), (4, 4, 300, 64, 16),
                                           (2, 1, 2000, 64, 96)])
def test_a_workspace_cut_from_a_larger_buffer(H, Hkv, T, d, off):
    q, k, v, dout, decay, S0, G, _ = inputs(2, H, Hkv, T, d, seed=T)
    want = (fs.fs_linear_attn(q, k, v, decay, state=S0),
            *fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G))
    n = max(fs.fs_linear_workspace(2, H, Hkv, T, d, "cuda", backward=b).numel() for b in (False, True))
    arena = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    ws = arena[off:off + n]
    got = (fs.fs_linear_attn(q, k, v, decay, state=S0, ws=ws),
           *fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G, ws=ws))
    fs.fs_check_status(ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (arena[:off] == 0).all() and (arena[off + n:] == 0).all()


@pytest.mark.parametrize("B,H,T,d", [(3, 16, 2500, 64), (5, 16, 2500, 128), (1, 2, 90000, 64), (20, 8, 700, 64)])
def test_one_workspace_for_the_largest_call_serves_all(B, H, T, d):
    dev = torch.device("cuda", torch.cuda.current_device())
    both = [fs.fs_linear_workspace(B, H, H, T, d, dev, backward=b) for b in (False, True)]
    for b, t in ((B, T), (B, T // 3), (1, T), (1, T // 2 + 1), (max(1, B // 2), T // 5), (B, 17), (1, 3)):
        q, k, v, dout, decay, S0, G, _ = inputs(b, H, H, t, d, seed=t)
        want = (fs.fs_linear_attn(q, k, v, decay, state=S0),
                *fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G))
        got = (fs.fs_linear_attn(q, k, v, decay, state=S0, ws=both[0]),
               *fs.fs_linear_attn_bwd(q, k, v, decay, dout, state=S0, dstate_out=G, ws=both[1]))
        assert all(torch.equal(x, y) for x, y in zip(got, want)), (b, t)
    for ws in both:
        fs.fs_check_status(ws)


@pytest.mark.parametrize("axis", [0, 2])
def test_sizes_past_32_bits_are_refused(axis):
    # axes as long as that exist by expansion alone; their low 32 bits would be a call of one token
    shape = [1, 1, 1, 64]
    shape[axis] = 2 ** 32 + 1
    x = torch.zeros((1, 1, 1, 64), device="cuda", dtype=torch.bfloat16).expand(shape)
    decay = torch.zeros(1, device="cuda")
    ws = fs.fs_linear_workspace(1, 1, 1, 1, 64, "cuda", backward=True)
    with pytest.raises(ValueError):
        fs.fs_linear_attn(x, x, x, decay, out=x, ws=ws)
    with pytest.raises(ValueError):
        fs.fs_linear_attn_bwd(x, x, x, decay, x, dq=x, dk=x, dv=x, ws=ws)
