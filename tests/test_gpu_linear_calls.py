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
