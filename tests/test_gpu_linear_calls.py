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


@pytest.mark.parametrize("B,H,Hkv,T,d", [(2, 2, 1, 200, 64), (1, 2, 2, 5000, 64), (4, 80, 40, 1500, 64), (2, 4, 2, 3000, 128)])
def test_waits_that_give_up(B, H, Hkv, T, d):
    # The limit runs out in other places each time, with copies and products under way; the call ends
    # with its status, written by the kernels, and the next one is right.  Values that are not finite,
    # so that the roles that look for them have work, too.
    q, k, v, dout, decay, S0, G, _ = inputs(B, H, Hkv, T, d, seed=7)
    for t in (v, k):
        t[0, 0, T // 2, 3] = float("inf")
    ws = fs.fs_linear_workspace(B, H, Hkv, T, d, q.device)
    wb = fs.fs_linear_workspace(B, H, Hkv, T, d, q.device, backward=True)
    bits = lambda *ts: [t.view(torch.int16) for t in ts]  # noqa: E731
    form, back = dict(state=S0, ws=ws), dict(state=S0, dstate_out=G, ws=wb)
    want = bits(fs.fs_linear_attn(q, k, v, decay, **form)), bits(*fs.fs_linear_attn_bwd(q, k, v, decay, dout, **back))
    fs.fs_check_status(ws), fs.fs_check_status(wb)
    gave_up = [0, 0]
    for cycles in (1, 100, 300, 1000, 2000, 4000, 8000, 16000, 32000, 64000, 10 ** 9):
        for i, (w, call, again) in enumerate((
                (ws, lambda: bits(fs.fs_selftest_linear_wait(q, k, v, decay, cycles, **form)),
                 lambda: bits(fs.fs_linear_attn(q, k, v, decay, **form))),
                (wb, lambda: bits(*fs.fs_selftest_linear_wait_bwd(q, k, v, decay, dout, cycles, **back)),
                 lambda: bits(*fs.fs_linear_attn_bwd(q, k, v, decay, dout, **back))))):
            got, status = call(), int(w[:4].view(torch.int32))
            assert status in (0, fs.FS_ERR_TIMEOUT)
            gave_up[i] += status != 0
            if status == 0:
                assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
            else:
                with pytest.raises(fs.FSError):
                    fs.fs_check_status(w)
            w[:4].zero_()
            assert all(torch.equal(a, b) for a, b in zip(again(), want[i]))
            fs.fs_check_status(w)
            if cycles == 10 ** 9:
                assert status == 0
    assert min(gave_up) > 0
