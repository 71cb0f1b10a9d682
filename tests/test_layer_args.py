"""Refusals of fs_linear_attn, fs_linear_attn_bwd, fs_block_norm and fs_block_norm_bwd before
anything is launched.  Runs without a GPU: every call here is refused."""
import ctypes
import math

import pytest
import torch

from long_context_lm_gb300 import fs

INVALID, UNSUPPORTED = fs.FS_ERR_INVALID_ARG, fs.FS_ERR_UNSUPPORTED
S = fs._Strides


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def linear(**kw):
    a = dict(q=0x1000, k=0x2000, v=0x3000, qs=None, ks=None, vs=None, decay=256, batch=2, H=4, Hkv=2, T=32, d=64,
             count=None, scale=0.125, state=None, state_out=None, out=0x4000, os=None, ws=256, n=1 << 40)
    a.update(kw)
    return fs.load().fs_linear_attn(vp(a["q"]), vp(a["k"]), vp(a["v"]), a["qs"], a["ks"], a["vs"], vp(a["decay"]),
                                    a["batch"], a["H"], a["Hkv"], a["T"], a["d"], vp(a["count"]), a["scale"],
                                    vp(a["state"]), vp(a["state_out"]), vp(a["out"]), a["os"], vp(a["ws"]), a["n"], None)


def linear_bwd(**kw):
    a = dict(q=0x1000, k=0x2000, v=0x3000, qs=None, ks=None, vs=None, decay=256, batch=2, H=4, Hkv=2, T=32, d=64,
             count=None, scale=0.125, state=None, dout=0x5000, ds=None, G=None, dq=0x6000, dk=0x7000, dv=0x8000,
             gq=None, gk=None, gv=None, dstate=None, ws=256, n=1 << 40)
    a.update(kw)
    return fs.load().fs_linear_attn_bwd(
        vp(a["q"]), vp(a["k"]), vp(a["v"]), a["qs"], a["ks"], a["vs"], vp(a["decay"]), a["batch"], a["H"], a["Hkv"],
        a["T"], a["d"], vp(a["count"]), a["scale"], vp(a["state"]), vp(a["dout"]), a["ds"], vp(a["G"]), vp(a["dq"]),
        vp(a["dk"]), vp(a["dv"]), a["gq"], a["gk"], a["gv"], vp(a["dstate"]), vp(a["ws"]), a["n"], None)


SHAPES = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(decay=None), INVALID),
    (dict(batch=0), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=3), INVALID),
    (dict(T=0), INVALID), (dict(d=0), INVALID), (dict(d=32), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(batch=1 << 14), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(q=0x1008), UNSUPPORTED),
    (dict(qs=S(8192, 2048, 60)), UNSUPPORTED), (dict(ks=S(8192, 2048, 0)), UNSUPPORTED),
    (dict(vs=S(-4096, 2048, 64)), INVALID), (dict(n=16), INVALID), (dict(ws=None), INVALID),
]


@pytest.mark.parametrize("kw,status", SHAPES)
@pytest.mark.parametrize("call", [linear, linear_bwd])
def test_linear_refusals(call, kw, status):
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(out=0x1000), INVALID), (dict(out=0x4008), UNSUPPORTED),
    (dict(os=S(0, 2048, 64)), INVALID), (dict(os=S(8192, 0, 64)), INVALID), (dict(state=0x10004), UNSUPPORTED),
    (dict(state=0x100000, state_out=0x100010), INVALID),
    (dict(state=0x100000, state_out=0x100000 + 2 * 4 * 64 * 64 * 4 - 16), INVALID),
])
def test_linear_forward_refusals(kw, status):
    assert linear(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dout=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID),
    (dict(dq=0x5000), INVALID), (dict(dk=0x1000), INVALID), (dict(dk=0x6000), INVALID), (dict(dv=0x7000), INVALID),
    (dict(gk=S(8192, 0, 64)), INVALID), (dict(T=1, ws=None), INVALID), (dict(ws=264), UNSUPPORTED),
    (dict(state=0x100000, dstate=0x100000), INVALID), (dict(G=0x100000, dstate=0x100000), INVALID),
])
def test_linear_backward_refusals(kw, status):
    assert linear_bwd(**kw) == status


def test_linear_workspaces():
    n = fs.load().fs_linear_workspace_bytes
    assert n(1, 2, 3, 64, 64, 0) == 0 and n(1, 2, 2, 64, 65, 0) == 0 and n(0, 2, 2, 64, 64, 1) == 0
    assert n(2, 4, 4, 1, 64, 0) >= 256
    # shared heads' gradients are summed from fp32 parts
    assert n(2, 4, 2, 1000, 64, 1) >= n(2, 4, 4, 1000, 64, 1) + 2 * 2 * 4 * 1000 * 64 * 4


def norm(**kw):
    a = dict(x=0x1000, xs=64, dtype=0, gate=None, gs=64, res=None, rs=64, rdtype=0, gain=None, next=None, M=4, D=64,
             groups=1, scale=1.0, eps=1e-6, z=0x2000, zs=64, y=None, ys=64)
    a.update(kw)
    return fs.load().fs_block_norm(vp(a["x"]), a["xs"], a["dtype"], vp(a["gate"]), a["gs"], vp(a["res"]), a["rs"],
                                   a["rdtype"], vp(a["gain"]), vp(a["next"]), a["M"], a["D"], a["groups"], a["scale"],
                                   a["eps"], vp(a["z"]), a["zs"], vp(a["y"]), a["ys"], None)


def norm_bwd(**kw):
    a = dict(x=0x1000, xs=64, dtype=0, gate=None, gs=64, res=None, rs=64, rdtype=0, gain=None, next=None, M=4, D=64,
             groups=1, scale=1.0, eps=1e-6, dz=0x2000, dzs=64, dy=None, dys=64, dx=0x3000, dxs=64, dgate=None, dgs=64,
             dres=None, drs=64, dgain=None, dnext=None, ws=None, n=0)
    a.update(kw)
    return fs.load().fs_block_norm_bwd(
        vp(a["x"]), a["xs"], a["dtype"], vp(a["gate"]), a["gs"], vp(a["res"]), a["rs"], a["rdtype"], vp(a["gain"]),
        vp(a["next"]), a["M"], a["D"], a["groups"], a["scale"], a["eps"], vp(a["dz"]), a["dzs"], vp(a["dy"]), a["dys"],
        vp(a["dx"]), a["dxs"], vp(a["dgate"]), a["dgs"], vp(a["dres"]), a["drs"], vp(a["dgain"]), vp(a["dnext"]),
        vp(a["ws"]), a["n"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(M=0), INVALID), (dict(D=0), INVALID), (dict(groups=-1), INVALID),
    (dict(groups=3), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(dtype=5), INVALID), (dict(rdtype=5), INVALID),
    (dict(dtype=1), UNSUPPORTED), (dict(D=16385, xs=20000, groups=0, zs=20000, dzs=20000, dxs=20000), UNSUPPORTED),
    (dict(xs=-64), INVALID), (dict(x=0x1001), INVALID), (dict(rdtype=1, res=0x4002), INVALID),
    (dict(gain=0x102), INVALID),
])
@pytest.mark.parametrize("call", [norm, norm_bwd])
def test_norm_refusals(call, kw, status):
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [(dict(z=None), INVALID), (dict(zs=63), INVALID), (dict(zs=0), INVALID),
                                       (dict(y=0x3000, ys=60), INVALID)])
def test_norm_forward_refusals(kw, status):
    assert norm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dz=None), INVALID), (dict(dx=None), INVALID), (dict(dgate=0x4000), INVALID), (dict(dnext=0x100), INVALID),
    (dict(dgain=0x100), INVALID), (dict(dgain=0x100, ws=256, n=64), INVALID), (dict(dxs=0), INVALID),
])
def test_norm_backward_refusals(kw, status):
    assert norm_bwd(**kw) == status


def test_binding_refuses_host_tensors_and_sizes_past_32_bits():
    x = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fs.fs_linear_attn(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError):
        fs.fs_linear_attn_bwd(x, x, x, torch.zeros(2), x)
    with pytest.raises(ValueError):
        fs.fs_block_norm(x)
    with pytest.raises(ValueError):
        fs.fs_block_norm_bwd(x, dz=x)
    with pytest.raises(ValueError):
        fs.fs_block_norm_workspace(2 ** 32 + 4, 64, "cpu")
    with pytest.raises(ValueError):
        fs.fs_linear_workspace(1, 2, 2, 2 ** 32 + 1, 64, "cpu")


@pytest.mark.parametrize("kw", [
    dict(os=S(8192, 2048, 56)),              # tokens
    dict(os=S(8192, 1984, 64)),              # heads
    dict(os=S(4096, 2048, 64)),              # sequences
])
def test_linear_rows_that_lie_on_one_another(kw):
    assert linear(**kw) == INVALID
    assert linear_bwd(gq=kw["os"]) == INVALID


@pytest.mark.parametrize("kw", [
    dict(y=0x2000),                                    # both outputs at one place
    dict(y=0x4000, res=0x4000),                        # y over the residual
    dict(z=0x4000, gate=0x4000),                       # z over the gate
    dict(z=0x1000, zs=128),                            # in place with other rows
    dict(z=0x1000, rdtype=1),                          # in place with another type
    dict(z=0x4000, res=0x4000, rs=128),
])
def test_norm_in_place_refusals(kw):
    assert norm(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(dx=0x2000),                                   # dx over dz
    dict(dx=0x4000, gate=0x4000),
    dict(dx=0x1000, dxs=128),
    dict(gate=0x4000, dgate=0x3000),                   # both outputs at one place
    dict(gate=0x4000, dgate=0x2000),
    dict(res=0x4000, dres=0x1000),
    dict(dy=0x5000, gain=0x100, next=0x200, dgain=0x600, dnext=0x600, ws=256, n=1 << 40),
])
def test_norm_backward_in_place_refusals(kw):
    assert norm_bwd(**kw) == INVALID


@pytest.mark.parametrize("scale", [1e-30, -1e-30, 1e-45, 1e30, -1e30])
@pytest.mark.parametrize("call", [linear, linear_bwd])
def test_linear_scales_that_states_cannot_be_held_over(call, scale):
    assert call(scale=scale) == INVALID
