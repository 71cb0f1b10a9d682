"""Refusals of fs_rope, fs_cache_* and fs_tree_attn before anything is
launched, and the host-only parts (the rotary plan, the row sizes).  Runs
without a GPU: every call here is refused or never reaches CUDA."""
import ctypes
import math

import pytest
import torch

from long_context_lm_gb300 import fs
import serving_ref as ref


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


@pytest.mark.parametrize("rot,kw", [
    (64, {}), (2, {}), (256, {}), (64, dict(scaling="linear", factor=8.0)),
    (96, dict(scaling="base", factor=3.5)), (64, dict(scaling="ramp", factor=40.0)),
    (32, dict(scaling="ramp", factor=8.0, original=32768, base=500000.0)),
    (64, dict(scaling="ramp", factor=4.0, original=16, beta_fast=2.0)),
])
def test_plan_holds_the_frequencies(rot, kw):
    # F_i / 2^64 turns a position: a double's last bit of f_i / 2 pi, and pow's
    plan = fs.fs_rope_plan(rot, **kw)
    assert plan.rot == rot
    for i, f in enumerate(ref.frequencies(rot, **kw)):
        assert plan.turns[i] / 2.0 ** 64 == pytest.approx(f / (2 * math.pi), rel=1e-14)


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), fs.FS_ERR_INVALID_ARG), (dict(rot=7), fs.FS_ERR_INVALID_ARG),
    (dict(rot=-2), fs.FS_ERR_INVALID_ARG), (dict(rot=258), fs.FS_ERR_UNSUPPORTED),
    (dict(rot=64, base=1.0), fs.FS_ERR_INVALID_ARG),
    (dict(rot=64, base=math.nan), fs.FS_ERR_INVALID_ARG),
    (dict(rot=64, factor=0.5), fs.FS_ERR_INVALID_ARG),
    (dict(rot=64, amplitude=-1.0), fs.FS_ERR_INVALID_ARG),
    (dict(rot=64, amplitude=math.inf), fs.FS_ERR_INVALID_ARG),
    (dict(rot=2, scaling="base", factor=2.0), fs.FS_ERR_INVALID_ARG),
    (dict(rot=64, scaling="ramp", factor=2.0, original=0), fs.FS_ERR_INVALID_ARG),
    (dict(rot=64, scaling="ramp", factor=2.0, beta_fast=0.5), fs.FS_ERR_INVALID_ARG),
])
def test_plan_refusals(kw, status):
    with pytest.raises(fs.FSError) as e:
        fs.fs_rope_plan(**kw)
    assert e.value.status == status


def test_unknown_names_are_refused():
    with pytest.raises(ValueError):
        fs.fs_rope_plan(64, layout="quarter")
    with pytest.raises(ValueError):
        fs.fs_rope_plan(64, scaling="square")
    with pytest.raises(ValueError):
        fs.fs_cache_alloc(1, 1, 16, 64, "int2", None)


def _rope(**kw):
    a = dict(q=256, qo=256, Hq=2, k=None, ko=None, Hk=0, dtype=0, batch=1, N=4, d=64, pos=256,
             stride=4, plan=fs.fs_rope_plan(64), inverse=0)
    a.update(kw)
    return fs.load().fs_rope(vp(a["q"]), vp(a["qo"]), a["Hq"], None, None, vp(a["k"]), vp(a["ko"]),
                             a["Hk"], None, None, a["dtype"], a["batch"], a["N"], a["d"],
                             vp(a["pos"]), a["stride"], 0, a["plan"], a["inverse"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), fs.FS_ERR_INVALID_ARG), (dict(qo=None), fs.FS_ERR_INVALID_ARG),
    (dict(plan=None), fs.FS_ERR_INVALID_ARG), (dict(N=0), fs.FS_ERR_INVALID_ARG),
    (dict(d=63), fs.FS_ERR_INVALID_ARG), (dict(d=32), fs.FS_ERR_INVALID_ARG),  # d < rot
    (dict(k=256), fs.FS_ERR_INVALID_ARG), (dict(Hk=1), fs.FS_ERR_INVALID_ARG),
    (dict(dtype=9), fs.FS_ERR_INVALID_ARG), (dict(inverse=2), fs.FS_ERR_INVALID_ARG),
    (dict(stride=-1), fs.FS_ERR_INVALID_ARG), (dict(q=257), fs.FS_ERR_INVALID_ARG),
    (dict(batch=1 << 14, N=1 << 14), fs.FS_ERR_UNSUPPORTED),
])
def test_rope_refusals(kw, status):
    assert _rope(**kw) == status


def _desc(**kw):
    a = dict(codes=256, scales=256, table=256, status=None, pages=4, page=16, Hkv=2, d=64, format=2,
             batch=3, max_pages=2)
    a.update(kw)
    return fs.fs_cache_t(a["codes"], a["scales"], a["table"], a["status"], a["pages"], a["page"],
                         a["Hkv"], a["d"], a["format"], a["batch"], a["max_pages"])


BAD_CACHES = [
    (dict(codes=None), fs.FS_ERR_INVALID_ARG), (dict(table=None), fs.FS_ERR_INVALID_ARG),
    (dict(scales=None), fs.FS_ERR_INVALID_ARG), (dict(pages=0), fs.FS_ERR_INVALID_ARG),
    (dict(page=0), fs.FS_ERR_INVALID_ARG), (dict(batch=0), fs.FS_ERR_INVALID_ARG),
    (dict(max_pages=0), fs.FS_ERR_INVALID_ARG), (dict(format=4), fs.FS_ERR_INVALID_ARG),
    (dict(format=-1), fs.FS_ERR_INVALID_ARG), (dict(page=48), fs.FS_ERR_UNSUPPORTED),
    (dict(page=512), fs.FS_ERR_UNSUPPORTED), (dict(d=80), fs.FS_ERR_UNSUPPORTED),
    (dict(codes=264), fs.FS_ERR_UNSUPPORTED), (dict(batch=40000), fs.FS_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 27), fs.FS_ERR_UNSUPPORTED), (dict(pages=1 << 30), fs.FS_ERR_UNSUPPORTED),
    (dict(Hkv=40000, batch=1, page=256, format=0, d=128), fs.FS_ERR_UNSUPPORTED),
]


def _append(c, **kw):
    a = dict(k=256, v=256, ks=None, T=4, start=256)
    a.update(kw)
    return fs.load().fs_cache_append(c, vp(a["k"]), vp(a["v"]), a["ks"], None, a["T"],
                                     vp(a["start"]), None, None)


def _read(c, **kw):
    a = dict(k=256, v=256, T=4, start=256, dtype=0)
    a.update(kw)
    return fs.load().fs_cache_read(c, vp(a["start"]), None, a["T"], a["dtype"], vp(a["k"]),
                                   vp(a["v"]), None)


def _accept(c, **kw):
    a = dict(start=256, path=256, A=4)
    a.update(kw)
    return fs.load().fs_cache_accept(c, vp(a["start"]), vp(a["path"]), None, a["A"], None)


def _tree(c, **kw):
    a = dict(q=256, past=256, H=4, T=8, window=0, scale=0.125, out=1 << 30, ws=256, wsb=1 << 40)
    a.update(kw)
    return fs.load().fs_tree_attn(vp(a["q"]), c, vp(a["past"]), None, None, a["H"], a["T"],
                                  a["window"], a["scale"], vp(a["out"]), vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
@pytest.mark.parametrize("call", [_append, _read, _accept, _tree])
def test_cache_refusals(call, kw, status):
    assert call(_desc(**kw)) == status


@pytest.mark.parametrize("call,kw,status", [
    (_append, dict(k=None), fs.FS_ERR_INVALID_ARG), (_append, dict(start=None), fs.FS_ERR_INVALID_ARG),
    (_append, dict(T=0), fs.FS_ERR_INVALID_ARG), (_append, dict(T=1 << 30), fs.FS_ERR_UNSUPPORTED),
    (_append, dict(k=258), fs.FS_ERR_UNSUPPORTED),
    (_append, dict(ks=(ctypes.c_longlong * 3)(512, 100, 64)), fs.FS_ERR_UNSUPPORTED),
    (_read, dict(v=None), fs.FS_ERR_INVALID_ARG), (_read, dict(dtype=2), fs.FS_ERR_INVALID_ARG),
    (_read, dict(T=-1), fs.FS_ERR_INVALID_ARG), (_read, dict(v=264), fs.FS_ERR_UNSUPPORTED),
    (_accept, dict(path=None), fs.FS_ERR_INVALID_ARG), (_accept, dict(A=0), fs.FS_ERR_INVALID_ARG),
    (_accept, dict(A=65), fs.FS_ERR_UNSUPPORTED),
    (_tree, dict(q=None), fs.FS_ERR_INVALID_ARG), (_tree, dict(past=None), fs.FS_ERR_INVALID_ARG),
    (_tree, dict(ws=None), fs.FS_ERR_INVALID_ARG), (_tree, dict(wsb=1), fs.FS_ERR_INVALID_ARG),
    (_tree, dict(T=0), fs.FS_ERR_INVALID_ARG), (_tree, dict(T=65), fs.FS_ERR_UNSUPPORTED),
    (_tree, dict(H=3), fs.FS_ERR_INVALID_ARG), (_tree, dict(window=63), fs.FS_ERR_INVALID_ARG),
    (_tree, dict(window=-1), fs.FS_ERR_INVALID_ARG), (_tree, dict(scale=0.0), fs.FS_ERR_INVALID_ARG),
    (_tree, dict(scale=math.nan), fs.FS_ERR_INVALID_ARG), (_tree, dict(out=264), fs.FS_ERR_UNSUPPORTED),
    (_tree, dict(out=256), fs.FS_ERR_INVALID_ARG), (_tree, dict(out=256 + 1024), fs.FS_ERR_INVALID_ARG),
])
def test_call_refusals(call, kw, status):
    assert call(_desc(), **kw) == status


def test_workspace_and_row_bytes():
    assert [fs.load().fs_cache_row_bytes(64, f) for f in range(5)] == [128, 64, 64, 32, 0]
    assert [fs.load().fs_cache_row_bytes(128, f) for f in range(4)] == [256, 128, 128, 64]
    assert fs.load().fs_cache_row_bytes(96, 0) == 0
    L = fs.load()
    assert L.fs_tree_workspace_bytes(_desc(), 4, 8) > 0
    assert L.fs_tree_workspace_bytes(_desc(), 3, 8) == 0   # H % Hkv
    assert L.fs_tree_workspace_bytes(_desc(), 4, 65) == 0
    assert L.fs_tree_workspace_bytes(_desc(d=32), 4, 8) == 0


def test_host_tensors_are_refused():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fs.fs_rope(x, None, 0, fs.fs_rope_plan(64))
    with pytest.raises(ValueError):
        fs.fs_cache(torch.zeros(4, 2, 2, 16, 64, dtype=torch.uint8), None,
                    torch.zeros(1, 2, dtype=torch.int32), "int8")


def test_reference_rounds_ties_to_even():
    # the 64-bit statement itself: borders between codes, by hand
    row = torch.zeros(64, dtype=torch.bfloat16)
    row[0], row[1], row[2], row[3] = 14.0, 1.0, 3.0, -5.0   # Q x / amax = 7, .5, 1.5, -2.5
    codes, scale = ref.quantise(row[None], "int4")
    assert codes[0, 0].item() == 7 and codes[0, 1].item() == (2 | (14 << 4)) and scale.item() == 2.0
    assert ref.values(codes, scale, "int4")[0, :4].tolist() == [14.0, 0.0, 4.0, -4.0]
    row[0], row[1], row[2], row[3] = 448.0, 17.0, 19.0, 2.0 ** -10
    codes, scale = ref.quantise(row[None], "e4m3")            # 16 | 18 | 20: ties to even codes
    assert ref.values(codes, scale, "e4m3")[0, :4].tolist() == [448.0, 16.0, 20.0, 0.0]
