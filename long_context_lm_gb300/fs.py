"""Thin Python binding of the C-ABI library ``libfs.so`` (``include/fs.h``).

Only argument marshalling happens here: tensors are checked for device,
dtype, shape and contiguity, their device pointers and the current CUDA
stream are handed to the library, and a non-zero status raises ``FSError``.
Every step of the computation runs in the library's CUDA kernels; there is no
CPU fallback, and a missing or unbuildable library raises.

Function names match the C entry points.  Tensors follow the C layouts:
q, k, v ``[batch, H, N, d]`` (bf16, or fp32 for ``fs_attention_fwd`` /
``fs_cell_summarize``); per-head ``lam``, ``sigma``, ``mix`` ``[H]`` fp32.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

(FS_OK, FS_ERR_INVALID_ARG, FS_ERR_UNSUPPORTED, FS_ERR_CUDA, FS_ERR_TIMEOUT, FS_ERR_RANGE,
 FS_ERR_SCRATCH_LIMIT, FS_ERR_STATE, FS_ERR_CACHE) = range(9)
FS_BF16, FS_FP32 = 0, 1
FS_MODE_FSL, FS_MODE_FS, FS_MODE_FSB = 0, 1, 2

SYMBOLS = ["fs_default_params", "fs_status_string", "fs_last_cuda_error", "fs_workspace_bytes",
           "fs_set_attention_timeline",
           "fs_prune_workspace_bytes", "fs_window_workspace_bytes", "fs_cell_summarize",
           "fs_prune_cells", "fs_select_cells", "fs_sparse_readout", "fs_window_attn",
           "fs_attention_fwd", "fs_attention_fwd_traced", "fs_workspace_view", "fs_check_status",
           "fs_prune_static_scratch_bytes", "fs_prune_cells_static", "fs_decode_step",
           "fs_selftest_wait_timeout", "fs_host_workspace_bytes", "fs_attention_fwd_host",
           "fs_window_attn_traced", "fs_decode_state_bytes", "fs_decode_state_init",
           "fs_decode_state_view", "fs_qkv_workspace_bytes", "fs_qkv_prologue",
           "fs_backward_workspace_bytes", "fs_attention_bwd",
           "fs_fsb_workspace_bytes", "fs_fsb_select",
           "fs_rope_make_plan", "fs_rope", "fs_cache_row_bytes", "fs_cache_append",
           "fs_cache_read", "fs_cache_accept", "fs_tree_workspace_bytes", "fs_tree_attn",
           "fs_selftest_tree_wait", "fs_linear_workspace_bytes", "fs_linear_attn",
           "fs_linear_attn_bwd", "fs_selftest_linear_wait", "fs_selftest_linear_wait_bwd",
           "fs_block_norm", "fs_block_norm_workspace_bytes", "fs_block_norm_bwd"]
FS_LINEAR_STEPS = 16
FS_ROPE_LAYOUTS = {"half": 0, "pairs": 1}
FS_ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3}
FS_CACHE_FORMATS = {"bf16": 0, "e4m3": 1, "int8": 2, "int4": 3}
FS_N_STAGES = 4
STAGE_NAMES = ["cells_prep", "prune", "select", "attention"]


class fs_params(ctypes.Structure):
    _fields_ = [("w", ctypes.c_int), ("s", ctypes.c_int), ("K", ctypes.c_int),
                ("P", ctypes.c_int), ("W", ctypes.c_int), ("Bq", ctypes.c_int),
                ("rope_base", ctypes.c_float), ("rms_eps", ctypes.c_float),
                ("mode", ctypes.c_int), ("beam", ctypes.c_int), ("tau", ctypes.c_float)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class fs_rope_params(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int), ("layout", ctypes.c_int), ("scaling", ctypes.c_int),
                ("original", ctypes.c_int), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("amplitude", ctypes.c_double)]


class fs_rope_plan_t(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int), ("layout", ctypes.c_int), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int), ("turns", ctypes.c_uint64 * 128)]


class fs_cache_t(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("pages", ctypes.c_int), ("page", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("d", ctypes.c_int), ("format", ctypes.c_int),
                ("batch", ctypes.c_int), ("max_pages", ctypes.c_int)]


class FSError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = f"{where}: {status_string(status)} (status {status})"
        if status == FS_ERR_CUDA:
            msg += ": " + load().fs_last_cuda_error().decode()
        super().__init__(msg)


_lock = threading.Lock()
_lib = None


def lib_path() -> str:
    return _build.LIB


def load(build_if_stale: bool = True):
    """Load libfs.so (compiling it in-tree first when it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if build_if_stale:
            _build.build()
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"{_build.LIB} is missing: build it with "
                               "`python -m long_context_lm_gb300.build`")
        L = ctypes.CDLL(_build.LIB)
        P, I, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        PP = ctypes.POINTER(fs_params)
        L.fs_default_params.argtypes = [PP]
        L.fs_default_params.restype = None
        L.fs_status_string.argtypes = [I]
        L.fs_status_string.restype = ctypes.c_char_p
        L.fs_last_cuda_error.argtypes = []
        L.fs_last_cuda_error.restype = ctypes.c_char_p
        L.fs_workspace_bytes.argtypes = [I, I, I, I, PP, I]
        L.fs_workspace_bytes.restype = Z
        L.fs_prune_workspace_bytes.argtypes = [I, I, I, PP]
        L.fs_prune_workspace_bytes.restype = Z
        L.fs_window_workspace_bytes.argtypes = [I, I, I, I, PP]
        L.fs_window_workspace_bytes.restype = Z
        L.fs_host_workspace_bytes.argtypes = [I, I, I, I, PP, I, I]
        L.fs_host_workspace_bytes.restype = Z
        L.fs_cell_summarize.argtypes = [P, I, I, I, I, I, I, P, P, P]
        L.fs_prune_cells.argtypes = [P, I, I, I, PP, P, P, P, Z, P]
        L.fs_select_cells.argtypes = [P, I, P, P, P, P, P, P, I, I, I, I, PP, P, P, P]
        L.fs_sparse_readout.argtypes = [P, P, P, I, P, I, I, I, I, PP, P, P]
        L.fs_window_attn.argtypes = [P, P, P, I, P, P, I, I, I, I, PP, P, P, Z, P]
        L.fs_window_attn_traced.argtypes = L.fs_window_attn.argtypes + [P]
        L.fs_attention_fwd.argtypes = [P, P, P, I, I, I, I, I, PP, P, P, P, P, P, Z, P]
        L.fs_attention_fwd_traced.argtypes = L.fs_attention_fwd.argtypes + [P]
        L.fs_attention_fwd_host.argtypes = [P, P, P, I, I, I, I, I, PP, P, P, P, P, I, P, Z, P]
        L.fs_workspace_view.argtypes = [I, I, I, I, PP, I] + [ctypes.POINTER(Z)] * 5
        L.fs_check_status.argtypes = [P, P]
        L.fs_set_attention_timeline.argtypes = [P, I]
        L.fs_selftest_wait_timeout.argtypes = [P, P]
        L.fs_prune_static_scratch_bytes.argtypes = []
        L.fs_prune_static_scratch_bytes.restype = Z
        L.fs_prune_cells_static.argtypes = [P, I, I, I, PP, P, P, P]
        L.fs_decode_state_bytes.argtypes = [I, I, I, PP]
        L.fs_decode_state_bytes.restype = Z
        L.fs_decode_state_view.argtypes = [I, I, I, PP, ctypes.POINTER(Z)]
        L.fs_qkv_workspace_bytes.argtypes = [I, I, I, I]
        L.fs_backward_workspace_bytes.argtypes = [I, I, I, I, PP]
        L.fs_fsb_workspace_bytes.argtypes = [I, I, I, PP]
        L.fs_fsb_workspace_bytes.restype = Z
        L.fs_fsb_select.argtypes = [P, P, P, P, P, P, I, I, I, I, PP, P, P, Z, P]
        L.fs_backward_workspace_bytes.restype = Z
        L.fs_attention_bwd.argtypes = [P, P, P, I, I, I, I, I, PP, P, P, P, P, P, P, P, P, P, Z, P]
        L.fs_qkv_workspace_bytes.restype = Z
        L.fs_qkv_prologue.argtypes = [P, P, P, I, I, I, I, F, P, P, P, P, Z, P]
        L.fs_decode_state_init.argtypes = [P, P, I, P, P, P, P, I, I, I, I, I, PP, P, Z, P]
        L.fs_decode_step.argtypes = [P, P, P, I, I, I, I, I, P, P, P, PP, P, Z, P, P, P]
        PC, S3 = ctypes.POINTER(fs_cache_t), ctypes.POINTER(ctypes.c_longlong)
        L.fs_rope_make_plan.argtypes = [ctypes.POINTER(fs_rope_params),
                                        ctypes.POINTER(fs_rope_plan_t)]
        L.fs_rope.argtypes = [P, P, I, S3, S3, P, P, I, S3, S3, I, I, I, I, P, ctypes.c_longlong, I,
                              ctypes.POINTER(fs_rope_plan_t), I, P]
        L.fs_cache_row_bytes.argtypes = [I, I]
        L.fs_cache_row_bytes.restype = Z
        L.fs_cache_append.argtypes = [PC, P, P, S3, S3, I, P, P, P]
        L.fs_cache_read.argtypes = [PC, P, P, I, I, P, P, P]
        L.fs_cache_accept.argtypes = [PC, P, P, P, I, P]
        L.fs_tree_workspace_bytes.argtypes = [PC, I, I]
        L.fs_tree_workspace_bytes.restype = Z
        L.fs_tree_attn.argtypes = [P, PC, P, P, P, I, I, I, F, P, P, Z, P]
        L.fs_selftest_tree_wait.argtypes = [P, PC, P, P, P, I, I, I, F, P, P, Z,
                                            ctypes.c_longlong, P]
        LL = ctypes.c_longlong
        L.fs_linear_workspace_bytes.argtypes = [I, I, I, I, I, I]
        L.fs_linear_workspace_bytes.restype = Z
        L.fs_linear_attn.argtypes = [P, P, P, S3, S3, S3, P, I, I, I, I, I, P, F, P, P, P, S3, P, Z, P]
        L.fs_linear_attn_bwd.argtypes = [P, P, P, S3, S3, S3, P, I, I, I, I, I, P, F, P, P, S3, P, P,
                                         P, P, S3, S3, S3, P, P, Z, P]
        L.fs_selftest_linear_wait.argtypes = [*L.fs_linear_attn.argtypes[:-1], LL, P]
        L.fs_selftest_linear_wait_bwd.argtypes = [*L.fs_linear_attn_bwd.argtypes[:-1], LL, P]
        L.fs_block_norm.argtypes = [P, LL, I, P, LL, P, LL, I, P, P, I, I, I, F, F, P, LL, P, LL, P]
        L.fs_block_norm_workspace_bytes.argtypes = [I, I]
        L.fs_block_norm_workspace_bytes.restype = Z
        L.fs_block_norm_bwd.argtypes = [P, LL, I, P, LL, P, LL, I, P, P, I, I, I, F, F, P, LL, P, LL, P,
                                        LL, P, LL, P, LL, P, P, P, Z, P]
        for name in SYMBOLS:
            if name not in ("fs_linear_workspace_bytes", "fs_block_norm_workspace_bytes",
                            "fs_cache_row_bytes", "fs_tree_workspace_bytes",
                            "fs_default_params", "fs_status_string", "fs_last_cuda_error",
                            "fs_workspace_bytes", "fs_prune_static_scratch_bytes",
                            "fs_prune_workspace_bytes", "fs_window_workspace_bytes",
                            "fs_host_workspace_bytes", "fs_decode_state_bytes",
                            "fs_qkv_workspace_bytes", "fs_backward_workspace_bytes",
                            "fs_fsb_workspace_bytes"):
                getattr(L, name).restype = I
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return load().fs_status_string(int(status)).decode()


def _check(status, where):
    if status != FS_OK:
        raise FSError(status, where)


def fs_default_params(**overrides) -> fs_params:
    p = fs_params()
    load().fs_default_params(ctypes.byref(p))
    for k, v in overrides.items():
        setattr(p, k, v)
    return p


def _params(params):
    if params is None:
        return fs_default_params()
    if isinstance(params, dict):
        return fs_default_params(**params)
    return params


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, name, dtypes):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _dtype_code(t):
    return FS_BF16 if t.dtype == torch.bfloat16 else FS_FP32


def _qkv_shape(q):
    if q.dim() != 4:
        raise ValueError("q/k/v must be [batch, H, N, d]")
    return tuple(q.shape)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def fs_workspace_bytes(batch, H, N, d, params=None, dtype=FS_BF16) -> int:
    p = _params(params)
    return load().fs_workspace_bytes(batch, H, N, d, ctypes.byref(p), dtype)


def fs_window_workspace_bytes(batch, H, N, d, params=None) -> int:
    p = _params(params)
    return load().fs_window_workspace_bytes(batch, H, N, d, ctypes.byref(p))


def fs_cell_summarize(k, s=32, kbar=None, amax=None, stream=None):
    L = load()
    _dev(k, "k", (torch.bfloat16, torch.float32))
    B, H, N, d = _qkv_shape(k)
    C = N // s
    kbar = kbar if kbar is not None else torch.empty((B, H, C, d), device=k.device, dtype=torch.float32)
    amax = amax if amax is not None else torch.empty((B, H, C), device=k.device, dtype=torch.float32)
    _dev(kbar, "kbar", (torch.float32,))
    _dev(amax, "amax", (torch.float32,))
    _check(L.fs_cell_summarize(_ptr(k), _dtype_code(k), B, H, N, d, s, _ptr(kbar), _ptr(amax),
                               _stream(stream)), "fs_cell_summarize")
    return kbar, amax


def fs_prune_cells(amax, N, params=None, stream=None):
    L = load()
    p = _params(params)
    _dev(amax, "amax", (torch.float32,))
    B, H, C = amax.shape
    nblk = N // p.Bq
    pool = torch.empty((B, H, nblk, p.P + p.W), device=amax.device, dtype=torch.int32)
    count = torch.empty((B, H, nblk), device=amax.device, dtype=torch.int32)
    wsb = L.fs_prune_workspace_bytes(B, H, N, ctypes.byref(p))
    if wsb == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_prune_workspace_bytes")
    ws = torch.empty(wsb, device=amax.device, dtype=torch.uint8)
    _check(L.fs_prune_cells(_ptr(amax), B, H, N, ctypes.byref(p), _ptr(pool), _ptr(count),
                            _ptr(ws), wsb, _stream(stream)), "fs_prune_cells")
    return pool, count


def fs_prune_cells_static(amax, N, params=None, pool=None, count=None, stream=None):
    """fs_prune_cells on the library's fixed scratch array (no workspace).
    ``pool`` / ``count`` may be given to avoid allocating outputs here."""
    L = load()
    p = _params(params)
    _dev(amax, "amax", (torch.float32,))
    B, H, C = amax.shape
    nblk = N // p.Bq
    if pool is None:
        pool = torch.empty((B, H, nblk, p.P + p.W), device=amax.device, dtype=torch.int32)
    if count is None:
        count = torch.empty((B, H, nblk), device=amax.device, dtype=torch.int32)
    _check(L.fs_prune_cells_static(_ptr(amax), B, H, N, ctypes.byref(p), _ptr(pool),
                                   _ptr(count), _stream(stream)), "fs_prune_cells_static")
    return pool, count


def fs_selftest_wait_timeout(ws, stream=None):
    """Launch the bounded-wait self-test into workspace ``ws`` (device uint8,
    >= 256 bytes); read the outcome with fs_check_status(ws)."""
    _check(load().fs_selftest_wait_timeout(_ptr(ws), _stream(stream)), "fs_selftest_wait_timeout")


def fs_decode_state_bytes(batch, H, d=64, params=None) -> int:
    p = _params(params)
    return load().fs_decode_state_bytes(batch, H, d, ctypes.byref(p))


def fs_decode_state_view(state, batch, H, params=None):
    """Views into a decode state: per (batch, head) slot cell ids [BH, nslots]
    int32, slot a_c [BH, nslots] f32, slot mean keys [BH, nslots, 64] f32,
    and the header ints [BH, n] (position, list counts, lists)."""
    L = load()
    p = _params(params)
    offs = (ctypes.c_size_t * 7)()
    _check(L.fs_decode_state_view(batch, H, 64, ctypes.byref(p), offs), "fs_decode_state_view")
    g, hb, oc, oa, ok, ns, nh = (int(x) for x in offs)
    heads = state[g:g + batch * H * hb].view(batch * H, hb)
    return dict(cell=heads[:, oc:oc + 4 * ns].contiguous().view(torch.int32),
                amax=heads[:, oa:oa + 4 * ns].contiguous().view(torch.float32),
                kbar=heads[:, ok:ok + 4 * 64 * ns].contiguous().view(torch.float32).view(-1, ns, 64),
                header=heads[:, :4 * nh].contiguous().view(torch.int32))


def fs_decode_state_init(batch, H, params=None, k=None, v=None, kbar=None, amax=None, pool=None,
                         pool_count=None, N0=0, state=None, device=None, stream=None):
    """Bounded decode state after the first N0 tokens (N0 = 0: an empty state).
    For N0 > 0, k, v [B,H,N,d] bf16 hold the prefix in rows < N0, and kbar,
    amax, pool, pool_count are fs_cell_summarize / fs_prune_cells of k.
    Returns the state (a device uint8 tensor of fs_decode_state_bytes)."""
    L = load()
    p = _params(params)
    nb = L.fs_decode_state_bytes(batch, H, 64, ctypes.byref(p))
    if nb == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_decode_state_bytes")
    if N0 > 0:
        for t_, n in ((k, "k"), (v, "v")):
            _dev(t_, n, (torch.bfloat16,))
        for t_, n in ((kbar, "kbar"), (amax, "amax")):
            _dev(t_, n, (torch.float32,))
        for t_, n in ((pool, "pool"), (pool_count, "pool_count")):
            _dev(t_, n, (torch.int32,))
        N = k.shape[2]
        device = k.device
    else:
        N = 128
        device = device or torch.device("cuda")
    if state is None:
        state = torch.empty(nb, device=device, dtype=torch.uint8)
    elif state.numel() * state.element_size() < nb:
        raise ValueError(f"state too small: {state.numel()} < {nb} bytes")
    _check(L.fs_decode_state_init(_ptr(k), _ptr(v), FS_BF16, _ptr(kbar), _ptr(amax), _ptr(pool),
                                  _ptr(pool_count), batch, H, N, int(N0), 64, ctypes.byref(p),
                                  _ptr(state), nb, _stream(stream)), "fs_decode_state_init")
    return state


def fs_decode_step(q_t, k_t, v_t, t, state, lam, sigma, mix, params=None, out=None,
                   sel=None, stream=None):
    """One decode step for token t from the bounded ``state`` (advanced in
    place).  q_t, k_t, v_t [B,H,d] bf16.  Returns out_t [B,H,d] f32."""
    L = load()
    p = _params(params)
    for t_, n in ((q_t, "q_t"), (k_t, "k_t"), (v_t, "v_t")):
        _dev(t_, n, (torch.bfloat16,))
    B, H, d = q_t.shape
    out = out if out is not None else torch.empty((B, H, d), device=q_t.device, dtype=torch.float32)
    _check(L.fs_decode_step(_ptr(q_t), _ptr(k_t), _ptr(v_t), FS_BF16, B, H, d, int(t), _ptr(lam),
                            _ptr(sigma), _ptr(mix), ctypes.byref(p), _ptr(state),
                            state.numel() * state.element_size(), _ptr(out), _ptr(sel),
                            _stream(stream)), "fs_decode_step")
    return out


def fs_fsb_select(q, k, kbar, amax, lam, sigma, params=None, stream=None):
    """FS-B selection (beam search over the two forests, token rerank):
    sel [B,H,N,K] int32.  params.mode must be FS_MODE_FSB."""
    L = load()
    p = _params(params)
    for t_, n in ((q, "q"), (k, "k")):
        _dev(t_, n, (torch.bfloat16,))
    for t_, n in ((kbar, "kbar"), (amax, "amax"), (lam, "lam"), (sigma, "sigma")):
        _dev(t_, n, (torch.float32,))
    B, H, N, d = _qkv_shape(q)
    wsb = L.fs_fsb_workspace_bytes(B, H, N, ctypes.byref(p))
    if wsb == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_fsb_workspace_bytes")
    ws = torch.empty(wsb, device=q.device, dtype=torch.uint8)
    sel = torch.empty((B, H, N, p.K), device=q.device, dtype=torch.int32)
    _check(L.fs_fsb_select(_ptr(q), _ptr(k), _ptr(kbar), _ptr(amax), _ptr(lam), _ptr(sigma), B, H,
                           N, d, ctypes.byref(p), _ptr(sel), _ptr(ws), wsb, _stream(stream)),
           "fs_fsb_select")
    return sel


def fs_backward_workspace_bytes(batch, H, N, d=64, params=None) -> int:
    p = _params(params)
    return load().fs_backward_workspace_bytes(batch, H, N, d, ctypes.byref(p))


def fs_attention_bwd(q, k, v, lam, sigma, mix, dout, params=None, ws=None, stream=None):
    """Gradients of L = sum(dout * fs_attention_fwd(q, k, v, ...)) with the
    forward's selections held fixed.  Returns dq, dk, dv [B,H,N,d] f32 and
    dmix [H] f32."""
    L = load()
    p = _params(params)
    for t_, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t_, n, (torch.bfloat16,))
    _dev(dout, "dout", (torch.float32,))
    for t_, n in ((lam, "lam"), (sigma, "sigma"), (mix, "mix")):
        _dev(t_, n, (torch.float32,))
    B, H, N, d = _qkv_shape(q)
    wsb = L.fs_backward_workspace_bytes(B, H, N, d, ctypes.byref(p))
    if wsb == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_backward_workspace_bytes")
    if ws is None:
        ws = torch.empty(wsb, device=q.device, dtype=torch.uint8)
    dq, dk, dv = (torch.empty((B, H, N, d), device=q.device, dtype=torch.float32) for _ in range(3))
    dmix = torch.empty(H, device=q.device, dtype=torch.float32)
    _check(L.fs_attention_bwd(_ptr(q), _ptr(k), _ptr(v), FS_BF16, B, H, N, d, ctypes.byref(p),
                              _ptr(lam), _ptr(sigma), _ptr(mix), _ptr(dout), _ptr(dq), _ptr(dk),
                              _ptr(dv), _ptr(dmix), _ptr(ws), wsb, _stream(stream)),
           "fs_attention_bwd")
    return dq, dk, dv, dmix


def fs_qkv_workspace_bytes(batch, N, D, H) -> int:
    return load().fs_qkv_workspace_bytes(batch, N, D, H)


def fs_qkv_prologue(x, w_qkv, H, gain=None, eps=1e-6, q=None, k=None, v=None, ws=None,
                    stream=None):
    """RMSNorm(x) . w_qkv^T split into q, k, v [batch, H, N, 64] bf16.
    x [batch, N, D] bf16, w_qkv [3*H*64, D] bf16, gain [D] f32 or None."""
    L = load()
    _dev(x, "x", (torch.bfloat16,))
    _dev(w_qkv, "w_qkv", (torch.bfloat16,))
    if gain is not None:
        _dev(gain, "gain", (torch.float32,))
    B, N, D = x.shape
    if tuple(w_qkv.shape) != (3 * H * 64, D):
        raise ValueError(f"w_qkv must be [{3 * H * 64}, {D}]")
    outs = []
    for t_ in (q, k, v):
        t_ = t_ if t_ is not None else torch.empty((B, H, N, 64), device=x.device,
                                                   dtype=torch.bfloat16)
        _dev(t_, "q/k/v", (torch.bfloat16,))
        outs.append(t_)
    wsb = L.fs_qkv_workspace_bytes(B, N, D, H)
    if wsb == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_qkv_workspace_bytes")
    if ws is None:
        ws = torch.empty(wsb, device=x.device, dtype=torch.uint8)
    _check(L.fs_qkv_prologue(_ptr(x), _ptr(gain), _ptr(w_qkv), B, N, D, H, float(eps),
                             _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _ptr(ws), wsb,
                             _stream(stream)), "fs_qkv_prologue")
    return tuple(outs)


def fs_select_cells(q, kbar, amax, pool, pool_count, lam, sigma, params=None,
                    with_scores=False, stream=None):
    L = load()
    p = _params(params)
    _dev(q, "q", (torch.bfloat16,))
    B, H, N, d = _qkv_shape(q)
    for t, n in ((kbar, "kbar"), (amax, "amax"), (lam, "lam"), (sigma, "sigma")):
        _dev(t, n, (torch.float32,))
    if pool is not None:
        _dev(pool, "pool", (torch.int32,))
        _dev(pool_count, "pool_count", (torch.int32,))
    sel = torch.empty((B, H, N, p.K), device=q.device, dtype=torch.int32)
    score = torch.empty((B, H, N, p.K), device=q.device, dtype=torch.float32) if with_scores else None
    _check(L.fs_select_cells(_ptr(q), FS_BF16, _ptr(kbar), _ptr(amax), _ptr(pool),
                             _ptr(pool_count), _ptr(lam), _ptr(sigma), B, H, N, d,
                             ctypes.byref(p), _ptr(sel), _ptr(score), _stream(stream)),
           "fs_select_cells")
    return (sel, score) if with_scores else sel


def fs_sparse_readout(q, k, v, sel, params=None, o_long=None, stream=None):
    L = load()
    p = _params(params)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n, (torch.bfloat16,))
    _dev(sel, "sel", (torch.int32,))
    B, H, N, d = _qkv_shape(q)
    o_long = o_long if o_long is not None else torch.empty((B, H, N, d), device=q.device, dtype=torch.float32)
    _check(L.fs_sparse_readout(_ptr(q), _ptr(k), _ptr(v), FS_BF16, _ptr(sel), B, H, N, d,
                               ctypes.byref(p), _ptr(o_long), _stream(stream)), "fs_sparse_readout")
    return o_long


def fs_window_attn(q, k, v, o_long=None, mix=None, params=None, out=None, stream=None,
                   ws=None, events=None):
    """Window branch (and mix with ``o_long`` when given).  ``events``: None,
    or 3 torch.cuda.Event objects (enable_timing) recorded before the operand
    preparation, before the attention kernel and after it."""
    L = load()
    p = _params(params)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n, (torch.bfloat16,))
    B, H, N, d = _qkv_shape(q)
    if o_long is not None:
        _dev(o_long, "o_long", (torch.float32,))
        _dev(mix, "mix", (torch.float32,))
    out = out if out is not None else torch.empty((B, H, N, d), device=q.device, dtype=torch.float32)
    wsb = L.fs_window_workspace_bytes(B, H, N, d, ctypes.byref(p))
    if wsb == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_window_workspace_bytes")
    if ws is None:
        ws = torch.empty(wsb, device=q.device, dtype=torch.uint8)
    elif ws.numel() * ws.element_size() < wsb:
        raise ValueError(f"workspace too small: {ws.numel()} < {wsb} bytes")
    args = [_ptr(q), _ptr(k), _ptr(v), FS_BF16, _ptr(o_long), _ptr(mix), B, H, N, d,
            ctypes.byref(p), _ptr(out), _ptr(ws), wsb, _stream(stream)]
    if events is None:
        _check(L.fs_window_attn(*args), "fs_window_attn")
    else:
        if len(events) != 3:
            raise ValueError("need 3 events")
        _check(L.fs_window_attn_traced(*args, _event_array(events)), "fs_window_attn_traced")
    return out


def _event_array(events):
    for e in events:
        if e.cuda_event == 0:  # torch creates the CUDA event lazily
            e.record()
    return (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])


def fs_attention_fwd(q, k, v, lam, sigma, mix, params=None, out=None, ws=None, stream=None):
    """Whole FS-L (or FS) forward.  Returns ``out`` [batch, H, N, d] fp32."""
    L = load()
    p = _params(params)
    dt = (torch.bfloat16, torch.float32)
    _dev(q, "q", dt)
    _dev(k, "k", (q.dtype,))
    _dev(v, "v", (q.dtype,))
    for t, n in ((lam, "lam"), (sigma, "sigma"), (mix, "mix")):
        _dev(t, n, (torch.float32,))
    B, H, N, d = _qkv_shape(q)
    code = _dtype_code(q)
    wsb = L.fs_workspace_bytes(B, H, N, d, ctypes.byref(p), code)
    if wsb == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_workspace_bytes")
    if ws is None:
        ws = torch.empty(wsb, device=q.device, dtype=torch.uint8)
    elif ws.numel() * ws.element_size() < wsb:
        raise ValueError(f"workspace too small: {ws.numel()} < {wsb} bytes")
    out = out if out is not None else torch.empty((B, H, N, d), device=q.device, dtype=torch.float32)
    _dev(out, "out", (torch.float32,))
    _check(L.fs_attention_fwd(_ptr(q), _ptr(k), _ptr(v), code, B, H, N, d, ctypes.byref(p),
                              _ptr(lam), _ptr(sigma), _ptr(mix), _ptr(out), _ptr(ws), wsb,
                              _stream(stream)), "fs_attention_fwd")
    return out


def fs_host_workspace_bytes(batch, H, N, d, params=None, dtype=FS_BF16, heads_per_chunk=2) -> int:
    p = _params(params)
    return load().fs_host_workspace_bytes(batch, H, N, d, ctypes.byref(p), dtype, heads_per_chunk)


def _host(t, name, dtypes):
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fs_attention_fwd_host(q, k, v, lam, sigma, mix, params=None, out=None, ws=None,
                          heads_per_chunk=2, stream=None):
    """fs_attention_fwd on host tensors q, k, v [batch, H, N, d] (pinned memory
    lets the copies overlap the compute); lam, sigma, mix are device tensors.
    Returns ``out`` [batch, H, N, d] fp32 on the host, readable after the
    stream is synchronised."""
    L = load()
    p = _params(params)
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        _host(t, nm, (torch.bfloat16, torch.float32))
    if not (q.dtype == k.dtype == v.dtype) or q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k, v must share dtype and shape")
    for t, nm in ((lam, "lam"), (sigma, "sigma"), (mix, "mix")):
        _dev(t, nm, (torch.float32,))
    B, H, N, d = _qkv_shape(q)
    code = FS_FP32 if q.dtype == torch.float32 else FS_BF16
    wsb = L.fs_host_workspace_bytes(B, H, N, d, ctypes.byref(p), code, heads_per_chunk)
    if wsb == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_host_workspace_bytes")
    dev = lam.device
    if ws is None:
        ws = torch.empty(wsb, device=dev, dtype=torch.uint8)
    elif ws.numel() * ws.element_size() < wsb:
        raise ValueError(f"workspace too small: {ws.numel()} < {wsb} bytes")
    if out is None:
        out = torch.empty((B, H, N, d), dtype=torch.float32, pin_memory=True)
    _host(out, "out", (torch.float32,))
    _check(L.fs_attention_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), code, B, H, N, d,
                                   ctypes.byref(p), _ptr(lam), _ptr(sigma), _ptr(mix),
                                   out.data_ptr(), heads_per_chunk, _ptr(ws), wsb,
                                   _stream(stream)), "fs_attention_fwd_host")
    return out


def fs_attention_fwd_traced(q, k, v, lam, sigma, mix, events, params=None, out=None, ws=None,
                            stream=None):
    """fs_attention_fwd recording ``events`` (FS_N_STAGES + 1 torch.cuda.Event
    objects, created with enable_timing) between its stages on the stream."""
    L = load()
    p = _params(params)
    if len(events) != FS_N_STAGES + 1:
        raise ValueError(f"need {FS_N_STAGES + 1} events")
    B, H, N, d = _qkv_shape(q)
    code = _dtype_code(q)
    wsb = L.fs_workspace_bytes(B, H, N, d, ctypes.byref(p), code)
    if wsb == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_workspace_bytes")
    if ws is None:
        ws = torch.empty(wsb, device=q.device, dtype=torch.uint8)
    elif ws.numel() * ws.element_size() < wsb:
        raise ValueError("workspace too small")
    out = out if out is not None else torch.empty((B, H, N, d), device=q.device, dtype=torch.float32)
    arr = _event_array(events)
    _check(L.fs_attention_fwd_traced(_ptr(q), _ptr(k), _ptr(v), code, B, H, N, d,
                                     ctypes.byref(p), _ptr(lam), _ptr(sigma), _ptr(mix),
                                     _ptr(out), _ptr(ws), wsb, _stream(stream), arr),
           "fs_attention_fwd_traced")
    return out


def fs_workspace_view(ws, batch, H, N, d, params=None, dtype=FS_BF16):
    """Views of the intermediates an fs_attention_fwd call left in ``ws``:
    dict with kbar, amax, pool, pool_count, sel."""
    L = load()
    p = _params(params)
    offs = [ctypes.c_size_t() for _ in range(5)]
    _check(L.fs_workspace_view(batch, H, N, d, ctypes.byref(p), dtype,
                               *[ctypes.byref(o) for o in offs]), "fs_workspace_view")
    C, nblk = N // p.s, N // p.Bq
    spec = [("kbar", (batch, H, C, d), torch.float32), ("amax", (batch, H, C), torch.float32),
            ("pool", (batch, H, nblk, p.P + p.W), torch.int32),
            ("pool_count", (batch, H, nblk), torch.int32),
            ("sel", (batch, H, N, p.K), torch.int32)]
    res = {}
    for (name, shape, dtype_), off in zip(spec, offs):
        n = 1
        for x in shape:
            n *= x
        nbytes = n * torch.tensor([], dtype=dtype_).element_size()
        res[name] = ws[off.value: off.value + nbytes].view(dtype_).view(shape)
    return res


def fs_set_attention_timeline(buf=None):
    """Record each CTA's start and end (device global timer, ns) of the calling
    thread's following attention launches into ``buf`` (a CUDA int64 tensor,
    two entries per CTA); ``None`` turns it off."""
    global _timeline_buf
    L = load()
    if buf is None:
        _check(L.fs_set_attention_timeline(None, 0), "fs_set_attention_timeline")
        _timeline_buf = None
        return
    if not (buf.is_cuda and buf.dtype == torch.int64 and buf.is_contiguous()):
        raise ValueError("timeline must be a contiguous CUDA int64 tensor")
    _check(L.fs_set_attention_timeline(_ptr(buf), buf.numel()), "fs_set_attention_timeline")
    _timeline_buf = buf  # the library keeps only the pointer: keep the memory alive


_timeline_buf = None


def fs_check_status(ws, stream=None):
    """Synchronise the stream and raise FSError if a kernel recorded an error
    (a bounded device wait that timed out) in the workspace header."""
    _check(load().fs_check_status(_ptr(ws), _stream(stream)), "fs_check_status")


# ---------------------------------------------------------------------------
# rotary positions, the paged cache, attention of drafted tokens
# ---------------------------------------------------------------------------

_Strides = ctypes.c_longlong * 3
_INT_MAX = 2 ** 31 - 1  # (ctypes would take the low 32 bits of more)


def _on(t, dev, name, dtype, shape=None):
    """Pointer of ``t``, a CUDA tensor of ``dtype`` on ``dev``, contiguous in ``shape`` when given."""
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and (t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous {list(shape)}, not {list(t.shape)}")
    return t.data_ptr()


def _rows(t, dev, name, dtype, shape):
    """Pointer and strides (None: contiguous) of a [batch, H, N, d] tensor of ``shape`` whose d
    values lie together."""
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), None
    a, b, c, e = t.stride()
    if e != 1 and shape[3] > 1:
        raise ValueError(f"{name}: the values of a head must be contiguous")
    return t.data_ptr(), _Strides(a, b, c)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _launch(dev, stream, fn, where, *args):
    """Calls ``fn`` for device ``dev`` on ``stream`` (default: the device's current one)."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev.index)
    elif stream.device != dev:
        raise ValueError(f"{where}: the stream is on {stream.device}, the tensors on {dev}")
    else:
        raw = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev.index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, raw)
    if rc != FS_OK:
        raise FSError(rc, where)


def _new(stream, make):
    """What ``make`` allocates, for use on ``stream`` (None: the current one)."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def fs_rope_plan(rot, layout="half", scaling="none", base=10000.0, factor=1.0, original=4096,
                 beta_fast=32.0, beta_slow=1.0, amplitude=1.0):
    """A model's rotary frequencies, worked out once on the host (fs_rope_make_plan):
    ``rot`` rotated elements of a head, ``layout`` "half" or "pairs", ``scaling`` "none",
    "linear", "base" or "ramp" by ``factor``."""
    if layout not in FS_ROPE_LAYOUTS or scaling not in FS_ROPE_SCALINGS:
        raise ValueError(f"unknown layout {layout!r} or scaling {scaling!r}")
    if max(int(rot), int(original)) > _INT_MAX or min(int(rot), int(original)) < -_INT_MAX:
        raise ValueError(f"rot {rot} or original {original} does not fit 32 bits")
    p = fs_rope_params(int(rot), FS_ROPE_LAYOUTS[layout], FS_ROPE_SCALINGS[scaling], int(original),
                       base, factor, beta_fast, beta_slow, amplitude)
    plan = fs_rope_plan_t()
    _check(load().fs_rope_make_plan(ctypes.byref(p), ctypes.byref(plan)), "fs_rope_make_plan")
    return plan


def fs_rope(q, k, pos, plan, inverse=False, q_out=None, k_out=None, stream=None):
    """Rotates q [batch, Hq, N, d] and k [batch, Hk, N, d] (k None: q alone), bf16 or fp32, any
    strides with the d values together, to the positions ``pos``: int32 [batch, N] or [N], or an
    int for positions pos, pos + 1, ...  ``inverse`` applies the transposed rotation, which takes
    the outputs' gradients to the inputs'.  ``q_out`` / ``k_out`` may be the inputs (in place).
    Returns (q_out, k_out)."""
    L = _lib or load()
    dev, dt = _cuda(q, "q"), q.dtype
    if dt is torch.bfloat16:
        code = FS_BF16
    elif dt is torch.float32:
        code = FS_FP32
    else:
        raise ValueError(f"q has dtype {dt}, expected bfloat16 or float32")
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [batch, Hq, N, d]")
    B, Hq, N, d = shape
    qp, qs = _rows(q, dev, "q", dt, shape)
    if q_out is None:
        q_out = _new(stream, lambda: torch.empty_like(q))
        qop, qos = (q_out.data_ptr(), None) if qs is None else _rows(q_out, dev, "q_out", dt, shape)
    else:
        qop, qos = _rows(q_out, dev, "q_out", dt, shape)
    kp = ks = kop = kos = None
    Hk = 0
    if k is not None:
        Hk = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
        shape = (B, Hk, N, d)
        kp, ks = _rows(k, dev, "k", dt, shape)
        if k_out is None:
            k_out = _new(stream, lambda: torch.empty_like(k))
            kop, kos = (k_out.data_ptr(), None) if ks is None else \
                _rows(k_out, dev, "k_out", dt, shape)
        else:
            kop, kos = _rows(k_out, dev, "k_out", dt, shape)
    pp, stride, pos0 = None, 0, 0
    if isinstance(pos, int):
        if not -2 ** 31 <= pos < 2 ** 31:
            raise ValueError(f"pos {pos} does not fit 32 bits")
        pos0 = pos
    elif isinstance(pos, torch.Tensor) and pos.dim() == 2:
        stride = N
        pp = _on(pos, dev, "pos", torch.int32, (B, N))
    else:
        pp = _on(pos, dev, "pos", torch.int32, (N,))
    _launch(dev, stream, L.fs_rope, "fs_rope", qp, qop, Hq, qs, qos, kp, kop, Hk, ks, kos, code, B,
            N, d, pp, stride, pos0, plan, 1 if inverse else 0)
    return q_out, k_out


class fs_cache:
    """A paged key/value cache: ``codes`` [pages, 2, Hkv, page, row bytes] uint8, ``scales``
    [pages, 2, Hkv, page] fp32 (ignored for "bf16"), ``table`` [batch, max_pages] int32 and the
    ``format`` ("bf16", "e4m3", "int8", "int4").  Holds the tensors; ``status`` is its error word
    (``fs_check_status(cache.status)`` raises if a call met a page or position outside)."""

    def __init__(self, codes, scales, table, format, status=None):
        if format not in FS_CACHE_FORMATS:
            raise ValueError(f"unknown cache format {format!r}")
        dev = _cuda(codes, "codes")
        if codes.dim() != 5 or codes.shape[1] != 2:
            raise ValueError("codes must be [pages, 2, Hkv, page, row bytes]")
        pages, _, Hkv, page, row = codes.shape
        cp = _on(codes, dev, "codes", torch.uint8, codes.shape)
        d = {"bf16": row // 2, "int4": row * 2}.get(format, row)
        if load().fs_cache_row_bytes(d, FS_CACHE_FORMATS[format]) != row:
            raise FSError(FS_ERR_UNSUPPORTED, "fs_cache")
        sp = None
        if format != "bf16":
            sp = _on(scales, dev, "scales", torch.float32, (pages, 2, Hkv, page))
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table must be [batch, max_pages]")
        tp = _on(table, dev, "table", torch.int32, table.shape)
        self.status = torch.zeros(64, dtype=torch.int32, device=dev) if status is None else status
        st = _on(self.status, dev, "status", torch.int32)
        self.codes, self.scales, self.table, self.format = codes, scales, table, format
        self.device, self.batch, self.Hkv, self.page, self.d = dev, table.shape[0], Hkv, page, d
        self.desc = fs_cache_t(cp, sp, tp, st, pages, page, Hkv, d, FS_CACHE_FORMATS[format],
                               table.shape[0], table.shape[1])


def fs_cache_alloc(pages, Hkv, page, d, format, table):
    """An empty ``fs_cache`` of ``pages`` pages on the device of ``table``."""
    if format not in FS_CACHE_FORMATS:
        raise ValueError(f"unknown cache format {format!r}")
    row = load().fs_cache_row_bytes(d, FS_CACHE_FORMATS[format])
    if row == 0:
        raise FSError(FS_ERR_UNSUPPORTED, "fs_cache_alloc")
    dev = _cuda(table, "table")
    codes = torch.zeros((pages, 2, Hkv, page, row), dtype=torch.uint8, device=dev)
    scales = None if format == "bf16" else torch.zeros((pages, 2, Hkv, page), device=dev)
    return fs_cache(codes, scales, table, format)


def _counts(cache, name, t):
    return None if t is None else _on(t, cache.device, name, torch.int32, (cache.batch,))


def fs_cache_append(cache, k, v, start, count=None, stream=None):
    """Writes k, v [batch, Hkv, T, d] bf16 (any 16-byte aligned strides) at positions
    start[b] .. start[b] + count[b] - 1 of every sequence (``count`` None: T)."""
    L = _lib or load()
    T = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
    shape = (cache.batch, cache.Hkv, T, cache.d)
    kp, ks = _rows(k, cache.device, "k", torch.bfloat16, shape)
    vp, vs = _rows(v, cache.device, "v", torch.bfloat16, shape)
    if start is None:
        raise ValueError("start must be given")
    _launch(cache.device, stream, L.fs_cache_append, "fs_cache_append", cache.desc, kp, vp, ks, vs,
            T, _counts(cache, "start", start), _counts(cache, "count", count))


def fs_cache_read(cache, start, count=None, k=None, v=None, T=None, dtype=torch.bfloat16,
                  stream=None):
    """Reads positions start[b] .. start[b] + count[b] - 1 of every sequence into k, v
    [batch, Hkv, T, d] (given, or new zeros of ``T`` rows in ``dtype``); rows past count[b] are
    left as they were.  Returns (k, v)."""
    L = _lib or load()
    if (k is None) != (v is None) or (k is None and T is None):
        raise ValueError("give k and v, or T")
    if k is None:
        k, v = _new(stream, lambda: torch.zeros((2, cache.batch, cache.Hkv, T, cache.d), dtype=dtype,
                                                device=cache.device)).unbind(0)
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or \
            k.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("k must be [batch, Hkv, T, d], bfloat16 or float32")
    shape = (cache.batch, cache.Hkv, k.shape[2], cache.d)
    kp = _on(k, cache.device, "k", k.dtype, shape)
    vp = _on(v, cache.device, "v", k.dtype, shape)
    if start is None:
        raise ValueError("start must be given")
    _launch(cache.device, stream, L.fs_cache_read, "fs_cache_read", cache.desc,
            _counts(cache, "start", start), _counts(cache, "count", count), k.shape[2],
            FS_BF16 if k.dtype == torch.bfloat16 else FS_FP32, kp, vp)
    return k, v


def fs_cache_accept(cache, start, path, count=None, stream=None):
    """Moves the row at start[b] + path[b, i] to start[b] + i for i < count[b] (``path``
    [batch, A <= 64] int32), every source read before any row is written."""
    L = _lib or load()
    if not isinstance(path, torch.Tensor) or path.dim() != 2 or start is None:
        raise ValueError("path must be [batch, A], start given")
    pp = _on(path, cache.device, "path", torch.int32, (cache.batch, path.shape[1]))
    _launch(cache.device, stream, L.fs_cache_accept, "fs_cache_accept", cache.desc,
            _counts(cache, "start", start), pp, _counts(cache, "count", count), path.shape[1])


def fs_tree_workspace(cache, batch, H, T):
    """A workspace for fs_tree_attn of this shape (one call at a time)."""
    if batch != cache.batch:
        raise ValueError(f"batch {batch}, but the cache's table has {cache.batch} sequences")
    n = load().fs_tree_workspace_bytes(cache.desc, H, T)
    if n == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_tree_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def fs_tree_attn(q, cache, past, tree=None, count=None, window=0, scale=None, out=None, ws=None,
                 stream=None):
    """Attention of drafted tokens q [batch, H, T <= 64, d] bf16, whose keys and values lie behind
    the past[b] tokens of the prefix in ``cache``.  ``tree`` [batch, T] int64: bit j of row i lets
    drafted token i see drafted token j (None: every token sees the drafted ones up to itself);
    ``count`` [batch]: drafted tokens of each sequence (None: T); ``window`` 0 or >= 64 last
    positions; ``scale`` default d ** -0.5.  Returns out [batch, H, T, d] bf16; rows past count[b]
    are left as they were (a new ``out`` starts as zeros when ``count`` is given)."""
    return _tree_attn((_lib or load()).fs_tree_attn, "fs_tree_attn", (), q, cache, past, tree, count,
                      window, scale, out, ws, stream)


def fs_selftest_tree_wait(q, cache, past, cycles, tree=None, count=None, window=0, scale=None,
                          out=None, ws=None, stream=None):
    """fs_tree_attn whose waits give up after ``cycles`` SM cycles (FS_ERR_TIMEOUT in
    ``cache.status``)."""
    return _tree_attn((_lib or load()).fs_selftest_tree_wait, "fs_selftest_tree_wait", (int(cycles),),
                      q, cache, past, tree, count, window, scale, out, ws, stream)


def _tree_attn(fn, where, more, q, cache, past, tree, count, window, scale, out, ws, stream):
    dev = cache.device
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be [batch, H, T, d]")
    B, H, T, d = q.shape
    qp = _on(q, dev, "q", torch.bfloat16, (cache.batch, H, T, cache.d))
    if past is None:
        raise ValueError("past must be given")
    tp = None if tree is None else _on(tree, dev, "tree", torch.int64, (B, T))
    if out is None:
        out = _new(stream, lambda: torch.empty_like(q) if count is None else torch.zeros_like(q))
    op = _on(out, dev, "out", torch.bfloat16, q.shape)
    if ws is None:
        ws = _new(stream, lambda: fs_tree_workspace(cache, B, H, T))
    wp = _on(ws, dev, "ws", torch.uint8)
    if not ws.is_contiguous():  # its bytes would not be ws.numel() bytes of memory
        raise ValueError("ws must be contiguous")
    _launch(dev, stream, fn, where, qp, cache.desc, _counts(cache, "past", past),
            _counts(cache, "count", count), tp, H, T, max(-1, min(int(window), _INT_MAX)),
            d ** -0.5 if scale is None else float(scale), op, wp, ws.numel(), *more)
    return out


# ---------------------------------------------------------------------------
# linear attention with a decay for each head, the norms around a block
# ---------------------------------------------------------------------------

def _scratch(ws, dev):
    """Pointer and bytes of a workspace."""
    p = _on(ws, dev, "ws", torch.uint8)
    if not ws.is_contiguous():  # its bytes would not be ws.numel() bytes of memory
        raise ValueError("ws must be contiguous")
    return p, ws.numel()


def fs_linear_workspace(batch, H, Hkv, T, d, device, backward=False):
    """A workspace for fs_linear_attn (or, ``backward``, fs_linear_attn_bwd) of this shape, or of a smaller
    batch or T, one call at a time; ``fs_check_status(ws)`` raises if a bounded wait of a call gave up."""
    if max(batch, H, Hkv, T, d) > _INT_MAX:
        raise ValueError("a size does not fit 32 bits")
    n = load().fs_linear_workspace_bytes(batch, H, Hkv, T, d, 1 if backward else 0)
    if n == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_linear_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()  # the error word, which no call clears
    return ws


def _linear_inputs(q, k, v, decay, count):
    dev, shape = _cuda(q, "q"), q.shape
    if len(shape) != 4:
        raise ValueError("q must be [batch, H, T, d]")
    B, H, T, d = shape
    qp, qs = _rows(q, dev, "q", torch.bfloat16, shape)
    Hkv = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
    if max(B, H, Hkv, T) > _INT_MAX:  # (expanded axes; ctypes would take their low 32 bits)
        raise ValueError("a size does not fit 32 bits")
    shape = (B, Hkv, T, d)
    kp, ks = _rows(k, dev, "k", torch.bfloat16, shape)
    vp, vs = _rows(v, dev, "v", torch.bfloat16, shape)
    gp = _on(decay, dev, "decay", torch.float32, (H,))
    cp = None if count is None else _on(count, dev, "count", torch.int32, (B,))
    return dev, Hkv, (qp, kp, vp, qs, ks, vs, gp, B, H, Hkv, T, d, cp)


def fs_linear_attn(q, k, v, decay, state=None, state_out=None, count=None, scale=None, out=None,
                   ws=None, stream=None):
    """Linear attention with a decay for each head: S = exp(decay) S + k v^T, out = scale q S, token
    after token.  q [batch, H, T, d], k, v [batch, Hkv, T, d] bf16, any 16-byte aligned strides with
    the d values together; ``decay`` [H] fp32, 0 or below; ``state`` [batch, H, d, d] fp32 before the
    first token (None: zeros); ``state_out`` receives the one after the last (may be ``state``);
    ``count`` [batch]: tokens of each sequence (None: T); ``scale`` default d ** -0.5.  T = 1 is a
    decoding step.  Returns out [batch, H, T, d] bf16; rows past count[b] are left as they were (a
    new ``out`` starts as zeros when ``count`` is given)."""
    return _linear_attn((_lib or load()).fs_linear_attn, "fs_linear_attn", (), q, k, v, decay, state,
                        state_out, count, scale, out, ws, stream)


def fs_selftest_linear_wait(q, k, v, decay, cycles, state=None, state_out=None, count=None, scale=None,
                            out=None, ws=None, stream=None):
    """fs_linear_attn whose waits give up after ``cycles`` SM cycles (FS_ERR_TIMEOUT in ``ws``)."""
    return _linear_attn((_lib or load()).fs_selftest_linear_wait, "fs_selftest_linear_wait", (int(cycles),),
                        q, k, v, decay, state, state_out, count, scale, out, ws, stream)


def _linear_attn(fn, where, more, q, k, v, decay, state, state_out, count, scale, out, ws, stream):
    dev, Hkv, args = _linear_inputs(q, k, v, decay, count)
    B, H, T, d = q.shape
    if out is None:
        out = _new(stream, lambda: torch.empty_like(q, memory_format=torch.contiguous_format)
                   if count is None else torch.zeros_like(q, memory_format=torch.contiguous_format))
    op, os_ = _rows(out, dev, "out", torch.bfloat16, q.shape)
    shape = (B, H, d, d)
    sp = None if state is None else _on(state, dev, "state", torch.float32, shape)
    tp = None if state_out is None else _on(state_out, dev, "state_out", torch.float32, shape)
    wp, wn = None, 0
    if ws is None and T > FS_LINEAR_STEPS:
        ws = _new(stream, lambda: fs_linear_workspace(B, H, Hkv, T, d, dev))
    if ws is not None:
        wp, wn = _scratch(ws, dev)
    _launch(dev, stream, fn, where, *args, d ** -0.5 if scale is None else float(scale), sp, tp, op, os_,
            wp, wn, *more)
    return out


def fs_linear_attn_bwd(q, k, v, decay, dout, state=None, dstate_out=None, count=None, scale=None,
                       dq=None, dk=None, dv=None, dstate=None, ws=None, stream=None):
    """Gradients of sum(dout * out) + sum(dstate_out * state_out) of fs_linear_attn: dq, dk and dv
    (bf16, as q, k and v), and the gradient of ``state`` into ``dstate`` [batch, H, d, d] fp32 where
    that is given.  Rows past count[b] are left as they were (new tensors start as zeros when
    ``count`` is given).  Returns (dq, dk, dv)."""
    return _linear_attn_bwd((_lib or load()).fs_linear_attn_bwd, "fs_linear_attn_bwd", (), q, k, v, decay, dout,
                            state, dstate_out, count, scale, dq, dk, dv, dstate, ws, stream)


def fs_selftest_linear_wait_bwd(q, k, v, decay, dout, cycles, state=None, dstate_out=None, count=None,
                                scale=None, dq=None, dk=None, dv=None, dstate=None, ws=None, stream=None):
    """fs_linear_attn_bwd whose waits give up after ``cycles`` SM cycles (FS_ERR_TIMEOUT in ``ws``)."""
    return _linear_attn_bwd((_lib or load()).fs_selftest_linear_wait_bwd, "fs_selftest_linear_wait_bwd",
                            (int(cycles),), q, k, v, decay, dout, state, dstate_out, count, scale, dq, dk, dv,
                            dstate, ws, stream)


def _linear_attn_bwd(fn, where, more, q, k, v, decay, dout, state, dstate_out, count, scale, dq, dk, dv,
                     dstate, ws, stream):
    dev, Hkv, args = _linear_inputs(q, k, v, decay, count)
    B, H, T, d = q.shape
    dp, ds = _rows(dout, dev, "dout", torch.bfloat16, q.shape)
    grads, ptrs, strides = [], [], []
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is None:
            t = _new(stream, lambda: torch.empty_like(like, memory_format=torch.contiguous_format)
                     if count is None else
                     torch.zeros_like(like, memory_format=torch.contiguous_format))
        p, s = _rows(t, dev, name, torch.bfloat16, like.shape)
        grads.append(t), ptrs.append(p), strides.append(s)
    shape = (B, H, d, d)
    sp, gp, tp = (None if t is None else _on(t, dev, name, torch.float32, shape) for name, t in
                  (("state", state), ("dstate_out", dstate_out), ("dstate", dstate)))
    if ws is None:
        ws = _new(stream, lambda: fs_linear_workspace(B, H, Hkv, T, d, dev, backward=True))
    wp, wn = _scratch(ws, dev)
    _launch(dev, stream, fn, where, *args, d ** -0.5 if scale is None else float(scale), sp, dp, ds, gp,
            *ptrs, *strides, tp, wp, wn, *more)
    return tuple(grads)


def _matrix(t, dev, name, dtype, shape):
    """Pointer and row stride of a [..., D] tensor of ``shape`` whose rows lie evenly apart."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev \
            and t.is_contiguous():
        return t.data_ptr(), shape[-1]
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    axes = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n > 1]
    for (_, outer), (n, inner) in zip(axes, axes[1:]):
        if outer != n * inner:
            raise ValueError(f"{name}: its rows must lie evenly apart, as a matrix's do")
    return t.data_ptr(), axes[-1][1] if axes else shape[-1]


_NORM_CODES = {torch.bfloat16: FS_BF16, torch.float32: FS_FP32}


def _like(t, dtype, stream):
    """A new contiguous tensor of t's shape."""
    if stream is None and t.dtype is dtype and t.is_contiguous():
        return torch.empty_like(t)
    return _new(stream, lambda: torch.empty(t.shape, dtype=dtype, device=t.device))


def _norm_inputs(x, gate, residual, gain, next_gain, groups, res_dtype):
    dev, dt = _cuda(x, "x"), x.dtype
    code, res_code = _NORM_CODES.get(dt), _NORM_CODES.get(res_dtype)
    if code is None or res_code is None:
        raise ValueError(f"x has dtype {dt}, the residual {res_dtype}: expected bfloat16 or float32")
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError("x must be [..., D]")
    D = shape[-1]
    M = x.numel() // D
    if M > _INT_MAX or not -_INT_MAX <= groups <= _INT_MAX:
        raise ValueError("a size does not fit 32 bits")
    xp, xs = _matrix(x, dev, "x", dt, shape)
    gp, gs = (None, 0) if gate is None else _matrix(gate, dev, "gate", dt, shape)
    rp, rs = (None, 0) if residual is None else _matrix(residual, dev, "residual", res_dtype, shape)
    a = None if gain is None else _on(gain, dev, "gain", torch.float32, (D,))
    b = None if next_gain is None else _on(next_gain, dev, "next_gain", torch.float32, (D,))
    return dev, (xp, xs, code, gp, gs, rp, rs, res_code, a, b, M, D, groups)


def fs_block_norm(x, gate=None, residual=None, groups=0, gain=None, next_norm=False, next_gain=None,
                  scale=1.0, eps=1e-6, z=None, y=None, stream=None):
    """The norms after and before a block, its gate and its residual scale, for x [..., D]:
    a = x, RMS-normalised in ``groups`` groups of its row (0: not), times ``gain`` [D] fp32, times
    silu(``gate``); z = ``residual`` + ``scale`` a; y = z RMS-normalised, times ``next_gain``
    (``next_norm``, or a given ``y``).  x, gate and y are bf16 or fp32, residual and z bf16 or fp32 of
    their own (z without a residual: x's type, or a given ``z``'s).  z may be x or the residual, y
    may be x or gate (in place).  Returns (z, y), y None without the second norm."""
    L = _lib or load()
    res_dtype = residual.dtype if residual is not None else z.dtype if z is not None else x.dtype
    dev, args = _norm_inputs(x, gate, residual, gain, next_gain, groups, res_dtype)
    if z is None:
        z = _like(x if residual is None else residual, res_dtype, stream)
        zp, zs = z.data_ptr(), args[11]
    else:
        zp, zs = _matrix(z, dev, "z", res_dtype, x.shape)
    yp, ys = None, 0
    if y is not None:
        yp, ys = _matrix(y, dev, "y", x.dtype, x.shape)
    elif next_norm:
        y = _like(x, x.dtype, stream)
        yp, ys = y.data_ptr(), args[11]
    elif next_gain is not None:
        raise ValueError("next_gain without next_norm")
    _launch(dev, stream, L.fs_block_norm, "fs_block_norm", *args, scale, eps, zp, zs, yp, ys)
    return z, y


def fs_block_norm_workspace(M, D, device):
    """A workspace for fs_block_norm_bwd of M rows of D elements (one call at a time)."""
    if max(M, D) > _INT_MAX:
        raise ValueError("a size does not fit 32 bits")
    n = load().fs_block_norm_workspace_bytes(M, D)
    if n == 0:
        raise FSError(FS_ERR_INVALID_ARG, "fs_block_norm_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def fs_block_norm_bwd(x, dz=None, dy=None, gate=None, residual=None, groups=0, gain=None,
                      next_gain=None, scale=1.0, eps=1e-6, dx=None, dgate=None, dresidual=None,
                      ws=None, stream=None):
    """Gradients of sum(dz * z) + sum(dy * y) of fs_block_norm with the same x, gate, residual,
    groups, gains, scale and eps (``dy`` None: without the second norm).  Returns a dict of the
    gradients of "x", "gate", "residual", "gain" and "next_gain", None where there is no such input.
    dx may be x or dy, dgate may be gate, dresidual may be dz or residual (in place)."""
    L = _lib or load()
    if dz is None and dy is None:
        raise ValueError("give dz or dy")
    res_dtype = residual.dtype if residual is not None else dz.dtype if dz is not None else x.dtype
    dev, args = _norm_inputs(x, gate, residual, gain, next_gain, groups, res_dtype)
    shape, M, D = x.shape, args[10], args[11]
    if dy is None and next_gain is not None:
        raise ValueError("next_gain without dy")
    dzp, dzs = (None, 0) if dz is None else _matrix(dz, dev, "dz", res_dtype, shape)
    dyp, dys = (None, 0) if dy is None else _matrix(dy, dev, "dy", x.dtype, shape)
    grads = []
    for name, t, of, dt in (("dx", dx, x, x.dtype), ("dgate", dgate, gate, x.dtype),
                            ("dresidual", dresidual, residual, res_dtype)):
        if of is None:
            if t is not None:
                raise ValueError(f"{name} without its input")
            grads.append((None, None, 0))
            continue
        if t is None:
            t = _like(of, dt, stream)
            grads.append((t, t.data_ptr(), D))
        else:
            grads.append((t, *_matrix(t, dev, name, dt, shape)))
    sums = [None if t is None else
            _new(stream, lambda: torch.empty(D, dtype=torch.float32, device=dev))
            for t in (gain, next_gain)]
    wp, wn = None, 0
    if gain is not None or next_gain is not None:
        if ws is None:
            ws = _new(stream, lambda: fs_block_norm_workspace(M, D, dev))
        wp, wn = _scratch(ws, dev)
    _launch(dev, stream, L.fs_block_norm_bwd, "fs_block_norm_bwd", *args, scale, eps, dzp,
            dzs, dyp, dys, *(x for _, p, s in grads for x in (p, s)),
            *(None if t is None else t.data_ptr() for t in sums), wp, wn)
    return {"x": grads[0][0], "gate": grads[1][0], "residual": grads[2][0], "gain": sums[0],
            "next_gain": sums[1]}
