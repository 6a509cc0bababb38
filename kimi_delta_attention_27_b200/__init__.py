"""B200 (sm_100a) Kimi Delta Attention library (prefill, backward, decode, and the operators around the
recurrence: short convolution, q/k norm and rotation, selective scan): Python binding.

The work happens in ``libkda.so`` (hand-written CUDA kernels behind the C ABI
declared in ``include/kda.h``). This module only marshals torch tensors into
that ABI: pointers, sizes, dtype codes and the current CUDA stream. There is
no fallback: if the library is missing or the tensors are not on a CUDA
device, the call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkda.so")

# entry points declared in include/kda.h
EXPORTS = ("kda_bwd", "kda_bwd_workspace", "kda_conv_bwd", "kda_conv_bwd_workspace", "kda_conv_decode",
           "kda_conv_fwd", "kda_decode", "kda_device_error", "kda_fwd", "kda_fwd_ex", "kda_fwd_noalloc",
           "kda_fwd_segmented", "kda_fwd_segmented_workspace", "kda_qk_bwd", "kda_qk_bwd_workspace", "kda_qk_fwd",
           "kda_scan_bwd", "kda_scan_bwd_workspace", "kda_scan_decode", "kda_scan_fwd", "kda_scan_fwd_workspace",
           "kda_status_string", "kda_version")

# kda_fwd_ex gate kinds and flags (include/kda.h)
KDA_GATE_FP32, KDA_GATE_BF16, KDA_GATE_SCALAR_FP32 = 0, 1, 2
KDA_FLAG_L2NORM_QK, KDA_FLAG_GATE_LOGSIGMOID = 1, 2

# kda_conv_*, kda_scan_* flags and kda_qk_* norm kinds (include/kda.h)
KDA_FLAG_CONV_SILU, KDA_FLAG_SCAN_SOFTPLUS = 1, 1
NORM_KINDS = {"none": 0, "l2": 1, "rms": 2}

# (sequence, head) pairs per kda_fwd_noalloc call (KDA_NOALLOC_MAX_UNITS in include/kda.h)
NOALLOC_MAX_UNITS = 32

KDA_DTYPE_NONE, KDA_DTYPE_BF16, KDA_DTYPE_FP32 = 0, 1, 2

_HERE = contextlib.nullcontext()
_lock = threading.Lock()
_lib = None


class KdaError(RuntimeError):
    """A non-zero kda_status returned by the library."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def load_library(path: str | None = None):
    """Load ``libkda.so`` (built by ``kimi_delta_attention_27_b200.build``)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA library not built: {p} is missing "
                               "(run python -m kimi_delta_attention_27_b200.build)")
        lib = ctypes.CDLL(p)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        fwd_args = [P, P, P, P, P, ctypes.c_float, P, i32, i32, i64, i32, i32, i32,
                    P, ctypes.c_int, P, ctypes.c_int, P, P]
        for name in ("kda_fwd", "kda_fwd_noalloc"):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = fwd_args
        lib.kda_fwd_ex.restype = ctypes.c_int
        lib.kda_fwd_ex.argtypes = [P, P, P, P, i32, P, ctypes.c_float, P, i32, i32, i64, i32, i32, i32,
                                   P, ctypes.c_int, P, ctypes.c_int, P, ctypes.c_uint32, P]
        lib.kda_fwd_segmented.restype = ctypes.c_int
        lib.kda_fwd_segmented.argtypes = [P, P, P, P, P, ctypes.c_float, i32, i64, i32, i32, i32, P, ctypes.c_int,
                                          P, ctypes.c_int, P, i64, P, ctypes.c_size_t, P]
        lib.kda_fwd_segmented_workspace.restype = ctypes.c_size_t
        lib.kda_fwd_segmented_workspace.argtypes = [i32, i64, i32, i64]
        lib.kda_bwd.restype = ctypes.c_int
        lib.kda_bwd.argtypes = [P, P, P, P, P, ctypes.c_float, P, i32, i32, i64, i32, i32, i32, P, ctypes.c_int,
                                P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.kda_bwd_workspace.restype = ctypes.c_size_t
        lib.kda_bwd_workspace.argtypes = [i64, i32, i32]
        lib.kda_decode.restype = ctypes.c_int
        lib.kda_decode.argtypes = [P, P, P, P, P, ctypes.c_float, i32, i32, i32, i32, P, P, ctypes.c_int, P, P]
        f32, u32, sz, dt = ctypes.c_float, ctypes.c_uint32, ctypes.c_size_t, ctypes.c_int
        conv = [P, dt, i64, P, P, u32]
        seqs = [P, i32, i32, i64]
        qk = [P, i64, P, i64, i64, i32, i32, i32, i32, f32, P, P, P, P, i32, i32, f32]
        scan = [P, i64, P, P, P, i64, P, i64, P, P, u32]
        for name, args in {
            "kda_conv_fwd": conv + seqs + [i32, i32, P, P, P, i64, P],
            "kda_conv_bwd": conv + seqs + [i32, i32, P, P, dt, i64, P, P, i64, P, P, P, P, sz, P],
            "kda_conv_decode": conv + [i32, i32, i32, P, P, P, i64, P],
            "kda_qk_fwd": qk + [P, i64, P, i64, P],
            "kda_qk_bwd": qk + [P, i64, P, i64, dt, P, i64, P, i64, P, P, P, sz, P],
            "kda_scan_fwd": scan + seqs + [i32, i32, i32, i32, P, dt, P, dt, P, i64, P, sz, P],
            "kda_scan_bwd": scan + seqs + [i32, i32, i32, i32, P, dt, P, i64, P, P, i64, P, P, P, i64, P, i64, P, P,
                                           P, P, sz, P],
            "kda_scan_decode": scan + [i32, i32, i32, i32, i32, P, P, dt, P, P],
        }.items():
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = args
        for name, args in {
            "kda_conv_bwd_workspace": [i64, i32, i32],
            "kda_qk_bwd_workspace": [i64, i32, i32, i32],
            "kda_scan_fwd_workspace": [i64, i32, i32, i32, i32],
            "kda_scan_bwd_workspace": [i64, i32, i32, i32, i32, i32],
        }.items():
            getattr(lib, name).restype = sz
            getattr(lib, name).argtypes = args
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_status_string.argtypes = [ctypes.c_int]
        lib.kda_version.restype = ctypes.c_int32
        lib.kda_version.argtypes = []
        lib.kda_device_error.restype = ctypes.c_int
        lib.kda_device_error.argtypes = []
        if path is None:
            _lib = lib
        return lib


def device_error() -> int:
    """Synchronise and read/clear the device-side error word (0 = no kernel gave up)."""
    return int(load_library().kda_device_error())


def status_string(status: int) -> str:
    return load_library().kda_status_string(int(status)).decode()


def _dtype_code(t) -> int:
    import torch
    if t is None:
        return KDA_DTYPE_NONE
    if t.dtype == torch.bfloat16:
        return KDA_DTYPE_BF16
    if t.dtype == torch.float32:
        return KDA_DTYPE_FP32
    return -1


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(name, t, dtype, ndim=None, shape=None):
    """Validate one tensor argument. ``shape`` (a tuple) is required exactly: the C
    ABI receives bare pointers and cannot tell an undersized buffer from a right one."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_devices(**tensors):
    """Every given tensor on one CUDA device (the first one's); returns that device."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on a CUDA device (no CPU path exists)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
    return dev


def kda_fwd(q, k, v, g, beta, scale: float | None = None, cu_seqlens=None,
            initial_state=None, final_state=None, out=None, final_state_dtype=None,
            stream=None, l2norm_qk: bool = False, gate_logsigmoid: bool = False):
    """Chunkwise KDA forward (see include/kda.h for the full contract).

    q, k, v: bf16 [B, T, H, 128]; g: log alpha, fp32 [B, T, H, 128] (kda_fwd), or
    bf16 [B, T, H, 128], or fp32 [B, T, H] (one decay per token and head: Gated
    DeltaNet); beta: fp32 [B, T, H]; cu_seqlens: int32 [N + 1] on the device (then
    B == 1) or None; initial_state: [N, H, 128, 128] bf16/fp32 or None.
    ``l2norm_qk``: the kernel L2-normalises q and k first; ``gate_logsigmoid``: g
    holds the gate's pre-activation and log alpha = logsigmoid(g). Any of these
    variants goes through kda_fwd_ex, the plain case through kda_fwd.
    ``final_state`` may be passed preallocated; otherwise one is allocated when
    ``final_state_dtype`` is given. ``out`` may be passed preallocated.
    Returns (out, final_state or None).
    """
    import torch
    kind = KDA_GATE_FP32
    if isinstance(g, torch.Tensor):
        if g.dtype == torch.bfloat16:
            kind = KDA_GATE_BF16
        elif g.dim() == 3:
            kind = KDA_GATE_SCALAR_FP32
    flags = (KDA_FLAG_L2NORM_QK if l2norm_qk else 0) | (KDA_FLAG_GATE_LOGSIGMOID if gate_logsigmoid else 0)
    entry = "kda_fwd" if kind == KDA_GATE_FP32 and flags == 0 else "kda_fwd_ex"
    return _fwd(entry, q, k, v, g, beta, scale, cu_seqlens, initial_state, final_state, out,
                final_state_dtype, stream, gate_kind=kind, flags=flags)


def kda_fwd_noalloc(q, k, v, g, beta, out, scale: float | None = None, cu_seqlens=None,
                    initial_state=None, final_state=None, stream=None):
    """``kda_fwd`` through the allocation-free entry point of include/kda.h.

    The caller provides ``out`` (and ``final_state`` if the final states are
    wanted): neither this wrapper nor the library allocates. At most
    ``NOALLOC_MAX_UNITS`` (sequence, head) pairs per call; calls whose work
    overlaps in time race on the library's fixed scratch. Returns
    (out, final_state or None).
    """
    if out is None:
        raise ValueError("kda_fwd_noalloc needs a preallocated out tensor")
    return _fwd("kda_fwd_noalloc", q, k, v, g, beta, scale, cu_seqlens, initial_state, final_state,
                out, None, stream)


def _fwd(entry, q, k, v, g, beta, scale, cu_seqlens, initial_state, final_state, out,
         final_state_dtype, stream, gate_kind=0, flags=0):
    import torch
    _check("q", q, torch.bfloat16, 4)
    B, T, H, Dk = q.shape
    Dv = v.shape[-1] if v.dim() == 4 else -1
    _check("k", k, torch.bfloat16, shape=q.shape)
    _check("v", v, torch.bfloat16, shape=(B, T, H, Dv))
    if gate_kind == KDA_GATE_SCALAR_FP32:
        _check("g", g, torch.float32, shape=(B, T, H))
    else:
        _check("g", g, torch.bfloat16 if gate_kind == KDA_GATE_BF16 else torch.float32, shape=q.shape)
    _check("beta", beta, torch.float32, shape=(B, T, H))
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, torch.int32, 1)
        N = cu_seqlens.numel() - 1
    else:
        N = B
    state_shape = (N, H, Dk, Dv)
    if initial_state is not None:
        _check("initial_state", initial_state, None, shape=state_shape)
    if out is not None:
        _check("out", out, torch.bfloat16, shape=(B, T, H, Dv))
    if final_state is not None:
        _check("final_state", final_state, None, shape=state_shape)
    dev = _check_devices(q=q, k=k, v=v, g=g, beta=beta, cu_seqlens=cu_seqlens, initial_state=initial_state,
                         out=out, final_state=final_state)
    if scale is None:
        scale = Dk ** -0.5
    lib = load_library()
    # the library works on the current device: make it q's
    stream, ctx = _stream_of(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((B, T, H, Dv), dtype=torch.bfloat16, device=dev)
        if final_state is None and final_state_dtype is not None:
            final_state = torch.empty(state_shape, dtype=final_state_dtype, device=dev)
        ic, fc = _dtype_code(initial_state), _dtype_code(final_state)
        if entry == "kda_fwd_ex":
            st = lib.kda_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), int(gate_kind), _ptr(beta), float(scale),
                                _ptr(cu_seqlens), int(N), int(B), int(T), int(H), int(Dk), int(Dv),
                                _ptr(initial_state), ic if ic >= 0 else 99,
                                _ptr(final_state), fc if fc >= 0 else 99,
                                _ptr(out), int(flags), ctypes.c_void_p(int(stream)))
        else:
            st = getattr(lib, entry)(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale),
                                     _ptr(cu_seqlens), int(N), int(B), int(T), int(H), int(Dk), int(Dv),
                                     _ptr(initial_state), ic if ic >= 0 else 99,
                                     _ptr(final_state), fc if fc >= 0 else 99,
                                     _ptr(out), ctypes.c_void_p(int(stream)))
    if st != 0:
        raise KdaError(st, lib.kda_status_string(st).decode())
    return out, final_state


def kda_fwd_segmented(q, k, v, g, beta, segment_len: int, scale: float | None = None, initial_state=None,
                      final_state=None, out=None, final_state_dtype=None, workspace=None, stream=None):
    """kda_fwd over fixed-length rows split into pieces of ``segment_len`` tokens that run at
    once (see include/kda.h, kda_fwd_segmented). q, k, v, g, beta, states and out as for
    ``kda_fwd`` without cu_seqlens. ``workspace`` (a uint8 CUDA tensor of at least
    ``segmented_workspace_bytes(...)`` bytes) is allocated here when not given.
    Returns (out, final_state or None)."""
    import torch
    _check("q", q, torch.bfloat16, 4)
    B, T, H, Dk = q.shape
    Dv = v.shape[-1] if v.dim() == 4 else -1
    _check("k", k, torch.bfloat16, shape=q.shape)
    _check("v", v, torch.bfloat16, shape=(B, T, H, Dv))
    _check("g", g, torch.float32, shape=q.shape)
    _check("beta", beta, torch.float32, shape=(B, T, H))
    state_shape = (B, H, Dk, Dv)
    if initial_state is not None:
        _check("initial_state", initial_state, None, shape=state_shape)
    if out is not None:
        _check("out", out, torch.bfloat16, shape=(B, T, H, Dv))
    if final_state is not None:
        _check("final_state", final_state, None, shape=state_shape)
    lib = load_library()
    need = int(lib.kda_fwd_segmented_workspace(int(B), int(T), int(H), int(segment_len)))
    if workspace is not None:
        _check("workspace", workspace, torch.uint8, 1)
    dev = _check_devices(q=q, k=k, v=v, g=g, beta=beta, initial_state=initial_state, out=out,
                         final_state=final_state, workspace=workspace)
    if scale is None:
        scale = Dk ** -0.5
    stream, ctx = _stream_of(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((B, T, H, Dv), dtype=torch.bfloat16, device=dev)
        if final_state is None and final_state_dtype is not None:
            final_state = torch.empty(state_shape, dtype=final_state_dtype, device=dev)
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        ic, fc = _dtype_code(initial_state), _dtype_code(final_state)
        st = lib.kda_fwd_segmented(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), int(B), int(T),
                                   int(H), int(Dk), int(Dv), _ptr(initial_state), ic if ic >= 0 else 99,
                                   _ptr(final_state), fc if fc >= 0 else 99, _ptr(out), int(segment_len),
                                   _ptr(workspace), int(workspace.numel()), ctypes.c_void_p(int(stream)))
    if st != 0:
        raise KdaError(st, lib.kda_status_string(st).decode())
    return out, final_state


def kda_bwd(q, k, v, g, beta, dout, scale: float | None = None, cu_seqlens=None, initial_state=None,
            dfinal_state=None, want_dinitial_state: bool = True, workspace=None, stream=None):
    """Gradients of sum(dout * out) + sum(dfinal_state * final_state) of ``kda_fwd`` with
    respect to q, k, v, g, beta and the initial state (see include/kda.h, kda_bwd).

    Inputs as for ``kda_fwd`` (fp32 per-channel g), plus dout bf16 [B, T, H, 128] and
    dfinal_state fp32 [N, H, 128, 128] or None. Returns a dict of fp32 tensors: dq, dk, dv,
    dg [B, T, H, 128], dbeta [B, T, H] and dh0 [N, H, 128, 128] (None unless asked).
    ``workspace`` (uint8, at least ``bwd_workspace_bytes(...)``) is allocated when not given."""
    import torch
    _check("q", q, torch.bfloat16, 4)
    B, T, H, Dk = q.shape
    Dv = v.shape[-1] if v.dim() == 4 else -1
    _check("k", k, torch.bfloat16, shape=q.shape)
    _check("v", v, torch.bfloat16, shape=(B, T, H, Dv))
    _check("g", g, torch.float32, shape=q.shape)
    _check("beta", beta, torch.float32, shape=(B, T, H))
    _check("dout", dout, torch.bfloat16, shape=(B, T, H, Dv))
    if cu_seqlens is not None:
        _check("cu_seqlens", cu_seqlens, torch.int32, 1)
        N = cu_seqlens.numel() - 1
    else:
        N = B
    state_shape = (N, H, Dk, Dv)
    if initial_state is not None:
        _check("initial_state", initial_state, None, shape=state_shape)
    if dfinal_state is not None:
        _check("dfinal_state", dfinal_state, torch.float32, shape=state_shape)
    if workspace is not None:
        _check("workspace", workspace, torch.uint8, 1)
    dev = _check_devices(q=q, k=k, v=v, g=g, beta=beta, dout=dout, cu_seqlens=cu_seqlens,
                         initial_state=initial_state, dfinal_state=dfinal_state, workspace=workspace)
    lib = load_library()
    rows = T if cu_seqlens is not None else B * T
    if scale is None:
        scale = Dk ** -0.5
    stream, ctx = _stream_of(dev, stream)
    ic = _dtype_code(initial_state)
    with ctx:
        if workspace is None:
            workspace = torch.empty(max(1, int(lib.kda_bwd_workspace(int(rows), int(N), int(H)))),
                                    dtype=torch.uint8, device=dev)
        out = {n: torch.empty((B, T, H, Dk if n != "dv" else Dv), dtype=torch.float32, device=dev)
               for n in ("dq", "dk", "dv", "dg")}
        out["dbeta"] = torch.empty((B, T, H), dtype=torch.float32, device=dev)
        out["dh0"] = torch.empty(state_shape, dtype=torch.float32, device=dev) if want_dinitial_state else None
        st = lib.kda_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), _ptr(cu_seqlens), int(N),
                         int(B), int(T), int(H), int(Dk), int(Dv), _ptr(initial_state), ic if ic >= 0 else 99,
                         _ptr(dout), _ptr(dfinal_state), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                         _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(workspace),
                         int(workspace.numel()), ctypes.c_void_p(int(stream)))
    if st != 0:
        raise KdaError(st, lib.kda_status_string(st).decode())
    return out


def bwd_workspace_bytes(total_tokens: int, num_seqs: int, num_heads: int) -> int:
    """Bytes of workspace kda_bwd needs."""
    return int(load_library().kda_bwd_workspace(int(total_tokens), int(num_seqs), int(num_heads)))


def segmented_workspace_bytes(batch: int, seq_len: int, num_heads: int, segment_len: int) -> int:
    """Bytes of workspace kda_fwd_segmented needs (0 for a bad segment_len)."""
    return int(load_library().kda_fwd_segmented_workspace(int(batch), int(seq_len), int(num_heads),
                                                          int(segment_len)))


def kda_decode(q, k, v, g, beta, state_in=None, state_out=None, scale: float | None = None, out=None,
               state_dtype=None, stream=None):
    """One recurrent step for a batch of requests (see include/kda.h, kda_decode).

    q, k, v: bf16 [B, H, 128]; g: fp32 [B, H, 128] (raw log alpha); beta: fp32 [B, H];
    state_in: [B, H, 128, 128] bf16/fp32 or None (zero states). ``state_out`` may be
    ``state_in`` itself (update in place) or a separate buffer; if it is None and
    ``state_dtype`` is given, one is allocated. ``out`` may be passed preallocated.
    Returns (out, state_out or None).
    """
    import torch
    _check("q", q, torch.bfloat16, 3)
    B, H, Dk = q.shape
    Dv = v.shape[-1] if v.dim() == 3 else -1
    _check("k", k, torch.bfloat16, shape=q.shape)
    _check("v", v, torch.bfloat16, shape=(B, H, Dv))
    _check("g", g, torch.float32, shape=q.shape)
    _check("beta", beta, torch.float32, shape=(B, H))
    state_shape = (B, H, Dk, Dv)
    if state_in is not None:
        _check("state_in", state_in, None, shape=state_shape)
    if state_out is not None:
        _check("state_out", state_out, None, shape=state_shape)
    if out is not None:
        _check("out", out, torch.bfloat16, shape=(B, H, Dv))
    dev = _check_devices(q=q, k=k, v=v, g=g, beta=beta, state_in=state_in, state_out=state_out, out=out)
    kept = state_dtype if state_out is None else state_out.dtype
    if state_in is not None and kept is not None and state_in.dtype != kept:
        raise ValueError("state_in and state_out must have the same dtype")
    if scale is None:
        scale = Dk ** -0.5
    lib = load_library()
    stream, ctx = _stream_of(dev, stream)
    with ctx:
        if state_out is None and state_dtype is not None:
            state_out = torch.empty(state_shape, dtype=state_dtype, device=dev)
        if out is None:
            out = torch.empty((B, H, Dv), dtype=torch.bfloat16, device=dev)
        st_t = state_in if state_in is not None else state_out
        code = _dtype_code(st_t)
        st = lib.kda_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(scale), int(B), int(H),
                            int(Dk), int(Dv), _ptr(state_in), _ptr(state_out), code if code >= 0 else 99,
                            _ptr(out), ctypes.c_void_p(int(stream)))
    if st != 0:
        raise KdaError(st, lib.kda_status_string(st).decode())
    return out, state_out


# ---------------------------------------------------------------- operators around the recurrence

def _check_rows(name, t, dtypes, shape, lead):
    """Validate a tensor whose token rows may be strided: the first ``lead`` dims are the rows, the others
    contiguous within one. Returns the row stride in elements."""
    import torch
    if type(t) is not torch.Tensor and not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape is not shape and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    width = math.prod(shape[lead:])
    if t.is_contiguous() or not t.numel():
        return width
    inner = 1
    for n, st in zip(reversed(t.shape[lead:]), reversed(t.stride()[lead:])):
        if n > 1 and st != inner:
            raise ValueError(f"{name} must be contiguous within a row")
        inner *= n
    stride, below = width, 1
    for n, st in zip(reversed(t.shape[:lead]), reversed(t.stride()[:lead])):
        if n > 1 and below == 1:
            stride = st
        elif n > 1 and st != stride * below:
            raise ValueError(f"{name}'s rows must be evenly spaced")
        below *= n
    if stride < width:
        raise ValueError(f"{name}'s rows must not overlap")
    return stride


def _check_param(name, t, shape):
    """Validate an optional contiguous fp32 tensor."""
    if t is not None:
        import torch
        _check_state(name, t, torch.float32, shape)


def _check_state(name, t, dtype, shape):
    """``_check`` for a tensor whose dtype and shape are known: one comparison each where all is well."""
    import torch
    if not (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _check(name, t, dtype, shape=shape)


def _one_device(first, *others):
    """``first``'s device, which must be a CUDA device that the others (or None) are on too."""
    at = first.get_device()
    if at < 0:
        raise ValueError("tensors must be on a CUDA device (no CPU path exists)")
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError(f"all tensors must be on {first.device}, got {t.device}")
    return first.device


def _stream_of(dev, stream):
    """(the handle to launch on, a context in which ``dev`` is the current device and the handle's stream the
    current stream): what is allocated in it belongs to the stream the kernels run on."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # the handle alone: 2 us less per call
    here = raw(dev.index) if raw else torch.cuda.current_stream(dev).cuda_stream
    handle = here if stream is None else int(stream)
    if handle != here:
        # handle 0 is the default stream, of which ExternalStream(0) would make one of torch's pool;
        # torch.cuda.stream makes the stream's device current, too
        other = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
        return handle, torch.cuda.stream(other)
    return handle, _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _like(t):
    """A contiguous tensor of t's shape, type and device (half the time of torch.empty with all three)."""
    import torch
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _addr(t):
    return None if t is None else t.data_ptr()


def _raise(lib, st):
    if st != 0:
        raise KdaError(st, lib.kda_status_string(st).decode())


def _scratch(need, given, dev):
    import torch
    if given is not None:
        _check("workspace", given, torch.uint8, 1)
        return given
    return torch.empty(need, dtype=torch.uint8, device=dev) if need else None


def _size(t):
    return 0 if t is None else t.numel()


def _num_seqs(cu_seqlens, B):
    import torch
    if cu_seqlens is None:
        return B
    _check("cu_seqlens", cu_seqlens, torch.int32, 1)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must have at least one entry")
    return cu_seqlens.numel() - 1


def _conv_args(x, weight, bias, lead):
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != lead + 1:
        raise ValueError(f"x must have {lead + 1} dims")
    C = x.shape[-1]
    xs = _check_rows("x", x, (torch.bfloat16, torch.float32), x.shape, lead)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must have 2 dims")
    W = weight.shape[1]
    _check_state("weight", weight, torch.float32, (C, W))
    _check_param("bias", bias, (C,))
    return C, W, xs


def kda_conv_fwd(x, weight, bias=None, silu: bool = True, cu_seqlens=None, initial_state=None, final_state=None,
                 out=None, want_final_state: bool = False, stream=None):
    """Short causal depthwise convolution with SiLU over a batch of sequences (see include/kda.h, kda_conv_fwd).

    x: bf16 or fp32 [B, T, C] (token rows may be strided); weight: fp32 [C, W], W 2 to 4; bias: fp32 [C] or
    None; cu_seqlens: int32 [N + 1] on the device (then B == 1) or None; initial_state: [N, W - 1, C] of x's
    type or None (zeros). ``final_state`` may be passed preallocated, or is allocated when
    ``want_final_state``. Returns (out, final_state or None)."""
    import torch
    C, W, xs = _conv_args(x, weight, bias, 2)
    B, T = x.shape[:2]
    N = _num_seqs(cu_seqlens, B)
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None:
            _check_state(name, t, x.dtype, (N, W - 1, C))
    os = C if out is None else _check_rows("out", out, (x.dtype,), x.shape, 2)
    dev = _one_device(x, weight, bias, cu_seqlens, initial_state,
                      final_state, out)
    lib = load_library()
    handle, ctx = _stream_of(dev, stream)
    with ctx:
        if out is None:
            out = _like(x)
        if final_state is None and want_final_state:
            final_state = torch.empty((N, W - 1, C), dtype=x.dtype, device=dev)
        _raise(lib, lib.kda_conv_fwd(_addr(x), _dtype_code(x), xs, _addr(weight), _addr(bias),
                                     KDA_FLAG_CONV_SILU if silu else 0, _addr(cu_seqlens), N, B, T, C, W,
                                     _addr(initial_state), _addr(final_state), _addr(out),
                                     os, handle))
    return out, final_state


def kda_conv_bwd(x, weight, dout, bias=None, silu: bool = True, cu_seqlens=None, initial_state=None,
                 dfinal_state=None, want_dinitial_state: bool = False, dx=None, workspace=None, stream=None):
    """Gradients of sum(dout * out) + sum(dfinal_state * final_state) of ``kda_conv_fwd`` (see include/kda.h,
    kda_conv_bwd). Inputs as for it, plus dout [B, T, C] (x's type, or fp32) and dfinal_state [N, W - 1, C] or
    None. Returns a dict: dx [B, T, C] (x's type), dweight fp32 [C, W], dbias fp32 [C] (None without a bias),
    dinitial_state [N, W - 1, C] (None unless asked). ``dx`` may be passed preallocated (strided)."""
    import torch
    C, W, xs = _conv_args(x, weight, bias, 2)
    B, T = x.shape[:2]
    N = _num_seqs(cu_seqlens, B)
    ds = _check_rows("dout", dout, (x.dtype, torch.float32), x.shape, 2)
    for name, t in (("initial_state", initial_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _check_state(name, t, x.dtype, (N, W - 1, C))
    dxs = C if dx is None else _check_rows("dx", dx, (x.dtype,), x.shape, 2)
    dev = _one_device(x, weight, bias, cu_seqlens, initial_state,
                      dout, dfinal_state, dx, workspace)
    lib = load_library()
    handle, ctx = _stream_of(dev, stream)
    with ctx:
        if dx is None:
            dx = _like(x)
        dweight = torch.empty((C, W), dtype=torch.float32, device=dev)
        dbias = torch.empty(C, dtype=torch.float32, device=dev) if bias is not None else None
        dinit = torch.empty((N, W - 1, C), dtype=x.dtype, device=dev) if want_dinitial_state else None
        ws = _scratch(int(lib.kda_conv_bwd_workspace(B * T, C, W)), workspace, dev)
        _raise(lib, lib.kda_conv_bwd(_addr(x), _dtype_code(x), xs, _addr(weight), _addr(bias),
                                     KDA_FLAG_CONV_SILU if silu else 0, _addr(cu_seqlens), N, B, T, C, W,
                                     _addr(initial_state), _addr(dout), _dtype_code(dout), ds, _addr(dfinal_state),
                                     _addr(dx), dxs, _addr(dweight),
                                     _addr(dbias), _addr(dinit), _addr(ws), _size(ws), handle))
    return dict(dx=dx, dweight=dweight, dbias=dbias, dinitial_state=dinit)


def kda_conv_decode(x, weight, state_in=None, state_out=None, bias=None, silu: bool = True, out=None, stream=None):
    """``kda_conv_fwd`` for one new token per request (see include/kda.h, kda_conv_decode).

    x: [B, C] (rows may be strided); states [B, W - 1, C] of x's type: ``state_in`` None means zeros,
    ``state_out`` may be ``state_in`` itself (in place) or None (not written). Returns (out, state_out)."""
    import torch
    C, W, xs = _conv_args(x, weight, bias, 1)
    B = x.shape[0]
    for name, t in (("state_in", state_in), ("state_out", state_out)):
        if t is not None:
            _check_state(name, t, x.dtype, (B, W - 1, C))
    os = C if out is None else _check_rows("out", out, (x.dtype,), x.shape, 1)
    dev = _one_device(x, weight, bias, state_in, state_out, out)
    lib = load_library()
    handle, ctx = _stream_of(dev, stream)
    with ctx:
        if out is None:
            out = _like(x)
        _raise(lib, lib.kda_conv_decode(_addr(x), _dtype_code(x), xs, _addr(weight), _addr(bias),
                                        KDA_FLAG_CONV_SILU if silu else 0, B, C, W, _addr(state_in), _addr(state_out),
                                        _addr(out), os, handle))
    return out, state_out


def _qk_args(q, k, norm, q_weight, k_weight, positions, inv_freq):
    import torch
    if norm not in NORM_KINDS:
        raise ValueError(f"norm must be one of {', '.join(NORM_KINDS)}, got {norm!r}")
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or (k is not None and (
            not isinstance(k, torch.Tensor) or k.dim() != 4)):
        raise ValueError("q and k must have 4 dims")
    B, T, Hq, D = q.shape
    qs = _check_rows("q", q, (torch.bfloat16,), q.shape, 2)
    Hk = 0 if k is None else k.shape[2]
    ks = 0 if k is None else _check_rows("k", k, (torch.bfloat16,), (B, T, Hk, D), 2)
    _check_param("q_weight", q_weight, (D,))
    _check_param("k_weight", k_weight, (D,))
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq come together")
    rot = 0
    if positions is not None:
        _check_state("positions", positions, torch.int32, (B, T))
        _check("inv_freq", inv_freq, torch.float32, 1)
        rot = 2 * inv_freq.numel()
    return B, T, Hq, Hk, D, qs, ks, rot


def kda_qk_fwd(q, k=None, norm: str = "l2", q_weight=None, k_weight=None, eps: float = 1e-6, positions=None,
               inv_freq=None, interleaved: bool = False, factor: float = 1.0, q_out=None, k_out=None, stream=None):
    """Norm of each head of q and k and its position rotation in one pass (see include/kda.h, kda_qk_fwd).

    q: bf16 [B, T, Hq, D], k: bf16 [B, T, Hk, D] or None (token rows may be strided), D 64, 128 or 256; norm:
    "l2", "rms" or "none"; weights: fp32 [D] or None; positions: int32 [B, T] and inv_freq: fp32
    [rot_dim / 2] rotate the first rot_dim channels (both None: no rotation), in pairs (2i, 2i + 1) if
    ``interleaved``, else (i, i + rot_dim / 2); ``factor`` multiplies cos and sin. ``q_out``/``k_out`` may be q and
    k themselves. Returns (q_out, k_out)."""
    import torch
    B, T, Hq, Hk, D, qs, ks, rot = _qk_args(q, k, norm, q_weight, k_weight, positions, inv_freq)
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    bf = (torch.bfloat16,)
    qos = Hq * D if q_out is None else _check_rows("q_out", q_out, bf, q.shape, 2)
    kos = Hk * D if k_out is None else _check_rows("k_out", k_out, bf, k.shape, 2)
    dev = _one_device(q, k, q_weight, k_weight, positions, inv_freq,
                      q_out, k_out)
    lib = load_library()
    handle, ctx = _stream_of(dev, stream)
    with ctx:
        if q_out is None:
            q_out = _like(q)
        if k_out is None and k is not None:
            k_out = _like(k)
        _raise(lib, lib.kda_qk_fwd(_addr(q), qs, _addr(k), ks, B * T, Hq, Hk, D, NORM_KINDS[norm], float(eps),
                                   _addr(q_weight), _addr(k_weight), _addr(positions), _addr(inv_freq), rot,
                                   int(bool(interleaved)), float(factor),
                                   _addr(q_out), qos, _addr(k_out), kos, handle))
    return q_out, k_out


def kda_qk_bwd(q, k, dq_out, dk_out, norm: str = "l2", q_weight=None, k_weight=None, eps: float = 1e-6,
               positions=None, inv_freq=None, interleaved: bool = False, factor: float = 1.0, workspace=None,
               stream=None):
    """Gradients of sum(dq_out * q_out) + sum(dk_out * k_out) of ``kda_qk_fwd`` (see include/kda.h, kda_qk_bwd).

    q, k and the options as it took them (k and dk_out None together); dq_out, dk_out both bf16 or both fp32 (as
    ``kda_bwd`` gives them). Returns a dict: dq, dk bf16, dq_weight, dk_weight fp32 [D] (None without that
    weight)."""
    import torch
    B, T, Hq, Hk, D, qs, ks, rot = _qk_args(q, k, norm, q_weight, k_weight, positions, inv_freq)
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out come together")
    if k is None and k_weight is not None:
        raise ValueError("k_weight without k")
    dqs = _check_rows("dq_out", dq_out, (torch.bfloat16, torch.float32), q.shape, 2)
    dks = 0 if k is None else _check_rows("dk_out", dk_out, (dq_out.dtype,), k.shape, 2)
    dev = _one_device(q, k, q_weight, k_weight, positions, inv_freq,
                      dq_out, dk_out, workspace)
    lib = load_library()
    handle, ctx = _stream_of(dev, stream)
    with ctx:
        dq = _like(q)
        dk = _like(k) if k is not None else None
        dqw = torch.empty(D, dtype=torch.float32, device=dev) if q_weight is not None else None
        dkw = torch.empty(D, dtype=torch.float32, device=dev) if k_weight is not None else None
        need = 0
        if dqw is not None or dkw is not None:
            need = int(lib.kda_qk_bwd_workspace(B * T, Hq, Hk, D))
        ws = _scratch(need, workspace, dev)
        _raise(lib, lib.kda_qk_bwd(_addr(q), qs, _addr(k), ks, B * T, Hq, Hk, D, NORM_KINDS[norm], float(eps),
                                   _addr(q_weight), _addr(k_weight), _addr(positions), _addr(inv_freq), rot,
                                   int(bool(interleaved)), float(factor), _addr(dq_out), dqs, _addr(dk_out), dks,
                                   _dtype_code(dq_out), _addr(dq), Hq * D, _addr(dk), Hk * D, _addr(dqw), _addr(dkw),
                                   _addr(ws), _size(ws), handle))
    return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)


def _scan_args(x, dt, A, B, C, D, dt_bias, lead):
    import torch
    bf = (torch.bfloat16,)
    for name, t in (("x", x), ("B", B)):
        if not isinstance(t, torch.Tensor) or t.dim() != lead + 2:
            raise ValueError(f"{name} must have {lead + 2} dims")
    H, P = x.shape[lead:]
    G, N = B.shape[lead:]
    rows = tuple(x.shape[:lead])
    strides = (_check_rows("x", x, bf, x.shape, lead), _check_rows("B", B, bf, rows + (G, N), lead),
               _check_rows("C", C, bf, rows + (G, N), lead))
    _check_state("dt", dt, torch.float32, rows + (H,))
    _check_state("A", A, torch.float32, (H,))
    _check_param("D", D, (H,))
    _check_param("dt_bias", dt_bias, (H,))
    return H, P, G, N, strides


def kda_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, dt_softplus: bool = False, cu_seqlens=None,
                 initial_state=None, final_state=None, out=None, final_state_dtype=None, workspace=None, stream=None):
    """Selective state space scan over a batch of sequences (see include/kda.h, kda_scan_fwd).

    x: bf16 [B, T, H, P]; dt: fp32 [B, T, H]; A: fp32 [H] (negative); B, C: bf16 [B, T, G, N], H a multiple of
    G (token rows of x, B, C may be strided: slices of one projection); D, dt_bias: fp32 [H] or None; the step is
    dt + dt_bias, or its softplus. States [N_seqs, H, N, P] bf16 or fp32; ``final_state`` may be
    ``initial_state`` (in place), or is allocated when ``final_state_dtype`` is given. P and N are 64 or 128.
    ``workspace`` (uint8, at least ``scan_workspace_bytes(...)``) is allocated when needed and not given.
    Returns (out, final_state or None)."""
    import torch
    H, P, G, N, (xs, bs, cs) = _scan_args(x, dt, A, B, C, D, dt_bias, 2)
    Bn, T = x.shape[:2]
    n = _num_seqs(cu_seqlens, Bn)
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None:
            _check_state(name, t, getattr(t, "dtype", None), (n, H, N, P))
    bf = (torch.bfloat16,)
    os = H * P if out is None else _check_rows("out", out, bf, x.shape, 2)
    dev = _one_device(x, dt, A, B, C, D, dt_bias, cu_seqlens,
                      initial_state, final_state, out, workspace)
    lib = load_library()
    handle, ctx = _stream_of(dev, stream)
    with ctx:
        if out is None:
            out = _like(x)
        if final_state is None and final_state_dtype is not None:
            final_state = torch.empty((n, H, N, P), dtype=final_state_dtype, device=dev)
        ws = _scratch(int(lib.kda_scan_fwd_workspace(Bn * T, n, H, P, N)), workspace, dev)
        ic, fc = _dtype_code(initial_state), _dtype_code(final_state)
        _raise(lib, lib.kda_scan_fwd(_addr(x), xs, _addr(dt), _addr(A), _addr(B), bs, _addr(C), cs, _addr(D), _addr(dt_bias),
                                     KDA_FLAG_SCAN_SOFTPLUS if dt_softplus else 0, _addr(cu_seqlens), n, Bn, T, H, G,
                                     P, N, _addr(initial_state), ic if ic >= 0 else 99, _addr(final_state),
                                     fc if fc >= 0 else 99, _addr(out), os,
                                     _addr(ws), _size(ws), handle))
    return out, final_state


def kda_scan_bwd(x, dt, A, B, C, dout, D=None, dt_bias=None, dt_softplus: bool = False, cu_seqlens=None,
                 initial_state=None, dfinal_state=None, want_dinitial_state: bool = True, dx=None, dB=None, dC=None,
                 workspace=None, stream=None):
    """Gradients of sum(dout * out) + sum(dfinal_state * final_state) of ``kda_scan_fwd`` (see include/kda.h,
    kda_scan_bwd). Inputs as for it, plus dout bf16 [B, T, H, P] and dfinal_state fp32 [N_seqs, H, N, P] or None.
    Returns a dict: dx, dB, dC bf16 (shapes of x, B, C; each may be passed preallocated, strided), ddt, dA, dD,
    ddt_bias fp32 (the last two None without D or dt_bias) and dh0 fp32 [N_seqs, H, N, P] (None unless asked)."""
    import torch
    H, P, G, N, (xs, bs, cs) = _scan_args(x, dt, A, B, C, D, dt_bias, 2)
    Bn, T = x.shape[:2]
    n = _num_seqs(cu_seqlens, Bn)
    bf = (torch.bfloat16,)
    ds = _check_rows("dout", dout, bf, x.shape, 2)
    if initial_state is not None:
        _check("initial_state", initial_state, None, shape=(n, H, N, P))
    if dfinal_state is not None:
        _check_state("dfinal_state", dfinal_state, torch.float32, (n, H, N, P))
    dxs = H * P if dx is None else _check_rows("dx", dx, bf, x.shape, 2)
    dbs = G * N if dB is None else _check_rows("dB", dB, bf, B.shape, 2)
    dcs = G * N if dC is None else _check_rows("dC", dC, bf, C.shape, 2)
    dev = _one_device(x, dt, A, B, C, D, dt_bias, dout, cu_seqlens,
                      initial_state, dfinal_state, dx, dB, dC,
                      workspace)
    lib = load_library()
    handle, ctx = _stream_of(dev, stream)
    with ctx:
        empty = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        f32 = torch.float32
        dx = _like(x) if dx is None else dx
        dB = _like(B) if dB is None else dB
        dC = _like(C) if dC is None else dC
        out = dict(dx=dx, dB=dB, dC=dC, ddt=_like(dt), dA=_like(A),
                   dD=empty((H,), f32) if D is not None else None,
                   ddt_bias=empty((H,), f32) if dt_bias is not None else None,
                   dh0=empty((n, H, N, P), f32) if want_dinitial_state else None)
        ws = _scratch(int(lib.kda_scan_bwd_workspace(Bn * T, n, H, G, P, N)), workspace, dev)
        ic = _dtype_code(initial_state)
        _raise(lib, lib.kda_scan_bwd(_addr(x), xs, _addr(dt), _addr(A), _addr(B), bs, _addr(C), cs, _addr(D), _addr(dt_bias),
                                     KDA_FLAG_SCAN_SOFTPLUS if dt_softplus else 0, _addr(cu_seqlens), n, Bn, T, H, G,
                                     P, N, _addr(initial_state), ic if ic >= 0 else 99, _addr(dout), ds,
                                     _addr(dfinal_state), _addr(dx), dxs,
                                     _addr(out["ddt"]), _addr(out["dA"]), _addr(dB),
                                     dbs, _addr(dC), dcs, _addr(out["dD"]), _addr(out["ddt_bias"]),
                                     _addr(out["dh0"]), _addr(ws), _size(ws), handle))
    return out


def scan_workspace_bytes(total_tokens: int, num_seqs: int, num_heads: int, head_dim: int, state_dim: int) -> int:
    """Bytes of workspace kda_scan_fwd needs (0 where it cuts no sequence)."""
    return int(load_library().kda_scan_fwd_workspace(int(total_tokens), int(num_seqs), int(num_heads), int(head_dim),
                                                     int(state_dim)))


def kda_scan_decode(x, dt, A, B, C, state_in=None, state_out=None, D=None, dt_bias=None, dt_softplus: bool = False,
                    out=None, state_dtype=None, stream=None):
    """``kda_scan_fwd`` for one new token per request (see include/kda.h, kda_scan_decode).

    x: bf16 [B, H, P], B, C: bf16 [B, G, N] (rows may be strided), dt: fp32 [B, H]; states [B, H, N, P] with
    ``kda_decode``'s rules: ``state_in`` None means zeros, ``state_out`` may be ``state_in`` itself, and is
    allocated when it is None and ``state_dtype`` is given. Returns (out, state_out or None)."""
    import torch
    H, P, G, N, (xs, bs, cs) = _scan_args(x, dt, A, B, C, D, dt_bias, 1)
    n = x.shape[0]
    for name, t in (("state_in", state_in), ("state_out", state_out)):
        if t is not None:
            _check_state(name, t, getattr(t, "dtype", None), (n, H, N, P))
    if state_in is not None and state_out is not None and state_in.dtype != state_out.dtype:
        raise ValueError("state_in and state_out must have the same dtype")
    if state_in is not None and state_out is None and state_dtype not in (None, state_in.dtype):
        raise ValueError("state_dtype must be state_in's")
    if out is not None:
        _check("out", out, torch.bfloat16, shape=x.shape)
    dev = _one_device(x, dt, A, B, C, D, dt_bias, state_in, state_out,
                      out)
    lib = load_library()
    handle, ctx = _stream_of(dev, stream)
    with ctx:
        if state_out is None and state_dtype is not None:
            state_out = torch.empty((n, H, N, P), dtype=state_dtype, device=dev)
        if out is None:
            out = _like(x)
        code = _dtype_code(state_in if state_in is not None else state_out)
        _raise(lib, lib.kda_scan_decode(_addr(x), xs, _addr(dt), _addr(A), _addr(B), bs, _addr(C), cs, _addr(D),
                                        _addr(dt_bias), KDA_FLAG_SCAN_SOFTPLUS if dt_softplus else 0, n, H, G, P, N,
                                        _addr(state_in), _addr(state_out), code if code >= 0 else 99, _addr(out),
                                        handle))
    return out, state_out
