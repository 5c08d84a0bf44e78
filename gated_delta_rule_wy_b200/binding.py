"""ctypes binding of libgdr2.so: the C ABI in ``include/gdr2.h`` with torch tensors.

Argument marshalling only. Every function here checks shapes, dtypes and
devices, allocates output tensors with PyTorch (device memory is the one
thing torch provides), passes raw device pointers and the current CUDA stream
to the library, and turns a non-OK status into ``GDR2Error``. There is no
fallback: if ``libgdr2.so`` is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdr2.so")

GDR2_OK, GDR2_ERR_INVALID_ARG, GDR2_ERR_UNSUPPORTED, GDR2_ERR_CUDA, GDR2_ERR_TIMEOUT = range(5)
GDR2_F32, GDR2_BF16 = 0, 1
CHUNK = 64
SSM_CHUNK = 16  # GDR2_SSM_CHUNK
_STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "TIMEOUT"}

# Every symbol include/gdr2.h declares (the ABI tests check the exports).
EXPORTED_SYMBOLS = ("gdr2_abi_version", "gdr2_last_error", "gdr2_forward_workspace_bytes", "gdr2_forward",
                    "gdr2_forward_gated", "gdr2_forward_varlen_workspace_bytes", "gdr2_forward_varlen",
                    "gdr2_forward_ex", "gdr2_short_conv_silu", "gdr2_gate_activations", "gdr2_segment_states",
                    "gdr2_short_conv_silu_backward_workspace_bytes", "gdr2_short_conv_silu_backward",
                    "gdr2_ssm_scan_workspace_bytes", "gdr2_ssm_scan", "gdr2_ssm_step",
                    "gdr2_ssm_scan_backward_workspace_bytes", "gdr2_ssm_scan_backward",
                    "gdr2_head_norm_rope", "gdr2_head_norm_rope_backward_workspace_bytes",
                    "gdr2_head_norm_rope_backward",
                    "gdr2_decode_step", "gdr2_decode_step_gated",
                    "gdr2_backward_workspace_bytes", "gdr2_backward", "gdr2_backward_gated", "gdr2_backward_noalloc",
                    "gdr2_sync_status", "gdr2_debug_force_timeout", "gdr2_debug_recip",
                    "gdr2_debug_forward_unfused")
NOALLOC_SCRATCH_BYTES = 64 << 20  # GDR2_NOALLOC_SCRATCH_BYTES


class GDR2Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"GDR2 {_STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_lock = threading.Lock()
_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libgdr2.so once and declare the signatures of include/gdr2.h."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with `python -m gated_delta_rule_wy_b200.build` "
                               "(there is no CPU fallback)")
        lib = ctypes.CDLL(p)
        I, P, Z = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        lib.gdr2_abi_version.restype = I
        lib.gdr2_abi_version.argtypes = []
        lib.gdr2_last_error.restype = ctypes.c_char_p
        lib.gdr2_last_error.argtypes = []
        lib.gdr2_forward_workspace_bytes.restype = Z
        lib.gdr2_forward_workspace_bytes.argtypes = [I, I, I, I, I, I]
        lib.gdr2_forward.restype = I
        lib.gdr2_forward.argtypes = [I, I, I, I, I, I] + [P] * 11 + [Z, P]
        lib.gdr2_decode_step.restype = I
        lib.gdr2_forward_varlen_workspace_bytes.restype = Z
        lib.gdr2_forward_varlen_workspace_bytes.argtypes = [I, I, I, I, I, I]
        lib.gdr2_forward_varlen.restype = I
        lib.gdr2_forward_varlen.argtypes = [I, I, I, I, I, I, I] + [P] * 12 + [Z, P]
        lib.gdr2_forward_ex.restype = I
        lib.gdr2_forward_ex.argtypes = [I, I, I, I, I, I, I] + [P] * 8 + [P, P, ctypes.c_float] + [P] * 4 + [Z, P]
        lib.gdr2_short_conv_silu.restype = I
        lib.gdr2_short_conv_silu.argtypes = [I] * 7 + [ctypes.c_float] + [P] * 7
        lib.gdr2_gate_activations.restype = I
        lib.gdr2_gate_activations.argtypes = [I] + [ctypes.c_longlong, P, P] * 3 + [P]
        F, LL = ctypes.c_float, ctypes.c_longlong
        lib.gdr2_short_conv_silu_backward_workspace_bytes.restype = Z
        lib.gdr2_short_conv_silu_backward_workspace_bytes.argtypes = [I] * 5
        lib.gdr2_short_conv_silu_backward.restype = I
        lib.gdr2_short_conv_silu_backward.argtypes = [I] * 7 + [F] + [P] * 9 + [Z, P]
        ssm_in = [P, LL, P, LL, P, P, LL, P, LL, P, P, LL, P]  # x, step, A, Bm, Cm, Dskip, z, step_bias
        lib.gdr2_ssm_scan_workspace_bytes.restype = Z
        lib.gdr2_ssm_scan_workspace_bytes.argtypes = [I] * 4
        lib.gdr2_ssm_scan.restype = I
        lib.gdr2_ssm_scan.argtypes = [I] * 6 + [P] + ssm_in + [P] * 5 + [Z, P]
        lib.gdr2_ssm_step.restype = I
        lib.gdr2_ssm_step.argtypes = [I] * 5 + ssm_in + [P] * 3
        lib.gdr2_ssm_scan_backward_workspace_bytes.restype = Z
        lib.gdr2_ssm_scan_backward_workspace_bytes.argtypes = [I] * 5
        lib.gdr2_ssm_scan_backward.restype = I
        lib.gdr2_ssm_scan_backward.argtypes = [I] * 6 + ssm_in + [P] * 14 + [Z, P]
        rope_in = [I] * 7 + [F, P, LL, P, LL, P, P, I, I, P, I, P, I]
        lib.gdr2_head_norm_rope.restype = I
        lib.gdr2_head_norm_rope.argtypes = rope_in + [P] * 3
        lib.gdr2_head_norm_rope_backward_workspace_bytes.restype = Z
        lib.gdr2_head_norm_rope_backward_workspace_bytes.argtypes = [I]
        lib.gdr2_head_norm_rope_backward.restype = I
        lib.gdr2_head_norm_rope_backward.argtypes = rope_in + [P] * 7 + [Z, P]
        lib.gdr2_segment_states.restype = I
        lib.gdr2_segment_states.argtypes = [I] * 5 + [P] * 6
        lib.gdr2_forward_gated.restype = I
        lib.gdr2_forward_gated.argtypes = [I, I, I, I, I, I, I] + [P] * 11 + [Z, P]
        lib.gdr2_decode_step_gated.restype = I
        lib.gdr2_decode_step_gated.argtypes = [I, I, I, I, I, I] + [P] * 9
        lib.gdr2_decode_step.argtypes = [I, I, I, I, I] + [P] * 9
        lib.gdr2_backward_workspace_bytes.restype = Z
        lib.gdr2_backward_workspace_bytes.argtypes = [I, I, I, I, I, I]
        lib.gdr2_backward.restype = I
        lib.gdr2_backward.argtypes = [I, I, I, I, I, I] + [P] * 18 + [Z, P]
        lib.gdr2_backward_gated.restype = I
        lib.gdr2_backward_gated.argtypes = [I, I, I, I, I, I, I] + [P] * 18 + [Z, P]
        lib.gdr2_backward_noalloc.restype = I
        lib.gdr2_backward_noalloc.argtypes = [I, I, I, I, I, I] + [P] * 18
        lib.gdr2_sync_status.restype = I
        lib.gdr2_sync_status.argtypes = [P]
        lib.gdr2_debug_force_timeout.restype = None
        lib.gdr2_debug_force_timeout.argtypes = [I]
        lib.gdr2_debug_forward_unfused.restype = None
        lib.gdr2_debug_forward_unfused.argtypes = [I]
        lib.gdr2_debug_recip.restype = I
        lib.gdr2_debug_recip.argtypes = [P, P, ctypes.c_longlong, P]
        _lib = lib
        return lib


def _tensors_in(args, kwargs):
    for a in list(args) + list(kwargs.values()):
        if isinstance(a, torch.Tensor):
            yield a
        elif isinstance(a, (list, tuple)):
            yield from (x for x in a if isinstance(x, torch.Tensor))


def _tensors_of(result):
    """The tensors that a call returns, one by one or in tuples and dicts."""
    if isinstance(result, torch.Tensor):
        yield result
    elif isinstance(result, (tuple, list, dict)):
        for part in result.values() if isinstance(result, dict) else result:
            yield from _tensors_of(part)


def _device_of(tensors):
    """The one device the tensors live on (None without tensors); raises if they span several."""
    devs = {t.device for t in tensors}
    if len(devs) > 1:
        names = ", ".join(sorted(str(d) for d in devs))
        raise ValueError(f"all tensors of a call must be on one CUDA device; got {names}")
    return next(iter(devs)) if devs else None


def _one_device(fn):
    """Run a library call on the device that holds its tensors.

    The library launches on the current CUDA device and stream, so tensors on another
    device would reach kernels as foreign pointers: the call is made under that device
    (its current stream unless one is given), after checking that every tensor argument
    and the stream share it. A given stream is the current one during the call, so that outputs and
    scratch are allocated in its order; the caller's own stream, on which outputs are read later, is recorded
    as a user of them, so that their memory is not handed to the given stream's next call before it has read them.
    """
    @functools.wraps(fn)
    def call(*args, **kwargs):
        stream = kwargs.get("stream")
        if stream is None:  # the common call: all tensors on the current device
            index = current = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1
            for a in (*args, *kwargs.values()):
                if isinstance(a, torch.Tensor):
                    index = a.get_device()
                    if index != current:
                        break
                elif isinstance(a, (list, tuple)):
                    index = -1
                    break
            if index == current >= 0:
                return fn(*args, **kwargs)
        dev = _device_of(_tensors_in(args, kwargs))
        if dev is None or dev.type != "cuda":
            return fn(*args, **kwargs)  # the argument checks reject host tensors
        if stream is not None and stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}: one CUDA device per call")
        if stream is not None:
            caller = torch.cuda.current_stream(dev)
            with torch.cuda.stream(stream):
                result = fn(*args, **kwargs)
            if caller != stream:
                for t in _tensors_of(result):
                    t.record_stream(caller)
            return result
        with torch.cuda.device(dev):
            return fn(*args, **kwargs)
    return call


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    """The raw stream, the current one of the current device unless one is given."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDR2_F32
    if t.dtype == torch.bfloat16:
        return GDR2_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _check(t, name, shape, dtype):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


GATE_SCALAR_B, GATE_SCALAR_W = 1, 2  # GDR2_GATE_* of include/gdr2.h


def _gates(b, w, lead):
    """Gate layout bits from the shapes: a gate shaped `lead` (no channel dim) is a scalar."""
    g = 0
    if tuple(b.shape) == tuple(lead):
        g |= GATE_SCALAR_B
    if tuple(w.shape) == tuple(lead):
        g |= GATE_SCALAR_W
    return g


def _epilogue(out_gate, norm_weight, o_shape, dv, dt, dev):
    """Checks the output gate and norm weight; True when either is given."""
    if out_gate is not None:
        _check(out_gate, "out_gate", o_shape, dt)
        if out_gate.device != dev:
            raise ValueError("out_gate must be on the inputs' device")
    if norm_weight is not None:
        _check(norm_weight, "norm_weight", (dv,), torch.float32)
        if norm_weight.device != dev:
            raise ValueError("norm_weight must be on the inputs' device")
    return out_gate is not None or norm_weight is not None


def _raise(lib, st):
    if st != GDR2_OK:
        raise GDR2Error(st, lib.gdr2_last_error().decode(errors="replace"))


def gdr2_abi_version() -> int:
    """GDR2_ABI_VERSION of the loaded libgdr2.so."""
    return load_library().gdr2_abi_version()


def gdr2_last_error() -> str:
    """Description of the calling thread's last non-OK status ('' if none)."""
    return load_library().gdr2_last_error().decode(errors="replace")


def gdr2_sync_status(stream=None) -> None:
    """Synchronise the stream and raise if a kernel gave up a bounded wait."""
    lib = load_library()
    _raise(lib, lib.gdr2_sync_status(_stream(stream)))


def gdr2_forward_workspace_bytes(B, T, H, dk, dv, dtype=torch.bfloat16) -> int:
    """Device scratch gdr2_forward needs (0 on the CUDA-core path: fp32, or d other than 128)."""
    lib = load_library()
    return int(lib.gdr2_forward_workspace_bytes(B, T, H, dk, dv, GDR2_BF16 if dtype == torch.bfloat16 else GDR2_F32))


@_one_device
def gdr2_forward(q, k, v, log_alpha, b, w, S0=None, *, final_state=True, save_states=False,
                 out=None, workspace=None, stream=None, out_gate=None, norm_weight=None, norm_eps=1e-6):
    """Chunkwise forward. Returns (o, S_T, saved_states); S_T / saved_states may be None.

    q, k, b: [B, T, H, dk]; v, w: [B, T, H, dv] (fp32 or bf16, one dtype);
    log_alpha: [B, T, H, dk] fp32; S0: [B, H, dk, dv] fp32 or None.
    b and/or w may instead be [B, T, H]: one gate value per token-head (scalar gates).
    out_gate ([B, T, H, dv], o's dtype) and norm_weight ([dv] fp32) apply the block's output
    epilogue o / rms(o) * norm_weight * silu(out_gate) in the kernel (bf16, d = 128 only).
    """
    lib = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    gates = _gates(b, w, (B, T, H))
    for name, t, shp in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)),
                         ("b", b, (B, T, H) if gates & GATE_SCALAR_B else (B, T, H, dk)),
                         ("v", v, (B, T, H, dv)), ("w", w, (B, T, H) if gates & GATE_SCALAR_W else (B, T, H, dv))):
        _check(t, name, shp, dt)
    _check(log_alpha, "log_alpha", (B, T, H, dk), torch.float32)
    _check(S0, "S0", (B, H, dk, dv), torch.float32)
    dev = q.device
    o = out if out is not None else torch.empty((B, T, H, dv), dtype=dt, device=dev)
    _check(o, "o", (B, T, H, dv), dt)
    S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if final_state else None
    nc = (T + CHUNK - 1) // CHUNK
    saved = torch.empty((B, H, nc, dk, dv), dtype=torch.float32, device=dev) if save_states else None
    need = gdr2_forward_workspace_bytes(B, T, H, dk, dv, dt)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if _epilogue(out_gate, norm_weight, (B, T, H, dv), dv, dt, dev):
        st = lib.gdr2_forward_ex(B, T, H, dk, dv, _dt(q), gates, None, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                 _ptr(b), _ptr(w), _ptr(S0), _ptr(out_gate), _ptr(norm_weight),
                                 ctypes.c_float(norm_eps), _ptr(o), _ptr(S_T), _ptr(saved), _ptr(workspace),
                                 ctypes.c_size_t(ws_bytes), _stream(stream))
    else:
        st = lib.gdr2_forward_gated(B, T, H, dk, dv, _dt(q), gates, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                    _ptr(b), _ptr(w), _ptr(S0), _ptr(o), _ptr(S_T), _ptr(saved), _ptr(workspace),
                                    ctypes.c_size_t(ws_bytes), _stream(stream))
    _raise(lib, st)
    return o, S_T, saved


def gdr2_forward_varlen_workspace_bytes(N, T, H, dk, dv, dtype=torch.bfloat16) -> int:
    """Device scratch gdr2_forward_varlen needs for N sequences of T tokens in all."""
    lib = load_library()
    return int(lib.gdr2_forward_varlen_workspace_bytes(N, T, H, dk, dv,
                                                       GDR2_BF16 if dtype == torch.bfloat16 else GDR2_F32))


@_one_device
def gdr2_forward_varlen(q, k, v, log_alpha, b, w, cu_seqlens, S0=None, *, final_state=True, save_states=False,
                        out=None, workspace=None, stream=None, out_gate=None, norm_weight=None, norm_eps=1e-6):
    """Forward over packed sequences. Returns (o, S_T, saved_states).

    q, k, b: [T, H, dk] (or [1, T, H, dk]); v, w: [T, H, dv]; bf16; log_alpha [T, H, dk] fp32;
    cu_seqlens: int32 [N + 1] on the device; S0: [N, H, dk, dv] fp32 or None; b and/or w may
    be [T, H] (scalar gates). saved_states,
    when asked for, is [H * (ceil(T / 64) + N), dk, dv] (see include/gdr2.h for the order).
    out_gate ([T, H, dv] bf16) and norm_weight ([dv] fp32): the output epilogue, as in gdr2_forward.
    """
    lib = load_library()
    sq4 = lambda t: None if t is None else (t[0] if t.dim() == 4 else t)  # noqa: E731
    q, k, v, log_alpha = (sq4(t) for t in (q, k, v, log_alpha))
    T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    sqg = lambda t: t[0] if t.dim() == 4 or (t.dim() == 3 and tuple(t.shape) == (1, T, H)) else t  # noqa: E731
    b, w = sqg(b), sqg(w)
    gates = _gates(b, w, (T, H))
    for name, t, shp in (("q", q, (T, H, dk)), ("k", k, (T, H, dk)),
                         ("b", b, (T, H) if gates & GATE_SCALAR_B else (T, H, dk)),
                         ("v", v, (T, H, dv)), ("w", w, (T, H) if gates & GATE_SCALAR_W else (T, H, dv))):
        _check(t, name, shp, dt)
    _check(log_alpha, "log_alpha", (T, H, dk), torch.float32)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() \
            or cu_seqlens.device != q.device:
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor on the inputs' device")
    N = cu_seqlens.numel() - 1
    _check(S0, "S0", (N, H, dk, dv), torch.float32)
    dev = q.device
    o = out if out is not None else torch.empty((T, H, dv), dtype=dt, device=dev)
    _check(sq4(o), "o", (T, H, dv), dt)
    S_T = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if final_state else None
    cap = H * ((T + CHUNK - 1) // CHUNK + N)
    saved = torch.empty((cap, dk, dv), dtype=torch.float32, device=dev) if save_states else None
    need = gdr2_forward_varlen_workspace_bytes(N, T, H, dk, dv, dt)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    out_gate = sq4(out_gate)
    if _epilogue(out_gate, norm_weight, (T, H, dv), dv, dt, dev):
        st = lib.gdr2_forward_ex(N, T, H, dk, dv, _dt(q), gates, _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v),
                                 _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(out_gate), _ptr(norm_weight),
                                 ctypes.c_float(norm_eps), _ptr(o), _ptr(S_T), _ptr(saved), _ptr(workspace),
                                 ctypes.c_size_t(ws_bytes), _stream(stream))
    else:
        st = lib.gdr2_forward_varlen(N, T, H, dk, dv, _dt(q), gates, _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(o), _ptr(S_T), _ptr(saved),
                                     _ptr(workspace), ctypes.c_size_t(ws_bytes), _stream(stream))
    _raise(lib, st)
    return o, S_T, saved


def _check_cu_seqlens(cu_seqlens, device):
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() \
            or cu_seqlens.device != device:
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor on the inputs' device")


@_one_device
def gdr2_short_conv_silu(x, weight, state=None, *, l2norm=False, eps=1e-6, cu_seqlens=None, final_state=False,
                         state_out=None, out=None, stream=None):
    """Block prologue of one branch: SiLU(causal depthwise convolution of x), then with
    l2norm the per-head L2 norm (query and key); without it, the value branch.

    x: [N, T, H, d] (dense) or [T, H, d] with cu_seqlens ([N + 1] int32); weight: [H * d, W]
    fp32 (a depthwise Conv1d weight [H * d, 1, W] too; the last tap is the current token);
    state: [N, W - 1, H, d] in x's dtype, the inputs before each sequence, or None (zeros).
    Returns (y, state_out): the state after the call when final_state or when a state_out
    tensor is given (state_out=state updates a decode step's state in place, T = 1), else None.
    """
    lib = load_library()
    if cu_seqlens is not None:
        T, H, d = x.shape
        _check_cu_seqlens(cu_seqlens, x.device)
        N = cu_seqlens.numel() - 1
    else:
        N, T, H, d = x.shape
    wgt = weight.reshape(weight.shape[0], weight.shape[-1]) if weight.dim() == 3 else weight
    W = int(wgt.shape[-1])
    dt = x.dtype
    _check(x, "x", tuple(x.shape), dt)
    _check(wgt, "weight", (H * d, W), torch.float32)
    _check(state, "state", (N, W - 1, H, d), dt)
    y = out if out is not None else torch.empty_like(x)
    _check(y, "out", tuple(x.shape), dt)
    if state_out is None and final_state:
        state_out = torch.empty((N, W - 1, H, d), dtype=dt, device=x.device)
    _check(state_out, "state_out", (N, W - 1, H, d), dt)
    ptr = lambda t: None if t is None or t.numel() == 0 else _ptr(t)  # noqa: E731
    st = lib.gdr2_short_conv_silu(N, T, H, d, _dt(x), W, int(bool(l2norm)), ctypes.c_float(eps), _ptr(cu_seqlens),
                                  ptr(x), ptr(wgt), ptr(state), ptr(state_out), ptr(y), _stream(stream))
    _raise(lib, st)
    return y, state_out


@_one_device
def gdr2_gate_activations(a=None, b=None, w=None, *, stream=None):
    """The decay and gate branches' activations, element by element, any of them None:
    log_alpha = -softplus(a) (fp32), sigmoid(b) and sigmoid(w) in the inputs' dtype."""
    lib = load_library()
    given = [t for t in (a, b, w) if t is not None]
    if not given:
        return None, None, None
    dt = given[0].dtype
    for name, t in (("a", a), ("b", b), ("w", w)):
        if t is not None:
            _check(t, name, tuple(t.shape), dt)
    la = None if a is None else torch.empty(tuple(a.shape), dtype=torch.float32, device=a.device)
    bo = None if b is None else torch.empty_like(b)
    wo = None if w is None else torch.empty_like(w)
    n = lambda t: 0 if t is None else t.numel()  # noqa: E731
    st = lib.gdr2_gate_activations(_dt(given[0]), n(a), _ptr(a), _ptr(la), n(b), _ptr(b), _ptr(bo), n(w), _ptr(w),
                                   _ptr(wo), _stream(stream))
    _raise(lib, st)
    return la, bo, wo


@_one_device
def gdr2_block_prologue(xq, xk, xv, conv_q, conv_k, conv_v, a, b, w, *, states=None, eps=1e-6, cu_seqlens=None,
                        final_state=False, stream=None):
    """The whole prologue: q, k = L2(SiLU(conv(x))) per head, v = SiLU(conv(x)), and the
    activations of a, b, w. states: (state_q, state_k, state_v) or None. Returns
    (q, k, v, log_alpha, b, w, new_states); new_states is a triple when final_state, else None."""
    sq, sk, sv = states if states is not None else (None, None, None)
    kw = dict(eps=eps, cu_seqlens=cu_seqlens, final_state=final_state, stream=stream)
    q, nq = gdr2_short_conv_silu(xq, conv_q, sq, l2norm=True, **kw)
    k, nk = gdr2_short_conv_silu(xk, conv_k, sk, l2norm=True, **kw)
    v, nv = gdr2_short_conv_silu(xv, conv_v, sv, l2norm=False, **kw)
    la, bo, wo = gdr2_gate_activations(a, b, w, stream=stream)
    return q, k, v, la, bo, wo, ((nq, nk, nv) if final_state else None)


@_one_device
def gdr2_short_conv_silu_backward(x, weight, dy, state=None, dstate_out=None, *, l2norm=False, eps=1e-6,
                                  want_dstate=None, workspace=None, stream=None):
    """Gradients of gdr2_short_conv_silu over dense sequences: of <y, dy> + <state_out, dstate_out>.

    x, dy: [N, T, H, d]; weight [H * d, W] fp32 (or [H * d, 1, W]); state, dstate_out:
    [N, W - 1, H, d] in x's dtype or None. Returns dict dx, dweight (weight's shape, fp32) and
    dstate (by default when a state is given, else None).
    """
    lib = load_library()
    N, T, H, d = x.shape
    wgt = weight.reshape(weight.shape[0], weight.shape[-1]) if weight.dim() == 3 else weight
    W = int(wgt.shape[-1])
    dt = x.dtype
    _check(x, "x", (N, T, H, d), dt)
    _check(dy, "dy", (N, T, H, d), dt)
    _check(wgt, "weight", (H * d, W), torch.float32)
    _check(state, "state", (N, W - 1, H, d), dt)
    _check(dstate_out, "dstate_out", (N, W - 1, H, d), dt)
    want = state is not None if want_dstate is None else want_dstate
    g = {"dx": torch.empty_like(x), "dweight": _like(weight), "dstate": x.new_empty((N, W - 1, H, d)) if want else None}
    if N * H == 0:
        g["dweight"].zero_()
    need = _scratch("gdr2_short_conv_silu_backward_workspace_bytes", x.device.index, N, T, H, d, W)
    workspace = _workspace(workspace, need, x.device)
    st = lib.gdr2_short_conv_silu_backward(N, T, H, d, _dt(x), W, int(bool(l2norm)), eps, _some(x),
                                           _some(wgt), _some(state), _some(dy), _some(dstate_out), _some(g["dx"]),
                                           _some(g["dweight"]), _some(g["dstate"]), _some(workspace),
                                           _nbytes(workspace), _stream(stream))
    _raise(lib, st)
    return g


def _some(t):
    """The data pointer; NULL for None (and for a tensor without elements, whose pointer is 0)."""
    return None if t is None else t.data_ptr()


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _like(t):
    """An uninitialised contiguous tensor of t's shape, dtype and device."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


@functools.lru_cache(maxsize=1024)
def _scratch(query, device, *sizes):
    """The bytes that the library's `query` asks for: a function of the sizes and of the (current) device alone."""
    return getattr(load_library(), query)(*sizes)


def _workspace(given, need, device):
    """The caller's workspace, or one of `need` bytes (None when nothing is needed)."""
    if given is not None:
        if not given.is_cuda or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        return given
    return torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None


def _rows(t, name, lead, width, dtype):
    """Checks a token tensor [*lead, width] whose rows may be views of a wider one (the last
    dimension dense, the same distance between all rows); returns that distance in elements."""
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape != (*lead, width):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(*lead, width)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.is_contiguous():  # so is a tensor without elements
        return width
    strides = t.stride()
    if width > 1 and strides[-1] != 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    return _row_distance(name, lead, strides, width)


def _ld(t, name, shape, dtype):
    """_rows of a tensor of `shape`, without a call or a tuple where it is contiguous."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return shape[-1]
    return _rows(t, name, tuple(shape[:-1]), shape[-1], dtype)


def _row_distance(name, lead, strides, width):
    """The one distance between rows of `width` elements over the leading dimensions, or a refusal."""
    ld, rows = None, 1  # distance between rows; the rows that the dimensions from here on hold
    for i in range(len(lead) - 1, -1, -1):
        n = lead[i]
        if n > 1:
            if ld is None:
                ld = strides[i]
            if strides[i] != ld * rows:
                raise ValueError(f"the rows of {name} must all be the same distance apart")
        rows *= n
    ld = width if ld is None else ld
    if ld < width:
        raise ValueError(f"the rows of {name} overlap")
    return ld


def _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, packed=None):
    """Checks the inputs that the scan, its step and its backward share; returns their sizes
    and the C arguments x .. step_bias."""
    shape, t = x.shape, x.dtype
    lead, C = tuple(shape[:-1]), shape[-1]
    N = A.shape[-1]
    states = (*lead, N)
    ldx, ldt, ldz = _ld(x, "x", shape, t), _ld(dt, "dt", shape, t), _ld(z, "z", shape, t)
    ldb, ldc = _ld(Bm, "Bm", states, t), _ld(Cm, "Cm", states, t)
    _check(A, "A", (C, N), torch.float32)
    if D is not None:
        _check(D, "D", (C,), torch.float32)
    if dt_bias is not None:
        _check(dt_bias, "dt_bias", (C,), torch.float32)
    if packed is not None:
        _check_cu_seqlens(packed, x.device)
    args = (_some(x), ldx, _some(dt), ldt, _some(A), _some(Bm), ldb, _some(Cm), ldc, _some(D), _some(z), ldz,
            _some(dt_bias))
    return lead, C, N, t, args


@_one_device
def gdr2_ssm_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, S0=None, *, softplus=True, cu_seqlens=None,
                  final_state=True, save_states=False, out=None, workspace=None, stream=None):
    """Selective state-space scan over whole sequences. Returns (y, S_T, saved_states).

    h_t = exp(s_t A) h_{t-1} + s_t Bm_t x_t with s_t = softplus(dt_t + dt_bias) (softplus=False:
    dt_t + dt_bias); y_t = (Cm_t . h_t + D x_t) * silu(z_t).
    x, dt, z: [B, T, C]; Bm, Cm: [B, T, N] (one dtype, fp32 or bf16; views of fused projections
    keep their row stride); with cu_seqlens (int32 [B + 1], nondecreasing from 0 to T; not checked: other values give
    unspecified outputs) [T, .], packed. A: [C, N], D, dt_bias:
    [C], S0, S_T: [B, C, N] fp32; N is 8, 16, 32 or 64. saved_states, when asked for (dense):
    [B, ceil(T / 16), C, N], for gdr2_ssm_scan_backward.
    """
    lib = load_library()
    if x.dim() != (2 if cu_seqlens is not None else 3):
        raise ValueError("x must be [B, T, C], or [T, C] with cu_seqlens")
    lead, C, N, t, args = _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, cu_seqlens)
    T = lead[-1]
    B = lead[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    dev = x.device
    _check(S0, "S0", (B, C, N), torch.float32)
    y = _like(x) if out is None else out
    _check(out, "out", x.shape, t)
    S_T = A.new_empty((B, C, N)) if final_state else None
    if save_states and cu_seqlens is not None:
        raise ValueError("save_states is for dense sequences (the backward takes no cu_seqlens)")
    saved = A.new_empty((B, -(-T // SSM_CHUNK), C, N)) if save_states else None
    need = _scratch("gdr2_ssm_scan_workspace_bytes", dev.index, B if cu_seqlens is None else 1, T, C, N)
    workspace = _workspace(workspace, need, dev)
    st = lib.gdr2_ssm_scan(B, T, C, N, _dt(x), int(bool(softplus)), _ptr(cu_seqlens), *args, _some(S0), _some(y),
                           _some(S_T), _some(saved), _some(workspace), _nbytes(workspace), _stream(stream))
    _raise(lib, st)
    return y, S_T, saved


@_one_device
def gdr2_ssm_step(x, dt, A, Bm, Cm, S, D=None, z=None, dt_bias=None, *, softplus=True, out=None, stream=None):
    """One token of gdr2_ssm_scan for B resident states: x, dt, z [B, C], Bm, Cm [B, N]; S
    [B, C, N] fp32 is updated in place. Returns y [B, C]."""
    lib = load_library()
    lead, C, N, t, args = _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias)
    if len(lead) != 1:
        raise ValueError("x must be [B, C]")
    _check(S, "S", (*lead, C, N), torch.float32)
    y = _like(x) if out is None else out
    _check(out, "out", x.shape, t)
    st = lib.gdr2_ssm_step(lead[0], C, N, _dt(x), int(bool(softplus)), *args, _some(S), _some(y), _stream(stream))
    _raise(lib, st)
    return y


@_one_device
def gdr2_ssm_scan_backward(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, S0=None, dS_T=None, saved_states=None,
                           *, softplus=True, want_dS0=True, workspace=None, stream=None):
    """Gradients of <y, dy> + <S_T, dS_T> of the dense gdr2_ssm_scan. Returns dict dx, ddt, dBm, dCm
    (x's dtype), dA, dD, ddt_bias, dS0 (fp32) and dz; those of absent inputs are None (dS0 by want_dS0).
    Without saved_states the states are formed again."""
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    (B, T), C, N, t, args = _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias)
    dev = x.device
    _check(dy, "dy", (B, T, C), t)
    _check(S0, "S0", (B, C, N), torch.float32)
    _check(dS_T, "dS_T", (B, C, N), torch.float32)
    _check(saved_states, "saved_states", (B, -(-T // SSM_CHUNK), C, N), torch.float32)
    g = {"dx": _like(x), "ddt": _like(dt), "dA": _like(A), "dBm": _like(Bm), "dCm": _like(Cm),
         "dD": None if D is None else _like(D), "dz": None if z is None else _like(z),
         "ddt_bias": None if dt_bias is None else _like(dt_bias),
         "dS0": A.new_empty((B, C, N)) if want_dS0 else None}
    need = _scratch("gdr2_ssm_scan_backward_workspace_bytes", dev.index, B, T, C, N, int(saved_states is not None))
    workspace = _workspace(workspace, need, dev)
    st = lib.gdr2_ssm_scan_backward(B, T, C, N, _dt(x), int(bool(softplus)), *args, _some(S0), _some(dy), _some(dS_T),
                                    _some(saved_states), *(_some(g[k]) for k in ("dx", "ddt", "dA", "dBm", "dCm", "dD",
                                                                                 "dz", "ddt_bias", "dS0")),
                                    _some(workspace), _nbytes(workspace), _stream(stream))
    _raise(lib, st)
    return g


_NORMS = {None: 0, "rms": 1, "l2": 2}


def _head_rows(v, name, shape, dtype):
    """As _rows, of tokens of heads that lie dense and side by side."""
    if v is None:
        return 0
    if not v.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if v.shape != shape:
        raise ValueError(f"{name} has shape {tuple(v.shape)}, expected {shape}")
    if v.dtype != dtype:
        raise TypeError(f"{name} has dtype {v.dtype}, expected {dtype}")
    H, d = shape[2:]
    if v.is_contiguous():
        return H * d
    strides = v.stride()
    if strides[-1] != 1 or (H > 1 and strides[-2] != d):
        raise ValueError(f"the heads of {name} must be dense and side by side")
    return _row_distance(name, shape[:2], strides, H * d)


def _rope_inputs(q, k, q_weight, k_weight, cos_sin, positions, norm, eps, interleaved, first_position):
    if norm not in _NORMS:
        raise ValueError(f"norm must be 'rms', 'l2' or None, not {norm!r}")
    if not -2 ** 31 <= first_position < 2 ** 31:  # a C int would take its low 32 bits
        raise ValueError(f"first_position {first_position} does not fit into 32 bits")
    B, T, Hq, d = q.shape
    Hk = 0 if k is None else k.shape[2]
    t = q.dtype
    ldq, ldk = _head_rows(q, "q", (B, T, Hq, d), t), _head_rows(k, "k", (B, T, Hk, d), t)
    _check(q_weight, "q_weight", (d,), torch.float32)
    _check(k_weight, "k_weight", (d,), torch.float32)
    R = P = 0
    if cos_sin is not None:
        P, R = cos_sin.shape
        _check(cos_sin, "cos_sin", (P, R), torch.float32)
    _check(positions, "positions", (B, T), torch.int32)
    return (B, T, Hq, Hk, d, _dt(q), _NORMS[norm], eps, _some(q), ldq, _some(k), ldk,
            _some(q_weight), _some(k_weight), R, int(bool(interleaved)), _some(cos_sin), P, _some(positions),
            int(first_position))


@_one_device
def gdr2_head_norm_rope(q, k=None, q_weight=None, k_weight=None, cos_sin=None, positions=None, *, norm="rms",
                        eps=1e-6, interleaved=False, first_position=0, q_out=None, k_out=None, stream=None):
    """Norm of queries and keys per head and rotation by position, in one pass. Returns (q_out, k_out).

    q: [B, T, Hq, d], k: [B, T, Hk, d] or None, views of a fused projection as they are (heads side by
    side, d 64, 128 or 256); norm "rms" (x / sqrt(mean x^2 + eps)), "l2" (sum) or None; weights [d] fp32
    or None. cos_sin [P, R] fp32 holds each position's R / 2 cosines and then sines (None: no rotation);
    the first R channels turn in pairs (j, j + R / 2), or (2j, 2j + 1) if interleaved. positions [B, T]
    int32, or None: token t is at first_position + t. A position outside the table leaves its token
    unturned and the next gdr2_sync_status raises.
    """
    lib = load_library()
    args = _rope_inputs(q, k, q_weight, k_weight, cos_sin, positions, norm, eps, interleaved, first_position)
    qo = _like(q) if q_out is None else q_out
    _check(q_out, "q_out", q.shape, q.dtype)
    ko = None
    if k is not None:
        ko = _like(k) if k_out is None else k_out
        _check(k_out, "k_out", k.shape, q.dtype)
    _raise(lib, lib.gdr2_head_norm_rope(*args, _some(qo), _some(ko), _stream(stream)))
    return qo, ko


@_one_device
def gdr2_head_norm_rope_backward(q, k, dq_out, dk_out=None, q_weight=None, k_weight=None, cos_sin=None, positions=None,
                                 *, norm="rms", eps=1e-6, interleaved=False, first_position=0, workspace=None,
                                 stream=None):
    """Gradients of gdr2_head_norm_rope from its inputs and the outputs' gradients (contiguous).
    Returns dict dq, dk, dq_weight, dk_weight (None for absent inputs)."""
    lib = load_library()
    args = _rope_inputs(q, k, q_weight, k_weight, cos_sin, positions, norm, eps, interleaved, first_position)
    d, dev = q.shape[-1], q.device
    _check(dq_out, "dq_out", tuple(q.shape), q.dtype)
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out: both or neither")
    if k is not None:
        _check(dk_out, "dk_out", tuple(k.shape), q.dtype)
    g = {n: None if t is None else _like(t)
         for n, t in (("dq", q), ("dk", k), ("dq_weight", q_weight), ("dk_weight", k_weight))}
    workspace = _workspace(workspace, lib.gdr2_head_norm_rope_backward_workspace_bytes(d), dev)
    st = lib.gdr2_head_norm_rope_backward(*args, _some(dq_out), _some(dk_out), _some(g["dq"]), _some(g["dk"]),
                                          _some(g["dq_weight"]), _some(g["dk_weight"]), _some(workspace),
                                          _nbytes(workspace), _stream(stream))
    _raise(lib, st)
    return g


@_one_device
def gdr2_segment_states(A, Bst, S0=None, *, final_state=True, stream=None):
    """States entering the segments of split sequences (see include/gdr2.h).

    A: [B, G, H, dk, dk] fp32 segment transitions; Bst: [B, G, H, dk, dv] fp32 segment
    offsets; S0: [B, H, dk, dv] fp32 or None. Returns (S_starts [B, G, H, dk, dv], S_T or None).
    """
    lib = load_library()
    B, G, H, dk, dv = Bst.shape
    _check(A, "A", (B, G, H, dk, dk), torch.float32)
    _check(Bst, "Bst", (B, G, H, dk, dv), torch.float32)
    _check(S0, "S0", (B, H, dk, dv), torch.float32)
    S_starts = torch.empty_like(Bst)
    S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=Bst.device) if final_state else None
    st = lib.gdr2_segment_states(B, G, H, dk, dv, _ptr(A), _ptr(Bst), _ptr(S0), _ptr(S_starts), _ptr(S_T),
                                 _stream(stream))
    _raise(lib, st)
    return S_starts, S_T


@_one_device
def gdr2_decode_step(q, k, v, log_alpha, b, w, S, *, out=None, stream=None):
    """One decode token; S [N, H, dk, dv] fp32 is updated in place. Returns o [N, H, dv].

    b and/or w may be [N, H]: one gate value per token-head (scalar gates).
    """
    lib = load_library()
    N, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    gates = _gates(b, w, (N, H))
    for name, t, shp in (("q", q, (N, H, dk)), ("k", k, (N, H, dk)),
                         ("b", b, (N, H) if gates & GATE_SCALAR_B else (N, H, dk)),
                         ("v", v, (N, H, dv)), ("w", w, (N, H) if gates & GATE_SCALAR_W else (N, H, dv))):
        _check(t, name, shp, dt)
    _check(log_alpha, "log_alpha", (N, H, dk), torch.float32)
    _check(S, "S", (N, H, dk, dv), torch.float32)
    o = out if out is not None else torch.empty((N, H, dv), dtype=dt, device=q.device)
    _check(o, "o", (N, H, dv), dt)
    st = lib.gdr2_decode_step_gated(N, H, dk, dv, _dt(q), gates, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                    _ptr(b), _ptr(w), _ptr(S), _ptr(o), _stream(stream))
    _raise(lib, st)
    return o


def gdr2_backward_workspace_bytes(B, T, H, dk, dv, dtype=torch.bfloat16) -> int:
    """Device scratch gdr2_backward needs for this problem."""
    lib = load_library()
    return int(lib.gdr2_backward_workspace_bytes(B, T, H, dk, dv, GDR2_BF16 if dtype == torch.bfloat16 else GDR2_F32))


@_one_device
def gdr2_backward(q, k, v, log_alpha, b, w, dO, S0=None, dS_T=None, saved_states=None, *,
                  want_dS0=True, workspace=None, stream=None):
    """Gradients of <o, dO> + <S_T, dS_T>. Returns dict dq, dk, dv, dlog_alpha, db, dw, dS0.

    b or w shaped [B, T, H] (one value per token-head) are scalar gates; their gradients
    have the same shape (the tensor-core path: bf16 with dk = dv = 128).
    """
    lib = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    gates = _gates(b, w, (B, T, H))
    for name, t, shp in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)),
                         ("b", b, (B, T, H) if gates & GATE_SCALAR_B else (B, T, H, dk)),
                         ("v", v, (B, T, H, dv)), ("w", w, (B, T, H) if gates & GATE_SCALAR_W else (B, T, H, dv)),
                         ("dO", dO, (B, T, H, dv))):
        _check(t, name, shp, dt)
    _check(log_alpha, "log_alpha", (B, T, H, dk), torch.float32)
    _check(S0, "S0", (B, H, dk, dv), torch.float32)
    _check(dS_T, "dS_T", (B, H, dk, dv), torch.float32)
    nc = (T + CHUNK - 1) // CHUNK
    _check(saved_states, "saved_states", (B, H, nc, dk, dv), torch.float32)
    dev = q.device
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dlog_alpha": torch.empty_like(log_alpha), "db": torch.empty_like(b), "dw": torch.empty_like(w),
         "dS0": torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if want_dS0 else None}
    need = gdr2_backward_workspace_bytes(B, T, H, dk, dv, dt)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    st = lib.gdr2_backward_gated(B, T, H, dk, dv, _dt(q), gates, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                 _ptr(b), _ptr(w), _ptr(S0), _ptr(dO), _ptr(dS_T), _ptr(saved_states),
                                 _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_alpha"]), _ptr(g["db"]),
                                 _ptr(g["dw"]), _ptr(g["dS0"]), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
                                 _stream(stream))
    _raise(lib, st)
    return g


@_one_device
def gdr2_backward_noalloc(q, k, v, log_alpha, b, w, dO, S0=None, dS_T=None, saved_states=None, *,
                          want_dS0=True, stream=None):
    """gdr2_backward through the entry point that allocates nothing on the device.

    The library uses its own fixed scratch array (NOALLOC_SCRATCH_BYTES per
    device) instead of a workspace; the gradient tensors returned here are
    ordinary torch allocations made by this binding, not by the library.
    """
    lib = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    for name, t, shp in (("q", q, (B, T, H, dk)), ("k", k, (B, T, H, dk)), ("b", b, (B, T, H, dk)),
                         ("v", v, (B, T, H, dv)), ("w", w, (B, T, H, dv)), ("dO", dO, (B, T, H, dv))):
        _check(t, name, shp, dt)
    _check(log_alpha, "log_alpha", (B, T, H, dk), torch.float32)
    _check(S0, "S0", (B, H, dk, dv), torch.float32)
    _check(dS_T, "dS_T", (B, H, dk, dv), torch.float32)
    nc = (T + CHUNK - 1) // CHUNK
    _check(saved_states, "saved_states", (B, H, nc, dk, dv), torch.float32)
    dev = q.device
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dlog_alpha": torch.empty_like(log_alpha), "db": torch.empty_like(b), "dw": torch.empty_like(w),
         "dS0": torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if want_dS0 else None}
    st = lib.gdr2_backward_noalloc(B, T, H, dk, dv, _dt(q), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                   _ptr(b), _ptr(w), _ptr(S0), _ptr(dO), _ptr(dS_T), _ptr(saved_states),
                                   _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_alpha"]),
                                   _ptr(g["db"]), _ptr(g["dw"]), _ptr(g["dS0"]), _stream(stream))
    _raise(lib, st)
    return g
