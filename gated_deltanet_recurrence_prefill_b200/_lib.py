"""ctypes binding of libgdn.so: torch tensors in, torch tensors out."""
from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(HERE, "libgdn.so")
_lib = None

STATUS = {
    0: "GDN_OK",
    1: "GDN_ERR_INVALID_ARG",
    2: "GDN_ERR_UNSUPPORTED",
    3: "GDN_ERR_MISALIGNED",
    4: "GDN_ERR_CUDA",
    5: "GDN_ERR_TIMEOUT",
    6: "GDN_ERR_WORKSPACE",
}

# exported symbol -> (restype, argtypes)
_vp, _i32, _i64, _f32, _sz = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t
SIGNATURES = {
    "gdn_abi_version": (C.c_int, []),
    "gdn_status_string": (C.c_char_p, [C.c_int]),
    "gdn_last_cuda_error": (C.c_int, []),
    "gdn_last_cuda_error_string": (C.c_char_p, []),
    "gdn_conv1d_silu": (C.c_int, [_vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                  _vp, _vp]),
    "gdn_prefill_workspace_size": (_sz, [_i32, _i64, _i32, _i32, _i32]),
    "gdn_prefill": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32,
                              _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "gdn_prefill_status": (C.c_int, [_vp, _vp]),
    "gdn_prefill_bf16": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32,
                                   _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "gdn_check_async": (C.c_int, [_vp, _vp, _vp]),
    "gdn_layer_prefill_host_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "gdn_layer_prefill_host": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _f32,
                                         _i32, _vp, _vp, _vp, _vp, _sz, _vp, _vp, _vp]),
    "gdn_prefill_noalloc": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32,
                                      _i32, _f32, _vp, _vp, _vp, _vp]),
    "gdn_decode_step": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                  _f32, _vp, _vp, _vp]),
    "gdn_decode_step_fused": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                        _i32, _i32, _f32, _i32, _vp, _vp, _vp]),
    "gdn_decode_step_bf16": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                       _i32, _f32, _vp, _vp, _vp]),
    "gdn_decode_step_fused_bf16": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                             _i32, _i32, _i32, _f32, _i32, _vp, _vp, _vp]),
    "gdn_gated_norm": (C.c_int, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _f32, _vp, _vp]),
    "gdn_selftest_bounded_wait": (C.c_int, [_i32, _i64, _vp, _vp]),
    "gdn_prefill_backward_workspace_size": (_sz, [_i32, _i64, _i32, _i32]),
    "gdn_prefill_backward": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32,
                                       _i32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _vp, _vp, _sz, _vp]),
    "gdn_gated_norm_backward_workspace_size": (_sz, [_i64, _i32, _i32, _i32]),
    "gdn_gated_norm_backward": (C.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _f32, _vp, _vp, _vp,
                                          _vp, _sz, _vp]),
    "gdn_conv1d_silu_backward_workspace_size": (_sz, [_i64, _i32, _i32, _i32]),
    "gdn_conv1d_silu_backward": (C.c_int, [_vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                           _vp, _vp, _vp, _vp, _sz, _vp]),
    "gdn_prefill_backward_chunked_workspace_size": (_sz, [_i32, _i64, _i32, _i32]),
    "gdn_prefill_backward_chunked": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32,
                                               _i32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                               _vp, _vp, _sz, _vp]),
    "gdn_decode_step_gated": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                        _i32, _f32, _vp, _i32, _vp, _vp, _vp, _f32, _vp, _vp]),
    "gdn_prefill_gated": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32,
                                    _i32, _f32, _vp, _vp, _vp, _vp, _vp, _f32, _vp, _vp, _sz, _vp]),
    "gdn_linear_prefill_workspace_size": (_sz, [_i32, _i64, _i32, _i32, _i32]),
    "gdn_linear_prefill": (C.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp, _i32, _i64, _i32, _i32, _i32,
                                     _f32, _vp, _vp, _vp, _i32, _vp, _sz, _vp]),
    "gdn_linear_prefill_backward_workspace_size": (_sz, [_i32, _i64, _i32, _i32, _i32]),
    "gdn_linear_prefill_backward": (C.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp, _i32, _i64, _i32,
                                              _i32, _i32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp,
                                              _sz, _vp]),
    "gdn_linear_decode_step": (C.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _f32, _i32,
                                         _vp, _i32, _vp, _i32, _vp]),
    "gdn_state_copy": (C.c_int, [_vp, _i32, _i32, _vp, _vp, _i32, _vp]),
    "gdn_state_workspace_size": (_sz, [_i32]),
    "gdn_state_fork": (C.c_int, [_vp, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _sz, _vp]),
    "gdn_state_compact": (C.c_int, [_vp, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "gdn_state_free": (C.c_int, [_vp, _i32, _vp, _i32, _vp]),
}


class StateBuffer(C.Structure):
    """gdn_state_buffer."""
    _fields_ = [("data", C.c_void_p), ("slot_bytes", C.c_int64)]


class GdnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = f"{fn} failed: {STATUS.get(status, status)}"
        if status == 4 and _lib is not None:
            msg += f" ({_lib.gdn_last_cuda_error_string().decode()})"
        super().__init__(msg)
        self.status = status


def lib_path() -> str:
    return _LIB_PATH


def lib():
    """Load libgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"libgdn.so not built at {_LIB_PATH}: run "
                              "`python -m gated_deltanet_recurrence_prefill_b200.build`")
        L = C.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _check(fn, status):
    if status != 0:
        raise GdnError(fn, status)


def _need(t, dtype, shape, name, device="cuda"):
    import torch
    if t is None:
        raise ValueError(f"{name} is required")
    if device == "cuda" and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device == "cpu" and t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    del torch
    return t


def conv1d_silu(qkv, conv_w, Hqk, Hv, d=128, cu_seqlens=None, conv_state_in=None,
                conv_state_out=None, out=None, stream=None):
    """Front end.  qkv [T, (2Hqk+Hv)d] bf16, conv_w [Ctot, 4] f32.
    Returns (q [T,Hqk,d], k [T,Hqk,d], v [T,Hv,d]) bf16."""
    import torch
    T = qkv.shape[0]
    ctot = (2 * Hqk + Hv) * d
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _need(qkv, torch.bfloat16, (T, ctot), "qkv")
    _need(conv_w, torch.float32, (ctot, 4), "conv_w")
    if cu_seqlens is not None:
        _need(cu_seqlens, torch.int32, (n_seq + 1,), "cu_seqlens")
    for nm, t in (("conv_state_in", conv_state_in), ("conv_state_out", conv_state_out)):
        if t is not None:
            _need(t, torch.float32, (n_seq, ctot, 3), nm)
    if out is None:
        q = torch.empty(T, Hqk, d, dtype=torch.bfloat16, device=qkv.device)
        k = torch.empty(T, Hqk, d, dtype=torch.bfloat16, device=qkv.device)
        v = torch.empty(T, Hv, d, dtype=torch.bfloat16, device=qkv.device)
    else:
        q, k, v = out
    st = lib().gdn_conv1d_silu(_ptr(qkv), _ptr(conv_w), _ptr(cu_seqlens), n_seq, T, Hqk, Hv, d,
                               _ptr(conv_state_in), _ptr(conv_state_out), _ptr(q), _ptr(k), _ptr(v),
                               _stream(stream))
    _check("gdn_conv1d_silu", st)
    return q, k, v


def _outputs(given, shapes, dev):
    """float32 output tensors of the given shapes (None: not wanted), taken from
    the caller's dict `given` where it has them (checked), else allocated."""
    import torch
    out = {}
    for name, shape in shapes.items():
        if shape is None:
            out[name] = None
        elif given is not None and given.get(name) is not None:
            _need(given[name], torch.float32, shape, name)
            out[name] = given[name]
        else:
            out[name] = torch.empty(*shape, dtype=torch.float32, device=dev)
    return out


def conv1d_silu_backward(qkv, conv_w, dq, dk, dv, Hqk, Hv, d=128, cu_seqlens=None, conv_state=None,
                         want_d_conv_state=True, workspace=None, stream=None, out=None):
    """gdn_conv1d_silu_backward: the front end's gradient given dL/dq, dL/dk
    [T, Hqk, d] and dL/dv [T, Hv, d] (float32).  Returns a dict of float32
    tensors d_qkv [T, Ctot], d_conv_w [Ctot, 4] and d_conv_state [N, Ctot, 3]
    (or None).  out: an optional dict of preallocated tensors under those names."""
    import torch
    T = qkv.shape[0]
    ctot = (2 * Hqk + Hv) * d
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _need(qkv, torch.bfloat16, (T, ctot), "qkv")
    _need(conv_w, torch.float32, (ctot, 4), "conv_w")
    _need(dq, torch.float32, (T, Hqk, d), "dq")
    _need(dk, torch.float32, (T, Hqk, d), "dk")
    _need(dv, torch.float32, (T, Hv, d), "dv")
    if cu_seqlens is not None:
        _need(cu_seqlens, torch.int32, (n_seq + 1,), "cu_seqlens")
    if conv_state is not None:
        _need(conv_state, torch.float32, (n_seq, ctot, 3), "conv_state")
    dev = qkv.device
    out = _outputs(out, dict(d_qkv=(T, ctot), d_conv_w=(ctot, 4),
                             d_conv_state=(n_seq, ctot, 3) if want_d_conv_state else None), dev)
    ws_bytes = int(lib().gdn_conv1d_silu_backward_workspace_size(T, Hqk, Hv, d))
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = lib().gdn_conv1d_silu_backward(
        _ptr(qkv), _ptr(conv_w), _ptr(cu_seqlens), n_seq, T, Hqk, Hv, d, _ptr(conv_state), _ptr(dq), _ptr(dk),
        _ptr(dv), _ptr(out["d_qkv"]), _ptr(out["d_conv_w"]), _ptr(out["d_conv_state"]), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    _check("gdn_conv1d_silu_backward", st)
    return out


def gated_norm_backward(o, z, norm_w, dy, eps=1e-6, workspace=None, stream=None, out=None):
    """gdn_gated_norm_backward: the gated norm's gradient given dL/dy [T, Hv, d]
    (float32).  o [T, Hv, d] float32, z [T, Hv, d] bf16, norm_w [layers, d] or
    [d] float32.  Returns a dict of float32 tensors d_o, d_z [T, Hv, d] and
    d_norm_w (shaped as norm_w).  out: an optional dict of preallocated tensors
    under those names (d_norm_w as [layers, d])."""
    import torch
    T, Hv, d = o.shape
    w2 = norm_w if norm_w.dim() == 2 else norm_w.view(1, -1)
    layers = w2.shape[0]
    _need(o, torch.float32, (T, Hv, d), "o")
    _need(z, torch.bfloat16, (T, Hv, d), "z")
    _need(w2, torch.float32, (layers, d), "norm_w")
    _need(dy, torch.float32, (T, Hv, d), "dy")
    dev = o.device
    out = _outputs(out, dict(d_o=(T, Hv, d), d_z=(T, Hv, d), d_norm_w=(layers, d)), dev)
    ws_bytes = int(lib().gdn_gated_norm_backward_workspace_size(T, Hv, d, layers))
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = lib().gdn_gated_norm_backward(
        _ptr(o), _ptr(z), _ptr(w2), _ptr(dy), T, Hv, d, layers, float(eps), _ptr(out["d_o"]), _ptr(out["d_z"]),
        _ptr(out["d_norm_w"]), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    _check("gdn_gated_norm_backward", st)
    if norm_w.dim() == 1:
        out["d_norm_w"] = out["d_norm_w"].view(-1)
    return out


def prefill_workspace_size(n_seq, T, Hqk, Hv, d=128) -> int:
    return int(lib().gdn_prefill_workspace_size(n_seq, T, Hqk, Hv, d))


def prefill(q, k, v, a, b, A_log, dt_bias, cu_seqlens=None, scale=None, initial_state=None,
            final_state=None, o=None, workspace=None, want_final_state=True, stream=None,
            o_dtype=None):
    """Chunked prefill.  Returns (o [T,Hv,d], final_state [N,Hv,d,d] f32 or None).
    o is float32 (gdn_prefill), or bf16 (gdn_prefill_bf16) when o_dtype is
    torch.bfloat16 or a bf16 `o` is passed."""
    import torch
    if o_dtype is None:
        o_dtype = o.dtype if o is not None else torch.float32
    if o_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("o must be float32 or bfloat16")
    T, Hqk, d = q.shape
    Hv = v.shape[1]
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _need(q, torch.bfloat16, (T, Hqk, d), "q")
    _need(k, torch.bfloat16, (T, Hqk, d), "k")
    _need(v, torch.bfloat16, (T, Hv, d), "v")
    _need(a, torch.float32, (T, Hv), "a")
    _need(b, torch.float32, (T, Hv), "b")
    _need(A_log, torch.float32, (Hv,), "A_log")
    _need(dt_bias, torch.float32, (Hv,), "dt_bias")
    if cu_seqlens is not None:
        _need(cu_seqlens, torch.int32, (n_seq + 1,), "cu_seqlens")
    if initial_state is not None:
        _need(initial_state, torch.float32, (n_seq, Hv, d, d), "initial_state")
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty(T, Hv, d, dtype=o_dtype, device=q.device)
    _need(o, o_dtype, (T, Hv, d), "o")
    if final_state is None and want_final_state:
        final_state = torch.empty(n_seq, Hv, d, d, dtype=torch.float32, device=q.device)
    ws_bytes = prefill_workspace_size(n_seq, T, Hqk, Hv, d)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    fn, name = ((lib().gdn_prefill_bf16, "gdn_prefill_bf16") if o_dtype == torch.bfloat16
                else (lib().gdn_prefill, "gdn_prefill"))
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
            _ptr(cu_seqlens), n_seq, T, Hqk, Hv, d, float(scale),
            _ptr(initial_state), _ptr(final_state), _ptr(o), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    _check(name, st)
    return o, final_state


_copy_streams = {}


def layer_prefill_host(h_qkv, h_a, h_b, conv_w, A_log, dt_bias, Hqk, Hv, h_o=None, h_final_state=None,
                       conv_state_in=None, initial_state=None, conv_state_out=None, n_blocks=8, scale=None,
                       workspace=None, stream=None, copy_streams=None):
    """gdn_layer_prefill_host: front end + prefill of one sequence from pinned
    host tensors (h_qkv [T, (2Hqk+Hv)d] bf16, h_a, h_b [T, Hv] f32) to pinned
    host tensors (h_o [T, Hv, d] f32, h_final_state [Hv, d, d] f32), the copies
    overlapped with the compute over n_blocks token ranges.  conv_w, A_log,
    dt_bias, conv_state_in / _out and initial_state are device tensors.
    copy_streams: (upload, download) torch streams; by default two streams kept
    per device.  Returns (h_o, h_final_state), ready once `stream` (default: the
    current stream) reaches the point after the call."""
    import torch
    d = 128
    T = h_qkv.shape[0]
    dev = conv_w.device
    _need(h_qkv, torch.bfloat16, (T, (2 * Hqk + Hv) * d), "h_qkv", device="cpu")
    _need(h_a, torch.float32, (T, Hv), "h_a", device="cpu")
    _need(h_b, torch.float32, (T, Hv), "h_b", device="cpu")
    if h_o is None:
        h_o = torch.empty(T, Hv, d, dtype=torch.float32).pin_memory()
    if h_final_state is None:
        h_final_state = torch.empty(Hv, d, d, dtype=torch.float32).pin_memory()
    _need(h_o, torch.float32, (T, Hv, d), "h_o", device="cpu")
    _need(h_final_state, torch.float32, (Hv, d, d), "h_final_state", device="cpu")
    if scale is None:
        scale = d ** -0.5
    ws_bytes = lib().gdn_layer_prefill_host_workspace_size(T, Hqk, Hv, d, n_blocks)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    if copy_streams is None:
        key = dev.index if dev.index is not None else torch.cuda.current_device()
        if key not in _copy_streams:
            _copy_streams[key] = (torch.cuda.Stream(device=dev), torch.cuda.Stream(device=dev))
        copy_streams = _copy_streams[key]
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    st = lib().gdn_layer_prefill_host(
        _ptr(h_qkv), _ptr(h_a), _ptr(h_b), _ptr(conv_w), _ptr(A_log), _ptr(dt_bias), _ptr(conv_state_in),
        _ptr(initial_state), T, Hqk, Hv, d, float(scale), n_blocks, _ptr(h_o), _ptr(h_final_state),
        _ptr(conv_state_out), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream),
        _stream(copy_streams[0]), _stream(copy_streams[1]))
    _check("gdn_layer_prefill_host", st)
    return h_o, h_final_state


def prefill_noalloc(q, k, v, a, b, A_log, dt_bias, cu_seqlens=None, scale=None,
                    initial_state=None, final_state=None, o=None, want_final_state=True,
                    stream=None):
    """gdn_prefill_noalloc: the chunked prefill without a caller-provided
    workspace, for callers that cannot allocate device memory (the library
    uses its own fixed 64 KiB device array; see include/gdn.h).  The output
    tensors are created here only when not passed in."""
    import torch
    T, Hqk, d = q.shape
    Hv = v.shape[1]
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _need(q, torch.bfloat16, (T, Hqk, d), "q")
    _need(k, torch.bfloat16, (T, Hqk, d), "k")
    _need(v, torch.bfloat16, (T, Hv, d), "v")
    _need(a, torch.float32, (T, Hv), "a")
    _need(b, torch.float32, (T, Hv), "b")
    _need(A_log, torch.float32, (Hv,), "A_log")
    _need(dt_bias, torch.float32, (Hv,), "dt_bias")
    if cu_seqlens is not None:
        _need(cu_seqlens, torch.int32, (n_seq + 1,), "cu_seqlens")
    if initial_state is not None:
        _need(initial_state, torch.float32, (n_seq, Hv, d, d), "initial_state")
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty(T, Hv, d, dtype=torch.float32, device=q.device)
    if final_state is None and want_final_state:
        final_state = torch.empty(n_seq, Hv, d, d, dtype=torch.float32, device=q.device)
    st = lib().gdn_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(A_log),
                                   _ptr(dt_bias), _ptr(cu_seqlens), n_seq, T, Hqk, Hv, d,
                                   float(scale), _ptr(initial_state), _ptr(final_state), _ptr(o),
                                   _stream(stream))
    _check("gdn_prefill_noalloc", st)
    return o, final_state


def prefill_status(workspace, stream=None) -> int:
    """Error word left by the last prefill on `workspace` (waits for the stream);
    workspace None: the array of gdn_prefill_noalloc on the current device."""
    return int(lib().gdn_prefill_status(_ptr(workspace), _stream(stream)))


def check_async(workspace, status_word, stream=None) -> None:
    """gdn_check_async: enqueue a copy of the workspace's error word (None: the
    array of gdn_prefill_noalloc) into `status_word`, a one-element int32 tensor
    on the device or in pinned host memory; returns without waiting."""
    import torch
    if status_word.numel() < 1 or status_word.dtype not in (torch.int32, torch.uint32):
        raise ValueError("status_word must be a one-element int32 tensor")
    if not status_word.is_cuda and not status_word.is_pinned():
        raise ValueError("status_word must be on the device or in pinned host memory")
    _check("gdn_check_async", lib().gdn_check_async(_ptr(workspace), _ptr(status_word), _stream(stream)))


def decode_step(q, k, v, a, b, A_log, dt_bias, state, n_seq, layers, scale=None, o=None,
                stream=None):
    """One decode step over U = n_seq*layers units; `state` [U,Hv,d,d] (float32,
    or bfloat16 for the bf16-state entry point) is updated in place.  Returns
    o [U,Hv,d] f32."""
    import torch
    U, Hqk, d = q.shape
    Hv = v.shape[1]
    if U != n_seq * layers:
        raise ValueError("q.shape[0] must equal n_seq * layers")
    _need(q, torch.bfloat16, (U, Hqk, d), "q")
    _need(k, torch.bfloat16, (U, Hqk, d), "k")
    _need(v, torch.bfloat16, (U, Hv, d), "v")
    _need(a, torch.float32, (U, Hv), "a")
    _need(b, torch.float32, (U, Hv), "b")
    _need(A_log, torch.float32, (layers, Hv), "A_log")
    _need(dt_bias, torch.float32, (layers, Hv), "dt_bias")
    bf16 = state.dtype == torch.bfloat16
    _need(state, torch.bfloat16 if bf16 else torch.float32, (U, Hv, d, d), "state")
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty(U, Hv, d, dtype=torch.float32, device=q.device)
    name = "gdn_decode_step_bf16" if bf16 else "gdn_decode_step"
    st = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(A_log),
                              _ptr(dt_bias), n_seq, layers, Hqk, Hv, d, float(scale), _ptr(state),
                              _ptr(o), _stream(stream))
    _check(name, st)
    return o


def decode_step_fused(qkv, conv_w, conv_state, a, b, A_log, dt_bias, state, n_seq, layers, Hqk, Hv,
                      slot=None, scale=None, o=None, stream=None):
    """One decode step with the front end fused in, for n_seq sequences x
    `layers` layers.  qkv [n_seq*layers, Ctot] bf16, conv_w [layers, Ctot, 4],
    conv_state [n_slots*layers, Ctot, 3] float32 and state [n_slots*layers, Hv,
    d, d] (float32, or bfloat16 for the bf16-state entry point), both updated in
    place, slot [n_seq] int32 or None.  Returns o [n_seq*layers, Hv, d] f32."""
    import torch
    d = state.shape[-1]
    U = n_seq * layers
    ctot = (2 * Hqk + Hv) * d
    n_slots = state.shape[0] // layers
    _need(qkv, torch.bfloat16, (U, ctot), "qkv")
    _need(conv_w, torch.float32, (layers, ctot, 4), "conv_w")
    _need(conv_state, torch.float32, (n_slots * layers, ctot, 3), "conv_state")
    bf16 = state.dtype == torch.bfloat16
    _need(state, torch.bfloat16 if bf16 else torch.float32, (n_slots * layers, Hv, d, d), "state")
    _need(a, torch.float32, (U, Hv), "a")
    _need(b, torch.float32, (U, Hv), "b")
    _need(A_log, torch.float32, (layers, Hv), "A_log")
    _need(dt_bias, torch.float32, (layers, Hv), "dt_bias")
    if slot is not None:
        _need(slot, torch.int32, (n_seq,), "slot")
    if o is None:
        o = torch.empty(U, Hv, d, dtype=torch.float32, device=state.device)
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    name = "gdn_decode_step_fused_bf16" if bf16 else "gdn_decode_step_fused"
    st = getattr(lib(), name)(_ptr(qkv), _ptr(conv_w), _ptr(conv_state), _ptr(a), _ptr(b),
                              _ptr(A_log), _ptr(dt_bias), _ptr(slot), n_seq, layers, Hqk, Hv,
                              d, scale, n_slots, _ptr(state), _ptr(o), _stream(stream))
    _check(name, st)
    return o


def gated_norm(o, z, norm_w, eps=1e-6, y=None, stream=None):
    """Gated output norm: y = norm_w * o / sqrt(mean_v o^2 + eps) * silu(z) per
    (token, value head).  o [T, Hv, d] float32, z [T, Hv, d] bf16, norm_w [d]
    or [layers, d] float32 (row t uses layer t % layers).  Returns y [T, Hv, d]
    bf16."""
    import torch
    T, Hv, d = o.shape
    w = norm_w if norm_w.dim() == 2 else norm_w.view(1, -1)
    layers = w.shape[0]
    _need(o, torch.float32, (T, Hv, d), "o")
    _need(z, torch.bfloat16, (T, Hv, d), "z")
    _need(w, torch.float32, (layers, d), "norm_w")
    if y is None:
        y = torch.empty(T, Hv, d, dtype=torch.bfloat16, device=o.device)
    st = lib().gdn_gated_norm(_ptr(o), _ptr(z), _ptr(w), T, Hv, d, layers, float(eps), _ptr(y),
                              _stream(stream))
    _check("gdn_gated_norm", st)
    return y


def prefill_gated(q, k, v, a, b, A_log, dt_bias, z, norm_w, eps=1e-6, cu_seqlens=None, scale=None,
                  initial_state=None, final_state=None, y=None, o=None, want_o=False,
                  workspace=None, want_final_state=True, stream=None):
    """gdn_prefill_gated: the chunked prefill with the gated output norm fused
    in.  z [T, Hv, d] bf16, norm_w [d] float32.  Returns (y [T, Hv, d] bf16,
    o [T, Hv, d] f32 or None, final_state or None); o is written only when
    passed in or want_o is set."""
    import torch
    T, Hqk, d = q.shape
    Hv = v.shape[1]
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _need(q, torch.bfloat16, (T, Hqk, d), "q")
    _need(k, torch.bfloat16, (T, Hqk, d), "k")
    _need(v, torch.bfloat16, (T, Hv, d), "v")
    _need(a, torch.float32, (T, Hv), "a")
    _need(b, torch.float32, (T, Hv), "b")
    _need(A_log, torch.float32, (Hv,), "A_log")
    _need(dt_bias, torch.float32, (Hv,), "dt_bias")
    _need(z, torch.bfloat16, (T, Hv, d), "z")
    _need(norm_w, torch.float32, (d,), "norm_w")
    if cu_seqlens is not None:
        _need(cu_seqlens, torch.int32, (n_seq + 1,), "cu_seqlens")
    if initial_state is not None:
        _need(initial_state, torch.float32, (n_seq, Hv, d, d), "initial_state")
    if scale is None:
        scale = d ** -0.5
    if y is None:
        y = torch.empty(T, Hv, d, dtype=torch.bfloat16, device=q.device)
    if o is None and want_o:
        o = torch.empty(T, Hv, d, dtype=torch.float32, device=q.device)
    if final_state is None and want_final_state:
        final_state = torch.empty(n_seq, Hv, d, d, dtype=torch.float32, device=q.device)
    ws_bytes = prefill_workspace_size(n_seq, T, Hqk, Hv, d)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    st = lib().gdn_prefill_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(A_log),
                                 _ptr(dt_bias), _ptr(cu_seqlens), n_seq, T, Hqk, Hv, d, float(scale),
                                 _ptr(initial_state), _ptr(final_state), _ptr(o), _ptr(z),
                                 _ptr(norm_w), float(eps), _ptr(y), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    _check("gdn_prefill_gated", st)
    return y, o, final_state


def decode_step_gated(q, k, v, a, b, A_log, dt_bias, state, n_seq, layers, z, norm_w, eps=1e-6,
                      scale=None, y=None, o=None, want_o=False, stream=None):
    """One decode step with the gated output norm fused in.  As decode_step,
    plus z [U, Hv, d] bf16 and norm_w [layers, d] f32.  Returns (y [U, Hv, d]
    bf16, o or None)."""
    import torch
    U, Hqk, d = q.shape
    Hv = v.shape[1]
    _need(q, torch.bfloat16, (U, Hqk, d), "q")
    _need(k, torch.bfloat16, (U, Hqk, d), "k")
    _need(v, torch.bfloat16, (U, Hv, d), "v")
    _need(a, torch.float32, (U, Hv), "a")
    _need(b, torch.float32, (U, Hv), "b")
    _need(A_log, torch.float32, (layers, Hv), "A_log")
    _need(dt_bias, torch.float32, (layers, Hv), "dt_bias")
    bf16 = state.dtype == torch.bfloat16
    _need(state, torch.bfloat16 if bf16 else torch.float32, (U, Hv, d, d), "state")
    _need(z, torch.bfloat16, (U, Hv, d), "z")
    _need(norm_w, torch.float32, (layers, d), "norm_w")
    if scale is None:
        scale = d ** -0.5
    if y is None:
        y = torch.empty(U, Hv, d, dtype=torch.bfloat16, device=q.device)
    if o is None and want_o:
        o = torch.empty(U, Hv, d, dtype=torch.float32, device=q.device)
    st = lib().gdn_decode_step_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(A_log),
                                     _ptr(dt_bias), n_seq, layers, Hqk, Hv, d, float(scale),
                                     _ptr(state), 1 if bf16 else 0, _ptr(o), _ptr(z), _ptr(norm_w),
                                     float(eps), _ptr(y), _stream(stream))
    _check("gdn_decode_step_gated", st)
    return y, o


def prefill_backward(q, k, v, a, b, A_log, dt_bias, d_o, d_final_state=None, cu_seqlens=None,
                     scale=None, initial_state=None, want_d_initial=True, workspace=None, stream=None, out=None):
    """gdn_prefill_backward: gradients of a loss with dL/do = d_o [T, Hv, d] and
    dL/dS_T = d_final_state [N, Hv, d, d] (or zero).  Returns a dict of float32
    tensors dq, dk [T, Hqk, d], dv [T, Hv, d], da, db [T, Hv], dA_log,
    ddt_bias [Hv] and d_initial_state [N, Hv, d, d] (or None).  out: an optional
    dict of preallocated tensors under those names (float32, contiguous)."""
    return _backward("gdn_prefill_backward", q, k, v, a, b, A_log, dt_bias, d_o, d_final_state, cu_seqlens,
                     scale, initial_state, want_d_initial, workspace, stream, out)


def prefill_backward_chunked(q, k, v, a, b, A_log, dt_bias, d_o, d_final_state=None, cu_seqlens=None,
                             scale=None, initial_state=None, want_d_initial=True, workspace=None, stream=None,
                             out=None):
    """gdn_prefill_backward_chunked: the same gradients through the chunked
    form (two chains over 64-token chunks, the rest chunk-parallel).  Arguments
    and result as for prefill_backward."""
    return _backward("gdn_prefill_backward_chunked", q, k, v, a, b, A_log, dt_bias, d_o, d_final_state,
                     cu_seqlens, scale, initial_state, want_d_initial, workspace, stream, out)


def _backward(entry, q, k, v, a, b, A_log, dt_bias, d_o, d_final_state, cu_seqlens, scale, initial_state,
              want_d_initial, workspace, stream, given=None):
    import torch
    T, Hqk, d = q.shape
    Hv = v.shape[1]
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _need(q, torch.bfloat16, (T, Hqk, d), "q")
    _need(k, torch.bfloat16, (T, Hqk, d), "k")
    _need(v, torch.bfloat16, (T, Hv, d), "v")
    _need(a, torch.float32, (T, Hv), "a")
    _need(b, torch.float32, (T, Hv), "b")
    _need(A_log, torch.float32, (Hv,), "A_log")
    _need(dt_bias, torch.float32, (Hv,), "dt_bias")
    _need(d_o, torch.float32, (T, Hv, d), "d_o")
    if cu_seqlens is not None:
        _need(cu_seqlens, torch.int32, (n_seq + 1,), "cu_seqlens")
    if initial_state is not None:
        _need(initial_state, torch.float32, (n_seq, Hv, d, d), "initial_state")
    if d_final_state is not None:
        _need(d_final_state, torch.float32, (n_seq, Hv, d, d), "d_final_state")
    if scale is None:
        scale = d ** -0.5
    dev = q.device
    shapes = dict(dq=(T, Hqk, d), dk=(T, Hqk, d), dv=(T, Hv, d), da=(T, Hv), db=(T, Hv), dA_log=(Hv,),
                  ddt_bias=(Hv,), d_initial_state=(n_seq, Hv, d, d) if want_d_initial else None)
    out = _outputs(given, shapes, dev)
    ws_bytes = getattr(lib(), entry + "_workspace_size")(n_seq, T, Hv, d)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = getattr(lib(), entry)(
        _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(cu_seqlens), n_seq, T,
        Hqk, Hv, d, float(scale), _ptr(initial_state), _ptr(d_o), _ptr(d_final_state), _ptr(out["dq"]),
        _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["da"]), _ptr(out["db"]), _ptr(out["dA_log"]),
        _ptr(out["ddt_bias"]), _ptr(out["d_initial_state"]), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(entry, st)
    return out


class _Launch:
    """The device and stream a call runs on: the device of its tensors (which must share one), made current for
    the call, and `stream` or that device's current stream, which allocations of the call then belong to.  With
    neither to be changed, entering it costs one look-up of the current stream."""

    __slots__ = ("device", "scopes")

    def __init__(self, stream, *tensors):
        import torch
        index = -1
        for t in tensors:
            if t is not None:
                i = t.get_device()
                if i < 0:
                    raise ValueError("all tensors must be CUDA tensors")
                if index < 0:
                    index = i
                elif i != index:
                    raise ValueError(f"all tensors must be on one device, got cuda:{index} and cuda:{i}")
        if stream is not None and stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
        self.device, self.scopes = index, None
        if index != torch.cuda.current_device():
            self.scopes = [torch.cuda.device(index)]
        if stream is not None:
            self.scopes = (self.scopes or []) + [torch.cuda.stream(stream)]

    def __enter__(self):
        import torch
        if self.scopes is not None:
            for s in self.scopes:
                s.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.device)

    def __exit__(self, *e):
        if self.scopes is not None:
            for s in reversed(self.scopes):
                s.__exit__(*e)


def _at(t):
    """The address of a tensor, NULL for None (as _ptr, without an object for each)."""
    return None if t is None else t.data_ptr()


def _want(t, dtype, shape, name):
    """_need for a tensor whose device is checked elsewhere: one comparison each where all is well."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _need(t, dtype, shape, name, device=None)
    return t


def _token_rows(t, T, H, d, name):
    """Checks a bf16 [T, H, d] tensor whose tokens may be any multiple of 8 elements apart (a view of a packed
    projection); returns that distance, 0 for a dense tensor."""
    import torch
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if t.shape != (T, H, d):
        raise ValueError(f"{name}: expected shape {(T, H, d)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return 0
    s = t.stride()
    if s[2] != 1 or (H > 1 and s[1] != d) or s[0] < H * d or s[0] % 8 != 0:
        raise ValueError(f"{name}: heads must be contiguous and tokens a multiple of 8 elements apart, got strides {s}")
    return s[0]


def _linear_shapes(q, k, v, g, cu_seqlens):
    import torch
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [T, heads, d]")
    T, Hqk, d = q.shape
    Hv = v.shape[1]
    n_seq = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    lds = (_token_rows(q, T, Hqk, d, "q"), _token_rows(k, T, Hqk, d, "k"), _token_rows(v, T, Hv, d, "v"))
    if g.dim() not in (1, 2):
        raise ValueError(f"g: expected shape {(T, Hv)} or {(Hv,)}, got {tuple(g.shape)}")
    _want(g, torch.float32, (T, Hv) if g.dim() == 2 else (Hv,), "g")
    if cu_seqlens is not None:
        _want(cu_seqlens, torch.int32, (n_seq + 1,), "cu_seqlens")
    return T, Hqk, Hv, d, n_seq, lds


def _given(t, dtype, shape, name, device):
    """An output: the caller's, checked, or a new one."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _want(t, dtype, shape, name)


def _workspace(workspace, size, device):
    """(the caller's workspace or a new one, its bytes)"""
    import torch
    if workspace is None:
        return torch.empty(size, dtype=torch.uint8, device=device), size
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def linear_prefill_workspace_size(n_seq, T, Hqk, Hv, d=128) -> int:
    return int(lib().gdn_linear_prefill_workspace_size(n_seq, T, Hqk, Hv, d))


def linear_prefill(q, k, v, g, cu_seqlens=None, scale=None, initial_state=None, final_state=None, o=None,
                   workspace=None, want_final_state=True, stream=None, o_dtype=None):
    """gdn_linear_prefill: linear attention with a decay per head, S_t = e^g S_{t-1} + v_t k_t^T, o_t = scale S_t q_t,
    over packed sequences.  q, k [T, Hqk, d], v [T, Hv, d] bf16 (dense, or views of a packed projection), g float32
    [T, Hv] or [Hv].  Returns (o [T, Hv, d] of o_dtype: bf16 by default, or float32; final_state [N, Hv, d, d] f32 or
    None)."""
    import torch
    T, Hqk, Hv, d, n_seq, lds = _linear_shapes(q, k, v, g, cu_seqlens)
    if o_dtype is None:
        o_dtype = o.dtype if o is not None else torch.bfloat16
    if o_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("o must be float32 or bfloat16")
    if initial_state is not None:
        _want(initial_state, torch.float32, (n_seq, Hv, d, d), "initial_state")
    if scale is None:
        scale = d ** -0.5
    with _Launch(stream, q, k, v, g, cu_seqlens, initial_state, final_state, o, workspace) as s:
        dev = q.device
        o = _given(o, o_dtype, (T, Hv, d), "o", dev)
        if final_state is not None or want_final_state:
            final_state = _given(final_state, torch.float32, (n_seq, Hv, d, d), "final_state", dev)
        ws, ws_bytes = _workspace(workspace, lib().gdn_linear_prefill_workspace_size(n_seq, T, Hqk, Hv, d), dev)
        st = lib().gdn_linear_prefill(_at(q), _at(k), _at(v), *lds, _at(g), g.dim() - 1, _at(cu_seqlens), n_seq,
                                      T, Hqk, Hv, d, float(scale), _at(initial_state), _at(final_state), _at(o),
                                      int(o_dtype == torch.bfloat16), _at(ws), ws_bytes, s)
    _check("gdn_linear_prefill", st)
    return o, final_state


def linear_prefill_backward(q, k, v, g, d_o, d_final_state=None, cu_seqlens=None, scale=None, initial_state=None,
                            want_d_initial=True, workspace=None, stream=None, out=None, grad_dtype=None):
    """gdn_linear_prefill_backward: gradients of a loss with dL/do = d_o [T, Hv, d] bf16 and dL/dS_T = d_final_state
    [N, Hv, d, d] float32 (or zero).  Returns a dict of dq, dk [T, Hqk, d], dv [T, Hv, d] (grad_dtype: bf16 by
    default, or float32), dg (float32, shaped as g) and d_initial_state [N, Hv, d, d] float32 (or None).  out: an
    optional dict of preallocated tensors under those names."""
    import torch
    T, Hqk, Hv, d, n_seq, lds = _linear_shapes(q, k, v, g, cu_seqlens)
    given = out or {}
    if grad_dtype is None:
        grad_dtype = next((given[n].dtype for n in ("dq", "dk", "dv") if given.get(n) is not None), torch.bfloat16)
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("the gradients must be float32 or bfloat16")
    _want(d_o, torch.bfloat16, (T, Hv, d), "d_o")
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None:
            _want(t, torch.float32, (n_seq, Hv, d, d), name)
    if scale is None:
        scale = d ** -0.5
    with _Launch(stream, q, k, v, g, d_o, cu_seqlens, initial_state, d_final_state, workspace, *given.values()) as s:
        dev = q.device
        out = {n: _given(given.get(n), dt, shape, n, dev) for n, dt, shape in (
            ("dq", grad_dtype, (T, Hqk, d)), ("dk", grad_dtype, (T, Hqk, d)), ("dv", grad_dtype, (T, Hv, d)),
            ("dg", torch.float32, tuple(g.shape)))}
        out["d_initial_state"] = _given(given.get("d_initial_state"), torch.float32, (n_seq, Hv, d, d),
                                        "d_initial_state", dev) if want_d_initial else None
        size = lib().gdn_linear_prefill_backward_workspace_size(n_seq, T, Hqk, Hv, d)
        ws, ws_bytes = _workspace(workspace, size, dev)
        st = lib().gdn_linear_prefill_backward(
            _at(q), _at(k), _at(v), *lds, _at(g), g.dim() - 1, _at(cu_seqlens), n_seq, T, Hqk, Hv, d,
            float(scale), _at(initial_state), _at(d_o), _at(d_final_state), _at(out["dq"]), _at(out["dk"]),
            _at(out["dv"]), int(grad_dtype == torch.bfloat16), _at(out["dg"]), _at(out["d_initial_state"]),
            _at(ws), ws_bytes, s)
    _check("gdn_linear_prefill_backward", st)
    return out


def linear_decode_step(q, k, v, g, state, n_seq, layers, slot=None, scale=None, o=None, stream=None, o_dtype=None):
    """gdn_linear_decode_step: one token of linear attention for n_seq sequences x `layers` layers.  q, k
    [n_seq*layers, Hqk, d], v [n_seq*layers, Hv, d] bf16, g float32 [n_seq*layers, Hv] or [layers, Hv], state
    [n_slots*layers, Hv, d, d] float32 or bf16, updated in place, slot [n_seq] int32 (-1: no sequence) or None.
    Returns o [n_seq*layers, Hv, d] (o_dtype: float32 by default, or bf16)."""
    import torch
    U, Hqk, d = q.shape
    Hv = v.shape[1]
    if U != n_seq * layers or layers <= 0:
        raise ValueError("q.shape[0] must equal n_seq * layers")
    _want(q, torch.bfloat16, (U, Hqk, d), "q")
    _want(k, torch.bfloat16, (U, Hqk, d), "k")
    _want(v, torch.bfloat16, (U, Hv, d), "v")
    per_unit = g.shape[0] != layers or n_seq == 1
    _want(g, torch.float32, (U if per_unit else layers, Hv), "g")
    n_slots = state.shape[0] // layers
    bf16 = state.dtype == torch.bfloat16
    _want(state, torch.bfloat16 if bf16 else torch.float32, (n_slots * layers, Hv, d, d), "state")
    if slot is not None:
        _want(slot, torch.int32, (n_seq,), "slot")
    if o_dtype is None:
        o_dtype = o.dtype if o is not None else torch.float32
    if o_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("o must be float32 or bfloat16")
    if scale is None:
        scale = d ** -0.5
    with _Launch(stream, q, k, v, g, state, slot, o) as s:
        o = _given(o, o_dtype, (U, Hv, d), "o", q.device)
        st = lib().gdn_linear_decode_step(_at(q), _at(k), _at(v), _at(g), int(per_unit), _at(slot), n_seq, layers,
                                          Hqk, Hv, d, float(scale), n_slots, _at(state), int(bf16), _at(o),
                                          int(o_dtype == torch.bfloat16), s)
    _check("gdn_linear_decode_step", st)
    return o


def _state_buffers(buffers, n_slots=None):
    """(gdn_state_buffer array, number of buffers, number of slots) of a cache's tensors [n_slots, ...]."""
    import torch
    if isinstance(buffers, torch.Tensor):
        buffers = [buffers]
    array = (StateBuffer * max(len(buffers), 1))()
    for i, b in enumerate(buffers):
        if b.dim() < 1 or not b.is_contiguous():
            raise ValueError("a cache's buffers must be contiguous, [n_slots, ...]")
        if n_slots is None:
            n_slots = b.shape[0]
        if b.shape[0] != n_slots:
            raise ValueError(f"a cache's buffers must have one number of slots, got {b.shape[0]} and {n_slots}")
        array[i].data = b.data_ptr()
        array[i].slot_bytes = b.numel() // max(n_slots, 1) * b.element_size()
    if n_slots is None:
        raise ValueError("a cache has at least one buffer")
    return array, len(buffers), n_slots, list(buffers)


def _index(t, n, name):
    import torch
    if t.dim() != 1:
        raise ValueError(f"{name} must be one-dimensional")
    return _want(t, torch.int32, (t.shape[0] if n is None else n,), name)


def state_copy(buffers, src, dst, stream=None):
    """gdn_state_copy: page[dst[i]] = page[src[i]] for all i at once (each source as it was before the call), a page
    being one slot of every tensor [n_slots, ...] in `buffers`.  src, dst [n] int32; an index outside the cache makes
    its entry void, and of several entries with one destination the last holds."""
    array, nb, n_slots, tensors = _state_buffers(buffers)
    _index(src, None, "src")
    n = src.shape[0]
    _index(dst, n, "dst")
    with _Launch(stream, src, dst, *tensors) as s:
        st = lib().gdn_state_copy(array, nb, n_slots, _at(src), _at(dst), n, s)
    _check("gdn_state_copy", st)


def _state_workspace(workspace, n_slots, device):
    return _workspace(workspace, lib().gdn_state_workspace_size(n_slots), device)


def state_fork(buffers, live, src, dst=None, workspace=None, stream=None):
    """gdn_state_fork: new pages for `src` [n] int32, each filled from that live slot or, for -1, with zeros, in the
    lowest free slots.  live [n_slots] int32 is updated.  Returns dst [n] int32 (-1 where none was free)."""
    import torch
    _index(live, None, "live")
    array, nb, n_slots, tensors = _state_buffers(buffers, live.shape[0])
    _index(src, None, "src")
    n = src.shape[0]
    with _Launch(stream, live, src, dst, workspace, *tensors) as s:
        dst = _given(dst, torch.int32, (n,), "dst", live.device)
        ws, ws_bytes = _state_workspace(workspace, n_slots, live.device)
        st = lib().gdn_state_fork(array, nb, n_slots, _at(live), _at(src), _at(dst), n, _at(ws), ws_bytes, s)
    _check("gdn_state_fork", st)
    return dst


def state_compact(buffers, live, moved=None, workspace=None, stream=None):
    """gdn_state_compact: moves the live pages into the first slots with the fewest moves.  live [n_slots] int32 is
    updated.  Returns moved [n_slots] int32, the new slot of each page (-1: free)."""
    import torch
    _index(live, None, "live")
    array, nb, n_slots, tensors = _state_buffers(buffers, live.shape[0])
    with _Launch(stream, live, moved, workspace, *tensors) as s:
        moved = _given(moved, torch.int32, (n_slots,), "moved", live.device)
        ws, ws_bytes = _state_workspace(workspace, n_slots, live.device)
        st = lib().gdn_state_compact(array, nb, n_slots, _at(live), _at(moved), _at(ws), ws_bytes, s)
    _check("gdn_state_compact", st)
    return moved


def state_free(live, slots, stream=None):
    """gdn_state_free: live[slots[i]] = 0 (indices outside the cache are ignored); the pages keep their contents."""
    _index(live, None, "live")
    _index(slots, None, "slots")
    with _Launch(stream, live, slots) as s:
        st = lib().gdn_state_free(_at(live), live.shape[0], _at(slots), slots.shape[0], s)
    _check("gdn_state_free", st)
