"""Thin Python binding of libmesa (include/mesa.h): argument marshalling only.

Every step of the Mesa layer runs in the library's HIP kernels; this module
allocates outputs with torch, passes raw device pointers and the current HIP
stream, and maps status codes to Python exceptions.  There is no fallback:
if libmesa.so is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmesa.so")

MESA_OK, MESA_ERR_INVALID_ARGUMENT, MESA_ERR_UNSUPPORTED, MESA_ERR_WORKSPACE_TOO_SMALL, MESA_ERR_HIP = range(5)
MESA_DTYPE_F32, MESA_DTYPE_BF16 = 0, 1
KERNEL_CHUNK_STATES, KERNEL_CG_OUTPUT, KERNEL_DECODE, KERNEL_QK_PREPROCESS = 0, 1, 2, 3
KERNEL_BWD_ADJOINT, KERNEL_BWD_STATES, KERNEL_BWD_KV, KERNEL_BWD_GATE, KERNEL_HAWK = 4, 5, 6, 7, 8
(KERNEL_DELTA_PREP, KERNEL_DELTA_SCAN, KERNEL_DELTA_STEP, KERNEL_DELTA_BWD_SCAN, KERNEL_DELTA_GRADS, KERNEL_GATE_NORM,
 KERNEL_GATE_NORM_BWD, KERNEL_RESIDUAL_NORM, KERNEL_RESIDUAL_NORM_BWD) = range(16, 25)
MESA_WARM_COLD, MESA_WARM_PREVIOUS, MESA_WARM_PROJECTED = 0, 1, 2

# Every symbol include/mesa.h declares, with its ctypes signature.
_P, _I, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "mesa_abi_version": ([], _I),
    "mesa_status_string": ([_I], ctypes.c_char_p),
    "mesa_last_error_message": ([], ctypes.c_char_p),
    "mesa_forward_workspace_bytes": ([_I, _I, _I, _I, _I, _I], _Z),
    "mesa_forward": ([_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                      _P, _P, _P, _P, _P, _Z, _P], _I),
    "mesa_forward_train": ([_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                            _P, _P, _P, _P, _Z, _P], _I),
    "mesa_forward_noalloc": ([_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                              _P, _P, _P, _P, _P], _I),
    "mesa_backward_workspace_bytes": ([_I, _I, _I, _I, _I, _I], _Z),
    "mesa_backward": ([_P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                       _P, _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "mesa_decode_step": ([_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F,
                          _P, _P, _P], _I),
    "mesa_decode_step_warm": ([_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I,
                               _P, _P, _P], _I),
    "mesa_qk_preprocess": ([_P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _P, _I, _P], _I),
    "mesa_hawk_workspace_bytes": ([_I, _I, _I], _Z),
    "mesa_hawk_scan": ([_P, _P, _P, _I, _P, _F, _P, _I, _I, _I, _P, _P, _P, _Z, _P], _I),
    "mesa_delta_workspace_bytes": ([_I, _I, _I, _I, _I, _I], _Z),
    "mesa_delta_forward": ([_P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _Z, _P], _I),
    "mesa_delta_backward_workspace_bytes": ([_I] * 7, _Z),
    "mesa_delta_backward": ([_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P,
                             _P, _Z, _P], _I),
    "mesa_delta_step": ([_P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P], _I),
    "mesa_gate_norm": ([_P, _I, _P, _I, _P, _F, _I, _I, _I, _I, _P, _P], _I),
    "mesa_gate_norm_backward_workspace_bytes": ([_I, _I, _I, _I], _Z),
    "mesa_gate_norm_backward": ([_P, _I, _P, _I, _P, _F, _P, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P], _I),
    "mesa_residual_norm": ([_P, _I, _P, _I, _P, _P, _F, _I, _I, _P, _P, _P], _I),
    "mesa_residual_norm_backward_workspace_bytes": ([_I, _I], _Z),
    "mesa_residual_norm_backward": ([_P, _I, _P, _I, _P, _P, _F, _P, _P, _I, _I, _P, _P, _P, _P, _P, _Z, _P], _I),
    "mesa_profile_enable": ([_I], _I),
    "mesa_profile_read": ([_I, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)], _I),
    "mesa_profile_reset": ([], _I),
    "mesa_kernel_name": ([_I], ctypes.c_char_p),
    # include/mesa_probe.h
    "mesa_probe_mfma_f32": ([_I, _I, _P, _P], _I),
    "mesa_probe_mfma_bf16": ([_I, _I, _P, _P], _I),
    "mesa_probe_copy": ([_P, _P, _Z, _P], _I),
}

_lib = None


class MesaError(RuntimeError):
    """A HIP runtime failure reported by libmesa."""


def lib():
    """The loaded libmesa (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status == MESA_OK:
        return
    L = lib()
    msg = f"{what}: {L.mesa_status_string(status).decode()}: {L.mesa_last_error_message().decode()}"
    if status in (MESA_ERR_INVALID_ARGUMENT, MESA_ERR_WORKSPACE_TOO_SMALL):
        raise ValueError(msg)
    if status == MESA_ERR_UNSUPPORTED:
        raise NotImplementedError(msg)
    raise MesaError(msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _qkv_dtype(t):
    import torch
    if t.dtype == torch.float32:
        return MESA_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return MESA_DTYPE_BF16
    raise ValueError(f"q/k/v dtype {t.dtype} is not float32 or bfloat16")


def _need(t, name, dtype=None, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _dims(t, name, ndim):
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {list(t.shape)}")
    return tuple(t.shape)


def _shapes(*specs):
    """Every (tensor, name, shape) must have exactly that shape.  Checked
    before any device or dtype check, so that a mis-shaped argument is named
    whatever else is wrong."""
    for t, name, shape in specs:
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _shape(t, name, shape, dtype=None, device=None):
    """A device tensor of exactly this shape (and dtype/device, when given)."""
    _shapes((t, name, shape))
    _need(t, name, dtype, device)


def _given(*specs):
    """The (tensor, name, shape) specs whose tensor was given."""
    return tuple(sp for sp in specs if sp[0] is not None)


def _forward_checks(q, k, v, gamma, lam, **outs):
    """Shapes, dtypes and devices of mesa_forward's inputs, and the shapes of
    the outputs the caller passed (out, iters, x_out, final_H, final_G);
    returns (B, H, T, dk, dv)."""
    import torch
    B, H, T, dk = _dims(q, "q", 4)
    dv = _dims(v, "v", 4)[-1]
    oshape = dict(out=(B, H, T, dv), iters=(B, H, T), x_out=(B, H, T, dk), final_H=(B, H, dk, dk),
                  final_G=(B, H, dv, dk))
    _shapes((k, "k", (B, H, T, dk)), (v, "v", (B, H, T, dv)), (gamma, "gamma", (B, H, T)),
            (lam, "lambda", (H, dk)), *_given(*((t, n, oshape[n]) for n, t in outs.items())))
    _qkv_dtype(q)
    for t, n, dt in ((q, "q", q.dtype), (k, "k", q.dtype), (v, "v", q.dtype), (gamma, "gamma", torch.float32),
                     (lam, "lambda", torch.float32)):
        _need(t, n, dt, q.device)
    return B, H, T, dk, dv


def _out(t, name, shape, dtype, device):
    """A caller-provided output: checked like an input, or allocated."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _shape(t, name, shape, dtype, device)
    return t


def mesa_forward_workspace_bytes(B, H, T, dk, dv, chunk) -> int:
    return int(lib().mesa_forward_workspace_bytes(B, H, T, dk, dv, chunk))


def mesa_forward(q, k, v, gamma, lam, max_iters, tol=0.0, chunk=64, *, out=None, iters=None,
                 return_iters=True, return_final=False, final_H=None, final_G=None,
                 workspace=None, stream=None):
    """Mesa-layer forward (see include/mesa.h, mesa_forward).

    q, k: [B,H,T,dk]; v: [B,H,T,dv] (float32 or bfloat16, same dtype);
    gamma: [B,H,T] float32; lam: [H,dk] float32.  Returns (out, iters,
    final_H, final_G); iters/final_* are None unless requested.
    """
    import torch
    B, H, T, dk, dv = _forward_checks(q, k, v, gamma, lam, out=out, iters=iters, final_H=final_H,
                                      final_G=final_G)
    dev = q.device
    dt = _qkv_dtype(q)
    out = _out(out, "out", (B, H, T, dv), torch.float32, dev)
    if iters is not None or return_iters:
        iters = _out(iters, "iters", (B, H, T), torch.int32, dev)
    if return_final or final_H is not None or final_G is not None:
        final_H = _out(final_H, "final_H", (B, H, dk, dk), torch.float32, dev)
        final_G = _out(final_G, "final_G", (B, H, dv, dk), torch.float32, dev)
    ws_bytes = mesa_forward_workspace_bytes(B, H, T, dk, dv, chunk) if max_iters > 0 else 0
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", None, dev)
    st = lib().mesa_forward(_ptr(q), _ptr(k), _ptr(v), dt, _ptr(gamma), _ptr(lam),
                            B, H, T, dk, dv, int(chunk), int(max_iters), float(tol),
                            _ptr(out), _ptr(iters), _ptr(final_H), _ptr(final_G),
                            _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
                            _stream(stream))
    _check(st, "mesa_forward")
    return out, iters, final_H, final_G


def mesa_forward_noalloc(q, k, v, gamma, lam, max_iters, tol=0.0, chunk=64, *, out, iters=None, final_H=None,
                         final_G=None, stream=None):
    """mesa_forward with the chunk states in the library's built-in device
    array (see include/mesa.h, mesa_forward_noalloc): the caller passes every
    output, and the call allocates nothing.  Returns (out, iters, final_H,
    final_G) as given."""
    B, H, T, dk, dv = _forward_checks(q, k, v, gamma, lam, out=out, iters=iters, final_H=final_H,
                                      final_G=final_G)
    import torch
    dev = q.device
    _need(out, "out", torch.float32, dev)
    for t, n, dt in ((iters, "iters", torch.int32), (final_H, "final_H", torch.float32),
                     (final_G, "final_G", torch.float32)):
        if t is not None:
            _need(t, n, dt, dev)
    st = lib().mesa_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _qkv_dtype(q), _ptr(gamma), _ptr(lam),
                                    B, H, T, dk, dv, int(chunk), int(max_iters), float(tol),
                                    _ptr(out), _ptr(iters), _ptr(final_H), _ptr(final_G), _stream(stream))
    _check(st, "mesa_forward_noalloc")
    return out, iters, final_H, final_G


def mesa_forward_train(q, k, v, gamma, lam, max_iters, tol=0.0, chunk=64, *, out=None, iters=None,
                       x_out=None, workspace=None, stream=None):
    """Forward that also returns the CG solutions x (see include/mesa.h,
    mesa_forward_train).  Returns (out, iters, x)."""
    import torch
    B, H, T, dk, dv = _forward_checks(q, k, v, gamma, lam, out=out, iters=iters, x_out=x_out)
    dev = q.device
    out = _out(out, "out", (B, H, T, dv), torch.float32, dev)
    iters = _out(iters, "iters", (B, H, T), torch.int32, dev)
    x_out = _out(x_out, "x_out", (B, H, T, dk), torch.float32, dev)
    nbytes = mesa_forward_workspace_bytes(B, H, T, dk, dv, chunk)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", None, dev)
    st = lib().mesa_forward_train(_ptr(q), _ptr(k), _ptr(v), _qkv_dtype(q), _ptr(gamma), _ptr(lam),
                                  B, H, T, dk, dv, chunk, int(max_iters), float(tol),
                                  _ptr(out), _ptr(iters), _ptr(x_out), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  _stream(stream))
    _check(st, "mesa_forward_train")
    return out, iters, x_out


def mesa_backward_workspace_bytes(B, H, T, dk, dv, chunk) -> int:
    return int(lib().mesa_backward_workspace_bytes(B, H, T, dk, dv, chunk))


def mesa_backward(k, v, gamma, lam, x, out, grad_out, max_iters, tol=0.0, chunk=64, *, workspace=None,
                  return_z_iters=True, stream=None):
    """Backward pass (see include/mesa.h, mesa_backward).  Returns a dict of
    grad_q, grad_k, grad_v, grad_gamma, grad_lambda (float32) and z_iters."""
    import torch
    B, H, T, dk = _dims(k, "k", 4)
    dv = _dims(v, "v", 4)[-1]
    dev = k.device
    _shapes((v, "v", (B, H, T, dv)), (gamma, "gamma", (B, H, T)), (lam, "lambda", (H, dk)),
            (x, "x", (B, H, T, dk)), (out, "out", (B, H, T, dv)), (grad_out, "grad_out", (B, H, T, dv)))
    _qkv_dtype(k)
    for t, n, dt in ((k, "k", k.dtype), (v, "v", k.dtype), (gamma, "gamma", torch.float32),
                     (lam, "lambda", torch.float32), (x, "x", torch.float32), (out, "out", torch.float32),
                     (grad_out, "grad_out", torch.float32)):
        _need(t, n, dt, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(grad_q=torch.empty((B, H, T, dk), **f32), grad_k=torch.empty((B, H, T, dk), **f32),
             grad_v=torch.empty((B, H, T, dv), **f32), grad_gamma=torch.empty((B, H, T), **f32),
             grad_lambda=torch.empty((H, dk), **f32))
    g["z_iters"] = torch.empty((B, H, T), dtype=torch.int32, device=dev) if return_z_iters else None
    nbytes = mesa_backward_workspace_bytes(B, H, T, dk, dv, chunk)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", None, dev)
    st = lib().mesa_backward(_ptr(k), _ptr(v), _qkv_dtype(k), _ptr(gamma), _ptr(lam), _ptr(x), _ptr(out),
                             _ptr(grad_out), B, H, T, dk, dv, chunk, int(max_iters), float(tol),
                             _ptr(g["grad_q"]), _ptr(g["grad_k"]), _ptr(g["grad_v"]), _ptr(g["grad_gamma"]),
                             _ptr(g["grad_lambda"]), _ptr(g["z_iters"]), _ptr(workspace),
                             workspace.numel() * workspace.element_size(),
                             _stream(stream))
    _check(st, "mesa_backward")
    return g


def _decode_checks(q, k, v, gamma, lam, state_H, state_G, state_x=None, out=None, iters=None):
    import torch
    N, H, dk = _dims(q, "q", 3)
    dv = _dims(v, "v", 3)[-1]
    dev = q.device
    specs = [(k, "k", (N, H, dk)), (v, "v", (N, H, dv)), (gamma, "gamma", (N, H)), (lam, "lambda", (H, dk)),
             (state_H, "state_H", (N, H, dk, dk)), (state_G, "state_G", (N, H, dv, dk)),
             *_given((out, "out", (N, H, dv)), (iters, "iters", (N, H)))]
    if state_x is not None:
        specs.append((state_x, "state_x", (N, H, dk)))
    _shapes(*specs)
    _qkv_dtype(q)
    for t, n, dt in ((q, "q", q.dtype), (k, "k", q.dtype), (v, "v", q.dtype), (gamma, "gamma", torch.float32),
                     (lam, "lambda", torch.float32), (state_H, "state_H", torch.float32),
                     (state_G, "state_G", torch.float32)):
        _need(t, n, dt, dev)
    if state_x is not None:
        _need(state_x, "state_x", torch.float32, dev)
    return N, H, dk, dv, dev


def mesa_decode_step(q, k, v, gamma, lam, state_H, state_G, max_iters, tol=0.0, *,
                     out=None, iters=None, return_iters=True, stream=None):
    """One decode step (see include/mesa.h, mesa_decode_step); state_H/G updated in place.

    q, k: [N,H,dk]; v: [N,H,dv]; gamma: [N,H]; lam: [H,dk];
    state_H: [N,H,dk,dk], state_G: [N,H,dv,dk] float32.  Returns (out, iters).
    """
    import torch
    N, H, dk, dv, dev = _decode_checks(q, k, v, gamma, lam, state_H, state_G, out=out, iters=iters)
    out = _out(out, "out", (N, H, dv), torch.float32, dev)
    if iters is not None or return_iters:
        iters = _out(iters, "iters", (N, H), torch.int32, dev)
    st = lib().mesa_decode_step(_ptr(q), _ptr(k), _ptr(v), _qkv_dtype(q), _ptr(gamma), _ptr(lam),
                                _ptr(state_H), _ptr(state_G), N, H, dk, dv, int(max_iters),
                                float(tol), _ptr(out), _ptr(iters), _stream(stream))
    _check(st, "mesa_decode_step")
    return out, iters


def mesa_decode_step_warm(q, k, v, gamma, lam, state_H, state_G, state_x, max_iters, tol=0.0,
                          warm_mode=MESA_WARM_PROJECTED, *, out=None, iters=None, return_iters=True,
                          stream=None):
    """One warm-started decode step (see include/mesa.h, mesa_decode_step_warm).

    As mesa_decode_step, plus state_x [N,H,dk] float32: the previous
    solutions on entry, this step's on exit.  Returns (out, iters).
    """
    import torch
    N, H, dk, dv, dev = _decode_checks(q, k, v, gamma, lam, state_H, state_G, state_x, out=out, iters=iters)
    out = _out(out, "out", (N, H, dv), torch.float32, dev)
    if iters is not None or return_iters:
        iters = _out(iters, "iters", (N, H), torch.int32, dev)
    st = lib().mesa_decode_step_warm(_ptr(q), _ptr(k), _ptr(v), _qkv_dtype(q), _ptr(gamma), _ptr(lam),
                                     _ptr(state_H), _ptr(state_G), _ptr(state_x), N, H, dk, dv,
                                     int(max_iters), float(tol), int(warm_mode), _ptr(out), _ptr(iters),
                                     _stream(stream))
    _check(st, "mesa_decode_step_warm")
    return out, iters


def mesa_qk_preprocess(x, conv_w, hist=None, *, out_dtype=None, out=None, return_hist=False,
                       hist_out=None, stream=None):
    """Causal convolution of width W over tokens + L2 normalisation (see include/mesa.h).

    x: [B,H,T,d] float32 or bfloat16; conv_w: [H,W,d] float32; hist: [B,H,W-1,d]
    in x's dtype or None.  Returns y (out_dtype, default x's dtype), and with
    return_hist also hist_out, the last W-1 input rows for the next piece.
    """
    import torch
    B, H, T, d = _dims(x, "x", 4)
    W = _dims(conv_w, "conv_w", 3)[1]
    dev = x.device
    _shapes((conv_w, "conv_w", (H, W, d)), *(((hist, "hist", (B, H, W - 1, d)),) if hist is not None else ()))
    _qkv_dtype(x)
    _need(x, "x", None, dev)
    _need(conv_w, "conv_w", torch.float32, dev)
    if hist is not None:
        _need(hist, "hist", x.dtype, dev)
    out_dtype = (x.dtype if out is None else out.dtype) if out_dtype is None else out_dtype
    out = _out(out, "out", (B, H, T, d), out_dtype, dev)
    if return_hist or hist_out is not None:
        hist_out = _out(hist_out, "hist_out", (B, H, W - 1, d), x.dtype, dev)
    st = lib().mesa_qk_preprocess(_ptr(x), _qkv_dtype(x), _ptr(conv_w), W, _ptr(hist), _ptr(hist_out),
                                  B, H, T, d, _ptr(out), _qkv_dtype(out), _stream(stream))
    _check(st, "mesa_qk_preprocess")
    return (out, hist_out) if return_hist else out


def mesa_hawk_scan(x, ga, gx, lam, c=8.0, h0=None, *, out=None, return_final=False, workspace=None,
                   stream=None):
    """The Hawk layer's gated linear recurrence (see include/mesa.h, mesa_hawk_scan).

    x, ga, gx: [B,T,D] float32 or bfloat16 (same dtype); lam: [D] float32;
    h0: [B,D] float32 or None.  Returns y [B,T,D] float32 (and h_final [B,D]).
    """
    import torch
    B, T, D = _dims(x, "x", 3)
    dev = x.device
    _shapes((ga, "ga", (B, T, D)), (gx, "gx", (B, T, D)), (lam, "lam", (D,)),
            *(((h0, "h0", (B, D)),) if h0 is not None else ()))
    _qkv_dtype(x)
    for t, n, dt in ((x, "x", x.dtype), (ga, "ga", x.dtype), (gx, "gx", x.dtype), (lam, "lam", torch.float32)):
        _need(t, n, dt, dev)
    if h0 is not None:
        _need(h0, "h0", torch.float32, dev)
    out = _out(out, "out", (B, T, D), torch.float32, dev)
    hf = torch.empty((B, D), dtype=torch.float32, device=dev) if return_final else None
    nbytes = int(lib().mesa_hawk_workspace_bytes(B, T, D))
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", None, dev)
    st = lib().mesa_hawk_scan(_ptr(x), _ptr(ga), _ptr(gx), _qkv_dtype(x), _ptr(lam), float(c), _ptr(h0), B, T, D,
                              _ptr(out), _ptr(hf), _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream))
    _check(st, "mesa_hawk_scan")
    return (out, hf) if return_final else out


def _tensors(dev, *specs):
    """Checks (tensor, name, shape, dtype) specs, tensors that are None left
    out: every shape before any device, dtype or layout."""
    for t, name, shape, _ in specs:
        if t is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    for t, name, _, dtype in specs:
        if t is not None and not (t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.device == dev):
            _need(t, name, dtype, dev)


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """The context in which a call allocates and enqueues: the tensors' device,
    and `stream` when one is given (which then owns what is allocated)."""
    import torch
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, expected {dev}")
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _at(t):
    return None if t is None else t.data_ptr()


def _here(dev):
    """The raw handle of dev's current stream."""
    import torch
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _scratch(workspace, nbytes, dev):
    """(workspace, its size): the caller's, checked, or a new one."""
    import torch
    if workspace is None:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev), max(nbytes, 16)
    _need(workspace, "workspace", None, dev)
    return workspace, workspace.numel() * workspace.element_size()


def _delta_sizes(q, v, ndim):
    """(B or N, Hk, H, the token axis, dk, dv) of a delta-rule call."""
    B, Hk, *t, dk = _dims(q, "q", ndim)
    _, H, *_, dv = _dims(v, "v", ndim)
    if H % Hk if Hk else H:
        raise ValueError(f"{H} value heads are not a multiple of {Hk} key heads")
    return B, Hk, H, t, dk, dv


def mesa_delta_workspace_bytes(B, H, T, dk, dv, dtype) -> int:
    return int(lib().mesa_delta_workspace_bytes(B, H, T, dk, dv, dtype))


def mesa_delta_forward(q, k, v, gamma, beta, state=None, *, out=None, return_final=False, final_state=None,
                       workspace=None, stream=None):
    """Gated delta rule over a sequence (see include/mesa.h, mesa_delta_forward).

    q, k: [B,Hk,T,dk]; v: [B,H,T,dv] (float32 or bfloat16, same dtype; H a
    multiple of Hk); gamma, beta: [B,H,T] float32; state: [B,H,dv,dk] float32
    or None.  Returns (out [B,H,T,dv] in q's dtype, final_state [B,H,dv,dk] or
    None); final_state may be the state passed in.
    """
    import torch
    B, Hk, H, (T,), dk, dv = _delta_sizes(q, v, 4)
    dev, dt, code, f32 = q.device, q.dtype, _qkv_dtype(q), torch.float32
    gates, states = (B, H, T), (B, H, dv, dk)
    _tensors(dev, (q, "q", (B, Hk, T, dk), dt), (k, "k", (B, Hk, T, dk), dt), (v, "v", (B, H, T, dv), dt),
             (gamma, "gamma", gates, f32), (beta, "beta", gates, f32), (state, "state", states, f32),
             (out, "out", (B, H, T, dv), dt), (final_state, "final_state", states, f32))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((B, H, T, dv), dtype=dt, device=dev)
        if return_final and final_state is None:
            final_state = torch.empty(states, dtype=f32, device=dev)
        L = lib()
        workspace, nbytes = _scratch(workspace, L.mesa_delta_workspace_bytes(B, H, T, dk, dv, code), dev)
        st = L.mesa_delta_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), code, gamma.data_ptr(), beta.data_ptr(),
                                  _at(state), B, Hk, H, T, dk, dv, out.data_ptr(), _at(final_state),
                                  workspace.data_ptr(), nbytes, _here(dev))
    _check(st, "mesa_delta_forward")
    return out, final_state


def mesa_delta_backward_workspace_bytes(B, Hk, H, T, dk, dv, dtype) -> int:
    return int(lib().mesa_delta_backward_workspace_bytes(B, Hk, H, T, dk, dv, dtype))


def mesa_delta_backward(q, k, v, gamma, beta, grad_out, state=None, *, grad_final=None, workspace=None, stream=None):
    """Gradients of mesa_delta_forward (see include/mesa.h, mesa_delta_backward).

    grad_out: [B,H,T,dv] in q's dtype; grad_final: [B,H,dv,dk] float32 or
    None.  Returns a dict of grad_q, grad_k [B,Hk,T,dk], grad_v (q's dtype),
    grad_gamma, grad_beta and grad_state (float32; None without a state).
    grad_gamma is 0 where gamma is: a gate of 0 marks a sequence's start in a
    packed row and is not differentiated.
    """
    import torch
    B, Hk, H, (T,), dk, dv = _delta_sizes(q, v, 4)
    dev, dt, code, f32 = q.device, q.dtype, _qkv_dtype(q), torch.float32
    gates, states = (B, H, T), (B, H, dv, dk)
    _tensors(dev, (q, "q", (B, Hk, T, dk), dt), (k, "k", (B, Hk, T, dk), dt), (v, "v", (B, H, T, dv), dt),
             (gamma, "gamma", gates, f32), (beta, "beta", gates, f32), (state, "state", states, f32),
             (grad_out, "grad_out", (B, H, T, dv), dt), (grad_final, "grad_final", states, f32))
    with _on(dev, stream):
        g = dict(grad_q=torch.empty_like(q), grad_k=torch.empty_like(k), grad_v=torch.empty_like(v),
                 grad_gamma=torch.empty_like(gamma), grad_beta=torch.empty_like(beta),
                 grad_state=None if state is None else torch.empty_like(state))
        L = lib()
        workspace, nbytes = _scratch(workspace, L.mesa_delta_backward_workspace_bytes(B, Hk, H, T, dk, dv, code), dev)
        st = L.mesa_delta_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), code, gamma.data_ptr(), beta.data_ptr(),
                                   _at(state), grad_out.data_ptr(), _at(grad_final), B, Hk, H, T, dk, dv,
                                   g["grad_q"].data_ptr(), g["grad_k"].data_ptr(), g["grad_v"].data_ptr(),
                                   g["grad_gamma"].data_ptr(), g["grad_beta"].data_ptr(), _at(g["grad_state"]),
                                   workspace.data_ptr(), nbytes, _here(dev))
    _check(st, "mesa_delta_backward")
    return g


def mesa_delta_step(q, k, v, gamma, beta, state, *, out=None, stream=None):
    """One token of the gated delta rule (see include/mesa.h, mesa_delta_step);
    state [N,H,dv,dk] float32 is updated in place.

    q, k: [N,Hk,dk]; v: [N,H,dv]; gamma, beta: [N,H].  Returns out [N,H,dv].
    """
    import torch
    N, Hk, H, _, dk, dv = _delta_sizes(q, v, 3)
    dev, dt, code, f32 = q.device, q.dtype, _qkv_dtype(q), torch.float32
    _tensors(dev, (q, "q", (N, Hk, dk), dt), (k, "k", (N, Hk, dk), dt), (v, "v", (N, H, dv), dt),
             (gamma, "gamma", (N, H), f32), (beta, "beta", (N, H), f32), (state, "state", (N, H, dv, dk), f32),
             (out, "out", (N, H, dv), dt))
    with _on(dev, stream):
        if out is None:
            out = torch.empty((N, H, dv), dtype=dt, device=dev)
        st = lib().mesa_delta_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), code, gamma.data_ptr(), beta.data_ptr(),
                                   state.data_ptr(), N, Hk, H, dk, dv, out.data_ptr(), _here(dev))
    _check(st, "mesa_delta_step")
    return out


def _rows_dtype(dtype, x, *rows):
    """The dtype of a norm's rows: the first given tensor's, which an explicit
    out_dtype must agree with, else out_dtype, else x's."""
    for t in rows:
        if t is not None:
            if dtype is not None and dtype is not t.dtype:
                raise ValueError(f"out_dtype is {dtype}, expected {t.dtype}")
            return t.dtype
    return x.dtype if dtype is None else dtype


def _gate_checks(x, gate, w, grad_y=None, y=None, dtype=None):
    """Checks a gate norm's tensors; returns (B, H, T, d, dtype of y)."""
    import torch
    B, H, T, d = _dims(x, "x", 4)
    rows = (B, T, H, d)
    dtype = _rows_dtype(dtype, x, gate, grad_y, y)
    _tensors(x.device, (x, "x", (B, H, T, d), x.dtype), (w, "w", (H, d), torch.float32), (gate, "gate", rows, dtype),
             (grad_y, "grad_y", rows, dtype), (y, "out", rows, dtype))
    return B, H, T, d, dtype


def mesa_gate_norm(x, gate, w, eps=1e-6, *, out=None, out_dtype=None, stream=None):
    """Per-head RMS norm of a layer's outputs times silu(gate) (see include/mesa.h, mesa_gate_norm).

    x: [B,H,T,d]; gate: [B,T,H,d] or None; w: [H,d] float32.  Returns y
    [B,T,H,d] in gate's dtype (without a gate out_dtype, default x's).
    """
    import torch
    B, H, T, d, dtype = _gate_checks(x, gate, w, y=out, dtype=out_dtype)
    dev = x.device
    with _on(dev, stream):
        if out is None:
            out = torch.empty((B, T, H, d), dtype=dtype, device=dev)
        st = lib().mesa_gate_norm(x.data_ptr(), _qkv_dtype(x), _at(gate), _qkv_dtype(out), w.data_ptr(), eps, B, H, T, d,
                                  out.data_ptr(), _here(dev))
    _check(st, "mesa_gate_norm")
    return out


def mesa_gate_norm_backward(x, gate, w, grad_y, eps=1e-6, *, workspace=None, stream=None):
    """Gradients of mesa_gate_norm from its inputs and grad_y [B,T,H,d].
    Returns a dict of grad_x, grad_gate (None without a gate) and grad_w."""
    import torch
    B, H, T, d, dtype = _gate_checks(x, gate, w, grad_y=grad_y)
    dev = x.device
    with _on(dev, stream):
        g = dict(grad_x=torch.empty_like(x), grad_gate=None if gate is None else torch.empty_like(gate),
                 grad_w=torch.empty((H, d), dtype=torch.float32, device=dev))
        L = lib()
        workspace, nbytes = _scratch(workspace, L.mesa_gate_norm_backward_workspace_bytes(B, H, T, d), dev)
        st = L.mesa_gate_norm_backward(x.data_ptr(), _qkv_dtype(x), _at(gate), _qkv_dtype(grad_y), w.data_ptr(), eps,
                                       grad_y.data_ptr(), B, H, T, d, g["grad_x"].data_ptr(), _at(g["grad_gate"]),
                                       g["grad_w"].data_ptr(), workspace.data_ptr(), nbytes, _here(dev))
    _check(st, "mesa_gate_norm_backward")
    return g


def _residual_checks(h, y, w, scale, grad_n=None, grad_h_out=None, n=None, h_out=None, dtype=None):
    """Checks a residual norm's tensors; returns (R, D, dtype of n)."""
    import torch
    R, D = _dims(h, "h", 2)
    if y is None and (scale is not None or h_out is not None):
        raise ValueError("scale and h_out need y")
    dtype = _rows_dtype(dtype, h, y, grad_n, n)
    rows, ht, f32 = (R, D), h.dtype, torch.float32
    _tensors(h.device, (h, "h", rows, ht), (y, "y", rows, dtype), (w, "w", (D,), f32), (scale, "scale", (D,), f32),
             (grad_n, "grad_n", rows, dtype), (grad_h_out, "grad_h_out", rows, ht), (n, "n", rows, dtype),
             (h_out, "h_out", rows, ht))
    return R, D, dtype


def mesa_residual_norm(h, y, w, scale=None, eps=1e-6, *, h_out=None, n=None, out_dtype=None, stream=None):
    """Residual addition with its scale, and the next block's RMS norm (see
    include/mesa.h, mesa_residual_norm).

    h: [R,D] residual; y: [R,D] block output or None; w, scale: [D] float32.
    Returns (h_out = h + scale y in h's dtype, n in y's dtype); without y, (h,
    its norm in out_dtype, default h's).  h_out may be h itself.
    """
    import torch
    R, D, dtype = _residual_checks(h, y, w, scale, n=n, h_out=h_out, dtype=out_dtype)
    dev = h.device
    with _on(dev, stream):
        if n is None:
            n = torch.empty((R, D), dtype=dtype, device=dev)
        if y is not None and h_out is None:
            h_out = torch.empty_like(h)
        st = lib().mesa_residual_norm(h.data_ptr(), _qkv_dtype(h), _at(y), _qkv_dtype(n), _at(scale), w.data_ptr(), eps,
                                      R, D, _at(h_out), n.data_ptr(), _here(dev))
    _check(st, "mesa_residual_norm")
    return (h if y is None else h_out), n


def mesa_residual_norm_backward(h, y, w, grad_n, scale=None, eps=1e-6, *, grad_h_out=None, workspace=None, stream=None):
    """Gradients of mesa_residual_norm from its inputs, grad_n and grad_h_out
    (the residual's gradient from what follows, or None).  Returns a dict of
    grad_h, grad_y, grad_w and grad_scale (None where the input is)."""
    import torch
    R, D, dtype = _residual_checks(h, y, w, scale, grad_n=grad_n, grad_h_out=grad_h_out)
    dev = h.device
    with _on(dev, stream):
        f32 = dict(dtype=torch.float32, device=dev)
        g = dict(grad_h=torch.empty_like(h), grad_y=None if y is None else torch.empty_like(y),
                 grad_w=torch.empty((D,), **f32), grad_scale=None if scale is None else torch.empty((D,), **f32))
        L = lib()
        workspace, nbytes = _scratch(workspace, L.mesa_residual_norm_backward_workspace_bytes(R, D), dev)
        st = L.mesa_residual_norm_backward(h.data_ptr(), _qkv_dtype(h), _at(y), _qkv_dtype(grad_n), _at(scale),
                                           w.data_ptr(), eps, grad_n.data_ptr(), _at(grad_h_out), R, D,
                                           g["grad_h"].data_ptr(), _at(g["grad_y"]), g["grad_w"].data_ptr(),
                                           _at(g["grad_scale"]), workspace.data_ptr(), nbytes, _here(dev))
    _check(st, "mesa_residual_norm_backward")
    return g


def profile_enable(on: bool = True):
    _check(lib().mesa_profile_enable(1 if on else 0), "mesa_profile_enable")


def profile_reset():
    _check(lib().mesa_profile_reset(), "mesa_profile_reset")


def profile_read(kernel_id: int):
    """(total milliseconds, launches) recorded for one kernel id since the last reset."""
    ms = ctypes.c_double(0)
    n = ctypes.c_int64(0)
    _check(lib().mesa_profile_read(kernel_id, ctypes.byref(ms), ctypes.byref(n)), "mesa_profile_read")
    return ms.value, n.value


def probe_mfma(dtype: str, n_workgroups: int, iters: int, sink, stream=None):
    """Launch the register-resident MFMA probe ("f32" or "bf16"); returns its flops."""
    fn = lib().mesa_probe_mfma_f32 if dtype == "f32" else lib().mesa_probe_mfma_bf16
    _check(fn(n_workgroups, iters, _ptr(sink), _stream(stream)), "mesa_probe_mfma")
    return n_workgroups * 4 * iters * 8 * (2048 if dtype == "f32" else 16384)


def probe_copy(src, dst, stream=None):
    """Launch the streaming-copy probe over src.numel() bytes of src (uint8) into dst."""
    _check(lib().mesa_probe_copy(_ptr(src), _ptr(dst), src.numel() * src.element_size(), _stream(stream)),
           "mesa_probe_copy")


def kernel_name(kernel_id: int) -> str:
    return lib().mesa_kernel_name(kernel_id).decode()
