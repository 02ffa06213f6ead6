"""Python binding of the B200 WKV operator library (``librwkv_wkv.so``).

Two layers, both argument marshalling only (every step of the operator runs in
the library's CUDA kernels):

* ``lib()`` returns the ctypes handle whose functions carry the exact C-ABI
  names and signatures of ``include/rwkv_wkv.h`` (``rwkv_wkv4_forward``,
  ``rwkv_wkv4_backward``, ``rwkv_wkv4_step``, ``rwkv_wkv5_forward``, ...).
* ``rwkv_wkv4_forward`` & co. below take torch CUDA tensors, allocate outputs
  and workspace with torch, pass raw device pointers and the current torch
  stream to the C call, and raise ``RwkvError`` on a non-OK status.

There is no fallback: if the library is missing or a call fails, this raises.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "LIB_PATH", "lib", "RwkvError", "RWKV_OK", "F32", "BF16", "ALGO_AUTO", "ALGO_SEQUENTIAL",
    "ALGO_CHUNKED", "CHUNK_LEN", "NOALLOC_MAX_LANES", "rwkv_wkv4_forward", "rwkv_wkv4_backward",
    "rwkv_wkv4_backward_noalloc", "rwkv_wkv4_step", "rwkv_wkv4_forward_gated", "rwkv_wkv4_backward_gated",
    "rwkv_wkv5_forward", "rwkv_wkv5_backward", "rwkv_wkv5_step", "rwkv_wkv6_forward", "rwkv_wkv6_backward",
    "rwkv_wkv6_step", "rwkv_causal_conv_forward", "rwkv_causal_conv_backward", "rwkv_causal_conv_step",
    "rwkv_selective_scan_forward", "rwkv_selective_scan_backward", "rwkv_selective_scan_step",
    "rwkv_layer_norm_forward", "rwkv_layer_norm_backward", "rwkv_check_device_error",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librwkv_wkv.so")

RWKV_OK = 0
F32, BF16 = 0, 1
ALGO_AUTO, ALGO_SEQUENTIAL, ALGO_CHUNKED = 0, 1, 2
CHUNK_LEN = 16  # checkpoint interval of the WKV-4 forward/backward pair
NOALLOC_MAX_LANES = 262144  # RWKV_NOALLOC_MAX_LANES: largest B*C of rwkv_wkv4_backward_noalloc

_lib = None


class RwkvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().rwkv_status_string(status).decode()
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


def lib():
    """ctypes handle of librwkv_wkv.so with argtypes set from the C header."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m rwkv_wkv_recurrence_b200._build` (needs nvcc)")
    h = ctypes.CDLL(LIB_PATH)
    I64, P, S, I = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    sig = {
        "rwkv_status_string": ([I], ctypes.c_char_p),
        "rwkv_version": ([], I),
        "rwkv_wkv4_num_checkpoints": ([I64, I64], I64),
        "rwkv_wkv4_forward_workspace_bytes": ([I64, I64, I64, I], S),
        "rwkv_wkv4_forward": ([I64, I64, I64, I, P, P, P, P, P, P, P, P, I64, I, P, S, P], I),
        "rwkv_wkv4_backward_workspace_bytes": ([I64, I64, I64, I64, I], S),
        "rwkv_wkv4_backward": ([I64, I64, I64, I, P, P, P, P, P, P, P, I64, P, P, P, P, P, S, P], I),
        "rwkv_wkv4_step": ([I64, I64, I, P, P, P, P, P, P, P, P], I),
        "rwkv_wkv4_forward_gated": ([I64, I64, I64, I, P, P, P, P, P, P, P, P, P, I64, I, P, S, P], I),
        "rwkv_wkv4_backward_gated": ([I64, I64, I64, I, P, P, P, P, P, P, P, P, I64, P, P, P, P, P, P, S, P], I),
        "rwkv_wkv5_forward_workspace_bytes": ([I64, I64, I64, I64], S),
        "rwkv_wkv5_forward": ([I64, I64, I64, I64, P, P, P, P, P, P, P, P, P, S, P], I),
        "rwkv_wkv4_backward_noalloc": ([I64, I64, I64, I, P, P, P, P, P, P, I64, P, P, P, P, P], I),
        "rwkv_wkv5_step": ([I64, I64, I64, P, P, P, P, P, P, P, P, P], I),
        "rwkv_wkv5_backward_workspace_bytes": ([I64, I64, I64, I64], S),
        "rwkv_wkv5_backward": ([I64, I64, I64, I64] + [P] * 15 + [S, P], I),
        "rwkv_wkv6_forward_workspace_bytes": ([I64, I64, I64, I64], S),
        "rwkv_wkv6_forward": ([I64, I64, I64, I64, P, P, P, P, P, P, P, P, P, S, P], I),
        "rwkv_wkv6_backward_workspace_bytes": ([I64, I64, I64, I64], S),
        "rwkv_wkv6_backward": ([I64, I64, I64, I64] + [P] * 15 + [S, P], I),
        "rwkv_wkv6_step": ([I64, I64, I64, P, P, P, P, P, P, P, P, P], I),
        "rwkv_causal_conv_forward": ([I64] * 4 + [I, P, P, I, P, I64, P, P, P, P], I),
        "rwkv_causal_conv_backward_workspace_bytes": ([I64] * 4, S),
        "rwkv_causal_conv_backward": ([I64] * 4 + [I, P, P, I, P, I64] + [P] * 8 + [S, P], I),
        "rwkv_causal_conv_step": ([I64] * 3 + [I, P, P, I, P, I64, P, P, P, P], I),
        "rwkv_selective_scan_forward_workspace_bytes": ([I64] * 4 + [I], S),
        "rwkv_selective_scan_forward": ([I64] * 4 + [I, P, P, P] + [P, I64] * 5 + [P, P, P, P, I64, I, P, S, P], I),
        "rwkv_selective_scan_backward_workspace_bytes": ([I64] * 5 + [I], S),
        "rwkv_selective_scan_backward": ([I64] * 4 + [I, P, P, P] + [P, I64] * 5 + [P] * 4 + [I64] + [P] * 10
                                         + [S, P], I),
        "rwkv_selective_scan_step": ([I64] * 3 + [I, P, P, P] + [P, I64] * 5 + [P] * 4, I),
        "rwkv_layer_norm_forward": ([I64] * 3 + [I, P, P, ctypes.c_float] + [P] * 4, I),
        "rwkv_layer_norm_backward_workspace_bytes": ([I64] * 3 + [I], S),
        "rwkv_layer_norm_backward": ([I64] * 3 + [I, P, P, ctypes.c_float] + [P] * 8 + [S, P], I),
        "rwkv_check_device_error": ([P], I),
        "rwkv_debug_set_wait_limit_ns": ([ctypes.c_uint64], I),
        "rwkv_debug_withhold_loads": ([I], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(h, name)
        f.argtypes = args
        f.restype = res
    _lib = h
    return h


# ------------------------------------------------------------------ helpers
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, status):
    if status != RWKV_OK:
        raise RwkvError(fn, status)


def _dtype_code(t):
    import torch

    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"WKV-4 tensors must be float32 or bfloat16, got {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("WKV tensors must be CUDA tensors (use .cuda())")
            if not t.is_contiguous():
                raise ValueError("WKV tensors must be contiguous")


def _f32(name, t, n):
    import torch

    if t.dtype != torch.float32 or t.numel() != n:
        raise ValueError(f"{name} must be float32 with {n} elements")


# ------------------------------------------------------------------ WKV-4
def rwkv_wkv4_forward(w, u, k, v, state_in=None, *, return_state=False, checkpoints=False,
                      algo=ALGO_AUTO, stream=None, out=None):
    """WKV-4 forward.  k, v [B,T,C] (fp32 or bf16); w, u [C] fp32.

    Returns y, plus the final state [3,B,C] if ``return_state`` and the
    checkpoints [ceil(T/16),3,B,C] for ``rwkv_wkv4_backward`` if ``checkpoints``.
    """
    import torch

    _need_cuda(w, u, k, v, state_in)
    B, T, C = k.shape
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v must have the same shape and dtype")
    _f32("w", w, C)
    _f32("u", u, C)
    if state_in is not None:
        _f32("state_in", state_in, 3 * B * C)
    h = lib()
    y = torch.empty_like(k) if out is None else out
    st = torch.empty((3, B, C), dtype=torch.float32, device=k.device) if return_state else None
    nck = int(h.rwkv_wkv4_num_checkpoints(T, CHUNK_LEN))
    ck = torch.empty((nck, 3, B, C), dtype=torch.float32, device=k.device) if checkpoints else None
    wsb = int(h.rwkv_wkv4_forward_workspace_bytes(B, T, C, algo))
    ws = torch.empty(wsb, dtype=torch.uint8, device=k.device) if wsb else None
    _check("rwkv_wkv4_forward",
           h.rwkv_wkv4_forward(B, T, C, _dtype_code(k), _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(y),
                               _ptr(state_in), _ptr(st), _ptr(ck), CHUNK_LEN, algo, _ptr(ws), wsb,
                               _stream(stream)))
    res = (y,)
    if return_state:
        res += (st,)
    if checkpoints:
        res += (ck,)
    return res[0] if len(res) == 1 else res


def rwkv_wkv4_backward(w, u, k, v, gy, ckpt=None, state_in=None, *, stream=None, out=None):
    """WKV-4 backward: returns (gk, gv, gw, gu) for L = sum(gy * y).

    ``ckpt`` are the forward's checkpoints (or None to recompute them)."""
    import torch

    _need_cuda(w, u, k, v, gy, ckpt, state_in)
    B, T, C = k.shape
    for name, t in (("v", v), ("gy", gy)):
        if t.shape != k.shape or t.dtype != k.dtype:
            raise ValueError(f"{name} must match k in shape and dtype")
    _f32("w", w, C)
    _f32("u", u, C)
    h = lib()
    if ckpt is not None:
        _f32("ckpt", ckpt, int(h.rwkv_wkv4_num_checkpoints(T, CHUNK_LEN)) * 3 * B * C)
    if state_in is not None:
        _f32("state_in", state_in, 3 * B * C)
    if out is None:
        gk, gv = torch.empty_like(k), torch.empty_like(v)
        gw = torch.empty(C, dtype=torch.float32, device=k.device)
        gu = torch.empty(C, dtype=torch.float32, device=k.device)
    else:
        gk, gv, gw, gu = out
    wsb = int(h.rwkv_wkv4_backward_workspace_bytes(B, T, C, CHUNK_LEN, 1 if ckpt is not None else 0))
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=k.device)
    _check("rwkv_wkv4_backward",
           h.rwkv_wkv4_backward(B, T, C, _dtype_code(k), _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(gy),
                                _ptr(state_in), _ptr(ckpt), CHUNK_LEN, _ptr(gk), _ptr(gv), _ptr(gw),
                                _ptr(gu), _ptr(ws), wsb, _stream(stream)))
    return gk, gv, gw, gu


def rwkv_wkv4_forward_gated(w, u, k, v, r, state_in=None, *, return_state=False, checkpoints=False,
                            algo=ALGO_AUTO, stream=None, out=None):
    """Receptance-gated WKV-4 forward: o = sigmoid(r) * WKV in one pass.  k, v, r
    [B,T,C] (fp32 or bf16); w, u [C] fp32.  Returns o (plus the state and the
    checkpoints as ``rwkv_wkv4_forward``)."""
    import torch

    _need_cuda(w, u, k, v, r, state_in)
    B, T, C = k.shape
    for name, t in (("v", v), ("r", r)):
        if t.shape != k.shape or t.dtype != k.dtype:
            raise ValueError(f"{name} must match k in shape and dtype")
    _f32("w", w, C)
    _f32("u", u, C)
    if state_in is not None:
        _f32("state_in", state_in, 3 * B * C)
    h = lib()
    o = torch.empty_like(k) if out is None else out
    st = torch.empty((3, B, C), dtype=torch.float32, device=k.device) if return_state else None
    nck = int(h.rwkv_wkv4_num_checkpoints(T, CHUNK_LEN))
    ck = torch.empty((nck, 3, B, C), dtype=torch.float32, device=k.device) if checkpoints else None
    wsb = int(h.rwkv_wkv4_forward_workspace_bytes(B, T, C, algo))
    ws = torch.empty(wsb, dtype=torch.uint8, device=k.device) if wsb else None
    _check("rwkv_wkv4_forward_gated",
           h.rwkv_wkv4_forward_gated(B, T, C, _dtype_code(k), _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(r), _ptr(o),
                                     _ptr(state_in), _ptr(st), _ptr(ck), CHUNK_LEN, algo, _ptr(ws), wsb,
                                     _stream(stream)))
    res = (o,)
    if return_state:
        res += (st,)
    if checkpoints:
        res += (ck,)
    return res[0] if len(res) == 1 else res


def rwkv_wkv4_backward_gated(w, u, k, v, r, go, ckpt=None, state_in=None, *, stream=None, out=None):
    """Backward of the gated forward: returns (gk, gv, gr, gw, gu) for
    L = sum(go * o), o = sigmoid(r) * WKV."""
    import torch

    _need_cuda(w, u, k, v, r, go, ckpt, state_in)
    B, T, C = k.shape
    for name, t in (("v", v), ("r", r), ("go", go)):
        if t.shape != k.shape or t.dtype != k.dtype:
            raise ValueError(f"{name} must match k in shape and dtype")
    _f32("w", w, C)
    _f32("u", u, C)
    h = lib()
    if ckpt is not None:
        _f32("ckpt", ckpt, int(h.rwkv_wkv4_num_checkpoints(T, CHUNK_LEN)) * 3 * B * C)
    if state_in is not None:
        _f32("state_in", state_in, 3 * B * C)
    if out is None:
        gk, gv, gr = torch.empty_like(k), torch.empty_like(v), torch.empty_like(r)
        gw = torch.empty(C, dtype=torch.float32, device=k.device)
        gu = torch.empty(C, dtype=torch.float32, device=k.device)
    else:
        gk, gv, gr, gw, gu = out
    wsb = int(h.rwkv_wkv4_backward_workspace_bytes(B, T, C, CHUNK_LEN, 1 if ckpt is not None else 0))
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=k.device)
    _check("rwkv_wkv4_backward_gated",
           h.rwkv_wkv4_backward_gated(B, T, C, _dtype_code(k), _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(r),
                                      _ptr(go), _ptr(state_in), _ptr(ckpt), CHUNK_LEN, _ptr(gk), _ptr(gv),
                                      _ptr(gr), _ptr(gw), _ptr(gu), _ptr(ws), wsb, _stream(stream)))
    return gk, gv, gr, gw, gu


def rwkv_wkv4_backward_noalloc(w, u, k, v, gy, ckpt, *, stream=None, out=None):
    """WKV-4 backward through the entry point that allocates no device memory
    and takes no workspace (its scratch is a fixed array inside the library,
    shared by all calls; see include/rwkv_wkv.h).  ``ckpt`` is required.
    Output tensors are still the caller's: pass ``out=(gk, gv, gw, gu)`` to
    keep this call free of allocations from Python too."""
    import torch

    _need_cuda(w, u, k, v, gy, ckpt)
    B, T, C = k.shape
    for name, t in (("v", v), ("gy", gy)):
        if t.shape != k.shape or t.dtype != k.dtype:
            raise ValueError(f"{name} must match k in shape and dtype")
    _f32("w", w, C)
    _f32("u", u, C)
    _f32("ckpt", ckpt, int(lib().rwkv_wkv4_num_checkpoints(T, CHUNK_LEN)) * 3 * B * C)
    if out is None:
        gk, gv = torch.empty_like(k), torch.empty_like(v)
        gw = torch.empty(C, dtype=torch.float32, device=k.device)
        gu = torch.empty(C, dtype=torch.float32, device=k.device)
    else:
        gk, gv, gw, gu = out
    _check("rwkv_wkv4_backward_noalloc",
           lib().rwkv_wkv4_backward_noalloc(B, T, C, _dtype_code(k), _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(gy),
                                            _ptr(ckpt), CHUNK_LEN, _ptr(gk), _ptr(gv), _ptr(gw), _ptr(gu),
                                            _stream(stream)))
    return gk, gv, gw, gu


def rwkv_wkv4_step(w, u, k, v, state, *, state_out=None, stream=None, out=None):
    """One decode token: k, v [B,C]; state [3,B,C] updated in place unless
    ``state_out`` is given.  Returns y [B,C]."""
    import torch

    _need_cuda(w, u, k, v, state, state_out)
    B, C = k.shape
    y = torch.empty_like(k) if out is None else out
    so = state if state_out is None else state_out
    _check("rwkv_wkv4_step",
           lib().rwkv_wkv4_step(B, C, _dtype_code(k), _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(y),
                                _ptr(state), _ptr(so), _stream(stream)))
    return y


# ------------------------------------------------------------------ WKV-5
def rwkv_wkv5_forward(r, k, v, omega, u, s_in=None, *, return_state=False, stream=None, out=None):
    """Eagle / RWKV-5 forward: r, k, v [B,T,H,N] bf16; omega, u [H,N] fp32."""
    import torch

    _need_cuda(r, k, v, omega, u, s_in)
    B, T, H, N = r.shape
    for t in (r, k, v):
        if t.dtype != torch.bfloat16 or t.shape != r.shape:
            raise ValueError("r, k, v must be bf16 of the same shape")
    _f32("omega", omega, H * N)
    _f32("u", u, H * N)
    h = lib()
    y = torch.empty_like(r) if out is None else out
    so = torch.empty((B, H, N, N), dtype=torch.float32, device=r.device) if return_state else None
    wsb = int(h.rwkv_wkv5_forward_workspace_bytes(B, T, H, N))
    ws = torch.empty(wsb, dtype=torch.uint8, device=r.device) if wsb else None
    _check("rwkv_wkv5_forward",
           h.rwkv_wkv5_forward(B, T, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(omega), _ptr(u), _ptr(y),
                               _ptr(s_in), _ptr(so), _ptr(ws), wsb, _stream(stream)))
    return (y, so) if return_state else y


def rwkv_wkv5_backward(r, k, v, omega, u, gy, s_in=None, gs_out=None, *, want_gs_in=False, stream=None):
    """Eagle / RWKV-5 backward: gradients of sum(gy * y) + sum(gs_out * s_out).  r, k, v, gy
    [B,T,H,N] bf16; omega, u [H,N] fp32; s_in, gs_out [B,H,N,N] fp32 or None.  Returns
    (gr, gk, gv, gomega, gu) and, with ``want_gs_in``, the gradient of s_in as well."""
    import torch

    _need_cuda(r, k, v, omega, u, gy, s_in, gs_out)
    B, T, H, N = r.shape
    for t in (r, k, v, gy):
        if t.dtype != torch.bfloat16 or t.shape != r.shape:
            raise ValueError("r, k, v, gy must be bf16 of the same shape")
    _f32("omega", omega, H * N)
    _f32("u", u, H * N)
    for name, t in (("s_in", s_in), ("gs_out", gs_out)):
        if t is not None:
            _f32(name, t, B * H * N * N)
    h = lib()
    gr, gk, gv = torch.empty_like(r), torch.empty_like(k), torch.empty_like(v)
    gomega = torch.empty((H, N), dtype=torch.float32, device=r.device)
    gu = torch.empty((H, N), dtype=torch.float32, device=r.device)
    gsi = torch.empty((B, H, N, N), dtype=torch.float32, device=r.device) if want_gs_in else None
    wsb = int(h.rwkv_wkv5_backward_workspace_bytes(B, T, H, N))
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=r.device)
    _check("rwkv_wkv5_backward",
           h.rwkv_wkv5_backward(B, T, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(omega), _ptr(u), _ptr(s_in), _ptr(gy),
                                _ptr(gs_out), _ptr(gr), _ptr(gk), _ptr(gv), _ptr(gomega), _ptr(gu), _ptr(gsi),
                                _ptr(ws), wsb, _stream(stream)))
    res = (gr, gk, gv, gomega, gu)
    return res + (gsi,) if want_gs_in else res


def rwkv_wkv6_backward(r, k, v, omega, u, gy, s_in=None, gs_out=None, *, want_gs_in=False, stream=None):
    """Finch / RWKV-6 backward: gradients of sum(gy * y) + sum(gs_out * s_out).  r, k, v, gy
    [B,T,H,N] bf16; omega [B,T,H,N] fp32 (per token); u [H,N] fp32; s_in, gs_out [B,H,N,N] fp32 or
    None.  Returns (gr, gk, gv, gomega [B,T,H,N], gu [H,N]) and, with ``want_gs_in``, the gradient
    of s_in as well."""
    import torch

    _need_cuda(r, k, v, omega, u, gy, s_in, gs_out)
    B, T, H, N = r.shape
    for t in (r, k, v, gy):
        if t.dtype != torch.bfloat16 or t.shape != r.shape:
            raise ValueError("r, k, v, gy must be bf16 of the same shape")
    _f32("omega", omega, B * T * H * N)
    _f32("u", u, H * N)
    for name, t in (("s_in", s_in), ("gs_out", gs_out)):
        if t is not None:
            _f32(name, t, B * H * N * N)
    h = lib()
    gr, gk, gv = torch.empty_like(r), torch.empty_like(k), torch.empty_like(v)
    gomega = torch.empty((B, T, H, N), dtype=torch.float32, device=r.device)
    gu = torch.empty((H, N), dtype=torch.float32, device=r.device)
    gsi = torch.empty((B, H, N, N), dtype=torch.float32, device=r.device) if want_gs_in else None
    wsb = int(h.rwkv_wkv6_backward_workspace_bytes(B, T, H, N))
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=r.device)
    _check("rwkv_wkv6_backward",
           h.rwkv_wkv6_backward(B, T, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(omega), _ptr(u), _ptr(s_in), _ptr(gy),
                                _ptr(gs_out), _ptr(gr), _ptr(gk), _ptr(gv), _ptr(gomega), _ptr(gu), _ptr(gsi),
                                _ptr(ws), wsb, _stream(stream)))
    res = (gr, gk, gv, gomega, gu)
    return res + (gsi,) if want_gs_in else res


def rwkv_wkv5_step(r, k, v, omega, u, state=None, *, state_out=None, stream=None, out=None):
    """Eagle / RWKV-5 decode step: r, k, v [B,H,N] bf16 (one token per stream);
    omega, u [H,N] fp32; state [B,H,N,N] fp32 or None (zero).  Returns
    (y [B,H,N] bf16, new state).  state_out may be `state` (in-place)."""
    import torch

    _need_cuda(r, k, v, omega, u, state, state_out)
    B, H, N = r.shape
    for t in (r, k, v):
        if t.dtype != torch.bfloat16 or t.shape != r.shape:
            raise ValueError("r, k, v must be bf16 of the same shape")
    _f32("omega", omega, H * N)
    _f32("u", u, H * N)
    y = torch.empty_like(r) if out is None else out
    so = state_out if state_out is not None else torch.empty((B, H, N, N), dtype=torch.float32, device=r.device)
    _check("rwkv_wkv5_step",
           lib().rwkv_wkv5_step(B, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(omega), _ptr(u), _ptr(y), _ptr(state),
                                _ptr(so), _stream(stream)))
    return y, so


# ------------------------------------------------------------------ WKV-6
def rwkv_wkv6_forward(r, k, v, omega, u, s_in=None, *, return_state=False, stream=None, out=None):
    """Finch / RWKV-6 forward (per-token decay): r, k, v [B,T,H,N] bf16;
    omega [B,T,H,N] fp32; u [H,N] fp32; s_in [B,H,N,N] fp32 or None."""
    import torch

    _need_cuda(r, k, v, omega, u, s_in)
    B, T, H, N = r.shape
    for t in (r, k, v):
        if t.dtype != torch.bfloat16 or t.shape != r.shape:
            raise ValueError("r, k, v must be bf16 of the same shape")
    if omega.dtype != torch.float32 or omega.shape != r.shape or not omega.is_contiguous():
        raise ValueError("omega must be a contiguous float32 tensor shaped like r")
    _f32("u", u, H * N)
    h = lib()
    y = torch.empty_like(r) if out is None else out
    so = torch.empty((B, H, N, N), dtype=torch.float32, device=r.device) if return_state else None
    wsb = int(h.rwkv_wkv6_forward_workspace_bytes(B, T, H, N))
    ws = torch.empty(wsb, dtype=torch.uint8, device=r.device) if wsb else None
    _check("rwkv_wkv6_forward",
           h.rwkv_wkv6_forward(B, T, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(omega), _ptr(u), _ptr(y),
                               _ptr(s_in), _ptr(so), _ptr(ws), wsb, _stream(stream)))
    return (y, so) if return_state else y


def rwkv_wkv6_step(r, k, v, omega, u, state=None, *, state_out=None, stream=None, out=None):
    """Finch / RWKV-6 decode step: r, k, v [B,H,N] bf16 and omega [B,H,N] fp32
    (one token per stream); u [H,N] fp32; state [B,H,N,N] fp32 or None (zero).
    Returns (y [B,H,N] bf16, new state).  state_out may be `state` (in-place)."""
    import torch

    _need_cuda(r, k, v, omega, u, state, state_out)
    B, H, N = r.shape
    for t in (r, k, v):
        if t.dtype != torch.bfloat16 or t.shape != r.shape:
            raise ValueError("r, k, v must be bf16 of the same shape")
    _f32("omega", omega, B * H * N)
    _f32("u", u, H * N)
    y = torch.empty_like(r) if out is None else out
    so = state_out if state_out is not None else torch.empty((B, H, N, N), dtype=torch.float32, device=r.device)
    _check("rwkv_wkv6_step",
           lib().rwkv_wkv6_step(B, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(omega), _ptr(u), _ptr(y), _ptr(state),
                                _ptr(so), _stream(stream)))
    return y, so


# ------------------------------------------------------------------ around the recurrence
# Decode calls these once per token and operator, so the checks below look at each tensor once and
# pass plain integers on: a call costs the host little more than its launch.
ACT_NONE, ACT_SILU = 0, 1
_fns = {}


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = getattr(lib(), name)
    return f


def _addr(t):
    return None if t is None else t.data_ptr()


def _io_code(name, t):
    import torch

    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _refuse(name, t, shape, dtype, index):
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected the device of the other tensors")
    raise ValueError(f"{name} must be contiguous")


def _dense(name, t, shape, dtype, index):
    """t (or None) is a contiguous tensor of this shape and type on device `index`; its address."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(name, t, shape, dtype, index)
    return t.data_ptr()


def _rows(name, t, shape, dtype, index):
    """Elements between the rows of t, whose last dimension is dense and whose rows lie at equal
    distances (a whole tensor, or a part of a wider one's last dimension)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _refuse(name, t, shape, dtype, index)
    width = shape[-1]
    if t.is_contiguous():
        return width
    stride = t.stride()
    if width > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    ld, inner = None, 1
    for size, st in zip(shape[-2::-1], stride[-2::-1]):
        if size == 1:
            continue
        if ld is None:
            ld = st
        elif st != ld * inner:
            raise ValueError(f"{name}: rows must lie at equal distances, got strides {stride}")
        inner *= size
    ld = width if ld is None else ld
    if ld < width:
        raise ValueError(f"{name}: rows overlap, got strides {stride}")
    return ld


def _dims(name, t, n):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(t.shape)}")
    return t.shape


class _Elsewhere:
    """A call that launches on another stream than the current one: its allocations belong to that
    stream, and the tensors the two share are recorded on both, so that memory freed after the call
    is not handed out again too early."""

    def __init__(self, stream):
        self.stream, self.outputs = stream, []

    def empty(self, x, shape, dtype, output):
        import torch

        with torch.cuda.stream(self.stream):
            t = x.new_empty(shape, dtype=dtype)
        if output:
            self.outputs.append(t)
        return t

    def done(self, *given):
        import torch

        current = torch.cuda.current_stream()
        for t in self.outputs:
            t.record_stream(current)
        for t in given:
            if t is not None:
                t.record_stream(self.stream)


def _launch(x, stream):
    """The device index of x, the stream handle a call launches on, and an ``_Elsewhere`` where that is
    not the current stream (else None)."""
    import torch

    index = x.get_device()
    if index < 0:
        raise ValueError("tensors must be CUDA tensors (use .cuda())")
    current = torch._C._cuda_getDevice()
    if index != current:
        raise ValueError(f"tensors are on {x.device}, the current device is cuda:{current}")
    raw = torch._C._cuda_getCurrentRawStream(index)
    if stream is None:
        return index, raw, None
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on {x.device}")
    if stream.cuda_stream == raw:
        return index, raw, None
    return index, stream.cuda_stream, _Elsewhere(stream)


def _like(x, other):
    """An output shaped and typed like x, contiguous."""
    import torch

    if other is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return other.empty(x, x.shape, x.dtype, True)


def _empty(x, shape, dtype, other):
    return x.new_empty(shape, dtype=dtype) if other is None else other.empty(x, shape, dtype, True)


def _workspace(x, nbytes, other):
    import torch

    if not nbytes:
        return None
    return x.new_empty(nbytes, dtype=torch.uint8) if other is None else other.empty(x, (nbytes,), torch.uint8, False)


def rwkv_causal_conv_forward(x, weight, bias=None, state_in=None, *, silu=False, return_state=False, stream=None,
                             out=None):
    """Causal convolution over time, one filter of W = 2, 3 or 4 taps per channel:
    y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j}), act the identity or (``silu``) silu.

    x [B,T,C] (fp32 or bf16; rows may be part of a wider tensor); weight [C,W], bias [C] fp32;
    state_in [B,W-1,C] like x, the tokens before the first, or None (zeros).  Returns y, plus the
    last W-1 tokens [B,W-1,C] if ``return_state``."""
    import torch

    (dev, raw, other), dt = _launch(x, stream), x.dtype
    code = _io_code("x", x)
    B, T, C = _dims("x", x, 3)
    W = _dims("weight", weight, 2)[1]
    p_weight = _dense("weight", weight, (C, W), torch.float32, dev)
    p_bias = _dense("bias", bias, (C,), torch.float32, dev)
    p_state_in = _dense("state_in", state_in, (B, W - 1, C), dt, dev)
    _dense("out", out, (B, T, C), dt, dev)
    ldx = _rows("x", x, (B, T, C), dt, dev)
    y = _like(x, other) if out is None else out
    st = _empty(x, (B, W - 1, C), dt, other) if return_state and W > 0 else None
    _check("rwkv_causal_conv_forward",
           _fn("rwkv_causal_conv_forward")(B, T, C, W, code, p_weight, p_bias,
                                           ACT_SILU if silu else ACT_NONE, _addr(x), ldx, _addr(y), p_state_in,
                                           _addr(st), raw))
    if other is not None:
        other.done(x, weight, bias, state_in, out)
    return (y, st) if return_state else y


def rwkv_causal_conv_backward(x, weight, gy, bias=None, state_in=None, gstate_out=None, *, silu=False,
                              want_gstate_in=False, stream=None):
    """Gradients of sum(gy * y) + sum(gstate_out * state_out) of ``rwkv_causal_conv_forward``:
    returns (gx, gweight, gbias) and, with ``want_gstate_in``, the gradient of state_in as well;
    gbias is None where bias is."""
    import torch

    (dev, raw, other), dt = _launch(x, stream), x.dtype
    code = _io_code("x", x)
    B, T, C = _dims("x", x, 3)
    W = _dims("weight", weight, 2)[1]
    p_weight = _dense("weight", weight, (C, W), torch.float32, dev)
    p_bias = _dense("bias", bias, (C,), torch.float32, dev)
    p_gy = _dense("gy", gy, (B, T, C), dt, dev)
    p_state_in = _dense("state_in", state_in, (B, W - 1, C), dt, dev)
    p_gstate_out = _dense("gstate_out", gstate_out, (B, W - 1, C), dt, dev)
    ldx = _rows("x", x, (B, T, C), dt, dev)
    gx = _like(x, other)
    gw = _empty(x, (C, W), torch.float32, other)
    gb = _empty(x, (C,), torch.float32, other) if bias is not None else None
    gs = _empty(x, (B, W - 1, C), dt, other) if want_gstate_in and W > 0 else None
    wsb = _fn("rwkv_causal_conv_backward_workspace_bytes")(B, T, C, W)
    ws = _workspace(x, wsb, other)
    _check("rwkv_causal_conv_backward",
           _fn("rwkv_causal_conv_backward")(B, T, C, W, code, p_weight, p_bias,
                                            ACT_SILU if silu else ACT_NONE, _addr(x), ldx, p_state_in, p_gy,
                                            p_gstate_out, _addr(gx), _addr(gw), _addr(gb), _addr(gs), _addr(ws),
                                            wsb, raw))
    if other is not None:
        other.done(x, weight, gy, bias, state_in, gstate_out)
    return (gx, gw, gb, gs) if want_gstate_in else (gx, gw, gb)


def rwkv_causal_conv_step(x, weight, state, bias=None, *, silu=False, state_out=None, stream=None, out=None):
    """One token for each of B streams: x [B,C]; state [B,W-1,C] like x, updated in place unless
    ``state_out`` is given.  Returns y [B,C]."""
    import torch

    (dev, raw, other), dt = _launch(x, stream), x.dtype
    code = _io_code("x", x)
    B, C = _dims("x", x, 2)
    W = _dims("weight", weight, 2)[1]
    p_weight = _dense("weight", weight, (C, W), torch.float32, dev)
    p_bias = _dense("bias", bias, (C,), torch.float32, dev)
    p_state = _dense("state", state, (B, W - 1, C), dt, dev)
    _dense("state_out", state_out, (B, W - 1, C), dt, dev)
    _dense("out", out, (B, C), dt, dev)
    ldx = _rows("x", x, (B, C), dt, dev)
    y = _like(x, other) if out is None else out
    so = state if state_out is None else state_out
    _check("rwkv_causal_conv_step",
           _fn("rwkv_causal_conv_step")(B, C, W, code, p_weight, p_bias, ACT_SILU if silu else ACT_NONE,
                                        _addr(x), ldx, _addr(y), p_state, _addr(so), raw))
    if other is not None:
        other.done(x, weight, state, bias, state_out, out)
    return y


def _scan_args(x, dt, b, c, a_log, d, dt_bias, z, dev):
    """Checks what the scan's calls share; returns N and the C calls' arguments from a_log to ldz."""
    import torch

    lead, C, ty = x.shape[:-1], x.shape[-1], x.dtype
    N = _dims("a_log", a_log, 2)[1]
    p_a_log = _dense("a_log", a_log, (C, N), torch.float32, dev)
    p_d = _dense("d", d, (C,), torch.float32, dev)
    p_dt_bias = _dense("dt_bias", dt_bias, (C,), torch.float32, dev)
    wide, state = lead + (C,), lead + (N,)
    return N, (p_a_log, p_d, p_dt_bias,
               _addr(x), _rows("x", x, wide, ty, dev), _addr(dt), _rows("dt", dt, wide, ty, dev),
               _addr(b), _rows("b", b, state, ty, dev), _addr(c), _rows("c", c, state, ty, dev),
               _addr(z), _rows("z", z, wide, ty, dev) if z is not None else C)


def rwkv_selective_scan_forward(x, dt, b, c, a_log, d=None, dt_bias=None, z=None, h_in=None, *, return_state=False,
                                checkpoints=False, algo=ALGO_AUTO, stream=None, out=None):
    """Selective scan: with D = softplus(dt + dt_bias) and A = -exp(a_log), per channel
    h_t = exp(D_t A) h_{t-1} + D_t x_t b_t,  y_t = c_t . h_t + d x_t, times silu(z_t) if z is given.

    x, dt, z [B,T,C] and b, c [B,T,N] (fp32 or bf16, all alike; rows may be parts of wider tensors);
    a_log [C,N], d, dt_bias [C] fp32; h_in [B,C,N] fp32 or None (zero); N 8, 16, 32 or 64.  Returns
    y, plus the final state [B,C,N] if ``return_state`` and the checkpoints [ceil(T/16),B,C,N] for
    ``rwkv_selective_scan_backward`` if ``checkpoints``."""
    import torch

    (dev, raw, other), ty = _launch(x, stream), x.dtype
    code = _io_code("x", x)
    B, T, C = _dims("x", x, 3)
    N, args = _scan_args(x, dt, b, c, a_log, d, dt_bias, z, dev)
    p_h_in = _dense("h_in", h_in, (B, C, N), torch.float32, dev)
    _dense("out", out, (B, T, C), ty, dev)
    y = _like(x, other) if out is None else out
    ho = _empty(x, (B, C, N), torch.float32, other) if return_state else None
    ck = _empty(x, ((T + CHUNK_LEN - 1) // CHUNK_LEN, B, C, N), torch.float32, other) if checkpoints else None
    wsb = _fn("rwkv_selective_scan_forward_workspace_bytes")(B, T, C, N, algo)
    ws = _workspace(x, wsb, other)
    _check("rwkv_selective_scan_forward",
           _fn("rwkv_selective_scan_forward")(B, T, C, N, code, *args, _addr(y), p_h_in, _addr(ho), _addr(ck),
                                              CHUNK_LEN, algo, _addr(ws), wsb, raw))
    if other is not None:
        other.done(x, dt, b, c, a_log, d, dt_bias, z, h_in, out)
    res = (y,)
    if return_state:
        res += (ho,)
    if checkpoints:
        res += (ck,)
    return res[0] if len(res) == 1 else res


def rwkv_selective_scan_backward(x, dt, b, c, a_log, gy, d=None, dt_bias=None, z=None, ckpt=None, h_in=None,
                                 gh_out=None, *, want_gh_in=False, stream=None):
    """Gradients of sum(gy * y) + sum(gh_out * h_out) of ``rwkv_selective_scan_forward``: returns
    (gx, gdt, gb, gc, ga_log, gd, gdt_bias, gz) and, with ``want_gh_in``, the gradient of h_in as
    well; gd, gdt_bias and gz are None where d, dt_bias and z are.  ``ckpt`` are the forward's
    checkpoints, or None to form them again (from ``h_in``)."""
    import torch

    (dev, raw, other), ty = _launch(x, stream), x.dtype
    code = _io_code("x", x)
    B, T, C = _dims("x", x, 3)
    N, args = _scan_args(x, dt, b, c, a_log, d, dt_bias, z, dev)
    f32 = torch.float32
    p_gy = _dense("gy", gy, (B, T, C), ty, dev)
    p_ckpt = _dense("ckpt", ckpt, ((T + CHUNK_LEN - 1) // CHUNK_LEN, B, C, N), f32, dev)
    p_h_in = _dense("h_in", h_in, (B, C, N), f32, dev)
    p_gh_out = _dense("gh_out", gh_out, (B, C, N), f32, dev)
    gx, gdt = _like(x, other), _like(x, other)
    gb, gc = _empty(x, (B, T, N), ty, other), _empty(x, (B, T, N), ty, other)
    gz = _like(x, other) if z is not None else None
    ga = _empty(x, (C, N), f32, other)
    gd = _empty(x, (C,), f32, other) if d is not None else None
    gbias = _empty(x, (C,), f32, other) if dt_bias is not None else None
    ghi = _empty(x, (B, C, N), f32, other) if want_gh_in else None
    wsb = _fn("rwkv_selective_scan_backward_workspace_bytes")(B, T, C, N, CHUNK_LEN, 1 if ckpt is not None else 0)
    ws = _workspace(x, wsb, other)
    _check("rwkv_selective_scan_backward",
           _fn("rwkv_selective_scan_backward")(B, T, C, N, code, *args, p_gy, p_h_in, p_gh_out,
                                               p_ckpt, CHUNK_LEN, _addr(gx), _addr(gdt), _addr(gb), _addr(gc),
                                               _addr(gz), _addr(ga), _addr(gd), _addr(gbias), _addr(ghi), _addr(ws),
                                               wsb, raw))
    if other is not None:
        other.done(x, dt, b, c, a_log, gy, d, dt_bias, z, ckpt, h_in, gh_out)
    res = (gx, gdt, gb, gc, ga, gd, gbias, gz)
    return res + (ghi,) if want_gh_in else res


def rwkv_selective_scan_step(x, dt, b, c, a_log, state, d=None, dt_bias=None, z=None, *, state_out=None, stream=None,
                             out=None):
    """One token for each of B streams: x, dt, z [B,C]; b, c [B,N]; state [B,C,N] fp32, updated in
    place unless ``state_out`` is given.  Returns y [B,C]."""
    import torch

    (dev, raw, other), ty = _launch(x, stream), x.dtype
    code = _io_code("x", x)
    B, C = _dims("x", x, 2)
    N, args = _scan_args(x, dt, b, c, a_log, d, dt_bias, z, dev)
    p_state = _dense("state", state, (B, C, N), torch.float32, dev)
    _dense("state_out", state_out, (B, C, N), torch.float32, dev)
    _dense("out", out, (B, C), ty, dev)
    y = _like(x, other) if out is None else out
    so = state if state_out is None else state_out
    _check("rwkv_selective_scan_step",
           _fn("rwkv_selective_scan_step")(B, C, N, code, *args, _addr(y), p_state, _addr(so), raw))
    if other is not None:
        other.done(x, dt, b, c, a_log, state, d, dt_bias, z, state_out, out)
    return y


def _norm_args(x, weight, bias, gate, groups, dev):
    """Checks what the norm's calls share; returns (M, N) for `groups` groups in x's last dimension."""
    import torch

    shape = x.shape
    if len(shape) == 0:
        raise ValueError("x must have at least one dimension")
    C = shape[-1]
    if groups < 1 or C % groups != 0:
        raise ValueError(f"groups must divide the last dimension {C}, got {groups}")
    _dense("x", x, shape, x.dtype, dev)
    _dense("weight", weight, (C,), torch.float32, dev)
    _dense("bias", bias, (C,), torch.float32, dev)
    _dense("gate", gate, shape, x.dtype, dev)
    return (x.numel() // C if C else 0), C // groups


def rwkv_layer_norm_forward(x, weight, bias=None, gate=None, *, groups=1, eps=1e-5, stream=None, out=None):
    """Layer norm over each of ``groups`` equal parts of x's last dimension [..., C]:
    (x - mean) / sqrt(var + eps) * weight + bias, times silu(gate) if a gate (like x) is given.
    x fp32 or bf16; weight, bias [C] fp32.  groups = H on an Eagle or Finch output [B,T,H*64] is
    the head-wise norm."""
    dev, raw, other = _launch(x, stream)
    code = _io_code("x", x)
    M, N = _norm_args(x, weight, bias, gate, groups, dev)
    _dense("out", out, x.shape, x.dtype, dev)
    y = _like(x, other) if out is None else out
    _check("rwkv_layer_norm_forward",
           _fn("rwkv_layer_norm_forward")(M, groups, N, code, _addr(weight), _addr(bias), eps, _addr(x), _addr(gate),
                                          _addr(y), raw))
    if other is not None:
        other.done(x, weight, bias, gate, out)
    return y


def rwkv_layer_norm_backward(x, weight, gy, bias=None, gate=None, *, groups=1, eps=1e-5, stream=None):
    """Gradients of sum(gy * y) of ``rwkv_layer_norm_forward``: returns (gx, gweight, gbias, ggate);
    gbias and ggate are None where bias and gate are."""
    import torch

    dev, raw, other = _launch(x, stream)
    code = _io_code("x", x)
    M, N = _norm_args(x, weight, bias, gate, groups, dev)
    p_gy = _dense("gy", gy, x.shape, x.dtype, dev)
    C = x.shape[-1]
    gx = _like(x, other)
    gw = _empty(x, (C,), torch.float32, other)
    gb = _empty(x, (C,), torch.float32, other) if bias is not None else None
    gg = _like(x, other) if gate is not None else None
    wsb = _fn("rwkv_layer_norm_backward_workspace_bytes")(M, groups, N, code)
    ws = _workspace(x, wsb, other)
    _check("rwkv_layer_norm_backward",
           _fn("rwkv_layer_norm_backward")(M, groups, N, code, _addr(weight), _addr(bias), eps, _addr(x), _addr(gate),
                                           p_gy, _addr(gx), _addr(gg), _addr(gw), _addr(gb), _addr(ws), wsb,
                                           raw))
    if other is not None:
        other.done(x, weight, gy, bias, gate)
    return gx, gw, gb, gg


def rwkv_check_device_error(stream=None):
    """Synchronise the stream and raise if a kernel's bounded wait timed out."""
    _check("rwkv_check_device_error", lib().rwkv_check_device_error(_stream(stream)))

