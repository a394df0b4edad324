"""GB300 (sm_103a) KDA mixer: Python binding of libk3kda.

The functions named ``k3kda_*`` are the C ABI of ``include/k3kda.h``, one for
one, taking torch CUDA tensors (or None) and marshalling their device pointers
and sizes; every step of the computation runs in the library's CUDA kernels.
PyTorch only provides device memory and the current stream.  A nonzero status
raises ``K3KDAError``.  If the CUDA library is missing and cannot be built,
importing the binding's functions raises: there is no CPU fallback.

Layouts (row-major, contiguous): q, k, g [T, H, dk]; v, gate, out [T, H, dv];
beta [T, H]; states [N, H, dk, dv] fp32; cu_seqlens int32 [N+1]; conv weights
[2*H*dk + H*dv, W] fp32; conv state [N, W-1, 2*H*dk + H*dv] fp32.

A call runs on the current stream, or on the one it is given.  Then what it allocates is that stream's
(outputs are kept for the current stream too), and the caller orders the two: the stream waits for the inputs,
the current stream for the outputs.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

__all__ = ["K3KDAError", "load_library", "library_path", "F32", "BF16", "L2_EPS",
           "k3kda_version", "k3kda_status_string", "k3kda_launch_count", "k3kda_short_conv",
           "k3kda_prefill_workspace_size", "k3kda_prefill_workspace_min", "k3kda_prefill", "k3kda_prefill_slots",
           "k3kda_decode_step_slots", "k3kda_prefill_noalloc", "k3kda_prefill_noalloc_status",
           "k3kda_decode_status", "k3kda_workspace_status",
           "k3kda_backward_workspace_size", "k3kda_backward", "backward",
           "k3kda_decode_step", "prefill", "decode_step", "short_conv",
           "k3mla_decode_workspace_size", "k3mla_decode_step", "k3mla_decode_step_slots", "mla_decode_step",
           "CACHE_BF16", "CACHE_I4", "RopeTable", "PagedCache", "rope_table", "rope", "rope_backward",
           "paged_pool", "paged_append", "paged_read", "paged_attend", "paged_attend_workspace",
           "k3mla_rope_table", "k3mla_rope", "k3mla_rope_backward", "k3mla_paged_block_bytes",
           "k3mla_paged_append", "k3mla_paged_read", "k3mla_paged_attend_workspace_size", "k3mla_paged_attend"]

F32, BF16 = 0, 1
CACHE_BF16, CACHE_I4 = 1, 2
L2_EPS = 1e-6
_STATUS = {0: "OK", -1: "INVALID_ARG", -2: "UNSUPPORTED", -3: "ALIGNMENT", -4: "WORKSPACE",
           -5: "CUDA", -6: "TIMEOUT"}

_lib = None
_lock = threading.Lock()


class K3KDAError(RuntimeError):
    def __init__(self, fn, status, detail=""):
        self.status = status
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)} ({status}) {detail}".rstrip())


def library_path() -> str:
    from . import build as _b
    return _b.LIB


def load_library(build_if_missing: bool = True):
    """Load libk3kda.so (building it with nvcc when missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        from . import build as _b
        if build_if_missing and not _b.up_to_date():
            _b.build()
        if not os.path.exists(_b.LIB):
            raise RuntimeError(f"libk3kda.so not found at {_b.LIB}; build it with "
                               "hybrid_linear_attention_rule_gb300.build.build()")
        lib = ctypes.CDLL(_b.LIB)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.k3kda_version.restype = I
        lib.k3kda_status_string.restype = ctypes.c_char_p
        lib.k3kda_status_string.argtypes = [I]
        lib.k3kda_last_error.restype = ctypes.c_char_p
        lib.k3kda_launch_count.restype = ctypes.c_longlong
        lib.k3kda_short_conv.argtypes = [P, I, P, P, P, I, I, I, I, I, P, I, P]
        lib.k3kda_short_conv.restype = I
        lib.k3kda_prefill_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
        lib.k3kda_prefill_workspace_size.restype = Z
        lib.k3kda_prefill_workspace_min.argtypes = [I, I, I, I, I, I, I, I]
        lib.k3kda_prefill_workspace_min.restype = Z
        lib.k3kda_prefill.argtypes = [P, P, P, I, P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P, I, P,
                                      P, Z, P]
        lib.k3kda_prefill.restype = I
        lib.k3kda_prefill_noalloc.argtypes = [P, P, P, I, P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P, I, P, P]
        lib.k3kda_prefill_noalloc.restype = I
        lib.k3kda_workspace_status.argtypes = [P, P]
        lib.k3kda_workspace_status.restype = I
        lib.k3kda_prefill_noalloc_status.argtypes = [P]
        lib.k3kda_prefill_noalloc_status.restype = I
        lib.k3kda_decode_status.argtypes = [P]
        lib.k3kda_decode_status.restype = I
        # internal test hook (not in the public header): see k3kda_test_arm_wait_timeout in api.cu
        lib.k3kda_test_arm_wait_timeout.argtypes = [I, ctypes.c_uint]
        lib.k3kda_test_arm_wait_timeout.restype = I
        lib.k3kda_decode_step.argtypes = [P, P, P, I, P, P, P, P, P, P, I, I, I, I, I, F, I, P, I, P]
        lib.k3kda_decode_step.restype = I
        lib.k3kda_prefill_slots.argtypes = [P, P, P, I, P, P, P, P, P, I, P, P, I, I, I, I, I, I, F, I, P, P,
                                            P, I, P, Z, P]
        lib.k3kda_prefill_slots.restype = I
        lib.k3kda_decode_step_slots.argtypes = [P, P, P, I, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, I,
                                                P]
        lib.k3kda_decode_step_slots.restype = I
        lib.k3kda_backward_workspace_size.argtypes = [I, I, I, I, I]
        lib.k3kda_backward_workspace_size.restype = ctypes.c_size_t
        lib.k3kda_backward.argtypes = [P, P, P, I, P, P, P, P, P, I, I, I, I, I, F, P, P, P, P, P, P, P, P, P,
                                       ctypes.c_size_t, P]
        lib.k3kda_backward.restype = I
        lib.k3mla_decode_workspace_size.argtypes = [I, I, I, I, I]
        lib.k3mla_decode_workspace_size.restype = Z
        lib.k3mla_decode_step.argtypes = [P, P, P, I, P, P, P, I, P, I, I, I, I, I, I, F, F, P, I, P, Z, P]
        lib.k3mla_decode_step.restype = I
        lib.k3mla_decode_step_slots.argtypes = [P, P, P, I, P, P, P, I, P, P, P, I, I, I, I, I, I, I, F, F, P, I, P,
                                                Z, P]
        lib.k3mla_decode_step_slots.restype = I
        D, R, V, C = ctypes.c_double, ctypes.POINTER(_RopeArgs), ctypes.POINTER(_View), ctypes.POINTER(_PagedArgs)
        lib.k3mla_rope_table.argtypes = [I, D, I, D, D, D, D, P, P]
        lib.k3mla_rope_table.restype = I
        lib.k3mla_rope.argtypes = [V, V, I, V, V, I, I, P, I, I, R, P]
        lib.k3mla_rope.restype = I
        lib.k3mla_rope_backward.argtypes = [V, V, I, V, V, I, I, I, P, I, I, R, P]
        lib.k3mla_rope_backward.restype = I
        lib.k3mla_paged_block_bytes.argtypes = [I, I, I, I]
        lib.k3mla_paged_block_bytes.restype = Z
        lib.k3mla_paged_append.argtypes = [C, V, V, I, P, P, I, R, P]
        lib.k3mla_paged_append.restype = I
        lib.k3mla_paged_read.argtypes = [C, V, V, I, P, P, I, P]
        lib.k3mla_paged_read.restype = I
        lib.k3mla_paged_attend_workspace_size.argtypes = [I, I, I, I]
        lib.k3mla_paged_attend_workspace_size.restype = Z
        lib.k3mla_paged_attend.argtypes = [C, V, I, I, P, P, I, I, R, F, V, P, I, P, Z, P]
        lib.k3mla_paged_attend.restype = I
        _lib = lib
        return lib


class _RopeArgs(ctypes.Structure):
    _fields_ = [("phase", ctypes.c_void_p), ("dim", ctypes.c_int), ("offset", ctypes.c_int), ("layout", ctypes.c_int),
                ("mscale", ctypes.c_float)]


class _View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


class _PagedArgs(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("block_table_host", ctypes.c_void_p), ("kv_len_host", ctypes.c_void_p), ("format", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("N", ctypes.c_int), ("heads", ctypes.c_int), ("dqk", ctypes.c_int), ("dv", ctypes.c_int)]


class _ConvArgs(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("conv_state", ctypes.c_void_p), ("W", ctypes.c_int)]


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_cuda:
        raise ValueError("k3kda: tensors must live on a CUDA device (no CPU path exists)")
    if not t.is_contiguous():
        raise ValueError("k3kda: tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"k3kda: unsupported element type {t.dtype}")


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """Where a call on `stream` allocates and fills what it needs: on that stream (None: the current one).  A block that the current
    stream's pool hands out may still be in use by that stream's pending kernels, which `stream` does not wait for."""
    return torch.cuda.stream(stream)


def _handed_out(stream, *tensors):
    """Outputs made on `stream` for the caller's current stream: their blocks are not handed out again before that has used them."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(torch.cuda.current_stream(t.device))


def _empty(shape, dtype, device, stream):
    """A call's output."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    _handed_out(stream, t)
    return t


def _check(fn, st):
    if st != 0:
        lib = load_library()
        raise K3KDAError(fn, st, lib.k3kda_last_error().decode() if st == -5 else "")


# ---- the C ABI, one for one ------------------------------------------------

def k3kda_version() -> int:
    return int(load_library().k3kda_version())


def k3kda_launch_count() -> int:
    return int(load_library().k3kda_launch_count())


def k3kda_status_string(status: int) -> str:
    return load_library().k3kda_status_string(int(status)).decode()


def k3kda_short_conv(x, weight, conv_state, cu_seqlens, N, T, D, W, apply_silu, out, stream=None):
    lib = load_library()
    st = lib.k3kda_short_conv(_ptr(x), _dtype(x), _ptr(weight), _ptr(conv_state), _ptr(cu_seqlens),
                              int(N), int(T), int(D), int(W), int(bool(apply_silu)), _ptr(out),
                              _dtype(out), _stream(stream))
    _check("k3kda_short_conv", st)


def k3kda_prefill_workspace_size(N, T, H, dk, dv, chunk, in_dtype, has_conv) -> int:
    return int(load_library().k3kda_prefill_workspace_size(int(N), int(T), int(H), int(dk), int(dv),
                                                           int(chunk), int(in_dtype), int(bool(has_conv))))


def k3kda_prefill_workspace_min(N, T, H, dk, dv, chunk, in_dtype, has_conv) -> int:
    return int(load_library().k3kda_prefill_workspace_min(int(N), int(T), int(H), int(dk), int(dv),
                                                          int(chunk), int(in_dtype), int(bool(has_conv))))


def k3kda_prefill(q, k, v, g, beta, initial_state, cu_seqlens, cu_seqlens_host, N, T, H, dk, dv, chunk,
                  scale, use_qk_l2norm, conv_weight, conv_state, conv_W, gate, out, final_state,
                  workspace, stream=None):
    """cu_seqlens_host: a CPU int32 tensor (or None), passed as the host copy."""
    lib = load_library()
    conv = None
    if conv_weight is not None:
        conv = ctypes.byref(_ConvArgs(_ptr(conv_weight), _ptr(conv_state), int(conv_W)))
    hcu = None
    if cu_seqlens_host is not None:
        if cu_seqlens_host.is_cuda or cu_seqlens_host.dtype != torch.int32 or not cu_seqlens_host.is_contiguous():
            raise ValueError("cu_seqlens_host must be a contiguous CPU int32 tensor")
        hcu = ctypes.c_void_p(cu_seqlens_host.data_ptr())
    st = lib.k3kda_prefill(_ptr(q), _ptr(k), _ptr(v), _dtype(q), _ptr(g), _ptr(beta), _ptr(initial_state),
                           _ptr(cu_seqlens), hcu, int(N), int(T), int(H), int(dk), int(dv), int(chunk),
                           float(scale), int(bool(use_qk_l2norm)), conv, _ptr(gate), _ptr(out), _dtype(out),
                           _ptr(final_state), _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream(stream))
    _check("k3kda_prefill", st)


def _host_i32(t, what):
    if t is None:
        return None
    if t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CPU int32 tensor")
    return ctypes.c_void_p(t.data_ptr())


def k3kda_prefill_slots(q, k, v, g, beta, state_pool, state_idx, state_idx_host, num_slots, cu_seqlens,
                        cu_seqlens_host, N, T, H, dk, dv, chunk, scale, use_qk_l2norm, conv_weight,
                        conv_state_pool, conv_W, gate, out, workspace, stream=None):
    """k3kda_prefill on slot-indexed state pools: sequence n reads and updates slot state_idx[n]."""
    lib = load_library()
    conv = None
    if conv_weight is not None:
        conv = ctypes.byref(_ConvArgs(_ptr(conv_weight), _ptr(conv_state_pool), int(conv_W)))
    st = lib.k3kda_prefill_slots(_ptr(q), _ptr(k), _ptr(v), _dtype(q), _ptr(g), _ptr(beta), _ptr(state_pool),
                                 _ptr(state_idx), _host_i32(state_idx_host, "state_idx_host"), int(num_slots),
                                 _ptr(cu_seqlens), _host_i32(cu_seqlens_host, "cu_seqlens_host"), int(N), int(T),
                                 int(H), int(dk), int(dv), int(chunk), float(scale), int(bool(use_qk_l2norm)), conv,
                                 _ptr(gate), _ptr(out), _dtype(out), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    _check("k3kda_prefill_slots", st)


def k3kda_decode_step_slots(q, k, v, g, beta, gate, conv_weight, conv_state_pool, state_pool, state_idx,
                            state_idx_host, num_slots, N, H, dk, dv, W, scale, use_qk_l2norm, out, stream=None):
    """k3kda_decode_step on slot-indexed state pools: sequence n reads and updates slot state_idx[n]."""
    lib = load_library()
    st = lib.k3kda_decode_step_slots(_ptr(q), _ptr(k), _ptr(v), _dtype(q), _ptr(g), _ptr(beta), _ptr(gate),
                                     _ptr(conv_weight), _ptr(conv_state_pool), _ptr(state_pool), _ptr(state_idx),
                                     _host_i32(state_idx_host, "state_idx_host"), int(num_slots), int(N), int(H),
                                     int(dk), int(dv), int(W), float(scale), int(bool(use_qk_l2norm)), _ptr(out),
                                     _dtype(out), _stream(stream))
    _check("k3kda_decode_step_slots", st)


def k3kda_backward_workspace_size(N, T, H, dk, dv):
    return int(load_library().k3kda_backward_workspace_size(int(N), int(T), int(H), int(dk), int(dv)))


def k3kda_backward(q, k, v, g, beta, initial_state, cu_seqlens, cu_seqlens_host, N, T, H, dk, dv, scale, dO,
                   dS_final, dq, dk_out, dv_out, dg, dbeta, dS0, workspace, stream=None):
    """Reverse-mode gradients of the ungated recurrence (see include/k3kda.h)."""
    lib = load_library()
    st = lib.k3kda_backward(_ptr(q), _ptr(k), _ptr(v), _dtype(q), _ptr(g), _ptr(beta), _ptr(initial_state),
                            _ptr(cu_seqlens), _host_i32(cu_seqlens_host, "cu_seqlens_host"), int(N), int(T), int(H),
                            int(dk), int(dv), float(scale), _ptr(dO), _ptr(dS_final), _ptr(dq), _ptr(dk_out),
                            _ptr(dv_out), _ptr(dg), _ptr(dbeta), _ptr(dS0), _ptr(workspace),
                            int(workspace.numel() * workspace.element_size()), _stream(stream))
    _check("k3kda_backward", st)


def backward(q, k, v, g, beta, dO, initial_state=None, dS_final=None, cu_seqlens=None, scale=None, stream=None):
    """Gradients (dict of fp32 tensors dq, dk, dv, dg, dbeta, dS0) of the ungated recurrence for the
    loss gradients dO [T, H, dv] (fp32) and dS_final [N, H, dk, dv] (optional); allocates its outputs
    and workspace with torch."""
    T, H, dk = q.shape
    dv = v.shape[-1]
    if cu_seqlens is None:
        cu_host = torch.tensor([0, T], dtype=torch.int32)
    else:
        cu_host = cu_seqlens.to("cpu", torch.int32)
    N = int(cu_host.numel()) - 1
    scale = float(dk) ** -0.5 if scale is None else float(scale)
    f32 = dict(dtype=torch.float32, device=q.device)
    with _on(stream):
        cu_dev = cu_host.to(q.device)
        out = dict(dq=torch.empty(T, H, dk, **f32), dk=torch.empty(T, H, dk, **f32), dv=torch.empty(T, H, dv, **f32),
                   dg=torch.empty(T, H, dk, **f32), dbeta=torch.empty(T, H, **f32), dS0=torch.empty(N, H, dk, dv, **f32))
        ws = torch.empty(k3kda_backward_workspace_size(N, T, H, dk, dv), dtype=torch.uint8, device=q.device)
    _handed_out(stream, *out.values())
    k3kda_backward(q, k, v, g, beta, initial_state, cu_dev, cu_host, N, T, H, dk, dv, scale, dO, dS_final,
                   out["dq"], out["dk"], out["dv"], out["dg"], out["dbeta"], out["dS0"], ws, stream)
    return out


def k3kda_prefill_noalloc(q, k, v, g, beta, initial_state, cu_seqlens, cu_seqlens_host, N, T, H, dk, dv,
                          chunk, scale, use_qk_l2norm, conv_weight, conv_state, conv_W, gate, out, final_state,
                          stream=None):
    """k3kda_prefill without a workspace: for callers that cannot allocate device memory where
    they run the mixer.  The scratch is a fixed 16 MiB array the library holds on each GPU; work
    that needs more raises K3KDAError (WORKSPACE).  The first call on a device sets up the array's
    address and should come before any stream capture; calls that overlap on the GPU race on it."""
    lib = load_library()
    conv = None
    if conv_weight is not None:
        conv = ctypes.byref(_ConvArgs(_ptr(conv_weight), _ptr(conv_state), int(conv_W)))
    hcu = None
    if cu_seqlens_host is not None:
        if cu_seqlens_host.is_cuda or cu_seqlens_host.dtype != torch.int32 or not cu_seqlens_host.is_contiguous():
            raise ValueError("cu_seqlens_host must be a contiguous CPU int32 tensor")
        hcu = ctypes.c_void_p(cu_seqlens_host.data_ptr())
    st = lib.k3kda_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _dtype(q), _ptr(g), _ptr(beta), _ptr(initial_state),
                                   _ptr(cu_seqlens), hcu, int(N), int(T), int(H), int(dk), int(dv), int(chunk),
                                   float(scale), int(bool(use_qk_l2norm)), conv, _ptr(gate), _ptr(out), _dtype(out),
                                   _ptr(final_state), _stream(stream))
    _check("k3kda_prefill_noalloc", st)


def k3kda_workspace_status(workspace, stream=None) -> int:
    return int(load_library().k3kda_workspace_status(_ptr(workspace), _stream(stream)))


def k3kda_prefill_noalloc_status(stream=None) -> int:
    return int(load_library().k3kda_prefill_noalloc_status(_stream(stream)))


def k3kda_decode_status(stream=None) -> int:
    return int(load_library().k3kda_decode_status(_stream(stream)))


def k3kda_decode_step(q, k, v, g, beta, gate, conv_weight, conv_state, state, N, H, dk, dv, W, scale,
                      use_qk_l2norm, out, stream=None):
    lib = load_library()
    st = lib.k3kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _dtype(q), _ptr(g), _ptr(beta), _ptr(gate),
                               _ptr(conv_weight), _ptr(conv_state), _ptr(state), int(N), int(H), int(dk),
                               int(dv), int(W), float(scale), int(bool(use_qk_l2norm)), _ptr(out),
                               _dtype(out), _stream(stream))
    _check("k3kda_decode_step", st)


# ---- conveniences: allocate outputs with torch, then call the ABI ----------

def prefill(q, k, v, g, beta, initial_state=None, cu_seqlens=None, chunk=64, scale=None,
            use_qk_l2norm=True, conv_weight=None, conv_state=None, gate=None, out_dtype=None,
            return_final_state=True, workspace=None, min_workspace=False, stream=None):
    """Allocate out / final_state / workspace and run k3kda_prefill.  cu_seqlens may be
    a CPU or CUDA int32 tensor (both copies are passed).  The workspace is the size of
    k3kda_prefill_workspace_size (the fastest path), or of k3kda_prefill_workspace_min
    with min_workspace=True.  Returns (out, final_state)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    dev = q.device
    if cu_seqlens is None:
        cu_h = torch.tensor([0, T], dtype=torch.int32)
    else:
        cu_h = cu_seqlens.to("cpu", torch.int32).contiguous()
    N = cu_h.numel() - 1
    W = 0 if conv_weight is None else conv_weight.shape[1]
    with _on(stream):
        cu_d = cu_h.to(dev)
        out = torch.empty((T, H, dv), dtype=out_dtype or q.dtype, device=dev)
        fs = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev) if return_final_state else None
        if workspace is None:
            size_fn = k3kda_prefill_workspace_min if min_workspace else k3kda_prefill_workspace_size
            nbytes = size_fn(N, T, H, dk, dv, chunk, _dtype(q), conv_weight is not None)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            workspace[:256].zero_()                 # the status word; the rest is written before it is read
    _handed_out(stream, out, fs)
    k3kda_prefill(q, k, v, g, beta, initial_state, cu_d, cu_h, N, T, H, dk, dv, chunk,
                  dk ** -0.5 if scale is None else scale, use_qk_l2norm, conv_weight, conv_state, W,
                  gate, out, fs, workspace, stream)
    return out, fs


def decode_step(q, k, v, g, beta, state, gate=None, conv_weight=None, conv_state=None, scale=None,
                use_qk_l2norm=True, out_dtype=None, stream=None):
    """Run k3kda_decode_step; state and conv_state are updated in place.  Returns out."""
    N, H, dk = q.shape
    dv = v.shape[2]
    out = _empty((N, H, dv), out_dtype or q.dtype, q.device, stream)
    W = 0 if conv_weight is None else conv_weight.shape[1]
    k3kda_decode_step(q, k, v, g, beta, gate, conv_weight, conv_state, state, N, H, dk, dv, W,
                      dk ** -0.5 if scale is None else scale, use_qk_l2norm, out, stream)
    return out


def short_conv(x, weight, conv_state=None, cu_seqlens=None, apply_silu=True, out_dtype=None, stream=None):
    """Run k3kda_short_conv over x [T, D]; conv_state is updated in place.  Returns out."""
    T, D = x.shape
    W = weight.shape[1]
    with _on(stream):
        cu = None if cu_seqlens is None else cu_seqlens.to(x.device, torch.int32)
    N = 1 if cu is None else cu.numel() - 1
    out = _empty((T, D), out_dtype or x.dtype, x.device, stream)
    k3kda_short_conv(x, weight, conv_state, cu, N, T, D, W, apply_silu, out, stream)
    return out


# ---- the gated attention (MLA) layers' decode token ------------------------

def k3mla_decode_workspace_size(N, H, dqk, dv, L_max) -> int:
    return int(load_library().k3mla_decode_workspace_size(int(N), int(H), int(dqk), int(dv), int(L_max)))


def k3mla_decode_step(q, k_new, v_new, gate, k_cache, v_cache, cache_len, N, H, dqk, dv, L_max, rope_dim, rope_theta,
                      scale, out, workspace, stream=None):
    """One decode token of the gated attention layers (see include/k3kda.h): RoPE, append, attention, gate."""
    lib = load_library()
    st = lib.k3mla_decode_step(_ptr(q), _ptr(k_new), _ptr(v_new), _dtype(q), _ptr(gate), _ptr(k_cache),
                               _ptr(v_cache), _dtype(k_cache), _ptr(cache_len), int(N), int(H), int(dqk), int(dv),
                               int(L_max),
                               int(rope_dim), float(rope_theta), float(scale), _ptr(out), _dtype(out),
                               _ptr(workspace), int(workspace.numel() * workspace.element_size()), _stream(stream))
    _check("k3mla_decode_step", st)


def k3mla_decode_step_slots(q, k_new, v_new, gate, k_cache_pool, v_cache_pool, cache_len_pool, cache_idx,
                            cache_idx_host, num_slots, N, H, dqk, dv, L_max, rope_dim, rope_theta, scale, out,
                            workspace, stream=None):
    """One decode token over a slot-indexed cache pool (see include/k3kda.h)."""
    lib = load_library()
    st = lib.k3mla_decode_step_slots(_ptr(q), _ptr(k_new), _ptr(v_new), _dtype(q), _ptr(gate), _ptr(k_cache_pool),
                                     _ptr(v_cache_pool), _dtype(k_cache_pool), _ptr(cache_len_pool), _ptr(cache_idx),
                                     _host_i32(cache_idx_host, "cache_idx_host"), int(num_slots), int(N), int(H),
                                     int(dqk), int(dv), int(L_max), int(rope_dim), float(rope_theta), float(scale),
                                     _ptr(out), _dtype(out), _ptr(workspace),
                                     int(workspace.numel() * workspace.element_size()), _stream(stream))
    _check("k3mla_decode_step_slots", st)


def mla_decode_step(q, k_new, v_new, k_cache, v_cache, cache_len, gate=None, scale=None, rope_dim=0,
                    rope_theta=10000.0, out_dtype=None, workspace=None, stream=None):
    """Decode one token for every sequence: q, k_new [N, H, dqk], v_new [N, H, dv]; caches
    [N, H, L_max, dqk | dv] and cache_len int32 [N] are updated in place.  Returns the output
    [N, H, dv] (allocated with torch, in out_dtype, default q's type)."""
    N, H, dqk = q.shape
    dv = v_new.shape[-1]
    L_max = k_cache.shape[2]
    scale = float(dqk) ** -0.5 if scale is None else float(scale)
    out = _empty((N, H, dv), out_dtype or q.dtype, q.device, stream)
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(k3mla_decode_workspace_size(N, H, dqk, dv, L_max), dtype=torch.uint8, device=q.device)
    k3mla_decode_step(q, k_new, v_new, gate, k_cache, v_cache, cache_len, N, H, dqk, dv, L_max, rope_dim, rope_theta,
                      scale, out, workspace, stream)
    return out


# ---- rotary positions and the paged cache ----------------------------------

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}
_FORMATS = {"bf16": CACHE_BF16, "i4": CACHE_I4}


# These calls are short on the GPU, so their marshalling is kept short too: few tensor attributes, the raw stream, argument
# structures that the handles keep.

def _raw_stream(stream, t):
    """The stream's address; by default the current one of the tensor's device."""
    return torch._C._cuda_getCurrentRawStream(t.device.index) if stream is None else stream.cuda_stream


def _view(t, what, d=None):
    """A [tokens, heads, channels] CUDA tensor of any token and head strides, its channels contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"k3mla: {what} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("k3mla: tensors must live on a CUDA device (no CPU path exists)")
    st = t.stride()
    if len(st) != 3 or (st[2] != 1 and t.shape[2] > 1):
        raise ValueError(f"k3mla: {what} must be [tokens, heads, channels] with contiguous channels")
    if d is not None and t.shape[2] != d:
        raise ValueError(f"k3mla: {what} has {t.shape[2]} channels, not {d}")
    return _View(t.data_ptr(), st[0], st[1])


def _i32(t, what, shape):
    """A contiguous int32 CUDA tensor of the given shape, or None; its address."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"k3mla: {what} must be a contiguous int32 CUDA tensor of shape {tuple(shape)}")
    return t.data_ptr()


class RopeTable:
    """The rotation's table: phases [dim/2] on the device (kept alive here), the rotated channels
    [offset, offset + dim), their pair layout ("half" or "interleaved") and the factor mscale."""

    def __init__(self, phase, dim, offset, layout, mscale):
        self.phase, self.dim, self.offset, self.layout, self.mscale = phase, dim, offset, layout, mscale
        self._args = _RopeArgs(phase.data_ptr(), dim, offset, _named(_LAYOUTS, layout, "layout"), mscale)

    def __setattr__(self, name, value):
        if hasattr(self, "_args"):
            raise AttributeError("k3mla: a RopeTable is fixed; make another")
        super().__setattr__(name, value)


def _named(names, key, what):
    try:
        return names[key]
    except KeyError:
        raise ValueError(f"k3mla: {what} is one of {sorted(names)}, not {key!r}") from None


def k3mla_rope_table(dim, theta, scaling="none", factor=1.0, original_length=0.0, beta_fast=32.0, beta_slow=1.0):
    """(phases as a CPU int64 tensor of the 64-bit patterns, mscale); see include/k3kda.h."""
    lib = load_library()
    phase = torch.zeros(max(int(dim) // 2, 1), dtype=torch.int64)
    mscale = ctypes.c_float(1.0)
    st = lib.k3mla_rope_table(int(dim), float(theta), _named(_SCALINGS, scaling, "scaling"), float(factor), float(original_length),
                              float(beta_fast), float(beta_slow), phase.data_ptr(), ctypes.byref(mscale))
    _check("k3mla_rope_table", st)
    return phase, mscale.value


def rope_table(dim, theta=10000.0, offset=0, layout="half", scaling="none", factor=1.0, original_length=0.0,
               beta_fast=32.0, beta_slow=1.0, device="cuda") -> RopeTable:
    """A rotation table for `dim` channels from `offset` on; scaling is "none", "linear", "ntk" or "by_parts"."""
    phase, mscale = k3mla_rope_table(dim, theta, scaling, factor, original_length, beta_fast, beta_slow)
    return RopeTable(phase.to(device), int(dim), int(offset), layout, mscale)


def _dense(shape, dtype, device, stream):
    """A new [tokens, heads, channels] output and its view (nothing about it needs a check)."""
    t = _empty(shape, dtype, device, stream)
    return t, _View(t.data_ptr(), shape[1] * shape[2], shape[2])


def _rope_call(name, q, qo, k, ko, positions, table, stream, *shared):
    """The library's call on inputs q, k and the outputs' views qo, ko."""
    T, hq, d = q.shape
    dt = _dtype(q)
    kv, hk = None, 0
    if k is not None:
        tk, hk, dk = k.shape
        if tk != T or dk != d or k.dtype != q.dtype:
            raise ValueError("k3mla: the two inputs differ in tokens, channels or type")
        kv = _view(k, "k")
    qv = _view(q, "q")
    st = getattr(_lib or load_library(), name)(qv, qo, hq, kv, ko, hk, *shared, dt, _i32(positions, "positions", (T,)), T, d,
                                               table._args, _raw_stream(stream, q))
    if st:
        _check(name, st)


def _rope_checked(name, q, q_out, k, k_out, k_heads_out, positions, table, stream, *shared):
    """The same with outputs that the caller gave."""
    if q_out.shape != q.shape or q_out.dtype != q.dtype:
        raise ValueError("k3mla: the first output has another shape or type than its input")
    if k is not None and (k_out.shape != (k.shape[0], k.shape[1] if k_heads_out is None else k_heads_out, k.shape[2]) or k_out.dtype != k.dtype):
        raise ValueError("k3mla: the second output has the wrong shape or type")
    _rope_call(name, q, _view(q_out, "q_out"), k, None if k is None else _view(k_out, "k_out"), positions, table, stream, *shared)


def k3mla_rope(q, q_out, k, k_out, positions, table, stream=None):
    """Rotate q [T, Hq, d] -> q_out and k [T, Hk, d] -> k_out (None: no k); an output may be its input."""
    _rope_checked("k3mla_rope", q, q_out, k, k_out, None, positions, table, stream)


def k3mla_rope_backward(dq_out, dq, dk_out, dk, k_shared, positions, table, stream=None):
    """The gradient of k3mla_rope; k_shared: k was one head for all, dk [T, 1, d] is the sum over heads."""
    _rope_checked("k3mla_rope_backward", dq_out, dq, dk_out, dk, 1 if k_shared else None, positions, table, stream,
                  1 if k_shared else 0)


def rope(q, positions, table, k=None, out=None, stream=None):
    """q [T, Hq, d] (and k [T, Hk, d]) turned by positions int32 [T].  Returns q's rotation, or (q's, k's);
    `out` (a tensor, or a pair with k) may be the inputs themselves.  Inputs may be strided views."""
    if out is None:
        dev, dt = q.device, q.dtype
        qo, qv = _dense(q.shape, dt, dev, stream)
        if k is None:
            _rope_call("k3mla_rope", q, qv, None, None, positions, table, stream)
            return qo
        ko, kv = _dense(k.shape, dt, dev, stream)
        _rope_call("k3mla_rope", q, qv, k, kv, positions, table, stream)
        return qo, ko
    qo, ko = (out, None) if k is None else out
    k3mla_rope(q, qo, k, ko, positions, table, stream)
    return out


def rope_backward(dq_out, positions, table, dk_out=None, k_shared=False, stream=None):
    """Gradients of rope's inputs: dq, or (dq, dk); with k_shared dk is [T, 1, d], the sum over heads."""
    dev, dt = dq_out.device, dq_out.dtype
    dq, qv = _dense(dq_out.shape, dt, dev, stream)
    if dk_out is None:
        _rope_call("k3mla_rope_backward", dq_out, qv, None, None, positions, table, stream, 0)
        return dq
    T, H, d = dk_out.shape
    dk, kv = _dense((T, 1 if k_shared else H, d), dt, dev, stream)
    _rope_call("k3mla_rope_backward", dq_out, qv, dk_out, kv, positions, table, stream, 1 if k_shared else 0)
    return dq, dk


def k3mla_paged_block_bytes(fmt, page_size, dqk, dv) -> int:
    return int(load_library().k3mla_paged_block_bytes(_FORMATS.get(fmt, fmt), int(page_size), int(dqk), int(dv)))


def paged_pool(num_pages, page_size, heads, dqk, dv, fmt="i4", device="cuda"):
    """An empty pool: uint8 [num_pages, heads, block bytes]."""
    n = k3mla_paged_block_bytes(fmt, page_size, dqk, dv)
    if n == 0:
        raise K3KDAError("k3mla_paged_block_bytes", -2)
    return torch.zeros((num_pages, heads, n), dtype=torch.uint8, device=device)


class PagedCache:
    """A paged key/value cache as the calls take it: pool uint8 [num_pages, heads, block bytes], block_table
    int32 [N, max_pages] and kv_len int32 [N] (lengths with the call's new tokens) on the device.  The tensors stay
    the caller's: write to them in place (kv_len.add_(1)) between calls.  block_table_host and
    kv_len_host: optional CPU copies that every call then checks."""

    def __init__(self, pool, block_table, kv_len, page_size, dqk, dv, fmt="i4", block_table_host=None, kv_len_host=None):
        if pool.dim() != 3 or pool.dtype != torch.uint8 or not pool.is_contiguous() or not pool.is_cuda:
            raise ValueError("k3mla: pool must be a contiguous uint8 CUDA tensor [num_pages, heads, block bytes]")
        block = k3mla_paged_block_bytes(fmt, page_size, dqk, dv)
        if block == 0:
            raise K3KDAError("k3mla_paged_block_bytes", -2, f"(format {fmt}, page_size {page_size}, dqk {dqk}, dv {dv})")
        if pool.shape[2] != block:
            raise ValueError(f"k3mla: a block has {block} bytes, the pool's have {pool.shape[2]}")
        N, width = block_table.shape
        tab, lens = _i32(block_table, "block_table", (N, width)), _i32(kv_len, "kv_len", (N,))
        if tuple(getattr(block_table_host, "shape", (N, width))) != (N, width) or tuple(getattr(kv_len_host, "shape", (N,))) != (N,):
            raise ValueError("k3mla: a host copy has another shape")
        self.pool, self.block_table, self.kv_len = pool, block_table, kv_len
        self.block_table_host, self.kv_len_host = block_table_host, kv_len_host
        self.N, self.heads, self.page_size, self.dqk, self.dv, self.fmt = N, pool.shape[1], page_size, dqk, dv, fmt
        self._args = _PagedArgs(pool.data_ptr(), tab, lens, _host_i32(block_table_host, "block_table_host"),
                                _host_i32(kv_len_host, "kv_len_host"), _FORMATS.get(fmt, fmt), pool.shape[0], page_size, width, N,
                                pool.shape[1], dqk, dv)

    def __setattr__(self, name, value):
        # the calls take the addresses that were given first
        if hasattr(self, "_args"):
            raise AttributeError("k3mla: a PagedCache's tensors are fixed; write to them in place, or make another")
        super().__setattr__(name, value)


def _packing(cache, cu_seqlens, cu_seqlens_host):
    if cu_seqlens_host is not None and cu_seqlens_host.numel() != cache.N + 1:
        raise ValueError("k3mla: cu_seqlens_host has another length")
    return (None if cu_seqlens is None else _i32(cu_seqlens, "cu_seqlens", (cache.N + 1,)),
            None if cu_seqlens_host is None else _host_i32(cu_seqlens_host, "cu_seqlens_host"))


def k3mla_paged_append(cache, k_new, v_new, cu_seqlens=None, cu_seqlens_host=None, rope=None, stream=None):
    """Append rows k_new [T, heads, dqk], v_new [T, heads, dv] (see include/k3kda.h); rope: a RopeTable or None."""
    T = k_new.shape[0]
    if v_new.shape[0] != T or k_new.shape[1] != cache.heads or v_new.shape[1] != cache.heads or k_new.dtype != v_new.dtype:
        raise ValueError("k3mla: k_new and v_new differ, or have other heads than the cache")
    cu, cuh = _packing(cache, cu_seqlens, cu_seqlens_host)
    st = (_lib or load_library()).k3mla_paged_append(
        cache._args, _view(k_new, "k_new", cache.dqk), _view(v_new, "v_new", cache.dv), _dtype(k_new), cu, cuh, T,
        None if rope is None else rope._args, _raw_stream(stream, k_new))
    if st:
        _check("k3mla_paged_append", st)


def k3mla_paged_read(cache, k_out, v_out, cu_seqlens=None, cu_seqlens_host=None, stream=None):
    """The last tokens' rows as values to k_out [T, heads, dqk] and v_out [T, heads, dv] (either may be None)."""
    some = k_out if k_out is not None else v_out
    if some is None or (k_out is not None and v_out is not None and (k_out.shape[:2] != v_out.shape[:2] or k_out.dtype != v_out.dtype)):
        raise ValueError("k3mla: k_out and v_out differ, or both are None")
    if some.shape[1] != cache.heads:
        raise ValueError("k3mla: the outputs have other heads than the cache")
    cu, cuh = _packing(cache, cu_seqlens, cu_seqlens_host)
    st = (_lib or load_library()).k3mla_paged_read(
        cache._args, None if k_out is None else _view(k_out, "k_out", cache.dqk),
        None if v_out is None else _view(v_out, "v_out", cache.dv), _dtype(some), cu, cuh, some.shape[0], _raw_stream(stream, some))
    if st:
        _check("k3mla_paged_read", st)


paged_append = k3mla_paged_append


def paged_read(cache, tokens, cu_seqlens=None, out_dtype=torch.bfloat16, stream=None):
    """The last `tokens` packed rows (all sequences together) as values: (k [tokens, heads, dqk], v [tokens, heads, dv])."""
    dev, heads = cache.pool.device, cache.heads
    k, kv = _dense((tokens, heads, cache.dqk), out_dtype, dev, stream)
    v, vv = _dense((tokens, heads, cache.dv), out_dtype, dev, stream)
    cu, _ = _packing(cache, cu_seqlens, None)
    st = (_lib or load_library()).k3mla_paged_read(cache._args, kv, vv, _dtype(k), cu, None, tokens, _raw_stream(stream, k))
    if st:
        _check("k3mla_paged_read", st)
    return k, v


def k3mla_paged_attend_workspace_size(Hq, heads, dqk, dv) -> int:
    return int(load_library().k3mla_paged_attend_workspace_size(int(Hq), int(heads), int(dqk), int(dv)))


def paged_attend_workspace(cache, Hq):
    """A zero-filled workspace for k3mla_paged_attend on this cache, for one call at a time; any later call may reuse it."""
    n = k3mla_paged_attend_workspace_size(Hq, cache.heads, cache.dqk, cache.dv)
    return torch.zeros(n, dtype=torch.uint8, device=cache.pool.device)


def k3mla_paged_attend(cache, q, gate, out, workspace, scale, cu_seqlens=None, cu_seqlens_host=None, max_new=1, rope=None,
                       stream=None):
    """Attention of the new tokens q [T, Hq, dqk] over the cache (see include/k3kda.h)."""
    T, Hq = q.shape[:2]
    want = (T, Hq, cache.dv)
    if gate is not None and (gate.shape != want or gate.dtype != q.dtype):
        raise ValueError("k3mla: gate is not [tokens, query heads, dv] of q's type")
    if out.shape != want:
        raise ValueError("k3mla: out is not [tokens, query heads, dv]")
    cu, cuh = _packing(cache, cu_seqlens, cu_seqlens_host)
    st = (_lib or load_library()).k3mla_paged_attend(
        cache._args, _view(q, "q", cache.dqk), _dtype(q), Hq, cu, cuh, T, int(max_new), None if rope is None else rope._args,
        scale, None if gate is None else _view(gate, "gate"), _ptr(out), _dtype(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _raw_stream(stream, q))
    if st:
        _check("k3mla_paged_attend", st)


def paged_attend(cache, q, cu_seqlens=None, max_new=None, rope=None, scale=None, gate=None, out=None, out_dtype=None,
                 workspace=None, stream=None):
    """Attention of the T packed new tokens q [T, Hq, dqk] over the cache, which holds them already (append first).
    max_new: the most new tokens of a sequence; it chooses the kernel, so a wrong one costs time only (default: 1 without
    cu_seqlens or with no more tokens than sequences, else T).  scale defaults to dqk^-1/2.  Returns out [T, Hq, dv].
    Without a workspace one is made for the call, and its status word (k3kda_workspace_status) goes with it."""
    if out is None:
        out = _empty((q.shape[0], q.shape[1], cache.dv), out_dtype or q.dtype, q.device, stream)
    if workspace is None:
        if stream is not None:                          # (without a workspace the call has always waited for the current stream)
            stream.wait_stream(torch.cuda.current_stream())
        with _on(stream):
            workspace = paged_attend_workspace(cache, q.shape[1])
    if max_new is None:
        max_new = 1 if cu_seqlens is None or q.shape[0] <= cache.N else q.shape[0]
    k3mla_paged_attend(cache, q, gate, out, workspace, cache.dqk ** -0.5 if scale is None else float(scale), cu_seqlens, None, max_new,
                       rope, stream)
    return out
