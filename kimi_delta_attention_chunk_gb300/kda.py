"""Thin ctypes binding of libkda.so (C ABI in include/kda.h).

Marshalling only: every function checks that the tensors live on the current
CUDA device, picks the dtype codes, and forwards raw device pointers, sizes and
the current CUDA stream to the library.  All arithmetic runs in the library's
kernels; there is no CPU or PyTorch fallback, and a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libkda.so"
_lock = threading.Lock()
_lib = None

KDA_F32, KDA_BF16 = 0, 1
_STATUS = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED", 3: "KDA_ERR_WORKSPACE",
           4: "KDA_ERR_CUDA", 5: "KDA_ERR_RANGE", 6: "KDA_ERR_TIMEOUT"}

# (name, restype, argtypes) of every exported symbol of include/kda.h
_vp, _fp, _i32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
_i, _f, _sz, _u32, _i64 = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_int64
SIGNATURES = {
    "kda_status_string": (ctypes.c_char_p, [_i]),
    "kda_abi_version": (_i, []),
    "kda_chunk_fwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "kda_chunk_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _f, _fp, _i32p, _i, _i, _i, _i, _i, _i,
                           _vp, _i, _fp, _vp, _sz, _i32p, _vp]),
    "kda_chunk_fwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _f, _fp, _i32p, _i, _i, _i, _i, _i,
                                   _i, _vp, _i, _fp, _vp]),
    "kda_chunk_fwd_fused": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _fp, _fp, _fp, _i, _fp, _fp, _f, _f,
                                 _f, _fp, _i32p, _i, _i, _i, _i, _i, _i, _vp, _i, _fp, _vp, _sz, _i32p,
                                 _vp]),
    "kda_trace_events": (None, [_vp, _vp, _vp]),
    "kda_set_wait_limit": (None, [_u32]),
    "kda_inject_wait_timeout": (None, [_i]),
    "kda_recurrent_step": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _f, _fp, _i, _i, _i, _i, _vp, _i,
                                _vp]),
    "kda_output_gate": (_i, [_fp, _vp, _i, _fp, _f, _i, _i, _i, _i, _vp, _i, _vp]),
    "kda_gate_proj_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "kda_gate_proj": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _i32p, _vp]),
    "kda_state_compose": (_i, [_fp, _fp, _fp, _fp, _i, _i, _i, _vp]),
    "kda_check_range": (_i, [_vp, _i, ctypes.c_int64, _f, _f, _vp, _vp]),
    "kda_recurrent_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "kda_chunk_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "kda_chunk_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _f, _fp, _i32p, _i, _i, _i, _i, _i, _i,
                           _fp, _fp, _fp, _fp, _fp, _fp, _fp, _fp, _vp, _sz, _i32p, _vp]),
    "kda_recurrent_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _f, _fp, _i32p, _i, _i, _i, _i, _i, _i,
                               _fp, _fp, _fp, _fp, _fp, _fp, _fp, _fp, _vp, _sz, _i32p, _vp]),
    "kda_recurrent_step_slots": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _f, _fp, _i32p, _i, _i, _i, _i, _i, _vp, _i,
                                      _i32p, _vp]),
    "kda_short_conv_fwd": (_i, [_vp, _i64, _fp, _fp, _i, _i, _vp, _i32p, _i, _i, _i, _i, _i, _vp, _vp, _vp]),
    "kda_short_conv_bwd_workspace_size": (_sz, [_i, _i, _i, _i]),
    "kda_short_conv_bwd": (_i, [_vp, _i64, _fp, _fp, _i, _i, _vp, _i32p, _i, _i, _i, _i, _i, _vp, _vp, _i, _vp, _fp,
                                _fp, _vp, _vp, _sz, _vp]),
    "kda_short_conv_step": (_i, [_vp, _i64, _fp, _fp, _i, _i, _vp, _i32p, _i, _i, _i, _i, _vp, _i32p, _vp]),
    "kda_ssm_step": (_i, [_vp, _i64, _vp, _i64, _fp, _vp, _i64, _vp, _i64, _fp, _vp, _i64, _fp, _i, _i, _fp, _i32p,
                          _i, _i, _i, _i, _i, _vp, _i32p, _vp]),
    "kda_ssm_scan_fwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "kda_ssm_scan_fwd": (_i, [_vp, _i64, _vp, _i64, _fp, _vp, _i64, _vp, _i64, _fp, _vp, _i64, _fp, _i, _i, _fp,
                              _i32p, _i, _i, _i, _i, _i, _i, _vp, _fp, _vp, _sz, _vp]),
    "kda_ssm_scan_bwd_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "kda_ssm_scan_bwd": (_i, [_vp, _i64, _vp, _i64, _fp, _vp, _i64, _vp, _i64, _fp, _vp, _i64, _fp, _i, _i, _fp,
                              _i32p, _i, _i, _i, _i, _i, _i, _vp, _fp, _i, _vp, _vp, _fp, _vp, _vp, _fp, _vp, _fp,
                              _fp, _vp, _sz, _vp]),
    "kda_pages_alloc": (_i, [_i32p, _i, _i, _i32p, _i32p, _vp]),
    "kda_pages_free": (_i, [_i32p, _i, _i32p, _i64, _i32p, _vp]),
    "kda_pages_fork": (_i, [_i32p, _i32p, _i, _i, _i, _i32p, _i, _i32p, _i32p, _i, _i32p, _i32p, _i32p, _vp]),
    "kda_pages_compact_workspace_size": (_sz, [_i]),
    "kda_pages_compact": (_i, [_i32p, _i, _i32p, _i64, _i32p, _i32p, _vp, _sz, _i32p, _vp]),
    "kda_pages_copy_workspace_size": (_sz, [_i, _i]),
    "kda_pages_copy": (_i, [_vp, _i, _i64, _i32p, _i32p, _i, _vp, _sz, _i32p, _vp]),
}


class KDAError(RuntimeError):
    """A libkda.so call returned a non-OK status."""

    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {_STATUS.get(status, status)}")
        self.status = status


def library_path() -> str:
    return os.environ.get("KDA_LIBRARY", os.path.join(_PKG, _LIB_NAME))


def load_library():
    """Load libkda.so (built by ``build.py``); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise ImportError(f"{path} is missing: build it with "
                                  "`python -m kimi_delta_attention_chunk_gb300.build`")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libkda must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libkda must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(fn: str, status: int):
    if status != 0:
        raise KDAError(fn, status)


def _dt_of(dtype) -> int:
    if dtype == torch.bfloat16:
        return KDA_BF16
    if dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {dtype}")


def _here(*tensors) -> int:
    """Every tensor given lies on one CUDA device, the current one; returns its index."""
    dev = -1
    for t in tensors:
        if t is None:
            continue
        i = t.get_device()
        if i < 0:
            raise ValueError("tensors passed to libkda must be CUDA tensors")
        if i != dev:
            if i != torch.cuda.current_device():
                raise ValueError(f"a tensor lies on {t.device}, the current device is {torch.cuda.current_device()}")
            dev = i
    return dev


def _at(t):
    """Address of a contiguous tensor that _here has looked at, None for none."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libkda must be contiguous")
    return t.data_ptr()


def _stream_of(dev: int) -> int:
    # the raw handle: a torch.cuda.Stream object a call would cost as much as a small kernel
    return torch._C._cuda_getCurrentRawStream(dev)


def _int32(*tensors):
    for t in tensors:
        if t is not None and t.dtype is not torch.int32:
            raise TypeError(f"expected an int32 tensor, got {t.dtype}")


def _ints(*sizes):
    """Sizes that the library takes as 32-bit integers (ctypes would drop their upper bits)."""
    if max(sizes) >= 1 << 31:
        raise ValueError(f"sizes must stay below 2**31, got {max(sizes)}")


def _f32(*tensors):
    for t in tensors:
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"expected a float32 tensor, got {t.dtype}")


def _like(ref, *tensors):
    """Every tensor given has ref's element type."""
    for t in tensors:
        if t is not None and t.dtype != ref.dtype:
            raise TypeError(f"expected {ref.dtype}, got {t.dtype}")


def _shape(name, t, shape):
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(name, t, lead: int):
    """(pointer, row stride in elements) of a tensor whose first ``lead`` dimensions number
    rows a fixed stride apart, each row's elements lying side by side."""
    if t is None:
        return None, 0
    shape, stride = t.shape, t.stride()
    if lead == 1:  # the single-token calls: [rows, width], or [rows, groups, width]
        width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
        if stride[-1] == 1 and (len(shape) == 2 or shape[1] == 1 or stride[1] == shape[2]):
            if shape[0] < 2:
                return t.data_ptr(), width
            if stride[0] >= width:
                return t.data_ptr(), stride[0]
    width = 1
    if t.is_contiguous():
        for d in shape[lead:]:
            width *= d
        return t.data_ptr(), width
    for d in reversed(range(lead, t.dim())):
        if t.shape[d] != 1 and t.stride(d) != width:
            raise ValueError(f"{name}: the elements of a row must lie side by side")
        width *= t.shape[d]
    ld, rows = None, 1
    for d in reversed(range(lead)):
        if t.shape[d] != 1 and t.numel():
            if ld is None:
                ld = t.stride(d)
            elif t.stride(d) != ld * rows:
                raise ValueError(f"{name}: rows must lie a fixed stride apart")
            rows *= t.shape[d]
    ld = width if ld is None else ld
    if ld < width:
        raise ValueError(f"{name}: rows must not overlap")
    return t.data_ptr(), ld


def workspace_size(in_dtype, B: int, T: int, H: int, K: int, V: int, N: int, packed: bool) -> int:
    """Device workspace bytes ``kda_chunk_fwd`` / ``kda_chunk_fwd_fused`` need."""
    return int(load_library().kda_chunk_fwd_workspace_size(_dt_of(in_dtype), B, T, H, K, V, N, int(packed)))


def bwd_workspace_size(in_dtype, B: int, T: int, H: int, K: int, V: int, N: int, packed: bool,
                       token_by_token: bool = False) -> int:
    """Device workspace bytes ``kda_chunk_bwd`` (or, with ``token_by_token``,
    ``kda_recurrent_bwd``) needs."""
    lib = load_library()
    fn = lib.kda_recurrent_bwd_workspace_size if token_by_token else lib.kda_chunk_bwd_workspace_size
    return int(fn(_dt_of(in_dtype), B, T, H, K, V, N, int(packed)))


def _workspace(nbytes: int, device, workspace):
    """The caller's workspace tensor (checked), or a fresh uint8 one of nbytes."""
    if workspace is None:
        if nbytes == 0:
            return None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, "
                         f"the call needs {nbytes}")
    return workspace, workspace.numel() * workspace.element_size()


def set_wait_limit(iterations: int = 0):
    """Testing hook: polls before a bounded device-side wait of the tensor-core
    prefill gives up (0 restores the default)."""
    load_library().kda_set_wait_limit(int(iterations))


def inject_wait_timeout(kernel: int):
    """Testing hook: the next tensor-core prefill or chunked backward call on this
    thread makes the first wait of its chunk-local (1), state (2), backward chain
    (3) or backward chunk (4) kernel one that nothing completes, so that it gives
    up and reports KDA_ERR_TIMEOUT."""
    load_library().kda_inject_wait_timeout(int(kernel))


def chunk_fwd(q, k, v, g, beta, scale: float | None = None, initial_state=None, cu_seqlens=None,
              output_final_state: bool = True, o_dtype=torch.float32, o=None, final_state=None,
              workspace=None, status=None):
    """Chunked KDA prefill.  q, k, g: [B,T,H,K]; v: [B,T,H,V]; beta: [B,T,H].

    Returns (o [B,T,H,V] in ``o_dtype``, final_state [N,H,K,V] fp32 or None).
    ``cu_seqlens`` (int32 [N+1], on the device) packs N sequences into B == 1.
    ``final_state`` may be the ``initial_state`` tensor itself (in-place update).
    ``workspace``: a device tensor of at least :func:`workspace_size` bytes (a
    fresh one from torch's allocator when None).  ``status``: an optional device
    int32 tensor that receives the call's device-side status (0, or 6 =
    KDA_ERR_TIMEOUT when a bounded wait gave up); read it after the stream work.
    """
    lib = load_library()
    B, T, H, K = q.shape
    V = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if o is None:
        o = torch.empty((B, T, H, V), dtype=o_dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
    ws, ws_bytes = _workspace(workspace_size(q.dtype, B, T, H, K, V, N, cu_seqlens is not None), q.device,
                              workspace)
    st = lib.kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q),
                           float(scale or 0.0), _ptr(initial_state), _ptr(cu_seqlens),
                           B, T, H, K, V, N, _ptr(o), _dt(o), _ptr(final_state), _ptr(ws), ws_bytes,
                           _ptr(status), _stream(q.device))
    _check("kda_chunk_fwd", st)
    return o, final_state


def chunk_fwd_noalloc(q, k, v, g, beta, scale: float | None = None, initial_state=None, cu_seqlens=None,
                      output_final_state: bool = True, o_dtype=torch.float32, o=None, final_state=None):
    """``chunk_fwd`` through ``kda_chunk_fwd_noalloc``: the library allocates no
    device memory for the call (its workspace is a fixed 64 MiB array, so only
    small calls fit; bf16 inputs with K = V = 128 only).  For callers whose
    device memory is all reserved by their own allocator.  ``o`` and
    ``final_state`` can be passed in so that nothing at all is allocated."""
    lib = load_library()
    B, T, H, K = q.shape
    V = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if o is None:
        o = torch.empty((B, T, H, V), dtype=o_dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
    st = lib.kda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q),
                                   float(scale or 0.0), _ptr(initial_state), _ptr(cu_seqlens),
                                   B, T, H, K, V, N, _ptr(o), _dt(o), _ptr(final_state), _stream(q.device))
    _check("kda_chunk_fwd_noalloc", st)
    return o, final_state


def chunk_fwd_fused(q_raw, k_raw, v_raw, gate_x, beta, conv_w, A_log, dt_bias,
                    scale: float | None = None, initial_state=None, cu_seqlens=None,
                    lower_bound: float = -5.0, l2_eps: float = 1e-6, conv_act: int = 0,
                    output_final_state: bool = True, o_dtype=torch.float32, o=None,
                    final_state=None, workspace=None, status=None):
    """Chunked prefill with the fused prologue (short conv, L2-norm, gate).

    conv_w: a sequence (conv_q [H*K,4], conv_k [H*K,4], conv_v [H*V,4]) of fp32
    tensors, or one [3, H*D, 4] tensor whose leading rows are used.  ``workspace``
    and ``status`` as for :func:`chunk_fwd`.
    """
    lib = load_library()
    B, T, H, K = q_raw.shape
    V = v_raw.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if isinstance(conv_w, torch.Tensor):
        cq = conv_w[0, : H * K].contiguous()
        ck = conv_w[1, : H * K].contiguous()
        cv = conv_w[2, : H * V].contiguous()
    else:
        cq, ck, cv = (w.contiguous() for w in conv_w)
    if o is None:
        o = torch.empty((B, T, H, V), dtype=o_dtype, device=q_raw.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, K, V), dtype=torch.float32, device=q_raw.device)
    ws, ws_bytes = _workspace(workspace_size(q_raw.dtype, B, T, H, K, V, N, cu_seqlens is not None),
                              q_raw.device, workspace)
    st = lib.kda_chunk_fwd_fused(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(gate_x), _ptr(beta),
                                 _dt(q_raw), _ptr(cq), _ptr(ck), _ptr(cv), int(conv_act), _ptr(A_log),
                                 _ptr(dt_bias), float(lower_bound), float(l2_eps), float(scale or 0.0),
                                 _ptr(initial_state), _ptr(cu_seqlens), B, T, H, K, V, N, _ptr(o),
                                 _dt(o), _ptr(final_state), _ptr(ws), ws_bytes, _ptr(status),
                                 _stream(q_raw.device))
    _check("kda_chunk_fwd_fused", st)
    return o, final_state


def trace_events(begin=None, split=None, end=None):
    """Have the next prefill call on this thread record these torch.cuda.Event
    objects on its stream: before its first kernel, after the chunk-local
    kernel, after its last kernel (tensor-core path only)."""
    lib = load_library()
    h = []
    for e in (begin, split, end):
        if e is None:
            h.append(None)
        else:
            if not e.cuda_event:  # torch creates the CUDA event on first record
                e.record()
            h.append(e.cuda_event)
    lib.kda_trace_events(*h)


def recurrent_step(q, k, v, g, beta, state, scale: float | None = None, o_dtype=torch.float32, o=None,
                   slots=None, status=None):
    """One decode token per sequence; ``state`` [N,H,K,V] fp32 is updated in place.

    q, k, g: [N,H,K]; v: [N,H,V]; beta: [N,H].  Returns o [N,H,V].  With ``slots``
    (device int32 [N]) ``state`` is a pool [P,H,K,V] and row i works on page
    ``slots[i]`` (-1: a padded row; its row of o is left as it is, so pass ``o`` to
    keep its contents); at most 2**18 rows.  ``status``: an optional device int32 word,
    5 = KDA_ERR_RANGE when a row's slot was out of range or an earlier row's.
    """
    lib = load_library()
    N, H, K = q.shape
    V = v.shape[-1]
    if o is None:
        o = torch.empty((N, H, V), dtype=o_dtype, device=q.device)
    if slots is not None:
        dev = _here(q, k, v, g, beta, state, o, slots, status)
        _check_slots(slots, status, N)
        dt = q.dtype
        if k.dtype is not dt or v.dtype is not dt or g.dtype is not dt or beta.dtype is not dt:
            raise TypeError(f"k, v, g and beta must be of q's type, {dt}")
        if state.dtype is not torch.float32:
            raise TypeError("state must be float32")
        if k.shape != (N, H, K) or g.shape != (N, H, K) or v.shape != (N, H, V) or beta.shape != (N, H) or o.shape != (N, H, V):
            raise ValueError(f"k and g must be [{N}, {H}, {K}], v and o [{N}, {H}, {V}], beta [{N}, {H}]")
        if state.shape[1:] != (H, K, V):
            raise ValueError(f"state must be [P, {H}, {K}, {V}]")
        _ints(state.shape[0], N, H)
        st = lib.kda_recurrent_step_slots(_at(q), _at(k), _at(v), _at(g), _at(beta), _dt(q), float(scale or 0.0),
                                          _at(state), _at(slots), state.shape[0], N, H, K, V, _at(o), _dt(o),
                                          _at(status), _stream_of(dev))
        _check("kda_recurrent_step_slots", st)
        return o
    if status is not None:
        raise ValueError("status goes with slots")
    st = lib.kda_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q),
                                float(scale or 0.0), _ptr(state), N, H, K, V, _ptr(o), _dt(o),
                                _stream(q.device))
    _check("kda_recurrent_step", st)
    return o


def output_gate(o, gate, weight=None, eps: float = 1e-6, out_dtype=torch.float32, out=None):
    """The layer's output gate, ``o / sqrt(mean(o^2) + eps) * weight * sigmoid(gate)``
    per (token, head) row of V values.

    o: [B,T,H,V] or [N,H,V] fp32; gate: same shape (bf16 or fp32); weight: [V] fp32
    or None.  ``out`` may be ``o`` itself for an fp32 result.  Returns out.
    """
    lib = load_library()
    if o.dim() == 3:
        (B, T), (H, V) = (1, o.shape[0]), o.shape[1:]
    else:
        B, T, H, V = o.shape
    if tuple(gate.shape) != tuple(o.shape):
        raise ValueError(f"gate has shape {tuple(gate.shape)}, expected {tuple(o.shape)}")
    if out is None:
        out = torch.empty(o.shape, dtype=out_dtype, device=o.device)
    st = lib.kda_output_gate(_ptr(o), _ptr(gate), _dt(gate), _ptr(weight), float(eps), B, T, H, V,
                             _ptr(out), _dt(out), _stream(o.device))
    _check("kda_output_gate", st)
    return out


def gate_proj_workspace_size(B: int, T: int, D: int, R: int, NH: int) -> int:
    """Device workspace bytes ``kda_gate_proj`` needs (the split partial sums and
    y = f_a x between its kernels)."""
    return int(load_library().kda_gate_proj_workspace_size(B, T, D, R, NH))


def gate_proj(x, f_a, f_b, b_proj, gate_x=None, beta=None, workspace=None, status=None):
    """The projections ahead of the gate: ``gate_x = f_b (f_a x)`` and
    ``beta = sigmoid(b_proj x)`` per token, bf16 in and out.

    x: [B,T,D] (or [T,D]); f_a [R,D]; f_b [HK,R]; b_proj [NH,D].  Returns
    (gate_x [B,T,HK], beta [B,T,NH]), the shapes ``chunk_fwd_fused`` takes as
    [B,T,H,K] and [B,T,H].  ``workspace``/``status`` as for :func:`chunk_fwd`.
    """
    lib = load_library()
    xs = x if x.dim() == 3 else x.unsqueeze(0)
    B, T, D = xs.shape
    R, HK, NH = f_a.shape[0], f_b.shape[0], b_proj.shape[0]
    if tuple(f_a.shape) != (R, D) or tuple(f_b.shape) != (HK, R) or tuple(b_proj.shape) != (NH, D):
        raise ValueError("f_a must be [R, D], f_b [HK, R] and b_proj [NH, D]")
    for t in (f_a, f_b, b_proj):
        if t.dtype != x.dtype:
            raise TypeError("x, f_a, f_b and b_proj must share one dtype")
    if gate_x is None:
        gate_x = torch.empty((B, T, HK), dtype=x.dtype, device=x.device)
    if beta is None:
        beta = torch.empty((B, T, NH), dtype=x.dtype, device=x.device)
    ws, ws_bytes = _workspace(gate_proj_workspace_size(B, T, D, R, NH), x.device, workspace)
    st = lib.kda_gate_proj(_ptr(xs), _ptr(f_a), _ptr(f_b), _ptr(b_proj), _dt(x), B, T, D, R, HK, NH,
                           _ptr(gate_x), _ptr(beta), _ptr(ws), ws_bytes, _ptr(status), _stream(x.device))
    _check("kda_gate_proj", st)
    return gate_x, beta


def state_compose(M, S, A=None, out=None):
    """out[h] = M[h] @ S[h] + A[h] for every head: M [..., H, K, K], S and A
    [..., H, K, V] fp32 (leading dims flattened into heads).  ``out`` may be A."""
    lib = load_library()
    K, V = S.shape[-2:]
    H = S.numel() // (K * V)
    if M.shape[-2:] != (K, K) or M.numel() != H * K * K:
        raise ValueError(f"M has shape {tuple(M.shape)}")
    if out is None:
        out = torch.empty_like(S)
    st = lib.kda_state_compose(_ptr(M), _ptr(S), _ptr(A), _ptr(out), H, K, V, _stream(S.device))
    _check("kda_state_compose", st)
    return out


def check_range(x, lo: float = -5.0, hi: float = 0.0, status=None, sync: bool = True):
    """Debug range check on the device (default: the log-decay precondition
    g in [-5, 0]).  With ``sync`` the stream is synchronised and KDAError
    (KDA_ERR_RANGE) is raised for an element outside [lo, hi] or NaN; without it
    the device status word (int32 tensor, 0 or 5) is returned for the caller to
    read later."""
    lib = load_library()
    if status is None:
        status = torch.empty(1, dtype=torch.int32, device=x.device)
    st = lib.kda_check_range(_ptr(x), _dt(x), x.numel(), float(lo), float(hi), _ptr(status),
                             _stream(x.device))
    _check("kda_check_range", st)
    if sync:
        code = int(status.item())
        _check("kda_check_range", code)
    return status


def chunk_bwd(q, k, v, g, beta, dO, dS_T=None, scale: float | None = None, initial_state=None,
              cu_seqlens=None, workspace=None, status=None, token_by_token: bool = False):
    """Gradients of <dO, o> + <dS_T, S_T> through :func:`chunk_fwd` (same shapes;
    dO fp32 [B,T,H,V], dS_T fp32 [N,H,K,V] or None).  Returns a dict of fp32
    tensors dq, dk, dv, dg, dbeta and dS0 ([N,H,K,V]).  ``workspace`` (at least
    :func:`bwd_workspace_size` bytes) and ``status`` as for :func:`chunk_fwd`
    (the status word reads 5 = KDA_ERR_RANGE when malformed offsets made the
    token-by-token path skip a sequence).  ``kda_chunk_bwd`` runs by default
    (chunk by chunk for bf16 with K = V = 128); ``token_by_token`` calls
    ``kda_recurrent_bwd``."""
    lib = load_library()
    B, T, H, K = q.shape
    V = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    dev = q.device
    f32 = torch.float32
    out = {"dq": torch.empty((B, T, H, K), dtype=f32, device=dev),
           "dk": torch.empty((B, T, H, K), dtype=f32, device=dev),
           "dv": torch.empty((B, T, H, V), dtype=f32, device=dev),
           "dg": torch.empty((B, T, H, K), dtype=f32, device=dev),
           "dbeta": torch.empty((B, T, H), dtype=f32, device=dev),
           "dS0": torch.empty((N, H, K, V), dtype=f32, device=dev)}
    ws, ws_bytes = _workspace(bwd_workspace_size(q.dtype, B, T, H, K, V, N, cu_seqlens is not None,
                                                 token_by_token), dev, workspace)
    name = "kda_recurrent_bwd" if token_by_token else "kda_chunk_bwd"
    st = getattr(lib, name)(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), float(scale or 0.0),
                            _ptr(initial_state), _ptr(cu_seqlens), B, T, H, K, V, N, _ptr(dO), _ptr(dS_T),
                            _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                            _ptr(out["dbeta"]), _ptr(out["dS0"]), _ptr(ws), ws_bytes, _ptr(status),
                            _stream(dev))
    _check(name, st)
    return out


def _check_slots(slots, status, N):
    if slots is not None and (slots.dtype is not torch.int32 or slots.shape != (N,)):
        raise TypeError(f"slots must be int32 [{N}]")
    if status is not None and status.dtype is not torch.int32:
        raise TypeError("status must be int32")


def _conv_check(x, weight, bias, conv_act):
    C, W = weight.shape
    _f32(weight, bias)
    if x.shape[-1] != C:
        raise ValueError(f"x has {x.shape[-1]} channels, expected {C}")
    _shape("bias", bias, (C,))
    if conv_act not in (0, 1):
        raise ValueError("conv_act is 0 (none) or 1 (SiLU)")
    return C, W


def _sequences(t, cu_seqlens):
    """N of a [B, T, ...] tensor with or without packed sequences."""
    if cu_seqlens is None:
        return t.shape[0]
    _int32(cu_seqlens)
    if t.shape[0] != 1:
        raise ValueError("packed sequences need B == 1")
    return cu_seqlens.numel() - 1


def short_conv_fwd(x, weight, bias=None, conv_act: int = 0, initial=None, cu_seqlens=None,
                   output_final: bool = True, y=None, final=None):
    """The short causal convolution as a call of its own: ``y_t = act(bias + sum_j
    weight[:, j] * line_{t-(W-1)+j})`` per sequence, line = [history | inputs].

    x: [B,T,C] (bf16 or fp32; rows may be slices of wider ones); weight: [C,W] fp32, W in
    2..4; bias: [C] fp32 or None; conv_act: 0 none, 1 SiLU; initial: [N,W-1,C] the last
    inputs before each sequence, oldest first (None: zeros); ``cu_seqlens`` as for
    :func:`chunk_fwd`.  Returns (y [B,T,C], final history [N,W-1,C] or None).  Rows that
    belong to no sequence are left as they are.
    """
    lib = _lib if _lib is not None else load_library()
    C, W = _conv_check(x, weight, bias, conv_act)
    B, T, _ = x.shape
    N = _sequences(x, cu_seqlens)
    _ints(B, T, C, W, N)
    dev = _here(x, weight, bias, initial, cu_seqlens, y, final)
    _like(x, initial, y, final)
    _shape("initial", initial, (N, W - 1, C))
    _shape("y", y, (B, T, C))
    _shape("final", final, (N, W - 1, C))
    if y is None:
        y = torch.empty((B, T, C), dtype=x.dtype, device=x.device)
    if final is None and output_final:
        final = torch.empty((N, W - 1, C), dtype=x.dtype, device=x.device)
    px, ldx = _rows("x", x, 2)
    st = lib.kda_short_conv_fwd(px, ldx, _at(weight), _at(bias), conv_act, _dt(x), _at(initial), _at(cu_seqlens),
                                B, T, C, W, N, _at(y), _at(final), _stream_of(dev))
    _check("kda_short_conv_fwd", st)
    return y, final


def short_conv_bwd(x, weight, dy, bias=None, conv_act: int = 0, initial=None, cu_seqlens=None, dfinal=None,
                   workspace=None):
    """Gradients of <dy, y> + <dfinal, final> through :func:`short_conv_fwd` (same
    arguments).  dy [B,T,C] and dfinal [N,W-1,C] share a type: x's, or fp32.  Returns a
    dict: dx [B,T,C] and dinitial [N,W-1,C] (None without ``initial``) in dy's type, dweight
    [C,W] and dbias [C] (None without ``bias``) fp32.  Rows that belong to no sequence have
    zeros in dx."""
    lib = _lib if _lib is not None else load_library()
    C, W = _conv_check(x, weight, bias, conv_act)
    B, T, _ = x.shape
    N = _sequences(x, cu_seqlens)
    _ints(B, T, C, W, N)
    dev = _here(x, weight, dy, bias, initial, cu_seqlens, dfinal, workspace)
    _like(x, initial)
    _like(dy, dfinal)
    _shape("dy", dy, (B, T, C))
    _shape("initial", initial, (N, W - 1, C))
    _shape("dfinal", dfinal, (N, W - 1, C))
    on = x.device
    out = {"dx": torch.empty((B, T, C), dtype=dy.dtype, device=on),
           "dweight": torch.empty((C, W), dtype=torch.float32, device=on),
           "dbias": torch.empty(C, dtype=torch.float32, device=on) if bias is not None else None,
           "dinitial": torch.empty((N, W - 1, C), dtype=dy.dtype, device=on) if initial is not None else None}
    ws, ws_bytes = _workspace(int(lib.kda_short_conv_bwd_workspace_size(B, T, C, W)), on, workspace)
    px, ldx = _rows("x", x, 2)
    st = lib.kda_short_conv_bwd(px, ldx, _at(weight), _at(bias), conv_act, _dt(x), _at(initial), _at(cu_seqlens),
                                B, T, C, W, N, _at(dy), _at(dfinal), _dt(dy), _at(out["dx"]), _at(out["dweight"]),
                                _at(out["dbias"]), _at(out["dinitial"]), _at(ws), ws_bytes, _stream_of(dev))
    _check("kda_short_conv_bwd", st)
    return out


def short_conv_step(x, history, weight, bias=None, conv_act: int = 0, slots=None, y=None, status=None):
    """One token of each of N sequences: x [N,C]; ``history`` [P,W-1,C] is updated in place
    (row i's page is ``slots[i]``, or i without slots; -1 is a padded row).  Returns y
    [N,C].  ``slots``/``status`` as for :func:`recurrent_step`."""
    lib = _lib if _lib is not None else load_library()
    C, W = _conv_check(x, weight, bias, conv_act)
    if x.dim() != 2:
        raise ValueError(f"x must be [N, {C}], got {tuple(x.shape)}")
    N = x.shape[0]
    P = history.shape[0]
    _ints(N, P, C, W)
    dev = _here(x, history, weight, bias, slots, y, status)
    if history.dtype is not x.dtype or history.shape != (P, W - 1, C):
        raise ValueError(f"history must be [P, {W - 1}, {C}] of {x.dtype}")
    if y is None:
        y = torch.empty((N, C), dtype=x.dtype, device=x.device)
    elif y.dtype is not x.dtype or y.shape != (N, C):
        raise ValueError(f"y must be {(N, C)} of {x.dtype}")
    _check_slots(slots, status, N)
    px, ldx = _rows("x", x, 1)
    st = lib.kda_short_conv_step(px, ldx, _at(weight), _at(bias), conv_act, _dt(x), _at(history), _at(slots), P, N, C, W, _at(y),
                                 _at(status), _stream_of(dev))
    _check("kda_short_conv_step", st)
    return y


def _ssm_check(u, delta, A, Bm, Cm, D, z, delta_bias):
    """(C, G, S) of a scan call whose u is [..., C] and Bm, Cm [..., G, S]."""
    C, S = A.shape
    rows, vecs, dt = u.shape, Bm.shape, u.dtype
    if rows[-1] != C or delta.shape != rows or (z is not None and z.shape != rows):
        raise ValueError(f"u, delta and z must be [..., {C}] alike")
    if vecs[-1] != S or vecs[:-2] != rows[:-1] or Cm.shape != vecs:
        raise ValueError(f"Bm and Cm must be {tuple(rows[:-1])} + [G, {S}] alike")
    if delta.dtype is not dt or Bm.dtype is not dt or Cm.dtype is not dt or (z is not None and z.dtype is not dt):
        raise TypeError(f"delta, Bm, Cm and z must be of u's type, {dt}")
    for v in (D, delta_bias):
        if v is not None and (v.dtype is not torch.float32 or v.shape != (C,)):
            raise TypeError(f"D and delta_bias must be float32 [{C}]")
    if A.dtype is not torch.float32:
        raise TypeError("A must be float32")
    return C, vecs[-2], S


def ssm_step(u, delta, A, Bm, Cm, state, D=None, z=None, delta_bias=None, softplus: bool = True, slots=None,
             y=None, status=None):
    """One token of each of N sequences through a selective state space layer: ``h <-
    exp(d A) h + d u B``, ``y = (C . h + D u) * silu(z)`` with ``d = softplus(delta +
    delta_bias)``.

    u, delta, z: [N,C]; A: [C,S] fp32, S in 8, 16, 32, 64; Bm, Cm: [N,G,S], channel c in
    group c // (C // G); D, delta_bias: [C] fp32; ``state`` fp32 [P,C,S] is updated in place.
    Returns y [N,C].  ``slots``/``status`` as for :func:`recurrent_step`."""
    lib = _lib if _lib is not None else load_library()
    C, G, S = _ssm_check(u, delta, A, Bm, Cm, D, z, delta_bias)
    if u.dim() != 2:
        raise ValueError(f"u must be [N, {C}], got {tuple(u.shape)}")
    N = u.shape[0]
    P = state.shape[0]
    _ints(N, P, C, G, S)
    dev = _here(u, delta, A, Bm, Cm, state, D, z, delta_bias, slots, y, status)
    if y is None:
        y = torch.empty((N, C), dtype=u.dtype, device=u.device)
    elif y.dtype is not u.dtype or y.shape != (N, C):
        raise ValueError(f"y must be {(N, C)} of {u.dtype}")
    if state.dtype is not torch.float32 or state.shape != (P, C, S):
        raise ValueError(f"state must be fp32 [P, {C}, {S}]")
    _check_slots(slots, status, N)
    (pu, ldu), (pd, ldd), (pz, ldz) = _rows("u", u, 1), _rows("delta", delta, 1), _rows("z", z, 1)
    (pb, ldb), (pc, ldc) = _rows("Bm", Bm, 1), _rows("Cm", Cm, 1)
    st = lib.kda_ssm_step(pu, ldu, pd, ldd, _at(A), pb, ldb, pc, ldc, _at(D), pz, ldz, _at(delta_bias), int(softplus),
                          KDA_BF16 if u.dtype is torch.bfloat16 else _dt(u), _at(state), _at(slots), P, N, C, G, S, _at(y),
                          _at(status), _stream_of(dev))
    _check("kda_ssm_step", st)
    return y


def _ssm_pointers(u, delta, A, Bm, Cm, D, z, delta_bias, softplus):
    (pu, ldu), (pd, ldd), (pz, ldz) = _rows("u", u, 2), _rows("delta", delta, 2), _rows("z", z, 2)
    (pb, ldb), (pc, ldc) = _rows("Bm", Bm, 2), _rows("Cm", Cm, 2)
    return pu, ldu, pd, ldd, _at(A), pb, ldb, pc, ldc, _at(D), pz, ldz, _at(delta_bias), int(softplus), _dt(u)


def ssm_scan_fwd(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, softplus: bool = True, initial_state=None,
                 cu_seqlens=None, output_final_state: bool = True, y=None, final_state=None, workspace=None):
    """:func:`ssm_step`'s recurrence over prompts.

    u, delta, z: [B,T,C] (bf16 or fp32; rows may be slices of wider ones); A: [C,S] fp32, S
    in 8, 16, 32, 64; Bm, Cm: [B,T,G,S]; D, delta_bias: [C] fp32 or None; ``initial_state``
    fp32 [N,C,S] (None: zeros); ``cu_seqlens`` as for :func:`chunk_fwd`.  Returns (y
    [B,T,C], final_state [N,C,S] fp32 or None).  Rows that belong to no sequence are left
    as they are."""
    lib = _lib if _lib is not None else load_library()
    C, G, S = _ssm_check(u, delta, A, Bm, Cm, D, z, delta_bias)
    B, T, _ = u.shape
    N = _sequences(u, cu_seqlens)
    _ints(B, T, C, G, S, N)
    dev = _here(u, delta, A, Bm, Cm, D, z, delta_bias, initial_state, cu_seqlens, y, final_state, workspace)
    _like(u, y)
    _f32(initial_state, final_state)
    _shape("initial_state", initial_state, (N, C, S))
    _shape("final_state", final_state, (N, C, S))
    _shape("y", y, (B, T, C))
    if y is None:
        y = torch.empty((B, T, C), dtype=u.dtype, device=u.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, C, S), dtype=torch.float32, device=u.device)
    ws, ws_bytes = _workspace(int(lib.kda_ssm_scan_fwd_workspace_size(B, T, C, G, S, N, int(cu_seqlens is not None))),
                              u.device, workspace)
    st = lib.kda_ssm_scan_fwd(*_ssm_pointers(u, delta, A, Bm, Cm, D, z, delta_bias, softplus), _at(initial_state),
                              _at(cu_seqlens), B, T, C, G, S, N, _at(y), _at(final_state), _at(ws), ws_bytes,
                              _stream_of(dev))
    _check("kda_ssm_scan_fwd", st)
    return y, final_state


def ssm_scan_bwd(u, delta, A, Bm, Cm, dy, D=None, z=None, delta_bias=None, softplus: bool = True,
                 initial_state=None, cu_seqlens=None, dfinal_state=None, workspace=None):
    """Gradients of <dy, y> + <dfinal_state, final_state> through :func:`ssm_scan_fwd` (same
    arguments).  dy [B,T,C] is of u's type or fp32.  Returns a dict: du, ddelta, dz [B,T,C]
    and dB, dC [B,T,G,S] in dy's type, dA [C,S], dD, ddelta_bias [C] and dinitial_state
    [N,C,S] fp32; the gradient of an argument that was not given is None.  Rows that belong
    to no sequence have zeros."""
    lib = _lib if _lib is not None else load_library()
    C, G, S = _ssm_check(u, delta, A, Bm, Cm, D, z, delta_bias)
    B, T, _ = u.shape
    N = _sequences(u, cu_seqlens)
    _ints(B, T, C, G, S, N)
    dev = _here(u, delta, A, Bm, Cm, dy, D, z, delta_bias, initial_state, cu_seqlens, dfinal_state, workspace)
    _f32(initial_state, dfinal_state)
    _shape("dy", dy, (B, T, C))
    _shape("initial_state", initial_state, (N, C, S))
    _shape("dfinal_state", dfinal_state, (N, C, S))
    rows, vecs = (B, T, C), (B, T, G, S)
    like, f32 = dy.new_empty, A.new_empty  # of the gradients' type, and fp32
    out = {"du": like(rows), "ddelta": like(rows), "dA": f32((C, S)), "dB": like(vecs), "dC": like(vecs),
           "dD": f32(C) if D is not None else None, "dz": like(rows) if z is not None else None,
           "ddelta_bias": f32(C) if delta_bias is not None else None,
           "dinitial_state": f32((N, C, S)) if initial_state is not None else None}
    ws, ws_bytes = _workspace(int(lib.kda_ssm_scan_bwd_workspace_size(B, T, C, G, S, N, int(cu_seqlens is not None))),
                              u.device, workspace)
    st = lib.kda_ssm_scan_bwd(*_ssm_pointers(u, delta, A, Bm, Cm, D, z, delta_bias, softplus), _at(initial_state),
                              _at(cu_seqlens), B, T, C, G, S, N, _at(dy), _at(dfinal_state), _dt(dy),
                              *(_at(out[k]) for k in ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias",
                                                       "dinitial_state")),
                              _at(ws), ws_bytes, _stream_of(dev))
    _check("kda_ssm_scan_bwd", st)
    return out


def pages_alloc(refs, n: int, pages=None, status=None):
    """Take ``n`` free pages, the lowest first: their numbers, int32 [n], -1 where there are
    no more; ``refs`` [P] (references of each page, 0: free) is updated.  ``status`` of
    every pages call: an optional device int32 word, 5 = KDA_ERR_RANGE when a request
    was refused (a refused request changes nothing)."""
    lib = _lib if _lib is not None else load_library()
    _ints(refs.numel(), n)
    dev = _here(refs, pages, status)
    _int32(refs, pages, status)
    _shape("pages", pages, (n,))
    if pages is None:
        pages = torch.empty(n, dtype=torch.int32, device=refs.device)
    _check("kda_pages_alloc", lib.kda_pages_alloc(_at(refs), refs.numel(), n, _at(pages), _at(status), _stream_of(dev)))
    return pages


def pages_free(refs, pages, status=None):
    """Give back one reference of each page listed in ``pages`` (int32, any shape; -1 entries
    are skipped)."""
    lib = _lib if _lib is not None else load_library()
    _ints(refs.numel())
    dev = _here(refs, pages, status)
    _int32(refs, pages, status)
    _check("kda_pages_free", lib.kda_pages_free(_at(refs), refs.numel(), _at(pages), pages.numel(), _at(status),
                                                _stream_of(dev)))


def pages_fork(tables, lens, refs, parents, children, page_tokens: int, status=None):
    """Sequence ``children[k]`` becomes a copy of ``parents[k]`` in the books: it shares the
    parent's full pages, and a last page that is not full is to be copied.  tables: int32
    [S,width] (-1 behind a sequence's pages); lens: int32 [S] tokens.  Returns (src, dst),
    int32 [n]: the copies to make in every pool with :func:`pages_copy` (-1: none).  Free
    the child's former pages first."""
    lib = _lib if _lib is not None else load_library()
    n = parents.numel()
    S, width = tables.shape
    _ints(S, width, page_tokens, refs.numel(), n)
    dev = _here(tables, lens, refs, parents, children, status)
    _int32(tables, lens, refs, parents, children, status)
    _shape("lens", lens, (S,))
    _shape("children", children, parents.shape)
    src = torch.empty(n, dtype=torch.int32, device=refs.device)
    dst = torch.empty(n, dtype=torch.int32, device=refs.device)
    st = lib.kda_pages_fork(_at(tables), _at(lens), S, width, int(page_tokens), _at(refs), refs.numel(), _at(parents),
                            _at(children), n, _at(src), _at(dst), _at(status), _stream_of(dev))
    _check("kda_pages_fork", st)
    return src, dst


def pages_compact(refs, tables=None, workspace=None, status=None):
    """Close up the pools: used pages behind the number of used pages move into the free
    places before it, in order; ``refs`` and the table entries follow (an entry that names a
    free page stays as it is and is reported).  Returns (src, dst), int32 [P // 2]: the
    copies to make in every pool with :func:`pages_copy` (-1: none)."""
    lib = _lib if _lib is not None else load_library()
    P = refs.numel()
    _ints(P)
    dev = _here(refs, tables, workspace, status)
    _int32(refs, tables, status)
    src = torch.empty(P // 2, dtype=torch.int32, device=refs.device)
    dst = torch.empty(P // 2, dtype=torch.int32, device=refs.device)
    ws, ws_bytes = _workspace(int(lib.kda_pages_compact_workspace_size(P)), refs.device, workspace)
    st = lib.kda_pages_compact(_at(refs), P, _at(tables), 0 if tables is None else tables.numel(), _at(src), _at(dst),
                               _at(ws), ws_bytes, _at(status), _stream_of(dev))
    _check("kda_pages_compact", st)
    return src, dst


def pages_copy(pool, src, dst, workspace=None, status=None):
    """Copy page ``src[i]`` of ``pool`` ([P, ...], any type, a page's bytes a multiple of 16)
    onto page ``dst[i]``; -1 entries are skipped.  A destination that a later pair writes or
    another pair reads is refused."""
    lib = _lib if _lib is not None else load_library()
    P, n = pool.shape[0], src.numel()
    _ints(P, n)
    dev = _here(pool, src, dst, workspace, status)
    _int32(src, dst, status)
    _shape("dst", dst, src.shape)
    page_bytes = pool.numel() // P * pool.element_size() if P else 16
    ws, ws_bytes = _workspace(int(lib.kda_pages_copy_workspace_size(P, n)), pool.device, workspace)
    st = lib.kda_pages_copy(_at(pool), P, page_bytes, _at(src), _at(dst), n, _at(ws), ws_bytes, _at(status),
                            _stream_of(dev))
    _check("kda_pages_copy", st)
