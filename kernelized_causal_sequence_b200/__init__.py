"""Python binding of liblinattn.so — B200 (sm_100a) kernelized linear attention
with the elu(x)+1 feature map.

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  PyTorch provides device memory (outputs, state and
workspace buffers) and the current CUDA stream.  The binding's functions carry
the C ABI's names (``include/linattn.h``):

    la_prefill_causal(q, k, v, decay=None, eps=1e-6, chunk=64, ...)
    la_forward_noncausal(q, k, v, eps=1e-6, ...)
    la_decode_step(q, k, v, state_S, state_z, decay=None, eps=1e-6, ...)

and, for the softmax layers of a hybrid stack,

    la_softmax_prefill(q, k, v, cu_seqlens, ...)
    la_kv4_append / la_kv4_read / la_kv4_decode / la_kv4_evict on a KV4Cache

If the shared library has not been built, importing works but every call
raises: there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import functools
import os
import typing

import torch

__all__ = [
    "LinAttnError", "lib", "la_prefill_causal", "la_forward_noncausal", "la_decode_step",
    "la_prefill_causal_mlstm", "la_decode_step_mlstm", "la_prefill_causal_flash",
    "la_prefill_causal_summary", "la_state_combine",
    "la_prefill_workspace_size", "la_noncausal_workspace_size", "la_status_string",
    "la_prefill_path", "la_launch_count", "la_workspace_status", "la_set_wait_limit_ns", "LA_F32", "LA_BF16", "LA_F16", "LA_STATE_NONE", "LA_STATE_OUT",
    "LA_STATE_INOUT", "LIB_PATH",
    "KV4Cache", "la_softmax_prefill", "la_kv4_append", "la_kv4_read", "la_kv4_decode", "la_kv4_evict",
    "la_softmax_prefill_workspace_size", "la_kv4_decode_workspace_size", "la_kv4_evict_workspace_size",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblinattn.so")

LA_F32, LA_BF16, LA_F16 = 0, 1, 2
LA_STATE_NONE, LA_STATE_OUT, LA_STATE_INOUT = 0, 1, 2
LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_CUDA, LA_ERR_TIMEOUT = 0, 1, 2, 3, 4

_DT = {torch.float32: LA_F32, torch.bfloat16: LA_BF16, torch.float16: LA_F16}

_lib = None
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class _Kv4CacheC(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("k_par", _vp), ("v_codes", _vp), ("v_par", _vp), ("B", _i), ("H_kv", _i),
                ("cap", _i), ("d", _i)]


class LinAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = f"{fn} returned {status}: {la_status_string(status)}"
        if status == LA_ERR_CUDA:
            msg += f" ({lib().la_last_error_string().decode()})"
        super().__init__(msg)
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m kernelized_causal_sequence_b200.build` (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        L.la_prefill_causal.restype = _i
        L.la_prefill_causal.argtypes = [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _f, _i, _vp,
                                        _vp, _i, _vp, _i, _vp, _sz, _vp]
        L.la_prefill_causal_ev.restype = _i
        L.la_prefill_causal_ev.argtypes = [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _f, _i, _vp,
                                           _vp, _i, _vp, _i, _vp, _sz, _vp, _vp]
        L.la_prefill_causal_gated.restype = _i
        L.la_prefill_causal_gated.argtypes = [_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _f, _i,
                                              _vp, _vp, _i, _vp, _i, _vp, _sz, _vp]
        L.la_prefill_causal_mlstm.restype = _i
        L.la_prefill_causal_mlstm.argtypes = [_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                              _vp, _vp, _i, _vp, _i, _vp, _sz, _vp]
        L.la_prefill_causal_flash.restype = _i
        L.la_prefill_causal_flash.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _i,
                                              _vp, _i, _vp, _sz, _vp]
        L.la_prefill_causal_summary.restype = _i
        L.la_prefill_causal_summary.argtypes = [_vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp,
                                                _vp, _sz, _vp]
        L.la_state_combine.restype = _i
        L.la_state_combine.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]
        L.la_prefill_workspace_size.restype = _sz
        L.la_prefill_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i]
        L.la_forward_noncausal.restype = _i
        L.la_forward_noncausal.argtypes = [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _f, _vp,
                                           _vp, _i, _vp, _i, _vp, _sz, _vp]
        L.la_noncausal_workspace_size.restype = _sz
        L.la_noncausal_workspace_size.argtypes = [_i, _i, _i, _i, _i]
        L.la_decode_step.restype = _i
        L.la_decode_step.argtypes = [_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _f, _vp, _vp, _vp,
                                     _i, _vp]
        L.la_decode_step_gated.restype = _i
        L.la_decode_step_gated.argtypes = [_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _f, _vp, _vp,
                                           _vp, _i, _vp]
        L.la_decode_step_mlstm.restype = _i
        L.la_decode_step_mlstm.argtypes = [_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _vp, _vp,
                                           _vp, _i, _vp]
        L.la_status_string.restype = ctypes.c_char_p
        L.la_status_string.argtypes = [_i]
        L.la_prefill_plan.restype = _i
        L.la_prefill_plan.argtypes = [_i, _i, _i, _i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i)]
        L.la_prefill_path.restype = _i
        L.la_prefill_path.argtypes = [_i, _i, _i, _i, _i]
        L.la_launch_count.restype = ctypes.c_uint64
        L.la_launch_count.argtypes = []
        L.la_last_error_string.restype = ctypes.c_char_p
        L.la_last_error_string.argtypes = []
        L.la_workspace_status.restype = _i
        L.la_workspace_status.argtypes = [_vp, ctypes.POINTER(_i), _vp]
        L.la_noalloc_status.restype = _i
        L.la_noalloc_status.argtypes = [ctypes.POINTER(_i), _vp]
        L.la_set_wait_limit_ns.restype = ctypes.c_uint64
        L.la_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        _cp = ctypes.POINTER(_Kv4CacheC)
        L.la_softmax_prefill.restype = _i
        L.la_softmax_prefill.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _i, _vp, _f, _vp, _i, _vp, _sz, _vp]
        L.la_softmax_prefill_workspace_size.restype = _sz
        L.la_softmax_prefill_workspace_size.argtypes = [_i, _i, _i, _i, _i]
        L.la_kv4_append.restype = _i
        L.la_kv4_append.argtypes = [_vp, _vp, _i, _i, _vp, _vp, _vp, _cp, _vp]
        L.la_kv4_read.restype = _i
        L.la_kv4_read.argtypes = [_cp, _i, _vp, _vp, _vp, _vp, _i, _vp]
        L.la_kv4_decode.restype = _i
        L.la_kv4_decode.argtypes = [_vp, _i, _i, _cp, _vp, _f, _vp, _vp, _vp, _i, _vp, _sz, _vp]
        L.la_kv4_decode_workspace_size.restype = _sz
        L.la_kv4_decode_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i]
        L.la_kv4_evict.restype = _i
        L.la_kv4_evict.argtypes = [_cp, _vp, _vp, _i, _i, _cp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.la_kv4_evict_workspace_size.restype = _sz
        L.la_kv4_evict_workspace_size.argtypes = [_i, _i, _i, _i]
        _lib = L
    return _lib


def la_launch_count() -> int:
    return int(lib().la_launch_count())


def la_workspace_status(workspace, stream=None):
    """(status, waiter) of the last call that used ``workspace``: status is
    LA_OK or LA_ERR_TIMEOUT (a bounded device-side wait of that call gave up),
    waiter the id of the first wait that gave up.  Synchronises the stream."""
    w = ctypes.c_int(0)
    st = lib().la_workspace_status(_ptr(workspace), ctypes.byref(w), _stream(stream))
    if st not in (LA_OK, LA_ERR_TIMEOUT):
        raise LinAttnError("la_workspace_status", st)
    return st, w.value


def la_set_wait_limit_ns(ns: int) -> int:
    """Limit of every bounded device-side wait of later calls (process-wide);
    returns the previous limit."""
    return int(lib().la_set_wait_limit_ns(int(ns)))


def la_status_string(status: int) -> str:
    return lib().la_status_string(int(status)).decode()


def la_prefill_workspace_size(B, H, T, d_k, d_v, chunk) -> int:
    return int(lib().la_prefill_workspace_size(B, H, T, d_k, d_v, chunk))


def la_prefill_plan(B, H, T, d_k, chunk):
    """(segments per head, tokens per segment) of la_prefill_causal's plan."""
    n, sl = ctypes.c_int(0), ctypes.c_int(0)
    _check("la_prefill_plan", lib().la_prefill_plan(B, H, T, d_k, chunk, ctypes.byref(n), ctypes.byref(sl)))
    return n.value, sl.value


def la_noncausal_workspace_size(B, H, Lk, d_k, d_v) -> int:
    return int(lib().la_noncausal_workspace_size(B, H, Lk, d_k, d_v))


def la_prefill_path(in_dtype, d_k, d_v, chunk, has_decay=False) -> int:
    if isinstance(in_dtype, torch.dtype):
        in_dtype = _DT[in_dtype]
    return int(lib().la_prefill_path(in_dtype, d_k, d_v, chunk, int(bool(has_decay))))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, st):
    if st != LA_OK:
        raise LinAttnError(fn, st)


def _workspace(nbytes, device):
    # 256-byte aligned by the caching allocator
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def la_prefill_causal(q, k, v, decay=None, eps=1e-6, chunk=64, state_S=None, state_z=None,
                      mode=None, out=None, out_dtype=None, workspace=None, stream=None,
                      events=None, gain=None):
    """Causal chunked prefill.  q, k: [B,H,T,d_k]; v: [B,H,T,d_v] (f32/bf16/f16, CUDA,
    contiguous); decay: [B,H,T] fp32 or None.  state_S [B,H,d_k,d_v] / state_z [B,H,d_k]
    fp32 with ``mode`` LA_STATE_NONE/OUT/INOUT (default: OUT if given, else NONE).
    ``gain``: [B,H,T] fp32 (>= 0) or None — the gated form, token t's new term
    scaled by gain[t] (la_prefill_causal_gated; the RFA gate is decay=g, gain=1-g).
    ``events``: None, or 4 recorded-once ``torch.cuda.Event(enable_timing=True)``
    objects that la_prefill_causal_ev records around the state pass, the scan and
    the output pass (not with ``gain``).  Returns ``out`` [B,H,T,d_v]."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=out_dtype, device=q.device)
    if mode is None:
        mode = LA_STATE_OUT if state_S is not None else LA_STATE_NONE
    if workspace is None:
        workspace = _workspace(la_prefill_workspace_size(B, H, T, dk, dv, chunk), q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], _ptr(decay), B, H, T, dk, dv, float(eps),
            int(chunk), _ptr(state_S), _ptr(state_z), int(mode), _ptr(out), _DT[out.dtype],
            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if gain is not None:
        if events is not None:
            raise ValueError("events are not recorded by the gated prefill")
        st = lib().la_prefill_causal_gated(*args[:5], _ptr(gain), *args[5:])
        _check("la_prefill_causal_gated", st)
    elif events is None:
        st = lib().la_prefill_causal(*args)
        _check("la_prefill_causal", st)
    else:
        if len(events) != 4:
            raise ValueError("events: 4 CUDA events")
        for e in events:   # torch creates the CUDA event at its first record
            if int(e.cuda_event) == 0:
                e.record()
        arr = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(int(e.cuda_event)) for e in events])
        st = lib().la_prefill_causal_ev(*args, arr)
        _check("la_prefill_causal_ev", st)
    return out


def la_prefill_causal_mlstm(q, k, v, forget=None, input_gate=None, chunk=64, state_S=None, state_z=None,
                            mode=None, out=None, out_dtype=None, workspace=None, stream=None):
    """Causal prefill with the mLSTM read-out: identity feature map, forget gate
    f and input gate i (``[B,H,T]`` fp32 or None), out = q^T S / max(|q^T z|, 1)."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=out_dtype, device=q.device)
    if mode is None:
        mode = LA_STATE_OUT if state_S is not None else LA_STATE_NONE
    if workspace is None:
        workspace = _workspace(la_prefill_workspace_size(B, H, T, dk, dv, chunk), q.device)
    st = lib().la_prefill_causal_mlstm(_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], _ptr(forget), _ptr(input_gate),
                                       B, H, T, dk, dv, int(chunk), _ptr(state_S), _ptr(state_z), int(mode),
                                       _ptr(out), _DT[out.dtype], _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream))
    _check("la_prefill_causal_mlstm", st)
    return out


def la_prefill_causal_flash(q, k, v, chunk=64, scaled=False, state_S=None, state_z=None, mode=None, out=None,
                            out_dtype=None, workspace=None, stream=None):
    """The FLASH chunk form: exact relu(q.k / s)^2 attention inside each chunk
    plus q^T (sum of the earlier chunks' k v^T) / s; s = chunk if ``scaled``
    (the listings' convention) else 1.  The state is the raw sum of k v^T
    (and of k) over all tokens.  Returns ``out`` [B,H,T,d_v]."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=out_dtype, device=q.device)
    if mode is None:
        mode = LA_STATE_OUT if state_S is not None else LA_STATE_NONE
    if workspace is None:
        workspace = _workspace(la_prefill_workspace_size(B, H, T, dk, dv, chunk), q.device)
    st = lib().la_prefill_causal_flash(_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], B, H, T, dk, dv, int(chunk),
                                       int(bool(scaled)), _ptr(state_S), _ptr(state_z), int(mode), _ptr(out),
                                       _DT[out.dtype], _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream))
    _check("la_prefill_causal_flash", st)
    return out


def la_prefill_causal_summary(k, v, decay=None, gain=None, chunk=64, sum_S=None, sum_z=None, sum_A=None,
                              workspace=None, stream=None):
    """A shard's summary: (dS [B,H,dk,dv], dz [B,H,dk], A [B,H]) fp32, the
    shard's contribution to the state from a zero entry state and its decay
    product (la_prefill_causal_summary)."""
    B, H, T, dk = k.shape
    dv = v.shape[-1]
    dev = k.device
    sum_S = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if sum_S is None else sum_S
    sum_z = torch.empty((B, H, dk), dtype=torch.float32, device=dev) if sum_z is None else sum_z
    sum_A = torch.empty((B, H), dtype=torch.float32, device=dev) if sum_A is None else sum_A
    if workspace is None:
        workspace = _workspace(max(256, la_prefill_workspace_size(B, H, max(T, 1), dk, dv, chunk)), dev)
    st = lib().la_prefill_causal_summary(_ptr(k), _ptr(v), _DT[k.dtype], _ptr(decay), _ptr(gain), B, H, T, dk, dv,
                                         int(chunk), _ptr(sum_S), _ptr(sum_z), _ptr(sum_A), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check("la_prefill_causal_summary", st)
    return sum_S, sum_z, sum_A


def la_state_combine(S_all, z_all, A_all, r, S_in=None, z_in=None, S_out=None, z_out=None, stream=None):
    """Entry state of shard r from the gathered summaries [R, B, H, ...]
    (la_state_combine).  Returns (S_out, z_out)."""
    R, B, H, dk, dv = S_all.shape
    dev = S_all.device
    S_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev) if S_out is None else S_out
    z_out = torch.empty((B, H, dk), dtype=torch.float32, device=dev) if z_out is None else z_out
    st = lib().la_state_combine(_ptr(S_all), _ptr(z_all), _ptr(A_all), R, int(r), B, H, dk, dv, _ptr(S_in),
                                _ptr(z_in), _ptr(S_out), _ptr(z_out), _stream(stream))
    _check("la_state_combine", st)
    return S_out, z_out


def la_decode_step_mlstm(q, k, v, state_S, state_z, forget=None, input_gate=None, out=None,
                         out_dtype=None, stream=None):
    """One mLSTM decode step (``forget``, ``input_gate``: [B,H] fp32 or None);
    the state is updated in place."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((B, H, dv), dtype=out_dtype, device=q.device)
    st = lib().la_decode_step_mlstm(_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], _ptr(forget), _ptr(input_gate),
                                    B, H, dk, dv, _ptr(state_S), _ptr(state_z), _ptr(out), _DT[out.dtype],
                                    _stream(stream))
    _check("la_decode_step_mlstm", st)
    return out


def la_forward_noncausal(q, k, v, eps=1e-6, state_S=None, state_z=None, mode=None, out=None,
                         out_dtype=None, workspace=None, stream=None, decay=None):
    """Non-causal form.  q: [B,H,Lq,d_k]; k: [B,H,Lk,d_k]; v: [B,H,Lk,d_v]."""
    B, H, Lq, dk = q.shape
    Lk, dv = v.shape[2], v.shape[3]
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((B, H, Lq, dv), dtype=out_dtype, device=q.device)
    if mode is None:
        mode = LA_STATE_OUT if state_S is not None else LA_STATE_NONE
    if workspace is None:
        workspace = _workspace(la_noncausal_workspace_size(B, H, Lk, dk, dv), q.device)
    st = lib().la_forward_noncausal(_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], _ptr(decay), B, H,
                                    Lq, Lk, dk, dv, float(eps), _ptr(state_S), _ptr(state_z),
                                    int(mode), _ptr(out), _DT[out.dtype], _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check("la_forward_noncausal", st)
    return out


def la_decode_step(q, k, v, state_S, state_z, decay=None, eps=1e-6, out=None, out_dtype=None,
                   stream=None, gain=None):
    """One decode step; q, k: [B,H,d_k]; v: [B,H,d_v]; state updated in place.
    ``decay``, ``gain``: [B,H] fp32 or None (gated step: S <- a S + b phi(k) v^T)."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    out_dtype = q.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((B, H, dv), dtype=out_dtype, device=q.device)
    st = lib().la_decode_step_gated(_ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], _ptr(decay), _ptr(gain), B, H,
                                    dk, dv, float(eps), _ptr(state_S), _ptr(state_z), _ptr(out),
                                    _DT[out.dtype], _stream(stream))
    _check("la_decode_step_gated" if gain is not None else "la_decode_step", st)
    return out


# ---- softmax attention for the other layers of a hybrid stack --------------
#
# These functions check what the C ABI cannot see (shapes, types, devices) and
# raise ValueError before anything is launched.  A call runs on ``stream``, or
# on the current stream of its tensors' device.  (A decode step is a few
# microseconds on the GPU, so the checks are written to be cheap: plain
# conditions, messages formed only on failure.)

class KV4Cache(typing.NamedTuple):
    """A key/value cache in 4 bits (the format: la_kv4_cache in linattn.h).

    k_codes, v_codes: [B, H_kv, cap, d / 2] uint8; k_par, v_par:
    [B, H_kv, cap, d / 32] int32; contiguous, on one device."""
    k_codes: torch.Tensor
    k_par: torch.Tensor
    v_codes: torch.Tensor
    v_par: torch.Tensor

    @classmethod
    def alloc(cls, B, H_kv, cap, d, device="cuda"):
        """An uninitialised cache for B sequences, H_kv heads of d channels and
        ``cap`` positions."""
        def half():
            return (torch.empty((B, H_kv, cap, d // 2), dtype=torch.uint8, device=device),
                    torch.empty((B, H_kv, cap, d // 32), dtype=torch.int32, device=device))
        return cls(*half(), *half())


_HALVES = (16, 32, 64)   # bytes of a row's codes


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _cache_c(cache, what="cache"):
    """The C view of a cache and its device index."""
    kc, kp, vc, vp = cache
    dev = kc.get_device()
    try:
        B, Hk, cap, half = shape = kc.shape
    except ValueError:
        B, Hk, cap, half = shape = (0, 0, 0, 0)
    par = (B, Hk, cap, half >> 4)
    if (half not in _HALVES or dev < 0 or vc.shape != shape or kp.shape != par or vp.shape != par
            or kc.dtype is not torch.uint8 or vc.dtype is not torch.uint8
            or kp.dtype is not torch.int32 or vp.dtype is not torch.int32
            or kp.get_device() != dev or vc.get_device() != dev or vp.get_device() != dev
            or not (kc.is_contiguous() and kp.is_contiguous() and vc.is_contiguous() and vp.is_contiguous())):
        raise ValueError(f"{what}: k_codes, v_codes [B, H_kv, cap, d / 2] uint8 and k_par, v_par [B, H_kv, cap, d / 32] "
                         "int32, contiguous, on one CUDA device, d 32, 64 or 128")
    return _Kv4CacheC(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), B, Hk, cap, half * 2), dev


def _ints(x, n, dev, what):
    if (x.dtype is not torch.int32 or x.dim() != 1 or x.get_device() != dev or not x.is_contiguous()
            or (n is not None and x.shape[0] != n)):
        raise ValueError(f"{what}: contiguous int32{'' if n is None else f' [{n}]'} on the tensors' device")


def _floats(x, shape, dev, what):
    if x.dtype is not torch.float32 or tuple(x.shape) != shape or x.get_device() != dev or not x.is_contiguous():
        raise ValueError(f"{what}: contiguous fp32 {list(shape)} on the cache's device")


def _packed(x, heads, N, d, dtype, dev, what):
    # a [heads, N, d] view whose channels are contiguous
    if (x.dim() != 3 or x.shape[0] != heads or x.shape[1] != N or x.shape[2] != d or x.dtype is not dtype
            or x.get_device() != dev or x.stride(2) != 1):
        raise ValueError(f"{what}: [{heads}, {N}, {d}] {dtype} with contiguous channels, on the device of the others")


def _strides(*xs):
    # NULL where all are contiguous
    for x in xs:
        if not x.is_contiguous():
            return (ctypes.c_int64 * (2 * len(xs)))(*[s for y in xs for s in y.stride()[:2]])
    return None


class _On:
    """The device and stream of one call.  With a stream other than the
    current one, what the call allocates comes from that stream's memory, and
    the caching allocator is told of every tensor that both streams touch."""
    __slots__ = ("ptr", "stream", "current", "guard")

    def __init__(self, dev, stream):
        self.stream = self.guard = None
        self.ptr = torch._C._cuda_getCurrentRawStream(dev)
        if stream is not None:
            _need(stream.device.index == dev, "stream: of another device than the tensors")
            if stream.cuda_stream != self.ptr:
                self.current = torch.cuda.current_stream(dev)
                self.ptr, self.stream, self.guard = stream.cuda_stream, stream, torch.cuda.stream(stream)
        if self.guard is None and torch.cuda.current_device() != dev:
            self.guard = torch.cuda.device(dev)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def uses(self, *given):
        """Tensors of the caller that this call reads or writes."""
        if self.stream is not None:
            for x in given:
                if x is not None:
                    x.record_stream(self.stream)

    def hands(self, *made):
        """Tensors that this call allocated for the caller."""
        if self.stream is not None:
            for x in made:
                x.record_stream(self.current)


def la_softmax_prefill_workspace_size(H, H_kv, N, d, n_seq) -> int:
    return int(lib().la_softmax_prefill_workspace_size(H, H_kv, N, d, n_seq))


@functools.lru_cache(maxsize=256)
def _decode_ws(B, H, H_kv, cap, d, with_weights):
    return int(lib().la_kv4_decode_workspace_size(B, H, H_kv, cap, d, with_weights))


def la_kv4_decode_workspace_size(B, H, H_kv, cap, d, with_weights=False) -> int:
    return _decode_ws(B, H, H_kv, cap, d, int(bool(with_weights)))


def la_kv4_evict_workspace_size(B, H_kv, cap, keep) -> int:
    return int(lib().la_kv4_evict_workspace_size(B, H_kv, cap, keep))


def _ws(workspace, need, device, dev):
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    _need(workspace.get_device() == dev and workspace.is_contiguous(), "workspace: contiguous, on the tensors' device")
    return workspace


def _out_like(x, dtype):
    # (x is contiguous)
    return torch.empty_like(x) if dtype is None else torch.empty_like(x, dtype=dtype)


def _addr(x):
    return None if x is None else x.data_ptr()


def la_softmax_prefill(q, k, v, cu_seqlens, scale=None, out=None, out_dtype=None, workspace=None, stream=None):
    """Causal softmax attention over a packed prompt with grouped heads.

    q: [H, N, d]; k, v: [H_kv, N, d] (f32/bf16/f16, views with any head and
    token strides that are multiples of 16 bytes); cu_seqlens: [n_seq + 1]
    int32 on the device, sequence s being tokens cu_seqlens[s] ..
    cu_seqlens[s + 1] - 1.  ``scale`` defaults to d ** -0.5.  Returns ``out``
    [H, N, d]; its rows behind the last sequence are left as they were."""
    _need(q.dim() == 3 and k.dim() == 3 and q.is_cuda and q.dtype in _DT, "q: [H, N, d] f32, bf16 or f16 on CUDA; k: [H_kv, N, d]")
    H, N, d = q.shape
    dev, dt, Hk = q.get_device(), q.dtype, k.shape[0]
    _packed(q, H, N, d, dt, dev, "q")
    _packed(k, Hk, N, d, dt, dev, "k")
    _packed(v, Hk, N, d, dt, dev, "v")
    _ints(cu_seqlens, None, dev, "cu_seqlens")
    n_seq = cu_seqlens.shape[0] - 1
    _need(n_seq >= 0, "cu_seqlens: at least one entry")
    if out is not None:
        _need(out.dtype in _DT and out_dtype in (None, out.dtype), "out: f32, bf16 or f16")
        _packed(out, H, N, d, out.dtype, dev, "out")
    with _On(dev, stream) as on:
        on.uses(q, k, v, cu_seqlens, out, workspace)
        if out is None:
            out = torch.empty((H, N, d), dtype=dt if out_dtype is None else out_dtype, device=q.device)
            on.hands(out)
        ws = _ws(workspace, 256, q.device, dev)
        st = lib().la_softmax_prefill(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), _DT[dt], H, Hk, N, d, cu_seqlens.data_ptr(), n_seq,
            _strides(q, k, v, out), d ** -0.5 if scale is None else scale, out.data_ptr(), _DT[out.dtype],
            ws.data_ptr(), ws.nbytes, on.ptr)
    _check("la_softmax_prefill", st)
    return out


def la_kv4_append(k, v, cache, start, cu_seqlens=None, stream=None):
    """Quantises tokens into the cache.  k, v: [H_kv, N, d] (views as for
    la_softmax_prefill); token t of sequence s goes to position start[s] +
    (t - cu_seqlens[s]); without ``cu_seqlens`` token t is sequence t's only
    one.  Positions outside the cache are dropped.  start: [B] int32."""
    c, dev = _cache_c(cache)
    dt = k.dtype
    _need(k.dim() == 3 and dt in _DT, "k: [H_kv, N, d] f32, bf16 or f16")
    N = k.shape[1]
    _packed(k, c.H_kv, N, c.d, dt, dev, "k")
    _packed(v, c.H_kv, N, c.d, dt, dev, "v")
    _ints(start, c.B, dev, "start")
    if cu_seqlens is not None:
        _ints(cu_seqlens, c.B + 1, dev, "cu_seqlens")
    else:
        _need(N == c.B, "without cu_seqlens: one token per sequence")
    with _On(dev, stream) as on:
        on.uses(k, v, start, cu_seqlens, *cache)
        st = lib().la_kv4_append(k.data_ptr(), v.data_ptr(), _DT[dt], N, _strides(k, v), _addr(cu_seqlens),
                                 start.data_ptr(), c, on.ptr)
    _check("la_kv4_append", st)


def la_kv4_read(cache, start, n_tokens, cu_seqlens=None, out_dtype=torch.float32, stream=None):
    """The cache's values at the positions la_kv4_append would write for the
    same ``start`` and ``cu_seqlens``: (k, v), each [H_kv, n_tokens, d].
    Positions outside the cache and tokens of no sequence give zeros."""
    c, dev = _cache_c(cache)
    _need(out_dtype in _DT and n_tokens >= 0, "out_dtype: f32, bf16 or f16; n_tokens >= 0")
    _ints(start, c.B, dev, "start")
    if cu_seqlens is not None:
        _ints(cu_seqlens, c.B + 1, dev, "cu_seqlens")
    else:
        _need(n_tokens == c.B, "without cu_seqlens: one token per sequence")
    with _On(dev, stream) as on:
        on.uses(start, cu_seqlens, *cache)
        k = torch.empty((c.H_kv, n_tokens, c.d), dtype=out_dtype, device=start.device)
        v = torch.empty_like(k)
        on.hands(k, v)
        st = lib().la_kv4_read(c, n_tokens, _addr(cu_seqlens), start.data_ptr(), k.data_ptr(), v.data_ptr(),
                               _DT[out_dtype], on.ptr)
    _check("la_kv4_read", st)
    return k, v


def la_kv4_decode(q, cache, lens, scale=None, weights_in=None, weights_out=None, out=None, out_dtype=None,
                  workspace=None, stream=None):
    """Softmax attention of one query token per sequence over the first
    lens[b] positions of the cache.  q: [B, H, d] contiguous; lens: [B] int32.
    ``scale`` defaults to d ** -0.5.  ``weights_out`` [B, H_kv, cap] fp32
    receives weights_in (zeros if None; may be the same tensor) plus each
    position's attention weight summed over the head's queries.  Returns
    ``out`` [B, H, d]; a length of 0 gives zeros."""
    c, dev = _cache_c(cache)
    B, Hk, cap, d, dt, shape = c.B, c.H_kv, c.cap, c.d, q.dtype, q.shape
    if (len(shape) != 3 or shape[0] != B or shape[2] != d or dt not in _DT or q.get_device() != dev
            or not q.is_contiguous()):
        raise ValueError("q: contiguous [B, H, d] of the cache's sequences and head dim, on its device")
    H = shape[1]
    _ints(lens, B, dev, "lens")
    if weights_in is not None:
        _floats(weights_in, (B, Hk, cap), dev, "weights_in")
    if weights_out is not None:
        _floats(weights_out, (B, Hk, cap), dev, "weights_out")
    if out is not None:
        _need(out.shape == shape and out.is_contiguous() and out.get_device() == dev and out.dtype in _DT
              and out_dtype in (None, out.dtype), "out: contiguous [B, H, d] on the cache's device")
    with _On(dev, stream) as on:
        on.uses(q, lens, weights_in, weights_out, out, workspace, *cache)
        if out is None:
            out = _out_like(q, out_dtype)
            on.hands(out)
        ws = _ws(workspace, _decode_ws(B, H, Hk, cap, d, 0 if weights_out is None else 1), q.device, dev)
        st = lib().la_kv4_decode(
            q.data_ptr(), _DT[dt], H, c, lens.data_ptr(), d ** -0.5 if scale is None else scale, _addr(weights_in),
            _addr(weights_out), out.data_ptr(), _DT[out.dtype], ws.data_ptr(), ws.nbytes, on.ptr)
    _check("la_kv4_decode", st)
    return out


def la_kv4_evict(cache, weights, lens, keep, recent=0, out=None, out_weights=None, stream=None):
    """Cuts every (sequence, head) down to ``keep`` positions: the ``recent``
    newest and the heaviest of the others (ties to the lower position), moved
    in their order to the front of ``out``, another cache of at least ``keep``
    positions (allocated with ``keep`` when None).  weights: [B, H_kv, cap]
    fp32.  Returns (kept, out_weights, out_lens): the old positions
    [B, H_kv, keep] int32 (-1 behind them), their weights [B, H_kv, out.cap]
    and the new lengths [B] int32; with ``out`` None (out, kept, out_weights,
    out_lens)."""
    c, dev = _cache_c(cache)
    B, Hk, cap = c.B, c.H_kv, c.cap
    keep, recent = int(keep), int(recent)
    _ints(lens, B, dev, "lens")
    _floats(weights, (B, Hk, cap), dev, "weights")
    _need(keep >= 1 and 0 <= recent <= keep, "keep >= 1, 0 <= recent <= keep")
    _need(Hk > 0 or B == 0, "cache: at least one head")
    device = lens.device
    cap_out = keep
    if out is not None:
        o, dev_o = _cache_c(out, "out")
        _need(dev_o == dev and o.B == B and o.H_kv == Hk and o.d == c.d and o.cap >= keep,
              "out: of the cache's sequences, heads and head dim, keep positions at least, on its device")
        cap_out = o.cap
    if out_weights is not None:
        _floats(out_weights, (B, Hk, cap_out), dev, "out_weights")
    with _On(dev, stream) as on:
        on.uses(weights, lens, out_weights, *cache, *(out or ()))
        dst = out
        if dst is None:
            dst = KV4Cache.alloc(B, Hk, keep, c.d, device)
            on.hands(*dst)
            o, _ = _cache_c(dst, "out")
        if out_weights is None:
            out_weights = torch.zeros((B, Hk, cap_out), dtype=torch.float32, device=device)
            on.hands(out_weights)
        kept = torch.empty((B, Hk, keep), dtype=torch.int32, device=device)
        out_lens = torch.empty(B, dtype=torch.int32, device=device)
        on.hands(kept, out_lens)
        # (with `kept` the library needs no workspace)
        st = lib().la_kv4_evict(c, weights.data_ptr(), lens.data_ptr(), keep, recent, o, out_weights.data_ptr(),
                                kept.data_ptr(), out_lens.data_ptr(), None, 0, on.ptr)
    _check("la_kv4_evict", st)
    return (dst, kept, out_weights, out_lens) if out is None else (kept, out_weights, out_lens)
