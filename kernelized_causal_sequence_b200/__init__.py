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
# on the current stream of its tensors' device.

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


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _cache_c(cache, what="cache"):
    kc, kp, vc, vp = cache
    _need(kc.dim() == 4 and kc.dtype == torch.uint8 and kc.is_cuda, f"{what}.k_codes: [B, H_kv, cap, d / 2] uint8 on CUDA")
    B, Hk, cap, half = kc.shape
    d = half * 2
    _need(d in (32, 64, 128), f"{what}: head dim 32, 64 or 128, not {d}")
    _need(vc.shape == kc.shape and vc.dtype == torch.uint8, f"{what}.v_codes: as k_codes")
    for x in (kp, vp):
        _need(x.dtype == torch.int32 and tuple(x.shape) == (B, Hk, cap, d // 32), f"{what}: k_par, v_par [B, H_kv, cap, d / 32] int32")
    for x in cache:
        _need(x.device == kc.device and x.is_contiguous(), f"{what}: contiguous tensors on one device")
    return _Kv4CacheC(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), B, Hk, cap, d)


def _ints(x, n, device, what):
    _need(x.dtype == torch.int32 and x.dim() == 1 and x.device == device and x.is_contiguous()
          and (n is None or x.numel() == n), f"{what}: contiguous int32" + ("" if n is None else f" [{n}]") + f" on {device}")


def _packed(x, like, heads, what):
    # a [heads, N, d] view whose channels are contiguous
    _need(x.dim() == 3 and (x.stride(2) == 1 or x.shape[2] == 1), f"{what}: [heads, N, d] with contiguous channels")
    if like is not None:
        _need(x.dtype == like.dtype and x.device == like.device and x.shape[1:] == like.shape[1:]
              and (heads is None or x.shape[0] == heads), f"{what}: does not match the other inputs")


def _strides(*xs):
    return (ctypes.c_int64 * (2 * len(xs)))(*[s for x in xs for s in x.stride()[:2]])


class _On:
    """The device and stream of one call.  With a stream other than the
    current one, what the call allocates comes from that stream's memory, and
    the caching allocator is told of every tensor that both streams touch."""

    def __init__(self, device, stream):
        self.current = torch.cuda.current_stream(device)
        self.stream = self.current if stream is None else stream
        self.other = self.stream.cuda_stream != self.current.cuda_stream
        _need(self.stream.device == device, "stream: of another device than the tensors")
        self.guard = None
        if self.other:
            self.guard = torch.cuda.stream(self.stream)
        elif torch.cuda.current_device() != device.index:
            self.guard = torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.stream.cuda_stream)

    def uses(self, *given):
        """Tensors of the caller that this call reads or writes."""
        if self.other:
            for x in given:
                if x is not None:
                    x.record_stream(self.stream)

    def hands(self, *made):
        """Tensors that this call allocated for the caller."""
        if self.other:
            for x in made:
                x.record_stream(self.current)


def la_softmax_prefill_workspace_size(H, H_kv, N, d, n_seq) -> int:
    return int(lib().la_softmax_prefill_workspace_size(H, H_kv, N, d, n_seq))


def la_kv4_decode_workspace_size(B, H, H_kv, cap, d, with_weights=False) -> int:
    return int(lib().la_kv4_decode_workspace_size(B, H, H_kv, cap, d, int(bool(with_weights))))


def la_kv4_evict_workspace_size(B, H_kv, cap, keep) -> int:
    return int(lib().la_kv4_evict_workspace_size(B, H_kv, cap, keep))


def _ws(workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    _need(workspace.device == device and workspace.is_contiguous(), f"workspace: contiguous, on {device}")
    return workspace


def la_softmax_prefill(q, k, v, cu_seqlens, scale=None, out=None, out_dtype=None, workspace=None, stream=None):
    """Causal softmax attention over a packed prompt with grouped heads.

    q: [H, N, d]; k, v: [H_kv, N, d] (f32/bf16/f16, views with any head and
    token strides that are multiples of 16 bytes); cu_seqlens: [n_seq + 1]
    int32 on the device, sequence s being tokens cu_seqlens[s] ..
    cu_seqlens[s + 1] - 1.  ``scale`` defaults to d ** -0.5.  Returns ``out``
    [H, N, d]; its rows behind the last sequence are left as they were."""
    _packed(q, None, None, "q")
    _need(q.is_cuda and q.dtype in _DT, "q: f32, bf16 or f16 on CUDA")
    H, N, d = q.shape
    _packed(k, q, None, "k")
    _packed(v, q, k.shape[0], "v")
    _ints(cu_seqlens, None, q.device, "cu_seqlens")
    n_seq = cu_seqlens.numel() - 1
    _need(n_seq >= 0, "cu_seqlens: at least one entry")
    if out is not None:
        _packed(out, None, None, "out")
        _need(out.shape == q.shape and out.device == q.device and out.dtype in _DT and out_dtype in (None, out.dtype),
              "out: [H, N, d] on the inputs' device")
    with _On(q.device, stream) as on:
        on.uses(q, k, v, cu_seqlens, out, workspace)
        if out is None:
            out = torch.empty((H, N, d), dtype=q.dtype if out_dtype is None else out_dtype, device=q.device)
            on.hands(out)
        ws = _ws(workspace, 256, q.device)
        _check("la_softmax_prefill", lib().la_softmax_prefill(
            _ptr(q), _ptr(k), _ptr(v), _DT[q.dtype], H, k.shape[0], N, d, _ptr(cu_seqlens), n_seq,
            _strides(q, k, v, out), d ** -0.5 if scale is None else float(scale), _ptr(out), _DT[out.dtype],
            _ptr(ws), ws.numel() * ws.element_size(), on.ptr))
    return out


def la_kv4_append(k, v, cache, start, cu_seqlens=None, stream=None):
    """Quantises tokens into the cache.  k, v: [H_kv, N, d] (views as for
    la_softmax_prefill); token t of sequence s goes to position start[s] +
    (t - cu_seqlens[s]); without ``cu_seqlens`` token t is sequence t's only
    one.  Positions outside the cache are dropped.  start: [B] int32."""
    c = _cache_c(cache)
    dev = cache.k_codes.device
    _packed(k, None, None, "k")
    _packed(v, k, c.H_kv, "v")
    _need(k.dtype in _DT and k.device == dev and k.shape[0] == c.H_kv and k.shape[2] == c.d,
          "k, v: [H_kv, N, d] of the cache's heads and head dim, on its device")
    _ints(start, c.B, dev, "start")
    if cu_seqlens is not None:
        _ints(cu_seqlens, c.B + 1, dev, "cu_seqlens")
    else:
        _need(k.shape[1] == c.B, "without cu_seqlens: one token per sequence")
    with _On(dev, stream) as on:
        on.uses(k, v, start, cu_seqlens, *cache)
        _check("la_kv4_append", lib().la_kv4_append(_ptr(k), _ptr(v), _DT[k.dtype], k.shape[1], _strides(k, v),
                                                    _ptr(cu_seqlens), _ptr(start), ctypes.byref(c), on.ptr))


def la_kv4_read(cache, start, n_tokens, cu_seqlens=None, out_dtype=torch.float32, stream=None):
    """The cache's values at the positions la_kv4_append would write for the
    same ``start`` and ``cu_seqlens``: (k, v), each [H_kv, n_tokens, d].
    Positions outside the cache and tokens of no sequence give zeros."""
    c = _cache_c(cache)
    dev = cache.k_codes.device
    _need(out_dtype in _DT and n_tokens >= 0, "out_dtype: f32, bf16 or f16; n_tokens >= 0")
    _ints(start, c.B, dev, "start")
    if cu_seqlens is not None:
        _ints(cu_seqlens, c.B + 1, dev, "cu_seqlens")
    else:
        _need(n_tokens == c.B, "without cu_seqlens: one token per sequence")
    with _On(dev, stream) as on:
        on.uses(start, cu_seqlens, *cache)
        k = torch.empty((c.H_kv, n_tokens, c.d), dtype=out_dtype, device=dev)
        v = torch.empty_like(k)
        on.hands(k, v)
        _check("la_kv4_read", lib().la_kv4_read(ctypes.byref(c), n_tokens, _ptr(cu_seqlens), _ptr(start), _ptr(k),
                                                _ptr(v), _DT[out_dtype], on.ptr))
    return k, v


def la_kv4_decode(q, cache, lens, scale=None, weights_in=None, weights_out=None, out=None, out_dtype=None,
                  workspace=None, stream=None):
    """Softmax attention of one query token per sequence over the first
    lens[b] positions of the cache.  q: [B, H, d] contiguous; lens: [B] int32.
    ``scale`` defaults to d ** -0.5.  ``weights_out`` [B, H_kv, cap] fp32
    receives weights_in (zeros if None; may be the same tensor) plus each
    position's attention weight summed over the head's queries.  Returns
    ``out`` [B, H, d]; a length of 0 gives zeros."""
    c = _cache_c(cache)
    dev = cache.k_codes.device
    _need(q.dim() == 3 and q.is_contiguous() and q.dtype in _DT and q.device == dev and q.shape[0] == c.B
          and q.shape[2] == c.d, "q: contiguous [B, H, d] of the cache's sequences and head dim, on its device")
    H = q.shape[1]
    _ints(lens, c.B, dev, "lens")
    for x in (weights_in, weights_out):
        if x is not None:
            _need(x.dtype == torch.float32 and tuple(x.shape) == (c.B, c.H_kv, c.cap) and x.device == dev
                  and x.is_contiguous(), "weights: contiguous [B, H_kv, cap] fp32")
    if out is not None:
        _need(out.shape == q.shape and out.is_contiguous() and out.device == dev and out.dtype in _DT
              and out_dtype in (None, out.dtype), "out: contiguous [B, H, d] on the cache's device")
    with _On(dev, stream) as on:
        on.uses(q, lens, weights_in, weights_out, out, workspace, *cache)
        if out is None:
            out = torch.empty((c.B, H, c.d), dtype=q.dtype if out_dtype is None else out_dtype, device=dev)
            on.hands(out)
        ws = _ws(workspace, la_kv4_decode_workspace_size(c.B, H, c.H_kv, c.cap, c.d, weights_out is not None), dev)
        _check("la_kv4_decode", lib().la_kv4_decode(
            _ptr(q), _DT[q.dtype], H, ctypes.byref(c), _ptr(lens), c.d ** -0.5 if scale is None else float(scale),
            _ptr(weights_in), _ptr(weights_out), _ptr(out), _DT[out.dtype], _ptr(ws),
            ws.numel() * ws.element_size(), on.ptr))
    return out


def la_kv4_evict(cache, weights, lens, keep, recent=0, out=None, out_weights=None, workspace=None, stream=None):
    """Cuts every (sequence, head) down to ``keep`` positions: the ``recent``
    newest and the heaviest of the others (ties to the lower position), moved
    in their order to the front of ``out``, another cache of at least ``keep``
    positions (allocated with ``keep`` when None).  weights: [B, H_kv, cap]
    fp32.  Returns (kept, out_weights, out_lens): the old positions
    [B, H_kv, keep] int32 (-1 behind them), their weights [B, H_kv, out.cap]
    and the new lengths [B] int32; with ``out`` None (out, kept, out_weights,
    out_lens)."""
    c = _cache_c(cache)
    dev = cache.k_codes.device
    keep, recent = int(keep), int(recent)
    _ints(lens, c.B, dev, "lens")
    _need(weights.dtype == torch.float32 and tuple(weights.shape) == (c.B, c.H_kv, c.cap) and weights.device == dev
          and weights.is_contiguous(), "weights: contiguous [B, H_kv, cap] fp32")
    _need(keep >= 1 and 0 <= recent <= keep, "keep >= 1, 0 <= recent <= keep")
    if out is not None:
        _need(_cache_c(out, "out").cap >= keep and out.k_codes.device == dev, "out: keep positions at least, on the cache's device")
    if out_weights is not None:
        cap_out = keep if out is None else out.k_codes.shape[2]
        _need(out_weights.dtype == torch.float32 and tuple(out_weights.shape) == (c.B, c.H_kv, cap_out)
              and out_weights.device == dev and out_weights.is_contiguous(),
              "out_weights: contiguous [B, H_kv, out.cap] fp32")
    with _On(dev, stream) as on:
        on.uses(weights, lens, out_weights, workspace, *cache, *(out or ()))
        dst = out
        if dst is None:
            dst = KV4Cache.alloc(c.B, c.H_kv, keep, c.d, dev)
            on.hands(*dst)
        o = _cache_c(dst, "out")
        if out_weights is None:
            out_weights = torch.zeros((c.B, c.H_kv, o.cap), dtype=torch.float32, device=dev)
            on.hands(out_weights)
        kept = torch.empty((c.B, c.H_kv, keep), dtype=torch.int32, device=dev)
        out_lens = torch.empty(c.B, dtype=torch.int32, device=dev)
        on.hands(kept, out_lens)
        ws = _ws(workspace, la_kv4_evict_workspace_size(c.B, c.H_kv, c.cap, keep), dev)
        _check("la_kv4_evict", lib().la_kv4_evict(ctypes.byref(c), _ptr(weights), _ptr(lens), keep, recent,
                                                  ctypes.byref(o), _ptr(out_weights), _ptr(kept), _ptr(out_lens),
                                                  _ptr(ws), ws.numel() * ws.element_size(), on.ptr))
    return (dst, kept, out_weights, out_lens) if out is None else (kept, out_weights, out_lens)
