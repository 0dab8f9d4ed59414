"""ctypes binding of libkda.so (include/kda.h).  Argument marshalling only.

Every step of the computation runs in the library's CUDA kernels.  PyTorch
supplies device memory and the current stream.  There is no fallback: if
libkda.so is missing or cannot load, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_F32, KDA_BF16 = 0, 1
KERNELS = {"auto": 0, "simt": 1, "tc": 2}
STATUS = {
    0: "KDA_OK", -1: "KDA_ERR_NULL", -2: "KDA_ERR_SHAPE", -3: "KDA_ERR_DTYPE",
    -4: "KDA_ERR_ALIGN", -5: "KDA_ERR_RANGE", -6: "KDA_ERR_CUDA", -7: "KDA_ERR_UNSUPPORTED",
    -8: "KDA_ERR_ALIAS", -9: "KDA_ERR_SCRATCH_LIMIT",
}


class KdaChunkDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
                ("num_seqs", ctypes.c_int), ("qkv_dtype", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("gate_dtype", ctypes.c_int),
                ("validate", ctypes.c_int), ("kernel", ctypes.c_int), ("segments", ctypes.c_int)]


class KdaDecodeDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("H", ctypes.c_int), ("dk", ctypes.c_int),
                ("dv", ctypes.c_int), ("qkv_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("gate_dtype", ctypes.c_int), ("validate", ctypes.c_int)]


class KdaLayerGates(ctypes.Structure):
    _fields_ = [("A_log", ctypes.c_void_p), ("g_min", ctypes.c_float), ("out_gate", ctypes.c_void_p),
                ("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float)]


class KdaScanDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int),
                ("num_seqs", ctypes.c_int), ("dtype", ctypes.c_int), ("gate_dtype", ctypes.c_int),
                ("write", ctypes.c_int), ("validate", ctypes.c_int)]


class KdaNormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int), ("dtype", ctypes.c_int),
                ("res_dtype", ctypes.c_int), ("post_norm", ctypes.c_int), ("post_eps", ctypes.c_float),
                ("pre_eps", ctypes.c_float)]


class KdaError(RuntimeError):
    def __init__(self, status: int, fn: str, detail: str = ""):
        self.status = status
        name = STATUS.get(status, str(status))
        super().__init__(f"{fn} returned {name}" + (f": {detail}" if detail else ""))


_lock = threading.Lock()
_lib = None


def load() -> ctypes.CDLL:
    """Load libkda.so (raises if it is absent: there is no CPU path)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libkda.so is not built ({LIB_PATH}); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        lib.kda_chunk_fwd.argtypes = [ctypes.POINTER(KdaChunkDesc), P, P, P, P, P, P, P, P, P, P]
        lib.kda_chunk_fwd.restype = ctypes.c_int
        lib.kda_chunk_fwd_ex.argtypes = [ctypes.POINTER(KdaChunkDesc), P, P, P, P, P, P, P, P, P,
                                         P, ctypes.c_size_t, P]
        lib.kda_chunk_fwd_ex.restype = ctypes.c_int
        lib.kda_chunk_fwd_workspace_size.argtypes = [ctypes.POINTER(KdaChunkDesc),
                                                     ctypes.POINTER(ctypes.c_size_t)]
        lib.kda_chunk_fwd_workspace_size.restype = ctypes.c_int
        lib.kda_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(KdaChunkDesc), P, P, P, P, P, P, P, P, P, P]
        lib.kda_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.kda_chunk_fwd_ckpt.argtypes = [ctypes.POINTER(KdaChunkDesc), P, P, P, P, P, P, P, P, P,
                                           ctypes.c_int, P, P, P, ctypes.c_size_t, P]
        lib.kda_chunk_fwd_ckpt.restype = ctypes.c_int
        lib.kda_decode_step.argtypes = [ctypes.POINTER(KdaDecodeDesc), P, P, P, P, P, P, P, P]
        lib.kda_decode_step.restype = ctypes.c_int
        lib.kda_layer_fwd.argtypes = [ctypes.POINTER(KdaChunkDesc), ctypes.POINTER(KdaLayerGates), P, P, P, P, P,
                                      P, P, P, P, P, ctypes.c_size_t, P]
        lib.kda_layer_fwd.restype = ctypes.c_int
        lib.kda_layer_decode_step.argtypes = [ctypes.POINTER(KdaDecodeDesc), ctypes.POINTER(KdaLayerGates), P, P,
                                              P, P, P, P, P, P]
        lib.kda_layer_decode_step.restype = ctypes.c_int
        lib.kda_chunk_bwd_workspace_size.argtypes = [ctypes.POINTER(KdaChunkDesc), ctypes.POINTER(ctypes.c_size_t)]
        lib.kda_chunk_bwd_workspace_size.restype = ctypes.c_int
        lib.kda_chunk_bwd.argtypes = [ctypes.POINTER(KdaChunkDesc), P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P,
                                      ctypes.c_size_t, P]
        lib.kda_chunk_bwd.restype = ctypes.c_int
        lib.kda_chunk_affine_pair.argtypes = [ctypes.POINTER(KdaChunkDesc), P, P, P, P, P, P, P, P]
        lib.kda_chunk_affine_pair.restype = ctypes.c_int
        lib.kda_affine_compose.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           P, P, P, P]
        lib.kda_affine_compose.restype = ctypes.c_int
        S, Z = ctypes.POINTER(KdaScanDesc), ctypes.POINTER(ctypes.c_size_t)
        F = ctypes.c_float
        lib.kda_scan_states_size.argtypes = [S, Z]
        lib.kda_scan_fwd.argtypes = [S, P, P, P, F, P, P, P, P, P, P]
        lib.kda_scan_bwd_workspace_size.argtypes = [S, ctypes.c_int, ctypes.c_int, Z]
        lib.kda_scan_bwd.argtypes = [S, P, P, P, F, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.kda_scan_step.argtypes = [S, P, P, P, F, P, P, P, P]
        NP = ctypes.POINTER(KdaNormDesc)
        lib.kda_block_norm_fwd.argtypes = [NP, P, P, P, P, P, P, P, P, P]
        lib.kda_block_norm_bwd_workspace_size.argtypes = [NP, Z]
        lib.kda_block_norm_bwd.argtypes = [NP, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        for fn in (lib.kda_scan_states_size, lib.kda_scan_fwd, lib.kda_scan_bwd_workspace_size, lib.kda_scan_bwd,
                   lib.kda_scan_step, lib.kda_block_norm_fwd, lib.kda_block_norm_bwd_workspace_size,
                   lib.kda_block_norm_bwd):
            fn.restype = ctypes.c_int
        lib.kda_status_string.argtypes = [ctypes.c_int]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_last_cuda_error.argtypes = []
        lib.kda_last_cuda_error.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, fn: str):
    if status != 0:
        lib = load()
        detail = lib.kda_status_string(status).decode()
        if status == -6:
            detail += " (" + lib.kda_last_cuda_error().decode() + ")"
        raise KdaError(status, fn, detail)


def chunk_desc(q, v, *, chunk=64, cu_seqlens=None, out_dtype=None, gate_dtype=None, validate=False,
               kernel="auto", segments=0, B=None) -> KdaChunkDesc:
    if q.dim() == 4:
        B_, T, H, dk = q.shape
    else:
        T, H, dk = q.shape
        B_ = 1
    if B is not None and q.dim() == 3:
        B_ = B
        T = T // B
    dv = v.shape[-1]
    d = KdaChunkDesc()
    d.B, d.T, d.H, d.dk, d.dv, d.chunk = B_, T, H, dk, dv, chunk
    d.num_seqs = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    d.qkv_dtype = _dt(q)
    d.out_dtype = KDA_BF16 if out_dtype == torch.bfloat16 else (
        KDA_F32 if out_dtype == torch.float32 else _dt(q))
    d.gate_dtype = gate_dtype if gate_dtype is not None else KDA_F32
    d.validate = int(bool(validate))
    d.kernel = KERNELS[kernel]
    d.segments = int(segments)
    return d


def kda_chunk_fwd(q, k, v, log_alpha, beta, initial_state=None, cu_seqlens=None, out=None,
                  final_state=None, *, chunk=64, kernel="auto", segments=0, validate=False,
                  out_dtype=None, want_final_state=True, B=None, stream=None, workspace=None):
    """Chunked KDA prefill through the C ABI.

    q, k, log_alpha: [B*T, H, dk] (or [B, T, H, dk]); v: [.., H, dv];
    beta: [B*T, H]; initial_state: [N, H, dk, dv] fp32 or None;
    cu_seqlens: int32 [N+1] on the device or None.  Returns (out, final_state).
    """
    lib = load()
    dev = q.device
    d = chunk_desc(q, v, chunk=chunk, cu_seqlens=cu_seqlens, out_dtype=out_dtype or q.dtype,
                   gate_dtype=_dt(log_alpha), validate=validate, kernel=kernel, segments=segments, B=B)
    if beta.dtype != log_alpha.dtype:
        raise TypeError("log_alpha and beta must share a dtype")
    Nseq = d.num_seqs if cu_seqlens is not None else d.B
    if out is None:
        out = torch.empty(q.shape[:-1] + (d.dv,), dtype=out_dtype or q.dtype, device=dev)
    if final_state is None and want_final_state:
        final_state = torch.empty(Nseq, d.H, d.dk, d.dv, dtype=torch.float32, device=dev)
    args = [ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
            _ptr(initial_state), _ptr(cu_seqlens), _ptr(out), _ptr(final_state)]
    if workspace is not None:
        st = lib.kda_chunk_fwd_ex(*args, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream, dev))
        _check(st, "kda_chunk_fwd_ex")
    else:
        st = lib.kda_chunk_fwd(*args, _stream_handle(stream, dev))
        _check(st, "kda_chunk_fwd")
    return out, final_state


def kda_chunk_fwd_noalloc(q, k, v, log_alpha, beta, initial_state=None, cu_seqlens=None, out=None,
                          final_state=None, *, chunk=64, kernel="auto", segments=0, out_dtype=None,
                          want_final_state=True, B=None, stream=None):
    """kda_chunk_fwd through the entry point that allocates no device memory:
    the long-sequence workspace comes from the library's static scratch array
    (KDA_STATIC_WORKSPACE_BYTES).  Output tensors are allocated here by torch
    only when not given; pass `out` and `final_state` to allocate nothing."""
    lib = load()
    dev = q.device
    d = chunk_desc(q, v, chunk=chunk, cu_seqlens=cu_seqlens, out_dtype=out_dtype or q.dtype,
                   gate_dtype=_dt(log_alpha), validate=False, kernel=kernel, segments=segments, B=B)
    Nseq = d.num_seqs if cu_seqlens is not None else d.B
    if out is None:
        out = torch.empty(q.shape[:-1] + (d.dv,), dtype=out_dtype or q.dtype, device=dev)
    if final_state is None and want_final_state:
        final_state = torch.empty(Nseq, d.H, d.dk, d.dv, dtype=torch.float32, device=dev)
    st = lib.kda_chunk_fwd_noalloc(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                   _ptr(initial_state), _ptr(cu_seqlens), _ptr(out), _ptr(final_state),
                                   _stream_handle(stream, dev))
    _check(st, "kda_chunk_fwd_noalloc")
    return out, final_state


def kda_chunk_fwd_ckpt(q, k, v, log_alpha, beta, every, initial_state=None, cu_seqlens=None,
                       cu_ckpt=None, out=None, final_state=None, ckpt=None, *, chunk=64, kernel="auto",
                       segments=0, validate=False, out_dtype=None, want_final_state=True, B=None,
                       stream=None, workspace=None):
    """kda_chunk_fwd that also stores the fp32 state after every `every`
    tokens of each sequence (prefix-cache checkpoints).

    cu_ckpt: int32 [N+1] on the device with cu_ckpt[n+1] - cu_ckpt[n] =
    len_n // every (required with cu_seqlens).  When `ckpt` is None it is
    allocated here with cu_ckpt[-1] slots (a device-to-host read) or, for a
    B x T batch, B * (T // every) slots.  Returns (out, final_state, ckpt).
    """
    lib = load()
    dev = q.device
    d = chunk_desc(q, v, chunk=chunk, cu_seqlens=cu_seqlens, out_dtype=out_dtype or q.dtype,
                   gate_dtype=_dt(log_alpha), validate=validate, kernel=kernel, segments=segments, B=B)
    Nseq = d.num_seqs if cu_seqlens is not None else d.B
    if out is None:
        out = torch.empty(q.shape[:-1] + (d.dv,), dtype=out_dtype or q.dtype, device=dev)
    if final_state is None and want_final_state:
        final_state = torch.empty(Nseq, d.H, d.dk, d.dv, dtype=torch.float32, device=dev)
    if ckpt is None:
        slots = int(cu_ckpt[-1].item()) if cu_seqlens is not None else d.B * (d.T // every if every > 0 else 0)
        ckpt = torch.empty(max(slots, 1), d.H, d.dk, d.dv, dtype=torch.float32, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.kda_chunk_fwd_ckpt(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                _ptr(initial_state), _ptr(cu_seqlens), _ptr(out), _ptr(final_state),
                                int(every), _ptr(cu_ckpt), _ptr(ckpt), _ptr(workspace), ws_bytes,
                                _stream_handle(stream, dev))
    _check(st, "kda_chunk_fwd_ckpt")
    return out, final_state, ckpt


def kda_chunk_fwd_workspace_size(desc: KdaChunkDesc) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    _check(lib.kda_chunk_fwd_workspace_size(ctypes.byref(desc), ctypes.byref(n)),
           "kda_chunk_fwd_workspace_size")
    return n.value


def kda_decode_step(q, k, v, log_alpha, beta, state_inout, out=None, *, validate=False,
                    out_dtype=None, stream=None):
    """One decode step through the C ABI: q,k,log_alpha [N,H,dk], v [N,H,dv],
    beta [N,H], state_inout [N,H,dk,dv] fp32 (updated in place).  Returns out."""
    lib = load()
    N, H, dk = q.shape
    dv = v.shape[-1]
    d = KdaDecodeDesc()
    d.N, d.H, d.dk, d.dv = N, H, dk, dv
    d.qkv_dtype = _dt(q)
    od = out_dtype or q.dtype
    d.out_dtype = _dt(torch.empty(0, dtype=od))
    d.gate_dtype = _dt(log_alpha)
    d.validate = int(bool(validate))
    if out is None:
        out = torch.empty(N, H, dv, dtype=od, device=q.device)
    st = lib.kda_decode_step(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                             _ptr(state_inout), _ptr(out), _stream_handle(stream, q.device))
    _check(st, "kda_decode_step")
    return out


def layer_gates(A_log, g_min=-5.0, out_gate=None, norm_weight=None, norm_eps=1e-6) -> KdaLayerGates:
    """The kda_layer_gates struct for the given device tensors."""
    lg = KdaLayerGates()
    lg.A_log = None if A_log is None else A_log.data_ptr()
    lg.g_min = float(g_min)
    lg.out_gate = None if out_gate is None else _ptr(out_gate).value
    lg.norm_weight = None if norm_weight is None else _ptr(norm_weight).value
    lg.norm_eps = float(norm_eps)
    return lg


def kda_layer_fwd(q, k, v, z, beta, A_log, g_min=-5.0, out_gate=None, norm_weight=None, norm_eps=1e-6,
                  initial_state=None, cu_seqlens=None, out=None, final_state=None, *, chunk=64, kernel="auto",
                  segments=0, validate=False, out_dtype=None, want_final_state=True, B=None, stream=None,
                  workspace=None):
    """KDA prefill inside the layer's gates through the C ABI: the log-decay is
    g_min * sigmoid(exp(A_log[h]) * z) (z: [.., H, dk] decay logits in q's
    dtype; A_log: [H] fp32) and, with out_gate ([.., H, dv], q's dtype), the
    output is sigmoid(out_gate) * RMSNorm(o) with norm_weight [dv] fp32 (None:
    ones) and norm_eps.  beta: fp32 or bf16.  Returns (out, final_state)."""
    lib = load()
    dev = q.device
    if z.dtype != q.dtype:
        raise TypeError("z must have q's dtype")
    if out_gate is not None and out_gate.dtype != q.dtype:
        raise TypeError("out_gate must have q's dtype")
    d = chunk_desc(q, v, chunk=chunk, cu_seqlens=cu_seqlens, out_dtype=out_dtype or q.dtype,
                   gate_dtype=_dt(beta), validate=validate, kernel=kernel, segments=segments, B=B)
    Nseq = d.num_seqs if cu_seqlens is not None else d.B
    if out is None:
        out = torch.empty(q.shape[:-1] + (d.dv,), dtype=out_dtype or q.dtype, device=dev)
    if final_state is None and want_final_state:
        final_state = torch.empty(Nseq, d.H, d.dk, d.dv, dtype=torch.float32, device=dev)
    lg = layer_gates(A_log, g_min, out_gate, norm_weight, norm_eps)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.kda_layer_fwd(ctypes.byref(d), ctypes.byref(lg), _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta),
                           _ptr(initial_state), _ptr(cu_seqlens), _ptr(out), _ptr(final_state),
                           _ptr(workspace), ws_bytes, _stream_handle(stream, dev))
    _check(st, "kda_layer_fwd")
    return out, final_state


def kda_layer_decode_step(q, k, v, z, beta, state_inout, A_log, g_min=-5.0, out_gate=None, norm_weight=None,
                          norm_eps=1e-6, out=None, *, validate=False, out_dtype=None, stream=None):
    """One decode step inside the layer's gates (see kda_layer_fwd): q, k, z
    [N,H,dk], v and out_gate [N,H,dv], beta [N,H], state_inout [N,H,dk,dv] fp32
    updated in place.  Returns out."""
    lib = load()
    N, H, dk = q.shape
    dv = v.shape[-1]
    d = KdaDecodeDesc()
    d.N, d.H, d.dk, d.dv = N, H, dk, dv
    d.qkv_dtype = _dt(q)
    od = out_dtype or q.dtype
    d.out_dtype = _dt(torch.empty(0, dtype=od))
    d.gate_dtype = _dt(beta)
    d.validate = int(bool(validate))
    if out is None:
        out = torch.empty(N, H, dv, dtype=od, device=q.device)
    lg = layer_gates(A_log, g_min, out_gate, norm_weight, norm_eps)
    st = lib.kda_layer_decode_step(ctypes.byref(d), ctypes.byref(lg), _ptr(q), _ptr(k), _ptr(v), _ptr(z),
                                   _ptr(beta), _ptr(state_inout), _ptr(out), _stream_handle(stream, q.device))
    _check(st, "kda_layer_decode_step")
    return out


def kda_chunk_bwd_workspace_size(desc: KdaChunkDesc) -> int:
    lib = load()
    n = ctypes.c_size_t(0)
    _check(lib.kda_chunk_bwd_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "kda_chunk_bwd_workspace_size")
    return n.value


def kda_chunk_bwd(q, k, v, log_alpha, beta, d_out, initial_state=None, d_final_state=None, cu_seqlens=None,
                  *, chunk=64, validate=False, want_d_initial_state=True, B=None, stream=None, workspace=None,
                  grads=None):
    """Gradients of kda_chunk_fwd through the C ABI for
    L = sum <d_out, out> + <d_final_state, final_state>.

    Arguments as kda_chunk_fwd plus d_out (out's shape and dtype) and
    d_final_state ([N,H,dk,dv] fp32 or None).  Returns a dict of fp32 tensors
    dq, dk, dv, dlog_alpha, dbeta and d_initial_state (None unless wanted).
    `grads` may pass that dict preallocated."""
    lib = load()
    dev = q.device
    d = chunk_desc(q, v, chunk=chunk, cu_seqlens=cu_seqlens, out_dtype=d_out.dtype, gate_dtype=_dt(log_alpha),
                   validate=validate, B=B)
    Nseq = d.num_seqs if cu_seqlens is not None else d.B
    if grads is None:
        f = dict(dtype=torch.float32, device=dev)
        grads = dict(dq=torch.empty(q.shape, **f), dk=torch.empty(k.shape, **f), dv=torch.empty(v.shape, **f),
                     dlog_alpha=torch.empty(log_alpha.shape, **f), dbeta=torch.empty(beta.shape, **f),
                     d_initial_state=(torch.empty(Nseq, d.H, d.dk, d.dv, **f) if want_d_initial_state else None))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.kda_chunk_bwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                           _ptr(initial_state), _ptr(cu_seqlens), _ptr(d_out), _ptr(d_final_state),
                           _ptr(grads["dq"]), _ptr(grads["dk"]), _ptr(grads["dv"]), _ptr(grads["dlog_alpha"]),
                           _ptr(grads["dbeta"]), _ptr(grads.get("d_initial_state")), _ptr(workspace), ws_bytes,
                           _stream_handle(stream, dev))
    _check(st, "kda_chunk_bwd")
    return grads


def kda_chunk_affine_pair(q, k, v, log_alpha, beta, cu_seqlens=None, pairs=None, *, B=None, validate=False,
                          stream=None):
    """The affine pair (S~, M) of each sequence of the call: returns pairs
    [2, N, H, dk, dv] fp32 with pairs[0] = S~ and pairs[1] = M."""
    lib = load()
    d = chunk_desc(q, v, cu_seqlens=cu_seqlens, gate_dtype=_dt(log_alpha), validate=validate, B=B)
    Nseq = d.num_seqs if cu_seqlens is not None else d.B
    if pairs is None:
        pairs = torch.empty(2, Nseq, d.H, d.dk, d.dv, dtype=torch.float32, device=q.device)
    st = lib.kda_chunk_affine_pair(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                   _ptr(cu_seqlens), _ptr(pairs), _stream_handle(stream, q.device))
    _check(st, "kda_chunk_affine_pair")
    return pairs


def kda_affine_compose(pairs, initial_state=None, entry_states=None, *, stream=None):
    """Entry states [N, P, H, dk, dv] of P consecutive segments from the pairs
    [2, N, P-1, H, dk, dv] of the first P-1 and the first entry state."""
    lib = load()
    _, N, Pm1, H, dk, dv = pairs.shape
    P = Pm1 + 1
    if entry_states is None:
        entry_states = torch.empty(N, P, H, dk, dv, dtype=torch.float32, device=pairs.device)
    st = lib.kda_affine_compose(N, H, dk, dv, P, _ptr(initial_state), _ptr(pairs) if Pm1 > 0 else None,
                                _ptr(entry_states), _stream_handle(stream, pairs.device))
    _check(st, "kda_affine_compose")
    return entry_states


# ------------------------------------------------ gated linear recurrence, norms
# These calls are short enough that marshalling shows, so each tensor is checked
# and turned into its address in one step, and descriptors are kept by their
# sizes and types.

WRITES = {"one": 0, "complement": 1}


def _stream_of(index):
    return torch.cuda.current_stream(index).cuda_stream


# Without the Python layers around them (0.4 us a call), where this build of torch has them: one without CUDA does not.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


def _arg(name, t, shape, dtype, index):
    """Address of an optional tensor, checked.  One without elements may have no
    address; the library reads nothing through it but refuses NULL, so it gets
    a non-null stand-in."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr() or 256
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on CUDA device {index}, not {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _new(t):
    """Address of a tensor that this call has just made."""
    return None if t is None else t.data_ptr() or 256


def _elsewhere(index, stream):
    """Whether a call has to be made on another device or stream than the current ones."""
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    return stream is not None or index != _current_device()


def _there(call, index, stream, tensors):
    """call() with `stream` (or device `index`) current, so that what it allocates
    belongs there.  On a side stream, every tensor of the call is kept from reuse
    until both streams are done with it."""
    if stream is None:
        with torch.cuda.device(index):
            return call()
    if stream.device.index != index:
        raise ValueError(f"the stream must be on CUDA device {index}, not {stream.device}")
    before = torch.cuda.current_stream(index)
    with torch.cuda.stream(stream):
        result = call()
    if stream != before:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        for t in result.values() if isinstance(result, dict) else result:
            if t is not None:
                t.record_stream(before)
                t.record_stream(stream)
    return result


class _Sized:
    """A descriptor, the pointer to it that calls take, and sizes that follow from it."""

    def __init__(self, desc):
        self.desc, self.ref, self.sizes = desc, ctypes.byref(desc), {}

    def size(self, fn, *args) -> int:
        key = (fn, *args)
        if key not in self.sizes:
            n = ctypes.c_size_t(0)
            _check(getattr(load(), fn)(self.ref, *args, ctypes.byref(n)), fn)
            self.sizes[key] = n.value
        return self.sizes[key]


@functools.lru_cache(maxsize=512)
def _scan_sized(*fields) -> _Sized:
    if max(fields) >= 1 << 31:  # (ctypes would cut it off)
        raise ValueError("a size passes 32 bits")
    return _Sized(KdaScanDesc(*fields))


@functools.lru_cache(maxsize=512)
def _norm_sized(rows, width, *rest) -> _Sized:
    if max(rows, width) >= 1 << 31:
        raise ValueError("a size passes 32 bits")
    return _Sized(KdaNormDesc(rows, width, *rest))


def _scan_call(x, decay, A_log, initial_state, cu_seqlens, write, B, validate):
    """The sized descriptor, the [N, H, d] state shape and the addresses of the
    inputs that every scan call has."""
    shape = x.shape
    if len(shape) == 3:
        tokens, H, d = shape
        batch = 1 if B is None else B
    elif len(shape) == 4:
        batch, T, H, d = shape
        tokens = batch * T
    else:
        raise ValueError("x must be [tokens, H, d] or [B, T, H, d]")
    if B is not None and (B != batch or B <= 0 or tokens % B):
        raise ValueError(f"{tokens} tokens are no batch of {B} sequences")
    if write not in WRITES:
        raise ValueError(f"write must be one of {sorted(WRITES)}")
    index, seqs, dt = x.get_device(), 0, x.dtype
    if cu_seqlens is not None:
        if batch != 1:
            raise ValueError("cu_seqlens needs B = 1")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be [N + 1] with N >= 1")
        seqs = cu_seqlens.numel() - 1
    sized = _scan_sized(batch, tokens // batch if batch else 0, H, d, seqs, _dt(x), _dt(decay), WRITES[write],
                        1 if validate else 0)
    state = (seqs or batch, H, d)
    return sized, state, (_arg("x", x, shape, dt, index),
                          _arg("decay", decay, shape, decay.dtype if A_log is None else dt, index),
                          _arg("A_log", A_log, (H,), torch.float32, index)), \
        _arg("initial_state", initial_state, state, torch.float32, index), \
        None if cu_seqlens is None else _arg("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, index)


def kda_scan_states_size(desc: KdaScanDesc) -> int:
    return _Sized(desc).size("kda_scan_states_size")


def kda_scan_fwd(x, decay, A_log=None, g_min=-5.0, initial_state=None, cu_seqlens=None, out=None, final_state=None,
                 states=None, *, write="one", validate=False, want_final_state=True, want_states=False, B=None,
                 stream=None):
    """Gated linear recurrence h_t = alpha_t h_{t-1} + w_t x_t through the C ABI.

    x, decay: [tokens, H, d] (or [B, T, H, d]); decay is log_alpha (fp32 or
    bf16), or with A_log ([H] fp32) the decay logits z in x's dtype;
    initial_state: [N, H, d] fp32 or None; write: "one" (w = 1) or
    "complement" (w = 1 - alpha).  Returns (out, final_state), and with
    want_states (or a `states` buffer) a third, the states for kda_scan_bwd."""
    lib = _lib or load()
    sized, state, ins, s0, cu = _scan_call(x, decay, A_log, initial_state, cu_seqlens, write, B, validate)
    index = x.get_device()
    if _elsewhere(index, stream):
        return _there(lambda: kda_scan_fwd(x, decay, A_log, g_min, initial_state, cu_seqlens, out, final_state, states,
                                           write=write, validate=validate, want_final_state=want_final_state,
                                           want_states=want_states, B=B),
                      index, stream, (x, decay, A_log, initial_state, cu_seqlens, out, final_state, states))
    given_out, given_final, kept = (_arg("out", out, x.shape, x.dtype, index),
                                    _arg("final_state", final_state, state, torch.float32, index), None)
    if out is None:
        out = torch.empty_like(x)
        given_out = _new(out)
    if final_state is None and want_final_state:
        final_state = (torch.empty(state, dtype=torch.float32, device=x.device) if initial_state is None
                       else torch.empty_like(initial_state))
        given_final = _new(final_state)
    if want_states or states is not None:
        n = sized.size("kda_scan_states_size") // 4
        if states is None:
            states = torch.empty(n, dtype=torch.float32, device=x.device)
            kept = _new(states)
        else:
            kept = _arg("states", states, (n,), torch.float32, index)
    st = lib.kda_scan_fwd(sized.ref, *ins, g_min, s0, cu, given_out, given_final, kept, _current_stream(index))
    if st:
        _check(st, "kda_scan_fwd")
    return (out, final_state) if states is None else (out, final_state, states)


def kda_scan_bwd(x, decay, d_out, A_log=None, g_min=-5.0, initial_state=None, d_final_state=None, cu_seqlens=None,
                 states=None, *, write="one", validate=False, want_d_initial_state=True, B=None, stream=None,
                 workspace=None, grads=None):
    """Gradients of kda_scan_fwd through the C ABI for
    L = sum <d_out, out> + <d_final_state, final_state>.

    states: what kda_scan_fwd(..., want_states=True) returned for the same
    arguments, or None (they are rebuilt).  Returns a dict: dx (x's dtype),
    d_decay (decay's dtype), dA_log ([H] fp32; None without A_log) and
    d_initial_state (fp32; None unless wanted).  Rows behind the last sequence
    of cu_seqlens are not written.  `grads` may pass that dict preallocated."""
    lib = _lib or load()
    sized, state, ins, s0, cu = _scan_call(x, decay, A_log, initial_state, cu_seqlens, write, B, validate)
    index, shape, f32 = x.get_device(), x.shape, torch.float32
    do = _arg("d_out", d_out, shape, x.dtype, index)
    dst = _arg("d_final_state", d_final_state, state, f32, index)
    if _elsewhere(index, stream):
        return _there(lambda: kda_scan_bwd(x, decay, d_out, A_log, g_min, initial_state, d_final_state, cu_seqlens,
                                           states, write=write, validate=validate,
                                           want_d_initial_state=want_d_initial_state, B=B, workspace=workspace,
                                           grads=grads),
                      index, stream, (x, decay, d_out, A_log, initial_state, d_final_state, cu_seqlens, states,
                                      workspace))
    kept = None
    if states is not None:
        kept = _arg("states", states, (sized.size("kda_scan_states_size") // 4,), f32, index)
    if grads is None:
        grads = {"dx": torch.empty_like(x), "d_decay": torch.empty_like(decay),
                 "dA_log": None if A_log is None else torch.empty_like(A_log),
                 "d_initial_state": (None if not want_d_initial_state else torch.empty_like(d_final_state)
                                     if d_final_state is not None else torch.empty(state, dtype=f32, device=x.device))}
        outs = [_new(t) for t in grads.values()]
    else:
        outs = (_arg("dx", grads["dx"], shape, x.dtype, index),
                _arg("d_decay", grads["d_decay"], shape, decay.dtype, index),
                _arg("dA_log", grads.get("dA_log"), state[1:2], f32, index),
                _arg("d_initial_state", grads.get("d_initial_state"), state, f32, index))
    if workspace is None:
        n = sized.size("kda_scan_bwd_workspace_size", int(A_log is not None), int(states is not None))
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    ws, ws_bytes = _workspace(workspace, index)
    st = lib.kda_scan_bwd(sized.ref, *ins, g_min, s0, cu, kept, do, dst, *outs, ws, ws_bytes, _current_stream(index))
    if st:
        _check(st, "kda_scan_bwd")
    return grads


def _workspace(t, index):
    if t is None:
        return None, 0
    return _arg("workspace", t, t.shape, t.dtype, index), t.numel() * t.element_size()


def kda_scan_step(x, decay, state_in, A_log=None, g_min=-5.0, state_out=None, out=None, *, write="one",
                  validate=False, stream=None):
    """One token of kda_scan_fwd for N sequences: x, decay [N, H, d], state_in
    [N, H, d] fp32.  The new state goes to state_out (None: in place of
    state_in).  Returns (out, state_out)."""
    lib = _lib or load()
    if x.dim() != 3 or x.shape[0] == 0:
        raise ValueError("x must be [N, H, d] with N >= 1")
    sized, state, ins, s0, _ = _scan_call(x, decay, A_log, state_in, None, write, x.shape[0], validate)
    index = x.get_device()
    if _elsewhere(index, stream):
        return _there(lambda: kda_scan_step(x, decay, state_in, A_log, g_min, state_out, out, write=write,
                                            validate=validate),
                      index, stream, (x, decay, state_in, A_log, state_out, out))
    if state_out is None:
        state_out, to = state_in, s0
    else:
        to = _arg("state_out", state_out, state, torch.float32, index)
    if out is None:
        out = torch.empty_like(x)
        given = _new(out)
    else:
        given = _arg("out", out, x.shape, x.dtype, index)
    st = lib.kda_scan_step(sized.ref, *ins, g_min, s0, to, given, _current_stream(index))
    if st:
        _check(st, "kda_scan_step")
    return out, state_out


def _norm_call(y, residual, gate, post_norm, post_weight, scale, pre_weight, post_eps, pre_eps):
    """The sized descriptor, out's dtype and the inputs' addresses."""
    shape = y.shape
    if not shape or shape[-1] < 1:
        raise ValueError("y must be [..., width] with width >= 1")
    index, width, dt = y.get_device(), shape[-1], y.dtype
    rdt = dt if residual is None else residual.dtype
    code = _dt(y)
    sized = _norm_sized(y.numel() // width, width, code, code if residual is None else _dt(residual),
                        1 if post_norm else 0, post_eps, pre_eps)
    row = shape[-1:]
    return sized, rdt, (_arg("y", y, shape, dt, index), _arg("residual", residual, shape, rdt, index),
                        _arg("gate", gate, shape, dt, index), _arg("post_weight", post_weight, row, torch.float32, index),
                        _arg("scale", scale, row, torch.float32, index),
                        _arg("pre_weight", pre_weight, row, torch.float32, index))


def kda_block_norm_fwd(y, residual=None, gate=None, *, post_norm=True, post_weight=None, scale=None, pre_weight=None,
                       post_eps=1e-6, pre_eps=1e-6, want_out=True, want_normed=False, out=None, normed=None,
                       stream=None):
    """Norms before and after a block through the C ABI, per row of y [..., width]:

        out    = residual + scale * sigmoid(gate) * RMSNorm(y; post_weight, post_eps)
        normed = RMSNorm(out; pre_weight, pre_eps)

    Every part is optional: post_norm=False leaves y as it is, None weights
    and scale are ones, no gate is 1, no residual is 0.  gate has y's dtype;
    residual (fp32 or bf16) sets out's.  Returns (out, normed), None for the
    one not wanted; out may be `residual` itself (update in place)."""
    lib = _lib or load()
    sized, rdt, ins = _norm_call(y, residual, gate, post_norm, post_weight, scale, pre_weight, post_eps, pre_eps)
    index, shape = y.get_device(), y.shape
    if _elsewhere(index, stream):
        return _there(lambda: kda_block_norm_fwd(y, residual, gate, post_norm=post_norm, post_weight=post_weight,
                                                 scale=scale, pre_weight=pre_weight, post_eps=post_eps,
                                                 pre_eps=pre_eps, want_out=want_out, want_normed=want_normed,
                                                 out=out, normed=normed),
                      index, stream, (y, residual, gate, post_weight, scale, pre_weight, out, normed))
    given_out, given_normed = _arg("out", out, shape, rdt, index), _arg("normed", normed, shape, y.dtype, index)
    if out is None and want_out:
        out = torch.empty_like(y if residual is None else residual)
        given_out = _new(out)
    if normed is None and want_normed:
        normed = torch.empty_like(y)
        given_normed = _new(normed)
    st = lib.kda_block_norm_fwd(sized.ref, *ins, given_out, given_normed, _current_stream(index))
    if st:
        _check(st, "kda_block_norm_fwd")
    return out, normed


def kda_block_norm_bwd(y, d_out, d_normed=None, residual=None, gate=None, *, post_norm=True, post_weight=None,
                       scale=None, pre_weight=None, post_eps=1e-6, pre_eps=1e-6, stream=None, workspace=None,
                       grads=None):
    """Gradients of kda_block_norm_fwd through the C ABI for
    L = <d_out, out> + <d_normed, normed> (either may be None).  Returns a dict:
    d_y, d_residual, d_gate in the dtypes of their tensors, d_post_weight,
    d_scale, d_pre_weight in fp32; None for each input that was not given.
    `grads` may pass that dict preallocated: then the entries it holds (d_y
    and, with a gate, d_gate are required) are written."""
    lib = _lib or load()
    sized, rdt, ins = _norm_call(y, residual, gate, post_norm, post_weight, scale, pre_weight, post_eps, pre_eps)
    index, shape, dt = y.get_device(), y.shape, y.dtype
    do = _arg("d_out", d_out, shape, rdt, index)
    dn = _arg("d_normed", d_normed, shape, dt, index)
    if _elsewhere(index, stream):
        return _there(lambda: kda_block_norm_bwd(y, d_out, d_normed, residual, gate, post_norm=post_norm,
                                                 post_weight=post_weight, scale=scale, pre_weight=pre_weight,
                                                 post_eps=post_eps, pre_eps=pre_eps, workspace=workspace, grads=grads),
                      index, stream, (y, d_out, d_normed, residual, gate, post_weight, scale, pre_weight, workspace))
    if grads is None:
        new = lambda like: None if like is None else torch.empty_like(like)  # noqa: E731
        grads = {"d_y": torch.empty_like(y), "d_residual": new(residual), "d_gate": new(gate),
                 "d_post_weight": new(post_weight), "d_scale": new(scale),
                 "d_pre_weight": None if d_normed is None else new(pre_weight)}
        outs = [_new(t) for t in grads.values()]
    else:
        get, row, f32 = grads.get, shape[-1:], torch.float32
        outs = [_arg("d_y", get("d_y"), shape, dt, index), _arg("d_residual", get("d_residual"), shape, rdt, index),
                _arg("d_gate", get("d_gate"), shape, dt, index)]
        outs += [_arg(n, get(n), row, f32, index) for n in ("d_post_weight", "d_scale", "d_pre_weight")]
    if workspace is None and any(outs[3:]):
        workspace = torch.empty(sized.size("kda_block_norm_bwd_workspace_size"), dtype=torch.uint8, device=y.device)
    ws, ws_bytes = _workspace(workspace, index)
    st = lib.kda_block_norm_bwd(sized.ref, *ins, do, dn, *outs, ws, ws_bytes, _current_stream(index))
    if st:
        _check(st, "kda_block_norm_bwd")
    return grads
