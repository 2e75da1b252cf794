"""Python binding of ``libgdn.so``, the gated delta rule (Gated DeltaNet) library for B200.

Argument marshalling only: every step of the computation runs in the library's CUDA kernels,
behind the C ABI declared in ``include/gdn.h``.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or a call fails, these functions raise.

Layouts (contiguous, last index fastest): q, k [B,T,Hk,dk]; v, o [B,T,Hv,dv]; log_alpha, beta
[B,T,Hv] fp32; states [B,Hv,dk,dv] fp32 holding S transposed (d_v contiguous).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

__all__ = ["GdnError", "lib", "library_path", "STATUS", "VARIANTS", "check_error",
           "chunk_fwd", "chunk_fwd_ba", "chunk_fwd_varlen", "chunk_fwd_variant",
           "chunk_fwd_workspace_bytes", "chunk_fwd_launches", "decode_step", "decode_layer_step",
           "gates", "gates_bwd", "prologue", "out_norm", "layer_fwd", "layer_fwd_varlen",
           "layer_fwd_static", "layer_workspace_bytes", "bwd", "bwd_varlen", "bwd_workspace_bytes",
           "bwd_launches", "layer_bwd", "layer_bwd_varlen", "layer_bwd_workspace_bytes",
           "ssm_conv", "ssm_conv_varlen", "ssm_scan", "ssm_scan_varlen",
           "ssm_scan_workspace_bytes", "ssm_step", "block_norm", "block_norm_bwd",
           "block_norm_bwd_workspace_bytes"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libgdn.so")
_lib = None

STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED", 3: "GDN_ERR_CUDA",
          4: "GDN_ERR_TIMEOUT"}
VARIANTS = {"auto": 0, "simt": 1, "tcgen05": 2}
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


class GdnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libgdn.so (built in-tree by ``__graft_entry__.build()``); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(_LIB_PATH)
        P, I, F, LL, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong, \
            ctypes.c_size_t
        L.gdn_status_string.argtypes = [I]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_version.argtypes = []
        L.gdn_version.restype = I
        L.gdn_check_error.argtypes = [P]
        L.gdn_check_error.restype = I
        L.gdn_chunk_fwd.argtypes = [P] * 9 + [SZ] + [I] * 7 + [F, I, I, P]
        L.gdn_chunk_fwd.restype = I
        L.gdn_chunk_fwd_ex.argtypes = [P] * 9 + [SZ] + [I] * 7 + [F, I, I, I, P]
        L.gdn_chunk_fwd_ex.restype = I
        L.gdn_chunk_fwd_ba.argtypes = [P] * 8 + [SZ] + [I] * 7 + [F, I, I, P]
        L.gdn_chunk_fwd_ba.restype = I
        L.gdn_chunk_fwd_workspace_bytes.argtypes = [I] * 8
        L.gdn_chunk_fwd_workspace_bytes.restype = SZ
        L.gdn_chunk_fwd_launches.argtypes = [I] * 10
        L.gdn_chunk_fwd_launches.restype = I
        L.gdn_chunk_fwd_varlen_workspace_bytes.argtypes = [I] * 8
        L.gdn_chunk_fwd_varlen_workspace_bytes.restype = SZ
        L.gdn_chunk_fwd_variant.argtypes = [I, I, I, I]
        L.gdn_chunk_fwd_variant.restype = I
        L.gdn_decode_step.argtypes = [P] * 7 + [I] * 5 + [F, I, I, P]
        L.gdn_decode_step.restype = I
        L.gdn_decode_layer_step.argtypes = [P] * 18 + [I] * 5 + [F, F, F, I, P]
        L.gdn_decode_layer_step.restype = I
        L.gdn_chunk_fwd_varlen.argtypes = [P] * 6 + [I, I] + [P] * 4 + [SZ] + [I] * 6 + \
            [F, I, I, P]
        L.gdn_chunk_fwd_varlen.restype = I
        L.gdn_gates.argtypes = [P, P, P, LL, I, I, P]
        L.gdn_gates.restype = I
        L.gdn_wait_timeout_selftest.argtypes = [LL, P]
        L.gdn_wait_timeout_selftest.restype = I
        L.gdn_prologue.argtypes = [P] * 9 + [I] * 6 + [F, I, P]
        L.gdn_prologue.restype = I
        L.gdn_prologue_ex.argtypes = [P] * 12 + [I] * 6 + [F, I, P]
        L.gdn_prologue_ex.restype = I
        L.gdn_out_norm.argtypes = [P, P, P, P, LL, I, F, I, P]
        L.gdn_out_norm.restype = I
        L.gdn_layer_fwd.argtypes = [P] * 14 + [SZ] + [I] * 7 + [F, F, F, I, I, P]
        L.gdn_layer_fwd.restype = I
        L.gdn_layer_fwd_ex.argtypes = [P] * 20 + [SZ] + [I] * 7 + [F, F, F, I, I, P]
        L.gdn_layer_fwd_ex.restype = I
        L.gdn_layer_fwd_varlen.argtypes = [P] * 5 + [I, I] + [P] * 16 + [SZ] + [I] * 6 + \
            [F, F, F, I, I, P]
        L.gdn_layer_fwd_varlen.restype = I
        L.gdn_layer_fwd_varlen_workspace_bytes.argtypes = [I] * 9
        L.gdn_layer_fwd_varlen_workspace_bytes.restype = SZ
        L.gdn_layer_workspace_bytes.argtypes = [I] * 7 + [I]
        L.gdn_layer_fwd_static.argtypes = [P] * 13 + [I] * 7 + [F, F, F, I, I, P]
        L.gdn_layer_fwd_static.restype = I
        L.gdn_layer_workspace_bytes.restype = SZ
        L.gdn_bwd.argtypes = [P] * 15 + [SZ] + [I] * 6 + [F, I, P]
        L.gdn_bwd.restype = I
        L.gdn_bwd_workspace_bytes.argtypes = [I] * 6
        L.gdn_bwd_varlen.argtypes = [P] * 6 + [I, I] + [P] * 10 + [SZ] + [I] * 5 + [F, I, P]
        L.gdn_bwd_varlen.restype = I
        L.gdn_bwd_varlen_workspace_bytes.argtypes = [I] * 7
        L.gdn_bwd_varlen_workspace_bytes.restype = SZ
        L.gdn_bwd_workspace_bytes.restype = SZ
        L.gdn_bwd_launches.argtypes = [I] * 6
        L.gdn_bwd_launches.restype = I
        L.gdn_layer_bwd.argtypes = [P] * 25 + [SZ] + [I] * 7 + [F, F, F, I, I, P]
        L.gdn_layer_bwd.restype = I
        L.gdn_layer_bwd_workspace_bytes.argtypes = [I] * 8
        L.gdn_layer_bwd_workspace_bytes.restype = SZ
        L.gdn_layer_bwd_varlen.argtypes = ([P] * 5 + [I, I] + [P] * 21 + [SZ] + [I] * 6 +
                                           [F, F, F, I, I, P])
        L.gdn_layer_bwd_varlen.restype = I
        L.gdn_layer_bwd_varlen_workspace_bytes.argtypes = [I] * 9
        L.gdn_layer_bwd_varlen_workspace_bytes.restype = SZ
        L.gdn_gates_bwd.argtypes = [P, P, P, P, LL, I, I, P]
        L.gdn_gates_bwd.restype = I
        L.gdn_ssm_conv.argtypes = [P, LL] + [P] * 5 + [I] * 4 + [P]
        L.gdn_ssm_conv_varlen.argtypes = [P, LL] + [P] * 3 + [I, I] + [P] * 3 + [I] * 3 + [P]
        L.gdn_ssm_scan.argtypes = [P, LL] * 5 + [P] * 7 + [SZ] + [I] * 7 + [P]
        L.gdn_ssm_scan_varlen.argtypes = [P, LL] * 5 + [P] * 4 + [I, I] + [P] * 4 + [SZ] + \
            [I] * 6 + [P]
        L.gdn_ssm_step.argtypes = [P, LL] * 3 + [P] * 9 + [I] * 6 + [P]
        L.gdn_block_norm.argtypes = [P] * 8 + [LL, I, F, I, I, P]
        L.gdn_block_norm_bwd.argtypes = [P] * 15 + [SZ, LL, I, F, I, I, P]
        for fn in (L.gdn_ssm_conv, L.gdn_ssm_conv_varlen, L.gdn_ssm_scan, L.gdn_ssm_scan_varlen,
                   L.gdn_ssm_step, L.gdn_block_norm, L.gdn_block_norm_bwd):
            fn.restype = I
        L.gdn_ssm_scan_workspace_bytes.argtypes = [I] * 7
        L.gdn_ssm_scan_workspace_bytes.restype = SZ
        L.gdn_ssm_scan_varlen_workspace_bytes.argtypes = [I] * 8
        L.gdn_ssm_scan_varlen_workspace_bytes.restype = SZ
        L.gdn_block_norm_bwd_workspace_bytes.argtypes = [LL, I]
        L.gdn_block_norm_bwd_workspace_bytes.restype = SZ
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _check(fn: str, status: int):
    if status != 0:
        raise GdnError(fn, status)


def _dev(*ts: Optional[torch.Tensor]) -> torch.device:
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("all tensors must be on one device")
    return dev


def _f32(*ts):
    for t in ts:
        if t is not None and t.dtype != torch.float32:
            raise ValueError("gates, states and weights must be float32")


def _io_dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return _DTYPES[t.dtype]


def chunk_fwd_variant(dk: int, dv: int, chunk: int, dtype: torch.dtype) -> str:
    """Which kernel family ``chunk_fwd`` runs for these sizes: 'simt' or 'tcgen05'."""
    v = lib().gdn_chunk_fwd_variant(dk, dv, chunk, _DTYPES[dtype])
    return {1: "simt", 2: "tcgen05"}[v]


def chunk_fwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, dtype) -> int:
    """Device scratch bytes ``chunk_fwd`` needs (0 for the CUDA-core family)."""
    return int(lib().gdn_chunk_fwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, _DTYPES[dtype]))


def chunk_fwd_launches(B, T, Hk, Hv, dk, dv, chunk, dtype, variant: str = "auto",
                       sms: int = 0) -> int:
    """Kernel launches of one ``chunk_fwd`` call (the library's own schedule decision) on a
    device of ``sms`` SMs, or on the current device when ``sms`` is 0."""
    n = lib().gdn_chunk_fwd_launches(B, T, Hk, Hv, dk, dv, chunk, _DTYPES[dtype],
                                     VARIANTS[variant], sms)
    if n < 0:
        raise ValueError("gdn_chunk_fwd_launches rejected the arguments")
    return n


def _workspace(need: int, dev, workspace: Optional[torch.Tensor]):
    """The caller-owned scratch of a call: the given tensor, or a fresh uint8 tensor from torch's
    allocator when none is given (torch's tensors are 256-byte aligned)."""
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    return workspace, workspace.numel() * workspace.element_size()


def chunk_fwd(q, k, v, log_alpha, beta, S0=None, *, chunk: int = 64, scale: float = 1.0,
              out: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
              want_state: bool = True, variant: str = "auto",
              out_dtype: Optional[torch.dtype] = None,
              workspace: Optional[torch.Tensor] = None
              ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked prefill forward: returns (o [B,T,Hv,dv], S_T [B,Hv,dk,dv] or None).  ``out_dtype``
    (default: q's dtype) may be float32 for bf16 inputs.  ``workspace``: a device uint8 tensor of
    at least ``chunk_fwd_workspace_bytes(...)`` bytes, else one is allocated for the call."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    if k.shape != q.shape or v.shape[:2] != (B, T) or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v shapes/dtypes disagree")
    if log_alpha.shape != (B, T, Hv) or beta.shape != (B, T, Hv):
        raise ValueError("gates must be [B, T, Hv]")
    _f32(log_alpha, beta, S0)
    odt = q.dtype if out_dtype is None else out_dtype
    o = torch.empty(v.shape, device=v.device, dtype=odt) if out is None else out
    sT = None
    if want_state:
        sT = torch.empty(B, Hv, dk, dv, device=q.device, dtype=torch.float32) \
            if state_out is None else state_out
    dev = _dev(q, k, v, log_alpha, beta, S0, o, sT, workspace)
    need = 0 if variant == "simt" else chunk_fwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk,
                                                                q.dtype)
    ws, wbytes = _workspace(need, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().gdn_chunk_fwd_ex(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(S0), _p(o),
                                    _p(sT), _p(ws), wbytes, B, T, Hk, Hv, dk, dv, chunk,
                                    float(scale), _io_dtype(q), _io_dtype(o), VARIANTS[variant],
                                    _stream(dev))
    _check("gdn_chunk_fwd", st)
    return o, sT


def bwd_workspace_bytes(B, T, Hk, Hv, dk, dv) -> int:
    """Caller-owned device scratch one ``bwd`` call needs."""
    return int(lib().gdn_bwd_workspace_bytes(B, T, Hk, Hv, dk, dv))


def bwd_launches(B, T, Hk, Hv, dk, dv) -> int:
    """Kernels one ``bwd`` call launches (the library's own count)."""
    n = lib().gdn_bwd_launches(B, T, Hk, Hv, dk, dv)
    if n < 0:
        raise ValueError("gdn_bwd_launches rejected the sizes")
    return n


def bwd(q, k, v, log_alpha, beta, S0, dO, dS_T=None, *, scale: float = 1.0,
        workspace: Optional[torch.Tensor] = None, want_dS0: bool = True) -> dict:
    """Gradients of sum <dO, o> + <dS_T, S_T> for the forward on the same inputs (gdn_bwd):
    fp32 dq, dk [B,T,Hk,dk] (summed over each key head's value heads), dv [B,T,Hv,dv],
    dlog_alpha, dbeta [B,T,Hv], dS0 [B,Hv,dk,dv] (None unless ``want_dS0``)."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    if (k.shape != q.shape or v.shape[:2] != (B, T) or dO.shape != v.shape
            or k.dtype != q.dtype or v.dtype != q.dtype or dO.dtype != q.dtype):
        raise ValueError("q, k, v, dO shapes/dtypes disagree")
    if log_alpha.shape != (B, T, Hv) or beta.shape != (B, T, Hv):
        raise ValueError("gates must be [B, T, Hv]")
    _f32(log_alpha, beta, S0, dS_T)
    f = dict(device=q.device, dtype=torch.float32)
    out = {"dq": torch.empty(B, T, Hk, dk, **f), "dk": torch.empty(B, T, Hk, dk, **f),
           "dv": torch.empty(B, T, Hv, dv, **f), "dlog_alpha": torch.empty(B, T, Hv, **f),
           "dbeta": torch.empty(B, T, Hv, **f),
           "dS0": torch.empty(B, Hv, dk, dv, **f) if want_dS0 else None}
    dev = _dev(q, k, v, log_alpha, beta, S0, dO, dS_T, workspace)
    ws, wbytes = _workspace(bwd_workspace_bytes(B, T, Hk, Hv, dk, dv), dev, workspace)
    with torch.cuda.device(dev):
        st = lib().gdn_bwd(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(S0), _p(dO),
                           _p(dS_T), _p(out["dq"]), _p(out["dk"]), _p(out["dv"]),
                           _p(out["dlog_alpha"]), _p(out["dbeta"]), _p(out["dS0"]), _p(ws),
                           wbytes, B, T, Hk, Hv, dk, dv, float(scale), _io_dtype(q),
                           _stream(dev))
    _check("gdn_bwd", st)
    return out


def bwd_varlen(q, k, v, log_alpha, beta, cu_seqlens, max_seqlen: int, S0, dO, dS_T=None, *,
               scale: float = 1.0) -> dict:
    """gdn_bwd over packed sequences (gdn_bwd_varlen): q, k [total, Hk, dk]; v, dO [total, Hv,
    dv]; gates [total, Hv]; cu_seqlens [nseq+1] int32 (device); S0, dS_T [nseq, Hv, dk, dv] or
    None.  Returns fp32 dq, dk [total, Hk, dk], dv [total, Hv, dv], dlog_alpha, dbeta [total, Hv],
    dS0 [nseq, Hv, dk, dv]."""
    total, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    nseq = cu_seqlens.numel() - 1
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    _f32(log_alpha, beta, S0, dS_T)
    f = dict(device=q.device, dtype=torch.float32)
    out = {"dq": torch.empty(total, Hk, dk, **f), "dk": torch.empty(total, Hk, dk, **f),
           "dv": torch.empty(total, Hv, dv, **f), "dlog_alpha": torch.empty(total, Hv, **f),
           "dbeta": torch.empty(total, Hv, **f), "dS0": torch.empty(nseq, Hv, dk, dv, **f)}
    dev = _dev(q, k, v, log_alpha, beta, cu_seqlens, S0, dO, dS_T)
    need = int(lib().gdn_bwd_varlen_workspace_bytes(nseq, int(max_seqlen), total, Hk, Hv, dk, dv))
    ws = torch.empty(max(need, 1), device=dev, dtype=torch.uint8)
    with torch.cuda.device(dev):
        st = lib().gdn_bwd_varlen(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(cu_seqlens),
                                  nseq, int(max_seqlen), _p(S0), _p(dO), _p(dS_T), _p(out["dq"]),
                                  _p(out["dk"]), _p(out["dv"]), _p(out["dlog_alpha"]),
                                  _p(out["dbeta"]), _p(out["dS0"]), _p(ws), need, total, Hk, Hv,
                                  dk, dv, float(scale), _io_dtype(q), _stream(dev))
    _check("gdn_bwd_varlen", st)
    return out


def chunk_fwd_ba(q, k, v, ba, S0=None, *, chunk: int = 64, scale: float = 1.0,
                 out: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
                 want_state: bool = True, out_dtype: Optional[torch.dtype] = None,
                 workspace: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``chunk_fwd`` with the gates computed from the in_proj_ba outputs ``ba`` [B,T,2*Hv] bf16
    (b then a): beta = sigmoid(b), log alpha = log sigmoid(a), inside the tensor-core pre-pass."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    if (k.shape != q.shape or v.shape[:2] != (B, T) or ba.shape != (B, T, 2 * Hv)
            or ba.dtype != torch.bfloat16):
        raise ValueError("q, k, v, ba shapes/dtypes disagree")
    _f32(S0)
    odt = q.dtype if out_dtype is None else out_dtype
    o = torch.empty(v.shape, device=v.device, dtype=odt) if out is None else out
    sT = None
    if want_state:
        sT = torch.empty(B, Hv, dk, dv, device=q.device, dtype=torch.float32) \
            if state_out is None else state_out
    dev = _dev(q, k, v, ba, S0, o, sT, workspace)
    need = chunk_fwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, q.dtype)
    ws, wbytes = _workspace(need, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().gdn_chunk_fwd_ba(_p(q), _p(k), _p(v), _p(ba), _p(S0), _p(o), _p(sT), _p(ws),
                                    wbytes, B, T, Hk, Hv, dk, dv, chunk, float(scale),
                                    _io_dtype(q), _io_dtype(o), _stream(dev))
    _check("gdn_chunk_fwd_ba", st)
    return o, sT


def decode_step(q, k, v, log_alpha, beta, S, *, scale: float = 1.0,
                out: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """One decode step: q,k [N,Hk,dk]; v [N,Hv,dv]; gates [N,Hv]; S [N,Hv,dk,dv] updated in
    place.  Returns o [N,Hv,dv] (``out_dtype``, default v's dtype; float32 for bf16 inputs)."""
    N, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    if k.shape != q.shape or v.shape[0] != N or S.shape != (N, Hv, dk, dv):
        raise ValueError("decode shapes disagree")
    _f32(log_alpha, beta, S)
    odt = v.dtype if out_dtype is None else out_dtype
    o = torch.empty(v.shape, device=v.device, dtype=odt) if out is None else out
    dev = _dev(q, k, v, log_alpha, beta, S, o)
    with torch.cuda.device(dev):
        st = lib().gdn_decode_step(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta), _p(S), _p(o),
                                   N, Hk, Hv, dk, dv, float(scale), _io_dtype(q), _io_dtype(o),
                                   _stream(dev))
    _check("gdn_decode_step", st)
    return o


def decode_layer_step(q_raw, k_raw, v_raw, z, hq_in, hk_in, hv_in, hq_out, hk_out, hv_out,
                      wq, wk, wv, log_alpha, beta, S, norm_w, *, Hk: int, Hv: int, dk: int,
                      dv: int, scale: float = 1.0, l2_eps: float = 1e-6, norm_eps: float = 1e-5,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One full-layer decode step (conv over the carried history + SiLU + L2, recurrence step
    with S updated in place, gated RMSNorm) in one kernel.  q_raw, k_raw [N,Hk*dk]; v_raw, z
    [N,Hv*dv]; histories [N,3,channels] (the _out set receives the moved-on history); conv taps
    [channels,4]; gates [N,Hv]; S [N,Hv,dk,dv]; norm_w [dv].  Returns y [N,Hv,dv]."""
    N = q_raw.shape[0]
    if (k_raw.shape != q_raw.shape or q_raw.shape[1] != Hk * dk or v_raw.shape != (N, Hv * dv)
            or z.shape != v_raw.shape or hq_in.shape != (N, 3, Hk * dk)
            or hk_in.shape != hq_in.shape or hv_in.shape != (N, 3, Hv * dv)
            or hq_out.shape != hq_in.shape or hk_out.shape != hk_in.shape
            or hv_out.shape != hv_in.shape or S.shape != (N, Hv, dk, dv)):
        raise ValueError("decode-layer shapes disagree")
    _f32(wq, wk, wv, log_alpha, beta, S, norm_w)
    y = torch.empty(N, Hv, dv, device=q_raw.device, dtype=q_raw.dtype) if out is None else out
    dev = _dev(q_raw, k_raw, v_raw, z, hq_in, hk_in, hv_in, hq_out, hk_out, hv_out, wq, wk, wv,
               log_alpha, beta, S, norm_w, y)
    with torch.cuda.device(dev):
        st = lib().gdn_decode_layer_step(
            _p(q_raw), _p(k_raw), _p(v_raw), _p(z), _p(hq_in), _p(hk_in), _p(hv_in), _p(hq_out),
            _p(hk_out), _p(hv_out), _p(wq), _p(wk), _p(wv), _p(log_alpha), _p(beta), _p(S),
            _p(norm_w), _p(y), N, Hk, Hv, dk, dv, float(scale), float(l2_eps), float(norm_eps),
            _io_dtype(q_raw), _stream(dev))
    _check("gdn_decode_layer_step", st)
    return y


def chunk_fwd_varlen(q, k, v, log_alpha, beta, cu_seqlens, max_seqlen: int, S0=None, *,
                     chunk: int = 64, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                     want_state: bool = True, out_dtype: Optional[torch.dtype] = None,
                     workspace: Optional[torch.Tensor] = None
                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Packed sequences: q,k [total,Hk,dk]; v [total,Hv,dv]; gates [total,Hv]; cu_seqlens
    [nseq+1] int32 on the device; S0 [nseq,Hv,dk,dv] or None.  Returns (o [total,Hv,dv],
    S_T [nseq,Hv,dk,dv] or None)."""
    total, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    nseq = cu_seqlens.numel() - 1
    if (k.shape != q.shape or v.shape[0] != total or log_alpha.shape != (total, Hv)
            or beta.shape != log_alpha.shape or cu_seqlens.dtype != torch.int32 or nseq < 0):
        raise ValueError("packed shapes disagree")
    _f32(log_alpha, beta)
    odt = q.dtype if out_dtype is None else out_dtype
    o = torch.empty(v.shape, device=v.device, dtype=odt) if out is None else out
    sT = (torch.empty(nseq, Hv, dk, dv, device=q.device, dtype=torch.float32)
          if want_state else None)
    dev = _dev(q, k, v, log_alpha, beta, cu_seqlens, o, workspace)
    need = int(lib().gdn_chunk_fwd_varlen_workspace_bytes(nseq, int(max_seqlen), Hk, Hv, dk, dv,
                                                          chunk, _DTYPES[q.dtype]))
    ws, wbytes = _workspace(need, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().gdn_chunk_fwd_varlen(_p(q), _p(k), _p(v), _p(log_alpha), _p(beta),
                                        _p(cu_seqlens), nseq, int(max_seqlen), _p(S0), _p(o),
                                        _p(sT), _p(ws), wbytes, total, Hk, Hv, dk, dv, chunk,
                                        float(scale), _io_dtype(q), _io_dtype(o), _stream(dev))
    _check("gdn_chunk_fwd_varlen", st)
    return o, sT


def gates(ba, Hv: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """in_proj_ba outputs [..., 2*Hv] (b then a) -> (log_alpha, beta) [..., Hv] fp32:
    beta = sigmoid(b), log alpha = -softplus(-a)."""
    if ba.shape[-1] != 2 * Hv:
        raise ValueError("ba must end in 2*Hv values")
    rows = ba.numel() // (2 * Hv)
    log_alpha = torch.empty(ba.shape[:-1] + (Hv,), device=ba.device, dtype=torch.float32)
    beta = torch.empty_like(log_alpha)
    dev = _dev(ba, log_alpha, beta)
    with torch.cuda.device(dev):
        st = lib().gdn_gates(_p(ba), _p(log_alpha), _p(beta), rows, Hv, _io_dtype(ba),
                             _stream(dev))
    _check("gdn_gates", st)
    return log_alpha, beta


def _hist_shapes(B, Hk, Hv, dk, dv, hist):
    """Check a conv history (hq, hk, hv) of [B, 3, Hk*dk], [B, 3, Hk*dk], [B, 3, Hv*dv]."""
    if hist is None:
        return (None, None, None)
    hq, hk, hv = hist
    if hq.shape != (B, 3, Hk * dk) or hk.shape != hq.shape or hv.shape != (B, 3, Hv * dv):
        raise ValueError("conv history shapes disagree")
    return hq, hk, hv


def prologue(q_raw, k_raw, v_raw, wq, wk, wv, Hk: int, Hv: int, dk: int, dv: int,
             l2_eps: float = 1e-6, hist=None):
    """Conv(4 taps) + SiLU + L2-normalisation of q/k heads.  Returns (q, k, v) shaped
    [B,T,Hk,dk], [B,T,Hk,dk], [B,T,Hv,dv].  ``hist`` (optional): the raw inputs (hq, hk, hv) of
    the three tokens before, [B,3,Hk*dk], [B,3,Hk*dk], [B,3,Hv*dv], oldest first."""
    B, T = q_raw.shape[:2]
    _f32(wq, wk, wv)
    hq, hk, hv = _hist_shapes(B, Hk, Hv, dk, dv, hist)
    q = torch.empty(B, T, Hk, dk, device=q_raw.device, dtype=q_raw.dtype)
    k = torch.empty_like(q)
    v = torch.empty(B, T, Hv, dv, device=q_raw.device, dtype=q_raw.dtype)
    dev = _dev(q_raw, k_raw, v_raw, wq, wk, wv, q, k, v, hq, hk, hv)
    with torch.cuda.device(dev):
        st = lib().gdn_prologue_ex(_p(q_raw), _p(k_raw), _p(v_raw), _p(hq), _p(hk), _p(hv),
                                   _p(wq), _p(wk), _p(wv), _p(q), _p(k), _p(v), B, T, Hk, Hv, dk,
                                   dv, float(l2_eps), _io_dtype(q_raw), _stream(dev))
    _check("gdn_prologue_ex", st)
    return q, k, v


def out_norm(o, z, w, eps: float = 1e-5) -> torch.Tensor:
    """y = RMSNorm(o) * w * SiLU(z) over the last dimension."""
    if z.shape != o.shape or z.dtype != o.dtype:
        raise ValueError("o and z must agree")
    _f32(w)
    dv = o.shape[-1]
    y = torch.empty_like(o)
    dev = _dev(o, z, w, y)
    with torch.cuda.device(dev):
        st = lib().gdn_out_norm(_p(o), _p(z), _p(w), _p(y), o.numel() // dv, dv, float(eps),
                                _io_dtype(o), _stream(dev))
    _check("gdn_out_norm", st)
    return y


def layer_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, dtype) -> int:
    return int(lib().gdn_layer_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, _DTYPES[dtype]))


def layer_fwd(q_raw, k_raw, v_raw, z, wq, wk, wv, log_alpha, beta, S0, norm_w, *, Hk: int,
              Hv: int, dk: int, dv: int, chunk: int = 64, scale: float = 1.0,
              l2_eps: float = 1e-6, norm_eps: float = 1e-5, want_state: bool = True,
              workspace: Optional[torch.Tensor] = None,
              out_dtype: Optional[torch.dtype] = None, hist=None, want_hist: bool = False):
    """Whole layer between the projections: returns (y [B,T,Hv,dv], S_T or None); y in
    ``out_dtype`` (default the inputs' dtype; float32 for bf16 inputs).  ``hist`` (optional): the
    raw inputs (hq, hk, hv) of the three tokens before this call, [B,3,Hk*dk], [B,3,Hk*dk],
    [B,3,Hv*dv], oldest first.  With ``want_hist`` the history after the call is returned too:
    (y, S_T, (hq, hk, hv))."""
    B, T = q_raw.shape[:2]
    _f32(wq, wk, wv, log_alpha, beta, S0, norm_w)
    hq, hk, hv = _hist_shapes(B, Hk, Hv, dk, dv, hist)
    y = torch.empty(B, T, Hv, dv, device=q_raw.device, dtype=out_dtype or q_raw.dtype)
    sT = torch.empty(B, Hv, dk, dv, device=q_raw.device, dtype=torch.float32) \
        if want_state else None
    ho = (None, None, None)
    if want_hist:
        ho = (torch.empty(B, 3, Hk * dk, device=q_raw.device, dtype=q_raw.dtype),
              torch.empty(B, 3, Hk * dk, device=q_raw.device, dtype=q_raw.dtype),
              torch.empty(B, 3, Hv * dv, device=q_raw.device, dtype=q_raw.dtype))
    need = layer_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, q_raw.dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=q_raw.device, dtype=torch.uint8)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    dev = _dev(q_raw, k_raw, v_raw, z, wq, wk, wv, log_alpha, beta, S0, norm_w, y, sT, hq, hk,
               hv, *ho)
    with torch.cuda.device(dev):
        st = lib().gdn_layer_fwd_ex(_p(q_raw), _p(k_raw), _p(v_raw), _p(z), _p(hq), _p(hk),
                                    _p(hv), _p(wq), _p(wk), _p(wv), _p(log_alpha), _p(beta),
                                    _p(S0), _p(norm_w), _p(y), _p(sT), _p(ho[0]), _p(ho[1]),
                                    _p(ho[2]), _p(workspace), wbytes, B, T, Hk, Hv, dk, dv, chunk,
                                    float(scale), float(l2_eps), float(norm_eps),
                                    _io_dtype(q_raw), _io_dtype(y), _stream(dev))
    _check("gdn_layer_fwd_ex", st)
    if want_hist:
        return y, sT, ho
    return y, sT


def layer_fwd_varlen(q_raw, k_raw, v_raw, z, cu_seqlens, max_seqlen: int, wq, wk, wv,
                     log_alpha, beta, S0, norm_w, *, Hk: int, Hv: int, dk: int, dv: int,
                     chunk: int = 64, scale: float = 1.0, l2_eps: float = 1e-6,
                     norm_eps: float = 1e-5, hist=None, want_hist: bool = False,
                     out_dtype: Optional[torch.dtype] = None):
    """The layer over packed requests: raw q, k [total, Hk*dk], v, z [total, Hv*dv], gates
    [total, Hv], cu_seqlens [nseq+1] int32 (device), S0 [nseq, Hv, dk, dv] or None, ``hist``
    (hq, hk, hv) [nseq, 3, C] or None.  Returns (y [total, Hv, dv], S_T) and, with
    ``want_hist``, the histories after the call."""
    total = q_raw.shape[0]
    nseq = cu_seqlens.numel() - 1
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    _f32(wq, wk, wv, log_alpha, beta, S0, norm_w)
    hq, hk, hv = _hist_shapes(nseq, Hk, Hv, dk, dv, hist)
    dev = q_raw.device
    y = torch.empty(total, Hv, dv, device=dev, dtype=out_dtype or q_raw.dtype)
    sT = torch.empty(nseq, Hv, dk, dv, device=dev, dtype=torch.float32)
    ho = (None, None, None)
    if want_hist:
        ho = (torch.empty(nseq, 3, Hk * dk, device=dev, dtype=q_raw.dtype),
              torch.empty(nseq, 3, Hk * dk, device=dev, dtype=q_raw.dtype),
              torch.empty(nseq, 3, Hv * dv, device=dev, dtype=q_raw.dtype))
    need = int(lib().gdn_layer_fwd_varlen_workspace_bytes(nseq, max_seqlen, total, Hk, Hv, dk, dv,
                                                          chunk, _DTYPES[q_raw.dtype]))
    ws = torch.empty(max(need, 1), device=dev, dtype=torch.uint8)
    d = _dev(q_raw, k_raw, v_raw, z, cu_seqlens, wq, wk, wv, log_alpha, beta, S0, norm_w, y, sT,
             hq, hk, hv, *ho)
    with torch.cuda.device(d):
        st = lib().gdn_layer_fwd_varlen(
            _p(q_raw), _p(k_raw), _p(v_raw), _p(z), _p(cu_seqlens), nseq, int(max_seqlen), _p(hq),
            _p(hk), _p(hv), _p(wq), _p(wk), _p(wv), _p(log_alpha), _p(beta), _p(S0), _p(norm_w),
            _p(y), _p(sT), _p(ho[0]), _p(ho[1]), _p(ho[2]), _p(ws), need, total, Hk, Hv, dk, dv,
            chunk, float(scale), float(l2_eps), float(norm_eps), _io_dtype(q_raw), _io_dtype(y),
            _stream(d))
    _check("gdn_layer_fwd_varlen", st)
    if want_hist:
        return y, sT, ho
    return y, sT


def layer_bwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, dtype) -> int:
    return int(lib().gdn_layer_bwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, _DTYPES[dtype]))


def layer_bwd(q_raw, k_raw, v_raw, z, wq, wk, wv, log_alpha, beta, S0, norm_w, dy, dS_T=None, *,
              Hk: int, Hv: int, dk: int, dv: int, chunk: int = 64, scale: float = 1.0,
              l2_eps: float = 1e-6, norm_eps: float = 1e-5, want_dS0: bool = True,
              workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of <dy, y> + <dS_T, S_T> for layer_fwd's inputs and weights (gdn_layer_bwd):
    fp32 dq_raw, dk_raw, dv_raw, dz, dwq, dwk, dwv, dlog_alpha, dbeta, dS0, dnorm_w."""
    B, T = q_raw.shape[:2]
    _f32(wq, wk, wv, log_alpha, beta, S0, norm_w, dS_T)
    f = dict(device=q_raw.device, dtype=torch.float32)
    out = {"dq_raw": torch.empty(q_raw.shape, **f), "dk_raw": torch.empty(k_raw.shape, **f),
           "dv_raw": torch.empty(v_raw.shape, **f), "dz": torch.empty(z.shape, **f),
           "dwq": torch.empty(wq.shape, **f), "dwk": torch.empty(wk.shape, **f),
           "dwv": torch.empty(wv.shape, **f), "dlog_alpha": torch.empty(log_alpha.shape, **f),
           "dbeta": torch.empty(beta.shape, **f),
           "dS0": torch.empty(B, Hv, dk, dv, **f) if want_dS0 else None,
           "dnorm_w": torch.empty(norm_w.shape, **f)}
    dev = _dev(q_raw, k_raw, v_raw, z, wq, wk, wv, log_alpha, beta, S0, norm_w, dy, dS_T,
               workspace)
    ws, wbytes = _workspace(layer_bwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, q_raw.dtype),
                            dev, workspace)
    with torch.cuda.device(dev):
        st = lib().gdn_layer_bwd(
            _p(q_raw), _p(k_raw), _p(v_raw), _p(z), _p(wq), _p(wk), _p(wv), _p(log_alpha),
            _p(beta), _p(S0), _p(norm_w), _p(dy), _p(dS_T), _p(out["dq_raw"]), _p(out["dk_raw"]),
            _p(out["dv_raw"]), _p(out["dz"]), _p(out["dwq"]), _p(out["dwk"]), _p(out["dwv"]),
            _p(out["dlog_alpha"]), _p(out["dbeta"]), _p(out["dS0"]), _p(out["dnorm_w"]), _p(ws),
            wbytes, B, T, Hk, Hv, dk, dv, chunk, float(scale), float(l2_eps), float(norm_eps),
            _io_dtype(q_raw), _io_dtype(dy), _stream(dev))
    _check("gdn_layer_bwd", st)
    return out


def layer_bwd_varlen(q_raw, k_raw, v_raw, z, cu_seqlens, max_seqlen: int, wq, wk, wv,
                     log_alpha, beta, S0, norm_w, dy, dS_T=None, *, Hk: int, Hv: int, dk: int,
                     dv: int, chunk: int = 64, scale: float = 1.0, l2_eps: float = 1e-6,
                     norm_eps: float = 1e-5, want_dS0: bool = True) -> dict:
    """layer_bwd over packed sequences (gdn_layer_bwd_varlen), laid out as layer_fwd_varlen's
    inputs (no carried history): the same fp32 gradients, token tensors [total, ...] and dS0
    [nseq, Hv, dk, dv]."""
    total = q_raw.shape[0]
    nseq = cu_seqlens.numel() - 1
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    _f32(wq, wk, wv, log_alpha, beta, S0, norm_w, dS_T)
    f = dict(device=q_raw.device, dtype=torch.float32)
    out = {"dq_raw": torch.empty(q_raw.shape, **f), "dk_raw": torch.empty(k_raw.shape, **f),
           "dv_raw": torch.empty(v_raw.shape, **f), "dz": torch.empty(z.shape, **f),
           "dwq": torch.empty(wq.shape, **f), "dwk": torch.empty(wk.shape, **f),
           "dwv": torch.empty(wv.shape, **f), "dlog_alpha": torch.empty(log_alpha.shape, **f),
           "dbeta": torch.empty(beta.shape, **f),
           "dS0": torch.empty(nseq, Hv, dk, dv, **f) if want_dS0 else None,
           "dnorm_w": torch.empty(norm_w.shape, **f)}
    need = int(lib().gdn_layer_bwd_varlen_workspace_bytes(nseq, int(max_seqlen), total, Hk, Hv,
                                                          dk, dv, chunk, _DTYPES[q_raw.dtype]))
    dev = _dev(q_raw, k_raw, v_raw, z, cu_seqlens, wq, wk, wv, log_alpha, beta, S0, norm_w, dy,
               dS_T)
    ws = torch.empty(max(need, 1), device=dev, dtype=torch.uint8)
    with torch.cuda.device(dev):
        st = lib().gdn_layer_bwd_varlen(
            _p(q_raw), _p(k_raw), _p(v_raw), _p(z), _p(cu_seqlens), nseq, int(max_seqlen),
            _p(wq), _p(wk), _p(wv), _p(log_alpha), _p(beta), _p(S0), _p(norm_w), _p(dy),
            _p(dS_T), _p(out["dq_raw"]), _p(out["dk_raw"]), _p(out["dv_raw"]), _p(out["dz"]),
            _p(out["dwq"]), _p(out["dwk"]), _p(out["dwv"]), _p(out["dlog_alpha"]),
            _p(out["dbeta"]), _p(out["dS0"]), _p(out["dnorm_w"]), _p(ws), need, total, Hk, Hv,
            dk, dv, chunk, float(scale), float(l2_eps), float(norm_eps), _io_dtype(q_raw),
            _io_dtype(dy), _stream(dev))
    _check("gdn_layer_bwd_varlen", st)
    return out


def gates_bwd(ba, dlog_alpha, dbeta) -> torch.Tensor:
    """Gradient [..., 2*Hv] fp32 of <dlog_alpha, log alpha> + <dbeta, beta> through gates(ba)."""
    Hv = ba.shape[-1] // 2
    rows = ba.numel() // (2 * Hv)
    _f32(dlog_alpha, dbeta)
    dba = torch.empty(ba.shape, device=ba.device, dtype=torch.float32)
    dev = _dev(ba, dlog_alpha, dbeta, dba)
    with torch.cuda.device(dev):
        st = lib().gdn_gates_bwd(_p(ba), _p(dlog_alpha), _p(dbeta), _p(dba), rows, Hv,
                                 _io_dtype(ba), _stream(dev))
    _check("gdn_gates_bwd", st)
    return dba


def layer_fwd_static(q_raw, k_raw, v_raw, z, wq, wk, wv, log_alpha, beta, S0, norm_w, *,
                     Hk: int, Hv: int, dk: int, dv: int, chunk: int = 64, scale: float = 1.0,
                     l2_eps: float = 1e-6, norm_eps: float = 1e-5, want_state: bool = True,
                     out_dtype: Optional[torch.dtype] = None):
    """layer_fwd with the library's built-in device scratch instead of a workspace (see
    gdn_layer_fwd_static in gdn.h: at most GDN_LAYER_STATIC_SCRATCH_BYTES of scratch, and calls
    on one device must not overlap on the GPU)."""
    B, T = q_raw.shape[:2]
    _f32(wq, wk, wv, log_alpha, beta, S0, norm_w)
    y = torch.empty(B, T, Hv, dv, device=q_raw.device, dtype=out_dtype or q_raw.dtype)
    sT = torch.empty(B, Hv, dk, dv, device=q_raw.device, dtype=torch.float32) \
        if want_state else None
    dev = _dev(q_raw, k_raw, v_raw, z, wq, wk, wv, log_alpha, beta, S0, norm_w, y, sT)
    with torch.cuda.device(dev):
        st = lib().gdn_layer_fwd_static(_p(q_raw), _p(k_raw), _p(v_raw), _p(z), _p(wq), _p(wk),
                                        _p(wv), _p(log_alpha), _p(beta), _p(S0), _p(norm_w),
                                        _p(y), _p(sT), B, T, Hk, Hv, dk, dv, chunk, float(scale),
                                        float(l2_eps), float(norm_eps), _io_dtype(q_raw),
                                        _io_dtype(y), _stream(dev))
    _check("gdn_layer_fwd_static", st)
    return y, sT


def check_error(device: Optional[torch.device] = None):
    """Synchronise the current stream and raise if a kernel recorded a timed-out wait."""
    dev = device or torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check("gdn_check_error", lib().gdn_check_error(_stream(dev)))


# ------------------------------------------------------------------------------------------------
# selective state space block
# ------------------------------------------------------------------------------------------------
# These calls also serve single tokens, where the host's time is the call's: their checks look at sizes
# and strides as plain tuples and at devices as plain numbers.
def _on(*ts: Optional[torch.Tensor]) -> int:
    """The one CUDA device (its number) of the tensors, any layout."""
    devs = {t.get_device() for t in ts if t is not None}
    dev = devs.pop()
    if dev < 0 or -1 in devs:
        raise ValueError("all tensors must be CUDA tensors")
    if devs:
        raise ValueError("all tensors must be on one device")
    return dev


def _dense(*ts: Optional[torch.Tensor]):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("states, histories, weights, offsets, outputs and norm inputs must be contiguous")


def _fp32(*ts: Optional[torch.Tensor]):
    for t in ts:
        if t is not None and t.dtype is not torch.float32:
            raise ValueError("gates, states and weights must be float32")


def _fit(*sizes: int):
    """Sizes that the C ABI takes as ints (ctypes would cut them to 32 bits without a word)."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError("sizes must be below 2^31")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _row_ld(t: Optional[torch.Tensor], lead: int, name: str) -> int:
    """Values between two tokens of ``t`` [tokens..., inner...] (``lead`` token dimensions), whose
    tokens are evenly spaced and whose inner dimensions lie without gaps: a slice of the columns of
    a contiguous tensor, or a contiguous tensor."""
    if t is None:
        return 0
    stride, shape = t.stride(), t.shape
    ld = stride[lead - 1]
    if stride[-1] == 1 and (lead == 1 or stride[0] == ld * shape[1]):      # the usual layouts
        if len(shape) == lead + 1:
            if ld >= shape[-1]:
                return ld
        elif stride[-2] == shape[-1] and len(shape) == lead + 2 and ld >= shape[-1] * shape[-2]:
            return ld
    want = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if stride[i] != want and shape[i] > 1:
            raise ValueError(f"{name}: the values of a token must be contiguous")
        want *= shape[i]
    if lead == 1:
        ld = stride[0] if shape[0] > 1 else max(want, 1)
    else:
        ld, span = max(want, 1), None
        for i in range(lead - 1, -1, -1):
            if shape[i] > 1:
                if span is None:
                    ld = span = stride[i]
                elif stride[i] != span:
                    raise ValueError(f"{name}: the tokens must be evenly spaced")
            if span is not None:
                span *= shape[i]
    if ld < want:
        raise ValueError(f"{name}: the tokens overlap")
    return ld


def _call(name: str, dev: int, *args):
    """Call the library on the current stream of device ``dev`` (made current where it is not)."""
    fn = getattr(_lib or lib(), name)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        raise GdnError(name, status)


def _conv(x, lead, w, bias, hist, nseq, want_hist, out, cu=None):
    C = x.shape[-1]
    _fit(*x.shape)
    if w.shape != (C, 4) or (bias is not None and bias.shape != (C,)):
        raise ValueError("w must be [C, 4] and bias [C]")
    if hist is not None and (hist.shape != (nseq, 3, C) or hist.dtype != x.dtype):
        raise ValueError("hist must be [sequences, 3, C] in x's dtype")
    if out is not None and (out.shape != x.shape or out.dtype != x.dtype):
        raise ValueError("out must have x's shape and dtype")
    _fp32(w, bias)
    io = _io_dtype(x)
    _dense(w, bias, hist, out)
    ld = _row_ld(x, lead, "x")
    dev = _on(x, w, bias, hist, out, cu)
    if out is None:
        out = x.new_empty(x.shape)
    hist_out = x.new_empty((nseq, 3, C)) if want_hist else None
    return out, hist_out, ld, io, dev


def ssm_conv(x, w, bias=None, *, hist=None, want_hist: bool = False,
             out: Optional[torch.Tensor] = None):
    """Short causal convolution of the state space block, then SiLU: x [B,T,C] (a slice of a wider
    row may be given), w [C,4] (tap 3 on the current token), bias [C] or None, ``hist`` [B,3,C] the
    raw rows before (None: zeros).  Returns out [B,T,C], or (out, hist_out) with ``want_hist``."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    B, T, C = x.shape
    out, hist_out, ld, io, dev = _conv(x, 2, w, bias, hist, B, want_hist, out)
    _call("gdn_ssm_conv", dev, x.data_ptr(), ld, w.data_ptr(), _ptr(bias), _ptr(hist), out.data_ptr(),
          _ptr(hist_out), B, T, C, io)
    return (out, hist_out) if want_hist else out


def _offsets(cu_seqlens) -> int:
    if cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 \
            or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous int32 [nseq + 1]")
    return cu_seqlens.shape[0] - 1


def ssm_conv_varlen(x, w, bias, cu_seqlens, max_seqlen: int, *, hist=None, want_hist: bool = False,
                    out: Optional[torch.Tensor] = None):
    """``ssm_conv`` over packed sequences: x [total,C], cu_seqlens [nseq+1] int32 (device), hist
    [nseq,3,C].  Rows in no sequence keep their ``out``."""
    if x.dim() != 2:
        raise ValueError("x must be [total, C]")
    nseq, max_seqlen = _offsets(cu_seqlens), int(max_seqlen)
    _fit(max_seqlen)
    out, hist_out, ld, io, dev = _conv(x, 1, w, bias, hist, nseq, want_hist, out, cu_seqlens)
    _call("gdn_ssm_conv_varlen", dev, x.data_ptr(), ld, w.data_ptr(), _ptr(bias), cu_seqlens.data_ptr(), nseq,
          max_seqlen, _ptr(hist), out.data_ptr(), _ptr(hist_out), x.shape[0], x.shape[1], io)
    return (out, hist_out) if want_hist else out


def ssm_scan_workspace_bytes(nseq, max_seqlen, H, G, P, N, dtype, total: Optional[int] = None) -> int:
    """Device scratch bytes ``ssm_scan`` / ``ssm_scan_varlen`` need (0: none); with ``total``, the rows of
    a packed call, no more than its rows make necessary."""
    _fit(nseq, max_seqlen, H, G, P, N, total or 0)
    if total is not None:
        return int(lib().gdn_ssm_scan_varlen_workspace_bytes(nseq, max_seqlen, total, H, G, P, N, _DTYPES[dtype]))
    return int(lib().gdn_ssm_scan_workspace_bytes(nseq, max_seqlen, H, G, P, N, _DTYPES[dtype]))


def _scan(x, dt, A_log, Bm, Cm, D, z, dt_bias, S0, lead, nseq, max_len, want_state, out, state_out,
          workspace, cu=None):
    shape = tuple(x.shape)
    H, P = shape[lead:]
    tok = shape[:lead]
    bs = tuple(Bm.shape)
    if dt.shape != tok + (H,) or len(bs) != lead + 2 or bs[:lead] != tok or Cm.shape != bs \
            or (z is not None and z.shape != shape):
        raise ValueError("x, dt, Bm, Cm, z shapes disagree")
    G, N = bs[lead:]
    _fit(max_len, G, N, *shape)
    ty = x.dtype
    if dt.dtype != ty or Bm.dtype != ty or Cm.dtype != ty or (z is not None and z.dtype != ty):
        raise ValueError("x, dt, Bm, Cm, z must have one dtype")
    for t in (A_log, D, dt_bias):
        if t is not None and t.shape != (H,):
            raise ValueError("A_log, D, dt_bias must be [H]")
    for t in (S0, state_out):
        if t is not None and t.shape != (nseq, H, N, P):
            raise ValueError("states must be [sequences, H, N, P]")
    if out is not None and (out.shape != shape or out.dtype != ty):
        raise ValueError("out must have x's shape and dtype")
    _fp32(A_log, D, dt_bias, S0, state_out)
    io = _io_dtype(x)
    _dense(A_log, D, dt_bias, S0, state_out, out, workspace)
    dev = _on(x, dt, Bm, Cm, z, A_log, D, dt_bias, S0, out, state_out, workspace, cu)
    lds = (_row_ld(x, lead, "x"), _row_ld(dt, lead, "dt"), _row_ld(Bm, lead, "Bm"), _row_ld(Cm, lead, "Cm"),
           _row_ld(z, lead, "z"))
    y = x.new_empty(shape) if out is None else out
    sT = state_out
    if sT is None and want_state:
        sT = A_log.new_empty((nseq, H, N, P))
    if cu is None:
        need = (_lib or lib()).gdn_ssm_scan_workspace_bytes(nseq, max_len, H, G, P, N, io)
    else:
        need = (_lib or lib()).gdn_ssm_scan_varlen_workspace_bytes(nseq, max_len, shape[0], H, G, P, N, io)
    ws, wbytes = _workspace(need, x.device, workspace)
    head = (x.data_ptr(), lds[0], dt.data_ptr(), lds[1], Bm.data_ptr(), lds[2], Cm.data_ptr(), lds[3], _ptr(z),
            lds[4], A_log.data_ptr(), _ptr(D), _ptr(dt_bias))
    return y, sT, ws, head, (_ptr(S0), y.data_ptr(), _ptr(sT), _ptr(ws), wbytes), (H, G, P, N, io), dev


def ssm_scan(x, dt, A_log, Bm, Cm, *, D=None, z=None, dt_bias=None, S0=None,
             want_state: bool = True, out: Optional[torch.Tensor] = None,
             state_out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None
             ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective scan over prompts: x [B,T,H,P], dt [B,T,H], Bm, Cm [B,T,G,N], z [B,T,H,P] or None
    in one dtype (column slices of wider rows may be given); A_log, D, dt_bias [H] fp32; S0
    [B,H,N,P] fp32 or None.  Returns (y [B,T,H,P], S_T [B,H,N,P] or None)."""
    if x.dim() != 4:
        raise ValueError("x must be [B, T, H, P]")
    B, T = x.shape[:2]
    y, sT, ws, head, mid, dims, dev = _scan(x, dt, A_log, Bm, Cm, D, z, dt_bias, S0, 2, B, T, want_state,
                                            out, state_out, workspace)
    _call("gdn_ssm_scan", dev, *head, *mid, B, T, *dims)
    return y, sT


def ssm_scan_varlen(x, dt, A_log, Bm, Cm, cu_seqlens, max_seqlen: int, *, D=None, z=None,
                    dt_bias=None, S0=None, want_state: bool = True,
                    out: Optional[torch.Tensor] = None,
                    state_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``ssm_scan`` over packed sequences: [total,...] token tensors, cu_seqlens [nseq+1] int32
    (device), states [nseq,H,N,P].  Rows in no sequence keep their ``out``."""
    if x.dim() != 3:
        raise ValueError("x must be [total, H, P]")
    nseq, max_seqlen = _offsets(cu_seqlens), int(max_seqlen)
    y, sT, ws, head, mid, dims, dev = _scan(x, dt, A_log, Bm, Cm, D, z, dt_bias, S0, 1, nseq, max_seqlen,
                                            want_state, out, state_out, workspace, cu_seqlens)
    _call("gdn_ssm_scan_varlen", dev, *head, cu_seqlens.data_ptr(), nseq, max_seqlen, *mid, x.shape[0], *dims)
    return y, sT


def ssm_step(u, dt, hist, w, bias, A_log, S, *, groups: int, D=None, z=None, dt_bias=None,
             hist_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None
             ) -> Tuple[torch.Tensor, torch.Tensor]:
    """One token of the state space block for n sequences: u [n, H*P + 2*groups*N] raw rows
    [x | B | C], dt [n,H], z [n,H,P] or None; hist [n,3,H*P + 2*groups*N] raw rows before; w, bias
    of the convolution; S [n,H,N,P] fp32, updated in place.  Returns (y [n,H,P], hist_out), the
    history moved on by one token (into ``hist_out`` if given, never into ``hist`` itself)."""
    if S.dim() != 4 or u.dim() != 2 or groups <= 0:
        raise ValueError("S must be [n, H, N, P], u [n, channels], groups positive")
    n, H, N, P = S.shape
    C = H * P + 2 * groups * N
    if u.shape != (n, C) or dt.shape != (n, H) or hist.shape != (n, 3, C) or w.shape != (C, 4) \
            or (bias is not None and bias.shape != (C,)) or (z is not None and z.shape != (n, H, P)):
        raise ValueError("u, dt, hist, w, bias, z shapes disagree with S and groups")
    for t in (A_log, D, dt_bias):
        if t is not None and t.shape != (H,):
            raise ValueError("A_log, D, dt_bias must be [H]")
    ty = u.dtype
    if hist_out is None:
        hist_out = hist.new_empty((n, 3, C))
    elif hist_out.shape != (n, 3, C):
        raise ValueError("hist_out has another shape")
    if out is None:
        out = u.new_empty((n, H, P))
    elif out.shape != (n, H, P):
        raise ValueError("out has another shape")
    if dt.dtype != ty or hist.dtype != ty or hist_out.dtype != ty or out.dtype != ty \
            or (z is not None and z.dtype != ty):
        raise ValueError("u, dt, hist, z and the outputs must have one dtype")
    _fp32(w, bias, A_log, D, dt_bias, S)
    _dense(hist, hist_out, w, bias, A_log, D, dt_bias, S, out)
    dev = _on(u, dt, hist, w, bias, A_log, S, D, z, dt_bias, hist_out, out)
    _call("gdn_ssm_step", dev, u.data_ptr(), _row_ld(u, 1, "u"), dt.data_ptr(), _row_ld(dt, 1, "dt"), _ptr(z),
          _row_ld(z, 1, "z"), hist.data_ptr(), hist_out.data_ptr(), w.data_ptr(), _ptr(bias), A_log.data_ptr(),
          _ptr(D), _ptr(dt_bias), S.data_ptr(), out.data_ptr(), n, H, groups, P, N, _io_dtype(u))
    return out, hist_out


# ------------------------------------------------------------------------------------------------
# the norms before and after a block
# ------------------------------------------------------------------------------------------------
def _norm_args(y, h, z, w_post, w_pre, res_scale):
    shape = y.shape
    D = shape[-1]
    _fit(D)
    if h.shape != shape or (z is not None and z.shape != shape):
        raise ValueError("y, h and z must have one shape")
    if z is not None and z.dtype != y.dtype:
        raise ValueError("y and z must have one dtype")
    for t in (w_post, w_pre, res_scale):
        if t is not None and t.shape != (D,):
            raise ValueError("w_post, w_pre and res_scale must be [D]")
    _fp32(w_post, w_pre, res_scale)
    _dense(y, h, z, w_post, w_pre, res_scale)
    return (y.numel() // D if D else 0), D, _io_dtype(y), _io_dtype(h)


def block_norm(y, h, *, w_post=None, w_pre=None, z=None, res_scale=None, eps: float = 1e-5
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The residual step around a block: h_out = h + res_scale * SiLU(z) * (RMSNorm(y) * w_post) and
    the next block's input x = RMSNorm(h_out) * w_pre.  y, z [..., D] in one dtype; h [..., D] in it
    or in float32; w_post, w_pre, res_scale [D] fp32, each optional.  Returns (h_out, x), x None
    without ``w_pre``."""
    rows, D, io, ho = _norm_args(y, h, z, w_post, w_pre, res_scale)
    dev = _on(y, h, z, w_post, w_pre, res_scale)
    h_out = torch.empty_like(h)
    x = None if w_pre is None else torch.empty_like(y)
    _call("gdn_block_norm", dev, y.data_ptr(), h.data_ptr(), _ptr(z), _ptr(w_post), _ptr(w_pre), _ptr(res_scale),
          h_out.data_ptr(), _ptr(x), rows, D, eps, io, ho)
    return h_out, x


def block_norm_bwd_workspace_bytes(rows: int, D: int) -> int:
    """Device scratch bytes one ``block_norm_bwd`` call needs."""
    _fit(D)
    return int(lib().gdn_block_norm_bwd_workspace_bytes(rows, D))


def block_norm_bwd(y, h_out, dh_out, dx=None, *, w_post=None, w_pre=None, z=None, res_scale=None,
                   eps: float = 1e-5, workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of <dh_out, h_out> + <dx, x> of ``block_norm`` from its y, its output h_out and z:
    dict of dy, dh, dz (in their inputs' dtypes) and dw_post, dw_pre, dres_scale (fp32); None for
    what the call does not have.  dh_out may be None where there is a ``w_pre``."""
    rows, D, io, ho = _norm_args(y, h_out, z, w_post, w_pre, res_scale)
    if (dx is None) != (w_pre is None) or (dx is not None and (dx.shape != y.shape or dx.dtype != y.dtype)):
        raise ValueError("dx comes with w_pre, in y's shape and dtype")
    if dh_out is None and w_pre is None:
        raise ValueError("dh_out is needed without w_pre")
    if dh_out is not None and (dh_out.shape != y.shape or dh_out.dtype != h_out.dtype):
        raise ValueError("dh_out must have h_out's shape and dtype")
    _dense(dh_out, dx, workspace)
    dev = _on(y, h_out, dh_out, dx, z, w_post, w_pre, res_scale, workspace)
    like = lambda t: None if t is None else torch.empty_like(t)
    g = {"dy": like(y), "dh": like(h_out), "dz": like(z), "dw_post": like(w_post), "dw_pre": like(w_pre),
         "dres_scale": like(res_scale)}
    ws, wbytes = _workspace((_lib or lib()).gdn_block_norm_bwd_workspace_bytes(rows, D), y.device, workspace)
    _call("gdn_block_norm_bwd", dev, y.data_ptr(), h_out.data_ptr(), _ptr(z), _ptr(dh_out), _ptr(dx), _ptr(w_post),
          _ptr(w_pre), _ptr(res_scale), g["dy"].data_ptr(), g["dh"].data_ptr(), _ptr(g["dz"]), _ptr(g["dw_post"]),
          _ptr(g["dw_pre"]), _ptr(g["dres_scale"]), _ptr(ws), wbytes, rows, D, eps, io, ho)
    return g
