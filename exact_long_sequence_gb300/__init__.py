"""GB300 (sm_103a) exact self-attention forward: Python binding of the C ABI.

This module only marshals arguments: every step of the computation runs in the
CUDA kernels of ``libexact_attn.so`` (see ``include/exact_attn.h``). PyTorch is
used for device memory and streams. There is no fallback: if the library is
not built, or no sm_103 GPU is present, the calls raise.

    import exact_long_sequence_gb300 as ela
    o, lse = ela.attn_fwd(q, k, v, causal=True)   # q, k, v: bf16 [B, H, N, d] on cuda

The operation is O = softmax(scale * Q K^T + mask) V with the per-row natural
log-sum-exp LSE, computed as the streaming tiled pass of "From Attention Graph
to FlashAttention - A Memory-Centric Compilation Approach in AICF", section 3.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

import torch

from . import workloads  # noqa: F401  (seeded synthetic inputs; no attention arithmetic)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libexact_attn.so")

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_MISALIGNED = 3
ATTN_ERR_CUDA = 4
ATTN_ERR_TIMEOUT = 5
ATTN_ERR_NO_DEVICE = 6

# Every symbol include/exact_attn.h declares.
EXPORTED_SYMBOLS = (
    "attn_fwd",
    "attn_fwd_host",
    "attn_fwd_host_workspace_bytes",
    "attn_fwd_split",
    "attn_fwd_split_workspace_bytes",
    "attn_fwd_split_segments",
    "attn_fwd_split_choice",
    "attn_plan",
    "attn_last_device_error",
    "attn_last_cuda_error",
    "attn_strerror",
    "attn_debug_wait_timeout",
    "attn_debug_arm_timeout",
    "attn_fwd_noalloc",
    "attn_noalloc_last_device_error",
    "attn_bwd",
    "attn_bwd_workspace_bytes",
    "attn_fwd_fp8",
    "attn_fwd_fp8_workspace_bytes",
    "attn_softmax_rows",
    "attn_softmax_rows_workspace_bytes",
    "attn_layernorm_rows",
    "attn_qk_norm_rope",
    "attn_qk_norm_rope_bwd",
    "attn_qk_norm_rope_bwd_workspace_bytes",
    "attn_fwd_prefix",
    "attn_fwd_prefix_workspace_bytes",
)


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str, lib=None):
        msg = f"{what}: status {status}"
        if lib is not None:
            msg += f" ({lib.attn_strerror(status).decode()})"
            if status == ATTN_ERR_CUDA:
                msg += f", cudaError {lib.attn_last_cuda_error()}"
        super().__init__(msg)
        self.status = status


class AttnPlan(ctypes.Structure):
    _fields_ = [
        ("Br", ctypes.c_int), ("Bc", ctypes.c_int), ("q_tiles", ctypes.c_int), ("kv_stages", ctypes.c_int),
        ("tmem_cols", ctypes.c_int), ("smem_bytes", ctypes.c_int), ("threads", ctypes.c_int),
        ("num_units", ctypes.c_int), ("grid", ctypes.c_int), ("heads_per_group", ctypes.c_int),
        ("flops", ctypes.c_double), ("io_bytes", ctypes.c_double), ("l2_bytes", ctypes.c_double),
        ("hbm_bytes", ctypes.c_double), ("io_opt_q_tiles", ctypes.c_int), ("io_opt_Bc", ctypes.c_int),
        ("io_opt_l2_bytes", ctypes.c_double), ("kv_in_flight_bytes", ctypes.c_double), ("l2_fit", ctypes.c_double),
    ]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


_lib = None


def load_library(path: str | None = None):
    """Load the CUDA library (built by ``__graft_entry__.build()``); raise if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(p)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    lib.attn_fwd.restype = i
    lib.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, ctypes.c_size_t, vp]
    lib.attn_fwd_host.restype = i
    lib.attn_fwd_host_workspace_bytes.argtypes = [i, i, i, i]
    lib.attn_fwd_host_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_fwd_split.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, ctypes.c_size_t, vp]
    lib.attn_fwd_split.restype = i
    lib.attn_fwd_split_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.attn_fwd_split_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_fwd_split_segments.argtypes = [i, i, i, i, i]
    lib.attn_fwd_split_segments.restype = i
    ip = ctypes.POINTER(ctypes.c_int)
    lib.attn_fwd_split_choice.argtypes = [i, i, i, i, i, i, ip, ip, ip, ip]
    lib.attn_fwd_split_choice.restype = i
    lib.attn_plan.argtypes = [i, i, i, i, i, i, ctypes.POINTER(AttnPlan)]
    lib.attn_plan.restype = i
    lib.attn_last_device_error.argtypes = [vp]
    lib.attn_last_device_error.restype = i
    lib.attn_last_cuda_error.argtypes = []
    lib.attn_last_cuda_error.restype = i
    lib.attn_strerror.argtypes = [i]
    lib.attn_strerror.restype = ctypes.c_char_p
    lib.attn_debug_wait_timeout.argtypes = [ctypes.c_uint64, vp]
    lib.attn_debug_wait_timeout.restype = i
    lib.attn_debug_arm_timeout.argtypes = [ctypes.c_uint64]
    lib.attn_debug_arm_timeout.restype = i
    lib.attn_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    lib.attn_fwd_noalloc.restype = i
    lib.attn_noalloc_last_device_error.argtypes = [vp]
    lib.attn_noalloc_last_device_error.restype = i
    lib.attn_bwd.argtypes = [vp] * 9 + [i, i, i, i, i, f, vp, ctypes.c_size_t, vp]
    lib.attn_bwd.restype = i
    lib.attn_bwd_workspace_bytes.argtypes = [i, i, i, i]
    lib.attn_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_fwd_fp8.argtypes = [vp] * 5 + [i, i, i, i, i, f, f, f, f, vp, ctypes.c_size_t, vp]
    lib.attn_fwd_fp8.restype = i
    lib.attn_fwd_fp8_workspace_bytes.argtypes = [i, i, i, i]
    lib.attn_fwd_fp8_workspace_bytes.restype = ctypes.c_size_t
    i64 = ctypes.c_int64
    lib.attn_softmax_rows.argtypes = [vp, vp, i64, i, vp, ctypes.c_size_t, vp]
    lib.attn_softmax_rows.restype = i
    lib.attn_softmax_rows_workspace_bytes.argtypes = [i64, i]
    lib.attn_softmax_rows_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_layernorm_rows.argtypes = [vp, vp, vp, vp, i64, i, f, vp]
    lib.attn_layernorm_rows.restype = i
    lib.attn_qk_norm_rope.argtypes = [vp] * 7 + [i64, i64, vp, vp, i] + [vp] * 4 + [i] * 5 + [f, i, vp]
    lib.attn_qk_norm_rope.restype = i
    lib.attn_qk_norm_rope_bwd.argtypes = ([vp] * 11 + [i64, i64, vp, vp, i] + [vp] * 6 + [i] * 5 + [f, i, vp,
                                                                                                   ctypes.c_size_t, vp])
    lib.attn_qk_norm_rope_bwd.restype = i
    lib.attn_qk_norm_rope_bwd_workspace_bytes.argtypes = [i]
    lib.attn_qk_norm_rope_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_fwd_prefix.argtypes = [vp] * 14 + [i] * 7 + [f, vp, ctypes.c_size_t, vp]
    lib.attn_fwd_prefix.restype = i
    lib.attn_fwd_prefix_workspace_bytes.argtypes = [i] * 7
    lib.attn_fwd_prefix_workspace_bytes.restype = ctypes.c_size_t
    if path is None:
        _lib = lib
    return lib


def _check(status: int, what: str):
    if status != ATTN_OK:
        raise AttnError(status, what, _lib)


def default_scale(d: int) -> float:
    """1/sqrt(d), computed in double and rounded once to fp32."""
    import torch

    return float(torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32).item())


# default_scale of the two head sizes, as it computes them
_SCALES = {d: struct.unpack("f", struct.pack("f", 1.0 / math.sqrt(d)))[0] for d in (64, 128)}


def _stream_handle(stream):
    import torch

    if stream is None:  # the current device's current stream, without building a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _empty(shape, dtype, device, stream, returned=True):
    """An uninitialised tensor for a call on `stream` (None: the current one), from that stream's memory: a
    block of the current stream may be one that its earlier work, still running, uses.  returned: the
    caller gets the tensor, and may free it while its own stream still reads it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if stream.device != device:
        raise ValueError(f"stream must be a stream of the tensors' device {device}")
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def split_workspace_bytes(B: int, H: int, N: int, d: int, causal: bool) -> int:
    """Device bytes attn_fwd_split needs for this shape on the current device (0: none)."""
    return int(load_library().attn_fwd_split_workspace_bytes(B, H, N, d, int(bool(causal))))


def split_choice(B: int, H: int, N: int, d: int, causal: bool, num_sms: int | None = None) -> dict:
    """The work split attn_fwd_split uses (host only): segments per split unit (1: none), the
    first split unit, the number of split units, and whether the dynamic schedule runs (a
    counter-zeroing kernel then precedes the attention kernel).  num_sms: the current device's
    by default."""
    import ctypes

    import torch

    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    out = [ctypes.c_int(0) for _ in range(4)]
    st = load_library().attn_fwd_split_choice(B, H, N, d, int(bool(causal)), int(num_sms),
                                              *[ctypes.byref(x) for x in out])
    _check(st, "attn_fwd_split_choice")
    return {"segs": out[0].value, "first": out[1].value, "units": out[2].value, "dynamic": bool(out[3].value)}


def split_segments(B: int, H: int, N: int, d: int, causal: bool) -> int:
    """K/V segments per split unit attn_fwd_split chooses (1: no split; 0: invalid or no device)."""
    return int(load_library().attn_fwd_split_segments(B, H, N, d, int(bool(causal))))


def attn_fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None, stream=None,
             split: bool = True, workspace=None, lib=None):
    """O, LSE = attention(q, k, v) on the GPU through the C ABI.

    q, k, v   : bf16 CUDA tensors [B, H, N, d], contiguous, d in {64, 128}
    out       : optional bf16 [B, H, N, d] output buffer; lse: optional fp32 [B, H, N]
    stream    : torch.cuda.Stream (default: the current stream); the call is asynchronous.
    split     : allow attn_fwd_split: the K/V split for problems with fewer work units than SMs,
                and the dynamic schedule for causal problems with more (False: always attn_fwd)
    workspace : optional uint8 CUDA tensor of at least split_workspace_bytes() bytes for the
                split (allocated here when needed and not given)
    lib       : a library handle from load_library(path) (a compile-time variant); default: the
                library built in-tree
    """
    import torch

    lib = lib or load_library()
    if q.dim() != 4 or q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k, v must share a [B, H, N, d] shape")
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors")
    B, H, N, d = q.shape
    if scale is None:
        scale = default_scale(d)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((B, H, N), torch.float32, q.device, stream)
    if out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor shaped like q")
    if lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    with torch.cuda.device(q.device):
        need = int(lib.attn_fwd_split_workspace_bytes(B, H, N, d, int(bool(causal)))) if split else 0
        if need == 0:
            st = lib.attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                              B, H, N, d, int(bool(causal)), float(scale), _stream_handle(stream))
            _check(st, "attn_fwd")
            return out, lse
        if workspace is None:
            workspace = _empty((need,), torch.uint8, q.device, stream, returned=False)
        if workspace.dtype != torch.uint8 or not workspace.is_cuda or workspace.numel() < need:
            raise ValueError(f"workspace must be a uint8 CUDA tensor of at least {need} bytes")
        st = lib.attn_fwd_split(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                B, H, N, d, int(bool(causal)), float(scale), workspace.data_ptr(),
                                workspace.numel(), _stream_handle(stream))
    _check(st, "attn_fwd_split")
    return out, lse


def attn_bwd(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None, workspace=None, stream=None):
    """dQ, dK, dV = gradients of attn_fwd for the upstream gradient `do`.

    q, k, v, o, do : bf16 CUDA tensors [B, H, N, d] (o, lse from attn_fwd on the same inputs)
    lse            : fp32 [B, H, N]
    """
    import torch

    lib = load_library()
    for t in (q, k, v, o, do):
        if t.shape != q.shape or t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v, o, do must be contiguous bf16 CUDA tensors of one [B, H, N, d] shape")
    B, H, N, d = q.shape
    if lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    if scale is None:
        scale = default_scale(d)
    dq, dk, dv = (_empty(q.shape, q.dtype, q.device, stream) for _ in range(3))
    need = lib.attn_bwd_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = _empty((need,), torch.uint8, q.device, stream, returned=False)
    with torch.cuda.device(q.device):
        st = lib.attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
                          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, int(bool(causal)), float(scale),
                          workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(st, "attn_bwd")
    return dq, dk, dv


def attn_fwd_fp8(q8, k8, v8, scales, causal: bool = False, scale: float | None = None, out=None, lse=None,
                 workspace=None, stream=None, lib=None):
    """FP8 forward: q8, k8, v8 are uint8 CUDA tensors [B, H, N, d] of E4M3 codes and
    `scales` = (q_scale, k_scale, v_scale), the real inputs being scale * e4m3(code).
    Returns (o bf16 [B, H, N, d], lse fp32 [B, H, N]).  d must be 128.  `lib`: a library handle
    from load_library(path) (a compile-time variant); default: the library built in-tree."""
    import torch

    lib = lib or load_library()
    for t in (q8, k8, v8):
        if t.shape != q8.shape or t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q8, k8, v8 must be contiguous uint8 (E4M3 code) CUDA tensors of one [B, H, N, d] shape")
    B, H, N, d = q8.shape
    if scale is None:
        scale = default_scale(d)
    if out is None:
        out = _empty(q8.shape, torch.bfloat16, q8.device, stream)
    if lse is None:
        lse = _empty((B, H, N), torch.float32, q8.device, stream)
    need = lib.attn_fwd_fp8_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = _empty((max(need, 16),), torch.uint8, q8.device, stream, returned=False)
    sq, sk, sv = (float(x) for x in scales)
    with torch.cuda.device(q8.device):
        st = lib.attn_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, N, d,
                              int(bool(causal)), float(scale), sq, sk, sv, workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(st, "attn_fwd_fp8")
    return out, lse


def softmax_rows(x, out=None, workspace=None, stream=None):
    """Row softmax over the last axis of a contiguous bf16 CUDA tensor (last axis a multiple of 8)."""
    import torch

    lib = load_library()
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 CUDA tensor")
    N = x.shape[-1]
    R = x.numel() // N
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    need = lib.attn_softmax_rows_workspace_bytes(R, N)
    if need and workspace is None:
        workspace = _empty((need,), torch.uint8, x.device, stream, returned=False)
    with torch.cuda.device(x.device):
        st = lib.attn_softmax_rows(x.data_ptr(), out.data_ptr(), R, N,
                                   workspace.data_ptr() if workspace is not None else None,
                                   workspace.numel() if workspace is not None else 0, _stream_handle(stream))
    _check(st, "attn_softmax_rows")
    return out


def layernorm_rows(x, gamma, beta, eps: float = 1e-5, out=None, stream=None):
    """Layer normalisation over the last axis (bf16 x, gamma, beta on CUDA; last axis a multiple of 8, <= 65536)."""
    import torch

    lib = load_library()
    for t in (x, gamma, beta):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("x, gamma, beta must be contiguous bf16 CUDA tensors")
    N = x.shape[-1]
    if gamma.shape != (N,) or beta.shape != (N,):
        raise ValueError("gamma and beta must have the row length")
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    with torch.cuda.device(x.device):
        st = lib.attn_layernorm_rows(x.data_ptr(), gamma.data_ptr(), beta.data_ptr(), out.data_ptr(),
                                     x.numel() // N, N, float(eps), _stream_handle(stream))
    _check(st, "attn_layernorm_rows")
    return out


_BF16 = torch.bfloat16
_pack2, _pack3 = struct.Struct("2q").pack, struct.Struct("3q").pack


def _elsewhere(index) -> bool:
    """Whether another device than `index` is current (the library works on the current one)."""
    return torch.cuda.current_device() != index


def _raw_stream(stream, index):
    """The handle of `stream`, or of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


class _NoSize(Exception):
    pass


def _found(size) -> int:
    """A workspace query's answer, to be kept; raises for 0 (an invalid shape, or no device state: device memory
    may be full just now), which is not."""
    if size == 0:
        raise _NoSize
    return int(size)


def _size(query, *key) -> int:
    """The answer of a query that keeps its answers; 0: none, and the call is then refused."""
    try:
        return query(*key)
    except _NoSize:
        return 0


def _view(name, t, shape, index):
    """Checks a bf16 view with its last axis contiguous; returns its address and the other axes' strides
    as the C call's host array (None: contiguous)."""
    if t.dtype is not _BF16 or t.get_device() != index or t.shape != shape:
        raise ValueError(f"{name} must be a bf16 tensor of shape {tuple(shape)} on q's device")
    if t.is_contiguous():
        return t.data_ptr(), None
    s = t.stride()
    if s[-1] != 1:
        raise ValueError(f"{name} must have its last axis contiguous")
    return t.data_ptr(), _pack3(*s[:3]) if len(s) == 4 else _pack2(*s[:2])


def _rotation(q, k, positions, inv_freq, sections, weights):
    """The checks both directions of qk_norm_rope share.  Returns the sections as a host array, their
    number, the positions [axes, B or 1, N], and their axis and batch strides."""
    if q.dim() != 4 or k.dim() != 4 or not q.is_cuda:
        raise ValueError("q and k must be CUDA tensors [B, H, N, d]")
    index = q.get_device()
    B, _, N, d = q.shape
    kB, _, kN, kd = k.shape
    if kB != B or kN != N or kd != d:
        raise ValueError("q and k must share B, N and d")
    if inv_freq.dtype != torch.float64 or inv_freq.get_device() != index or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 tensor of one axis on q's device")
    if sections is None:
        sections = (inv_freq.shape[0],)
    if sum(sections) != inv_freq.shape[0]:
        raise ValueError("sections must add up to the number of frequencies")
    if positions.dtype != torch.int32 or positions.get_device() != index:
        raise ValueError("positions must be an int32 tensor on q's device")
    A = len(sections)
    while positions.dim() < 3 and (positions.dim() < 2 or A == 1):  # [N] or [B, N]: one axis
        positions = positions.unsqueeze(0)
    if positions.dim() != 3 or positions.shape[0] != A or positions.shape[1] not in (1, B) or positions.shape[2] != N:
        raise ValueError("positions must be [axes, B, N] (B may be 1; [B, N] or [N] for a single axis)")
    pa, pb, pn = positions.stride()
    if N > 1 and pn != 1:
        raise ValueError("positions must be contiguous along the tokens")
    for w in weights:
        if w is not None and (w.dtype != torch.bfloat16 or w.get_device() != index or w.shape != (d,) or
                              not w.is_contiguous()):
            raise ValueError("norm weights must be contiguous bf16 tensors [d] on q's device")
    return (ctypes.c_int * A)(*sections), A, positions, pa, 0 if positions.shape[1] == 1 else pb


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, sections=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Queries and keys made ready for attn_fwd: RMS norm of each head and rotary positions, one pass.

    q, k       : bf16 CUDA views [B, Hq, N, d] and [B, Hk, N, d], d contiguous (64 or 128), other strides
                 multiples of 8: for example slices of a projection's output, transposed
    positions  : int32 CUDA [axes, B, N] (B may be 1); [B, N] or [N] for a single axis
    inv_freq   : float64 CUDA, radians per position of each rotated pair (at most d / 2, a multiple of 8)
    q_weight, k_weight : bf16 [d] norm weights; None: that tensor is rotated without a norm
    sections   : how many pairs turn by each position axis, in order (default: all by one axis)
    interleaved: pairs are neighbours (2i, 2i + 1) instead of halves (i, i + pairs)
    q_out, k_out : optional bf16 views of the outputs' shapes (a cache's rows, or q and k themselves);
                 default: new contiguous tensors, the layout attn_fwd reads
    Returns (q_out, k_out)."""
    lib = load_library()
    sec, A, positions, pa, pb = _rotation(q, k, positions, inv_freq, sections, (q_weight, k_weight))
    B, Hq, N, d = q.shape
    Hk = k.shape[1]
    index = q.get_device()
    if _elsewhere(index):
        with torch.cuda.device(index):
            return qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, sections, eps, interleaved, q_out, k_out,
                                stream)
    if q_out is None:
        q_out = _empty((B, Hq, N, d), torch.bfloat16, q.device, stream)
    if k_out is None:
        k_out = _empty((B, Hk, N, d), torch.bfloat16, q.device, stream)
    qp, qs = _view("q", q, q.shape, index)
    kp, ks = _view("k", k, k.shape, index)
    qop, qos = _view("q_out", q_out, q.shape, index)
    kop, kos = _view("k_out", k_out, k.shape, index)
    st = lib.attn_qk_norm_rope(qp, qs, kp, ks, None if q_weight is None else q_weight.data_ptr(),
                               None if k_weight is None else k_weight.data_ptr(), positions.data_ptr(), pa, pb,
                               inv_freq.data_ptr(), sec, A, qop, qos, kop, kos, B, Hq, Hk, N, d,
                               float(eps), 1 if interleaved else 0, _raw_stream(stream, index))
    _check(st, "attn_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_bwd_workspace_bytes(d: int) -> int:
    """Device bytes qk_norm_rope_bwd needs with a norm, on the current device."""
    return int(load_library().attn_qk_norm_rope_bwd_workspace_bytes(d))


@functools.lru_cache(maxsize=16)
def _bwd_workspace_bytes(index, d) -> int:
    return _found(load_library().attn_qk_norm_rope_bwd_workspace_bytes(d))


def qk_norm_rope_bwd(dq_out, dk_out, q, k, positions, inv_freq, q_weight=None, k_weight=None, sections=None,
                     eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None):
    """Gradients of qk_norm_rope for upstream gradients of its outputs (attn_bwd's dQ and dK).

    dq_out, dk_out : bf16 CUDA views shaped like q and k; q, k and the rest: as given to qk_norm_rope
    dq, dk     : optional bf16 views for the gradients of q and k (default: new contiguous tensors)
    workspace  : optional uint8 CUDA tensor of qk_norm_rope_bwd_workspace_bytes(d) bytes
    Returns (dq, dk, dq_weight, dk_weight), the weights' gradients fp32 [d], None without a weight."""
    lib = load_library()
    sec, A, positions, pa, pb = _rotation(q, k, positions, inv_freq, sections, (q_weight, k_weight))
    B, Hq, N, d = q.shape
    Hk = k.shape[1]
    index = q.get_device()
    if _elsewhere(index):
        with torch.cuda.device(index):
            return qk_norm_rope_bwd(dq_out, dk_out, q, k, positions, inv_freq, q_weight, k_weight, sections, eps,
                                    interleaved, dq, dk, workspace, stream)
    if dq is None:
        dq = _empty((B, Hq, N, d), torch.bfloat16, q.device, stream)
    if dk is None:
        dk = _empty((B, Hk, N, d), torch.bfloat16, q.device, stream)
    dwq = None if q_weight is None else _empty((d,), torch.float32, q.device, stream)
    dwk = None if k_weight is None else _empty((d,), torch.float32, q.device, stream)
    if workspace is None and (dwq is not None or dwk is not None):
        workspace = _empty((_size(_bwd_workspace_bytes, index, d),), torch.uint8, q.device, stream, returned=False)
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.get_device() != index or
                                  not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    gqp, gqs = _view("dq_out", dq_out, q.shape, index)
    gkp, gks = _view("dk_out", dk_out, k.shape, index)
    qp, qs = _view("q", q, q.shape, index)
    kp, ks = _view("k", k, k.shape, index)
    dqp, dqs = _view("dq", dq, q.shape, index)
    dkp, dks = _view("dk", dk, k.shape, index)
    st = lib.attn_qk_norm_rope_bwd(
        gqp, gqs, gkp, gks, qp, qs, kp, ks, None if q_weight is None else q_weight.data_ptr(),
        None if k_weight is None else k_weight.data_ptr(), positions.data_ptr(), pa, pb, inv_freq.data_ptr(), sec, A,
        dqp, dqs, dkp, dks, None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(),
        B, Hq, Hk, N, d, float(eps), 1 if interleaved else 0, None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel(), _raw_stream(stream, index))
    _check(st, "attn_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


def prefix_workspace_bytes(R: int, Hq: int, Hk: int, T: int, P: int, C: int, d: int) -> int:
    """Device bytes attn_fwd_prefix needs for this shape on the current device (0: invalid shape)."""
    return int(load_library().attn_fwd_prefix_workspace_bytes(R, Hq, Hk, T, P, C, d))


@functools.lru_cache(maxsize=256)
def _prefix_workspace_bytes(index, *shape) -> int:
    """The query's answer for a device (the current one) and a shape."""
    return _found(load_library().attn_fwd_prefix_workspace_bytes(*shape))


def attn_fwd_prefix(q, k_prefix=None, v_prefix=None, k_own=None, v_own=None, own_lens=None, scale: float | None = None,
                    out=None, lse=None, workspace=None, stream=None):
    """O, LSE of T new tokens of R requests over a prefix all of them share and each request's own keys.

    q         : bf16 CUDA [R, Hq, T, d], d in {64, 128}
    k_prefix, v_prefix : bf16 [Hk, P, d], Hk a divisor of Hq; None: no prefix
    k_own, v_own : bf16 [R, Hk, C, d], caches of capacity C; None: no own keys
    own_lens  : int32 [R] on the device: own keys of each request, the T new tokens among them as the
                last; 0: the prefix alone; negative: padding, the request's rows are left as they were.
                Token t sees the own keys j < own_lens - (T - 1 - t).
    out, lse  : optional bf16 view like q and fp32 [R, Hq, T] (default: new contiguous tensors)
    workspace : optional uint8 CUDA tensor of prefix_workspace_bytes() bytes
    All bf16 tensors are views with d contiguous and other strides positive multiples of 8, so token-major
    caches may be given transposed.  Returns (out, lse)."""
    lib = load_library()
    if q.dim() != 4 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [R, Hq, T, d]")
    index = q.get_device()
    R, Hq, T, d = q.shape
    P = C = 0
    kp = vp = ko = vo = lens = kps = vps = kos = vos = None
    if k_prefix is None and k_own is None:
        raise ValueError("give a prefix, own keys, or both")
    if (k_prefix is None and v_prefix is not None) or (k_own is None and v_own is not None):
        raise ValueError("values need their keys")
    Hk = k_prefix.shape[0] if k_prefix is not None else k_own.shape[1] if k_own.dim() == 4 else 0
    if k_prefix is not None:
        if k_prefix.dim() != 3 or v_prefix is None:
            raise ValueError("k_prefix and v_prefix must be [Hk, P, d]")
        P = k_prefix.shape[1]
        kp, kps = _view("k_prefix", k_prefix, (Hk, P, d), index)
        vp, vps = _view("v_prefix", v_prefix, (Hk, P, d), index)
    if k_own is not None:
        if k_own.dim() != 4 or v_own is None or own_lens is None:
            raise ValueError("own keys need k_own and v_own [R, Hk, C, d] and own_lens")
        C = k_own.shape[2]
        shape = (R, Hk, C, d)
        ko, kos = _view("k_own", k_own, shape, index)
        vo, vos = _view("v_own", v_own, shape, index)
    if own_lens is not None:
        if own_lens.dtype != torch.int32 or own_lens.get_device() != index or own_lens.shape != (R,) or \
                not own_lens.is_contiguous():
            raise ValueError("own_lens must be a contiguous int32 tensor [R] on q's device")
        lens = own_lens.data_ptr()
    if scale is None:
        scale = _SCALES.get(d) or default_scale(d)
    if _elsewhere(index):
        with torch.cuda.device(index):
            return attn_fwd_prefix(q, k_prefix, v_prefix, k_own, v_own, own_lens, scale, out, lse, workspace, stream)
    if out is None:
        out = _empty((R, Hq, T, d), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _empty((R, Hq, T), torch.float32, q.device, stream)
    elif lse.dtype != torch.float32 or lse.get_device() != index or lse.shape != (R, Hq, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 tensor [R, Hq, T] on q's device")
    if workspace is None:
        workspace = _empty((_size(_prefix_workspace_bytes, index, R, Hq, Hk, T, P, C, d),), torch.uint8, q.device, stream,
                           returned=False)
    elif workspace.dtype != torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    qp, qs = _view("q", q, q.shape, index)
    op, os_ = _view("out", out, q.shape, index)
    st = lib.attn_fwd_prefix(qp, qs, kp, kps, vp, vps, ko, kos, vo, vos, lens, op, os_, lse.data_ptr(), R, Hq, Hk, T,
                             P, C, d, float(scale), workspace.data_ptr() or None, workspace.numel(),
                             _raw_stream(stream, index))
    _check(st, "attn_fwd_prefix")
    return out, lse


def attn_fwd_noalloc(q, k, v, out, lse, causal: bool = False, scale: float | None = None, stream=None):
    """attn_fwd through the entry point that never allocates device memory.

    For callers that cannot let the library cudaMalloc (their own pool owns all
    of device memory, or their path cannot take cudaMalloc's implicit device
    synchronisation): the kernel's error word lives in a fixed array compiled
    into the library instead. The caller passes the outputs `out` (bf16, shaped
    like q) and `lse` (fp32 [B, H, N]); calls that overlap on the GPU race on
    the shared word, so serialise them.
    """
    lib = load_library()
    B, H, N, d = q.shape
    if scale is None:
        scale = default_scale(d)
    for t in (q, k, v, out):
        if t.shape != q.shape or not t.is_contiguous():
            raise ValueError("q, k, v, out must be contiguous tensors of one [B, H, N, d] shape")
    if lse.shape != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous [B, H, N] tensor")
    st = lib.attn_fwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                              B, H, N, d, int(bool(causal)), float(scale), _stream_handle(stream))
    _check(st, "attn_fwd_noalloc")
    return out, lse


def attn_fwd_host(q_h, k_h, v_h, causal: bool = False, scale: float | None = None, out_h=None, lse_h=None,
                  workspace=None, stream=None):
    """Same operation on HOST tensors (pin them for asynchronous copies): the library
    copies Q, K, V in, runs the kernel and copies O, LSE out on `stream`. Synchronise the
    stream before reading the outputs."""
    import torch

    lib = load_library()
    B, H, N, d = q_h.shape
    if scale is None:
        scale = default_scale(d)
    if out_h is None:
        out_h = torch.empty_like(q_h, pin_memory=q_h.is_pinned())
    if lse_h is None:
        lse_h = torch.empty((B, H, N), dtype=torch.float32, pin_memory=q_h.is_pinned())
    need = lib.attn_fwd_host_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = _empty((need,), torch.uint8, torch.device("cuda", torch.cuda.current_device()), stream, returned=False)
    st = lib.attn_fwd_host(q_h.data_ptr(), k_h.data_ptr(), v_h.data_ptr(), out_h.data_ptr(), lse_h.data_ptr(),
                           B, H, N, d, int(bool(causal)), float(scale), workspace.data_ptr(),
                           workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(st, "attn_fwd_host")
    return out_h, lse_h


def host_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().attn_fwd_host_workspace_bytes(B, H, N, d))


def attn_plan(B: int, H: int, N: int, d: int, causal: bool, num_sms: int = 0) -> dict:
    """The planner's tiling for a shape (host only; num_sms=0 asks the current GPU)."""
    lib = load_library()
    plan = AttnPlan()
    _check(lib.attn_plan(B, H, N, d, int(bool(causal)), num_sms, ctypes.byref(plan)), "attn_plan")
    return plan.as_dict()


def last_device_error(stream=None, lib=None) -> int:
    """Synchronise `stream` and return (and clear) the kernel error status."""
    return (lib or load_library()).attn_last_device_error(_stream_handle(stream))


def debug_wait_timeout(timeout_ns: int, stream=None) -> int:
    """Launch the bounded-wait test kernel (waits on a barrier nobody arrives on)."""
    return load_library().attn_debug_wait_timeout(int(timeout_ns), _stream_handle(stream))


def debug_arm_timeout(timeout_ns: int) -> int:
    """Arm the one-shot abort hook: the next forward launch runs with this wait limit and
    withholds one of CTA 0's query-tile copies, so its wait runs out (test use only)."""
    return load_library().attn_debug_arm_timeout(int(timeout_ns))


def noalloc_last_device_error(stream=None) -> int:
    """Synchronise `stream` and return (and clear) attn_fwd_noalloc's error status."""
    return load_library().attn_noalloc_last_device_error(_stream_handle(stream))
