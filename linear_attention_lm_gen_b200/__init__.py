"""JetBlock token mixer on B200: Python binding of the C ABI in include/jet.h.

Argument marshalling only: every step of the mixer runs in the CUDA kernels
of ``libjet.so`` (built in-tree by ``build.py``). torch supplies device memory
and the current stream. There is no CPU path: if the library is missing or
no CUDA device is present, the calls raise.

Function names match the C entry points:
  jet_kernel_gen, jet_dyn_conv_v, jet_gdn_prefill_workspace_size,
  jet_gdn_prefill_workspace_min, jet_gdn_prefill, jet_gdn_prefill_noalloc, jet_gdn_decode_step,
  jet_jetblock_decode_step, jet_conv_gdn_decode_step, jet_jetblock_prefill_workspace_size,
  jet_jetblock_prefill, jet_jetblock_decode_slots, jet_jetblock_prefill_varlen_workspace_size,
  jet_jetblock_prefill_varlen, jet_jetblock_prefill_range_workspace_size,
  jet_jetblock_prefill_range, jet_gdn_range_compose, jet_gdn_range_correct,
  jet_attn_rope_append, jet_attn_paged_workspace_size, jet_attn_paged, jet_cache_copy,
  jet_cache_compact_workspace_size, jet_cache_compact,
  jet_device_error, jet_status_string, jet_launch_count.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import warnings
from array import array

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libjet.so")

JET_F32, JET_BF16 = 0, 1
STATUS = {0: "JET_OK", 1: "JET_ERR_INVALID_ARG", 2: "JET_ERR_UNSUPPORTED", 3: "JET_ERR_MISALIGNED",
          4: "JET_ERR_CUDA", 5: "JET_ERR_TIMEOUT", 6: "JET_ERR_DEVICE", 7: "JET_ERR_WORKSPACE",
          8: "JET_ERR_TOO_LARGE", 9: "JET_ERR_LIBRARY"}
EXPORTS = ("jet_kernel_gen", "jet_dyn_conv_v", "jet_gdn_prefill_workspace_size", "jet_gdn_prefill_workspace_min",
           "jet_gdn_prefill",
           "jet_gdn_prefill_noalloc", "jet_gdn_decode_step", "jet_jetblock_decode_step", "jet_conv_gdn_decode_step",
           "jet_jetblock_prefill_workspace_size", "jet_jetblock_prefill", "jet_jetblock_decode_slots",
           "jet_jetblock_prefill_varlen_workspace_size", "jet_jetblock_prefill_varlen",
           "jet_jetblock_prefill_range_workspace_size", "jet_jetblock_prefill_range", "jet_gdn_range_compose",
           "jet_gdn_range_correct", "jet_jetblock_layer_workspace_size", "jet_jetblock_layer",
           "jet_attn_rope_append", "jet_attn_paged_workspace_size", "jet_attn_paged", "jet_cache_copy",
           "jet_cache_compact_workspace_size", "jet_cache_compact", "jet_device_error",
           "jet_status_string", "jet_launch_count")
NOALLOC_SCRATCH_BYTES = 16 << 20


class JetError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")


_lib = None
_bind = None          # the fast path of the decode step's calls (csrc/bind.cpp); without it the checks here do


def _load_bind():
    """The module _bind, or None, with a warning, if it is missing or was built for another torch or Python."""
    from .build import bind_abi
    try:
        m = importlib.import_module("._bind", __name__)
        found, abi = getattr(m, "abi", "an unknown one"), bind_abi()
        if found == abi:
            return m
        why = f"it was built for {found}, this is {abi}"
    except ImportError as e:
        why = str(e)
    warnings.warn(f"_bind.so cannot be used ({why}): attention and cache calls take longer on the host; "
                  "run linear_attention_lm_gen_b200/build.py", RuntimeWarning, stacklevel=3)
    return None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libjet.so (raises if it has not been built) and, if it can be used, the binding's _bind.so."""
    global _lib, _bind
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libjet.so not built at {path}: run linear_attention_lm_gen_b200/build.py")
    _bind = _load_bind()
    _lib = declare(ctypes.CDLL(path))
    return _lib


def declare(L: ctypes.CDLL) -> ctypes.CDLL:
    """Set the argument and result types of the C entry points on a loaded library."""
    P, I, Z, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64
    L.jet_kernel_gen.argtypes = [P, P, P, P, I, I, I, I, I, I, I, P]
    L.jet_dyn_conv_v.argtypes = [P] * 8 + [I] * 8 + [P]
    L.jet_gdn_prefill_workspace_size.argtypes = [I] * 7
    L.jet_gdn_prefill_workspace_size.restype = Z
    L.jet_gdn_prefill_workspace_min.argtypes = [I] * 7
    L.jet_gdn_prefill_workspace_min.restype = Z
    L.jet_gdn_prefill.argtypes = [P] * 9 + [Z] + [I] * 7 + [P]
    L.jet_gdn_prefill_noalloc.argtypes = [P] * 8 + [I] * 7 + [P]
    L.jet_gdn_decode_step.argtypes = [P] * 7 + [I] * 5 + [P]
    L.jet_jetblock_decode_step.argtypes = [P] * 13 + [I] * 8 + [P]
    L.jet_conv_gdn_decode_step.argtypes = [P] * 10 + [I] * 5 + [P]
    L.jet_jetblock_prefill_workspace_size.argtypes = [I] * 7
    L.jet_jetblock_prefill_workspace_size.restype = Z
    L.jet_jetblock_prefill.argtypes = [P] * 14 + [Z] + [I] * 10 + [P]
    L.jet_jetblock_decode_slots.argtypes = [P] * 11 + [I] + [P] * 3 + [I] * 8 + [P]
    L.jet_jetblock_prefill_varlen_workspace_size.argtypes = [P, I, I, I, I, I, I]
    L.jet_jetblock_prefill_varlen_workspace_size.restype = Z
    L.jet_jetblock_prefill_varlen.argtypes = [P] * 14 + [Z] + [P] + [I] * 9 + [P]
    L.jet_jetblock_prefill_range_workspace_size.argtypes = [I] * 7
    L.jet_jetblock_prefill_range_workspace_size.restype = Z
    L.jet_jetblock_prefill_range.argtypes = [P] * 16 + [Z] + [I] * 10 + [P]
    L.jet_gdn_range_compose.argtypes = [P] * 4 + [I] * 5 + [P]
    L.jet_gdn_range_correct.argtypes = [P] * 3 + [I] * 6 + [P]
    L.jet_jetblock_layer_workspace_size.argtypes = [I] * 6
    L.jet_jetblock_layer_workspace_size.restype = Z
    L.jet_jetblock_layer.argtypes = [P] * 17 + [Z] + [I] * 9 + [P]
    Q, F = ctypes.c_int64, ctypes.c_float
    L.jet_attn_rope_append.argtypes = [P, Q] * 3 + [P, P, F, P, I, I, P, Q, P, P, Q, Q, Q, P, P, P] + [I] * 9 + [P]
    L.jet_attn_paged_workspace_size.argtypes = [I] * 6
    L.jet_attn_paged_workspace_size.restype = Z
    L.jet_attn_paged.argtypes = [P, Q, P, P, Q, Q, Q, P, P, P, P, P, Z] + [I] * 10 + [F, I, P]
    L.jet_cache_copy.argtypes = [P, P, P, I, I, P, P, I, P]
    L.jet_cache_compact_workspace_size.argtypes = [I]
    L.jet_cache_compact_workspace_size.restype = Z
    L.jet_cache_compact.argtypes = [P, P, P, I, I, I, P, P, I, I, P, P, P, Z, P]
    L.jet_device_error.argtypes = [P]
    L.jet_status_string.argtypes = [I]
    L.jet_status_string.restype = ctypes.c_char_p
    L.jet_launch_count.argtypes = []
    L.jet_launch_count.restype = U
    for f in ("jet_kernel_gen", "jet_dyn_conv_v", "jet_gdn_prefill", "jet_gdn_prefill_noalloc",
              "jet_gdn_decode_step", "jet_jetblock_decode_step", "jet_conv_gdn_decode_step", "jet_jetblock_prefill",
              "jet_jetblock_decode_slots", "jet_jetblock_prefill_varlen", "jet_jetblock_prefill_range",
              "jet_gdn_range_compose",
              "jet_gdn_range_correct", "jet_jetblock_layer", "jet_attn_rope_append", "jet_attn_paged", "jet_cache_copy",
              "jet_cache_compact", "jet_device_error"):
        getattr(L, f).restype = I
    for f in ("jet_attn_rope_append", "jet_attn_paged", "jet_cache_copy", "jet_cache_compact"):
        setattr(L, "at_" + f, ctypes.cast(getattr(L, f), P).value)
    return L


# ---------------------------------------------------------------- marshalling
def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return JET_BF16
    if t.dtype == torch.float32:
        return JET_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or float32)")


def _ptr(t, name, dtype=None, shape=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn, st):
    if st != 0:
        raise JetError(fn, st)


# ---------------------------------------------------------------- entry points
def jet_kernel_gen(x, W1, W2, H: int, conv_w=None, *, stream=None):
    """x [B,T,D], W1 [D,32], W2 [32,H*4] -> conv taps [B,T,H,4] float32."""
    L = load_library()
    B, T, D = x.shape
    dt = _dt(x)
    if conv_w is None:
        conv_w = torch.empty((B, T, H, 4), device=x.device, dtype=torch.float32)
    st = L.jet_kernel_gen(_ptr(x, "x"), _ptr(W1, "W1", x.dtype, (D, 32)), _ptr(W2, "W2", x.dtype, (32, H * 4)),
                          _ptr(conv_w, "conv_w", torch.float32, (B, T, H, 4)), B, T, D, H, 32, 4, dt, _stream(stream))
    _check("jet_kernel_gen", st)
    return conv_w


def jet_dyn_conv_v(x, W1, W2, v, hist_in=None, v_out=None, hist_out=None, conv_w_out=None, *, stream=None):
    """Generator + dynamic causal conv on V. v [B,T,H,dv] -> v' (same shape).
    Returns (v_out, hist_out); hist_out is None unless a buffer is given."""
    L = load_library()
    B, T, D = x.shape
    _, _, H, dv = v.shape
    dt = _dt(x)
    if v_out is None:
        v_out = torch.empty_like(v)
    st = L.jet_dyn_conv_v(_ptr(x, "x"), _ptr(W1, "W1", x.dtype, (D, 32)), _ptr(W2, "W2", x.dtype, (32, H * 4)),
                          _ptr(v, "v", x.dtype, (B, T, H, dv)),
                          _ptr(hist_in, "hist_in", x.dtype, (B, 3, H, dv)), _ptr(v_out, "v_out", x.dtype, (B, T, H, dv)),
                          _ptr(hist_out, "hist_out", x.dtype, (B, 3, H, dv)),
                          _ptr(conv_w_out, "conv_w_out", torch.float32, (B, T, H, 4)),
                          B, T, D, H, dv, 32, 4, dt, _stream(stream))
    _check("jet_dyn_conv_v", st)
    return v_out, hist_out


def jet_gdn_prefill_workspace_size(B, T, H, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Workspace bytes of the fastest prefill plan (chunk images + segment buffers)."""
    L = load_library()
    return int(L.jet_gdn_prefill_workspace_size(B, T, H, dk, dv, chunk,
                                                JET_BF16 if dtype == torch.bfloat16 else JET_F32))


def jet_gdn_prefill_workspace_min(B, T, H, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Smallest workspace jet_gdn_prefill accepts (segment buffers only)."""
    L = load_library()
    return int(L.jet_gdn_prefill_workspace_min(B, T, H, dk, dv, chunk,
                                               JET_BF16 if dtype == torch.bfloat16 else JET_F32))


def jet_gdn_prefill(q, k, v, g, beta, S0=None, o=None, S_out=None, workspace=None, *, stream=None):
    """Chunked Gated DeltaNet prefill. q,k [B,T,H,dk], v [B,T,H,dv], g,beta [B,T,H]
    float32, S0 [B,H,dv,dk] float32 or None. Returns (o, S_out)."""
    L = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    if o is None:
        o = torch.empty((B, T, H, dv), device=q.device, dtype=q.dtype)
    if S_out is None:
        S_out = torch.empty((B, H, dv, dk), device=q.device, dtype=torch.float32)
    need = jet_gdn_prefill_workspace_size(B, T, H, dk, dv, 64, q.dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = L.jet_gdn_prefill(_ptr(q, "q"), _ptr(k, "k", q.dtype, q.shape), _ptr(v, "v", q.dtype, (B, T, H, dv)),
                           _ptr(g, "g", torch.float32, (B, T, H)), _ptr(beta, "beta", torch.float32, (B, T, H)),
                           _ptr(S0, "S0", torch.float32, (B, H, dv, dk)), _ptr(o, "o", q.dtype, (B, T, H, dv)),
                           _ptr(S_out, "S_out", torch.float32, (B, H, dv, dk)), _ptr(workspace, "workspace"),
                           ws_bytes, B, T, H, dk, dv, 64, dt, _stream(stream))
    _check("jet_gdn_prefill", st)
    return o, S_out


def jet_gdn_prefill_noalloc(q, k, v, g, beta, S0, o, S_out, *, stream=None):
    """jet_gdn_prefill without a workspace argument, for callers that cannot
    allocate: the library uses its own fixed scratch array (16 MiB per GPU).
    o and S_out must be given (nothing is allocated here either). Calls whose
    work overlaps on the GPU share that array and must be ordered by the caller."""
    L = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    st = L.jet_gdn_prefill_noalloc(_ptr(q, "q"), _ptr(k, "k", q.dtype, q.shape), _ptr(v, "v", q.dtype, (B, T, H, dv)),
                                   _ptr(g, "g", torch.float32, (B, T, H)), _ptr(beta, "beta", torch.float32, (B, T, H)),
                                   _ptr(S0, "S0", torch.float32, (B, H, dv, dk)), _ptr(o, "o", q.dtype, (B, T, H, dv)),
                                   _ptr(S_out, "S_out", torch.float32, (B, H, dv, dk)),
                                   B, T, H, dk, dv, 64, _dt(q), _stream(stream))
    _check("jet_gdn_prefill_noalloc", st)
    return o, S_out


def jet_jetblock_prefill_workspace_size(B, T, H, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Workspace bytes of jet_jetblock_prefill (taps + the prefill's fastest plan)."""
    L = load_library()
    return int(L.jet_jetblock_prefill_workspace_size(B, T, H, dk, dv, chunk,
                                                     JET_BF16 if dtype == torch.bfloat16 else JET_F32))


def jet_jetblock_prefill(x, W1, W2, q, k, v, g, beta, hist_in=None, hist_out=None, S0=None, o=None, S_out=None,
                         workspace=None, *, stream=None):
    """Generator + dynamic conv + chunked Gated DeltaNet over a prompt. x [B,T,D],
    q,k [B,T,H,dk], v [B,T,H,dv] raw, g,beta [B,T,H] float32, hist_in / hist_out
    [B,3,H,dv] or None, S0 [B,H,dv,dk] float32 or None. Returns (o, S_out)."""
    L = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    D = x.shape[-1]
    hidden, HW = W2.shape
    width = HW // H
    dt = _dt(q)
    if o is None:
        o = torch.empty((B, T, H, dv), device=q.device, dtype=q.dtype)
    if S_out is None:
        S_out = torch.empty((B, H, dv, dk), device=q.device, dtype=torch.float32)
    if workspace is None:
        workspace = torch.empty(max(1, jet_jetblock_prefill_workspace_size(B, T, H, dk, dv, 64, q.dtype)),
                                device=q.device, dtype=torch.uint8)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = L.jet_jetblock_prefill(
        _ptr(x, "x", q.dtype, (B, T, D)), _ptr(W1, "W1", q.dtype, (D, hidden)), _ptr(W2, "W2", q.dtype, (hidden, HW)),
        _ptr(q, "q"), _ptr(k, "k", q.dtype, q.shape), _ptr(v, "v", q.dtype, (B, T, H, dv)),
        _ptr(hist_in, "hist_in", q.dtype, (B, 3, H, dv)), _ptr(hist_out, "hist_out", q.dtype, (B, 3, H, dv)),
        _ptr(g, "g", torch.float32, (B, T, H)), _ptr(beta, "beta", torch.float32, (B, T, H)),
        _ptr(S0, "S0", torch.float32, (B, H, dv, dk)), _ptr(o, "o", q.dtype, (B, T, H, dv)),
        _ptr(S_out, "S_out", torch.float32, (B, H, dv, dk)), _ptr(workspace, "workspace"), ws_bytes,
        B, T, D, H, dk, dv, hidden, width, 64, dt, _stream(stream))
    _check("jet_jetblock_prefill", st)
    return o, S_out


def _cu(cu_seqlens):
    """Sequence offsets as a host int32 array (a list, tuple or CPU tensor)."""
    import numpy as np
    if isinstance(cu_seqlens, torch.Tensor):
        if cu_seqlens.is_cuda:
            raise TypeError("cu_seqlens must be on the host: the launch plan is made from it")
        cu_seqlens = cu_seqlens.tolist()
    return np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))


def jet_jetblock_prefill_varlen_workspace_size(cu_seqlens, H, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Workspace bytes of jet_jetblock_prefill_varlen for these sequence offsets."""
    L = load_library()
    cu = _cu(cu_seqlens)
    return int(L.jet_jetblock_prefill_varlen_workspace_size(cu.ctypes.data_as(ctypes.c_void_p), len(cu) - 1, H, dk,
                                                            dv, chunk, JET_BF16 if dtype == torch.bfloat16 else JET_F32))


def jet_jetblock_prefill_varlen(x, W1, W2, q, k, v, g, beta, cu_seqlens, hist_in=None, hist_out=None, S0=None, o=None,
                                S_out=None, workspace=None, *, stream=None):
    """The mixer over several prompts of different lengths in one call, packed
    along the token axis: x [total,D], q,k [total,H,dk], v [total,H,dv] raw,
    g,beta [total,H] float32; cu_seqlens (host) the nseq + 1 offsets;
    hist_in / hist_out [nseq,3,H,dv], S0 [nseq,H,dv,dk] or None. Returns
    (o [total,H,dv], S_out [nseq,H,dv,dk])."""
    L = load_library()
    cu = _cu(cu_seqlens)
    nseq = len(cu) - 1
    total, H, dk = q.shape
    dv = v.shape[-1]
    D = x.shape[-1]
    hidden, HW = W2.shape
    width = HW // H
    if o is None:
        o = torch.empty((total, H, dv), device=q.device, dtype=q.dtype)
    if S_out is None:
        S_out = torch.empty((nseq, H, dv, dk), device=q.device, dtype=torch.float32)
    if workspace is None:
        workspace = torch.empty(max(16, jet_jetblock_prefill_varlen_workspace_size(cu, H, dk, dv, 64, q.dtype)),
                                device=q.device, dtype=torch.uint8)
    st = L.jet_jetblock_prefill_varlen(
        _ptr(x, "x", q.dtype, (total, D)), _ptr(W1, "W1", q.dtype, (D, hidden)), _ptr(W2, "W2", q.dtype, (hidden, HW)),
        _ptr(q, "q"), _ptr(k, "k", q.dtype, q.shape), _ptr(v, "v", q.dtype, (total, H, dv)),
        _ptr(hist_in, "hist_in", q.dtype, (nseq, 3, H, dv)), _ptr(hist_out, "hist_out", q.dtype, (nseq, 3, H, dv)),
        _ptr(g, "g", torch.float32, (total, H)), _ptr(beta, "beta", torch.float32, (total, H)),
        _ptr(S0, "S0", torch.float32, (nseq, H, dv, dk)), _ptr(o, "o", q.dtype, (total, H, dv)),
        _ptr(S_out, "S_out", torch.float32, (nseq, H, dv, dk)), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), cu.ctypes.data_as(ctypes.c_void_p), nseq, D, H, dk, dv, hidden,
        width, 64, _dt(q), _stream(stream))
    _check("jet_jetblock_prefill_varlen", st)
    return o, S_out


def jet_jetblock_prefill_range_workspace_size(B, T, H, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Workspace bytes of jet_jetblock_prefill_range (taps + chunk images)."""
    L = load_library()
    return int(L.jet_jetblock_prefill_range_workspace_size(B, T, H, dk, dv, chunk,
                                                           JET_BF16 if dtype == torch.bfloat16 else JET_F32))


def jet_jetblock_prefill_range(x, W1, W2, q, k, v, g, beta, hist_in=None, hist_out=None, S0=None, first=False,
                               o=None, E_out=None, A_out=None, Qe_out=None, workspace=None, *, stream=None):
    """The mixer over one token range of a sequence split across GPUs.
    first=True: the range starts at S0 (or zero) for real and gets no
    transition; otherwise it runs from a zero start and also returns its
    transition A [B,H,dk,dk] and output-correction operand Qe. Returns
    (o, E, A, Qe); A and Qe are None for a first range."""
    L = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    D = x.shape[-1]
    hidden, HW = W2.shape
    width = HW // H
    dev = q.device
    if o is None:
        o = torch.empty((B, T, H, dv), device=dev, dtype=q.dtype)
    if E_out is None:
        E_out = torch.empty((B, H, dv, dk), device=dev, dtype=torch.float32)
    if not first:
        if A_out is None:
            A_out = torch.empty((B, H, dk, dk), device=dev, dtype=torch.float32)
        if Qe_out is None:
            Qe_out = torch.empty((B, H, (T + 63) // 64, 64, dk), device=dev, dtype=q.dtype)
    if workspace is None:
        workspace = torch.empty(max(16, jet_jetblock_prefill_range_workspace_size(B, T, H, dk, dv, 64, q.dtype)),
                                device=dev, dtype=torch.uint8)
    st = L.jet_jetblock_prefill_range(
        _ptr(x, "x", q.dtype, (B, T, D)), _ptr(W1, "W1", q.dtype, (D, hidden)), _ptr(W2, "W2", q.dtype, (hidden, HW)),
        _ptr(q, "q"), _ptr(k, "k", q.dtype, q.shape), _ptr(v, "v", q.dtype, (B, T, H, dv)),
        _ptr(hist_in, "hist_in", q.dtype, (B, 3, H, dv)), _ptr(hist_out, "hist_out", q.dtype, (B, 3, H, dv)),
        _ptr(g, "g", torch.float32, (B, T, H)), _ptr(beta, "beta", torch.float32, (B, T, H)),
        _ptr(S0, "S0", torch.float32, (B, H, dv, dk)), _ptr(o, "o", q.dtype, (B, T, H, dv)),
        _ptr(E_out, "E_out", torch.float32, (B, H, dv, dk)),
        _ptr(A_out, "A_out", torch.float32, (B, H, dk, dk)),
        _ptr(Qe_out, "Qe_out", q.dtype, (B, H, (T + 63) // 64, 64, dk)),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        B, T, D, H, dk, dv, hidden, width, 64, _dt(q), _stream(stream))
    _check("jet_jetblock_prefill_range", st)
    return o, E_out, A_out, Qe_out


def jet_gdn_range_compose(E, A, Sb=None, S_out=None, *, stream=None):
    """Start states of R ranges from their (E, A) pairs: E [R,B,H,dv,dk] and
    A [R,B,H,dk,dk] float32. Returns (Sb [R,B,H,dv,dk] bf16, entries 1.. are the
    ranges' start states; S_out [B,H,dv,dk] float32, the final state)."""
    L = load_library()
    R, B, H, dv, dk = E.shape
    if Sb is None:
        Sb = torch.empty((R, B, H, dv, dk), device=E.device, dtype=torch.bfloat16)
    if S_out is None:
        S_out = torch.empty((B, H, dv, dk), device=E.device, dtype=torch.float32)
    st = L.jet_gdn_range_compose(_ptr(E, "E", torch.float32), _ptr(A, "A", torch.float32, (R, B, H, dk, dk)),
                                 _ptr(Sb, "Sb", torch.bfloat16, (R, B, H, dv, dk)),
                                 _ptr(S_out, "S_out", torch.float32, (B, H, dv, dk)), R, B, H, dk, dv,
                                 _stream(stream))
    _check("jet_gdn_range_compose", st)
    return Sb, S_out


def jet_gdn_range_correct(Qe, Sb, o, *, stream=None):
    """o [B,T,H,dv] += the start-state term of a range: Qe from its range pass,
    Sb [B,H,dv,dk] bf16 its start state. Returns o."""
    L = load_library()
    B, T, H, dv = o.shape
    dk = Sb.shape[-1]
    st = L.jet_gdn_range_correct(_ptr(Qe, "Qe", o.dtype, (B, H, (T + 63) // 64, 64, dk)),
                                 _ptr(Sb, "Sb", torch.bfloat16, (B, H, dv, dk)), _ptr(o, "o"), B, T, H, dk, dv,
                                 _dt(o), _stream(stream))
    _check("jet_gdn_range_correct", st)
    return o


def jet_gdn_decode_step(q, k, v, g, beta, S, o=None, *, stream=None):
    """One decode step, S [B,H,dv,dk] float32 updated in place. q,k [B,H,dk],
    v [B,H,dv], g,beta [B,H]. Returns o [B,H,dv]."""
    L = load_library()
    B, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    if o is None:
        o = torch.empty((B, H, dv), device=q.device, dtype=q.dtype)
    st = L.jet_gdn_decode_step(_ptr(q, "q"), _ptr(k, "k", q.dtype, q.shape), _ptr(v, "v", q.dtype, (B, H, dv)),
                               _ptr(g, "g", torch.float32, (B, H)), _ptr(beta, "beta", torch.float32, (B, H)),
                               _ptr(S, "S", torch.float32, (B, H, dv, dk)), _ptr(o, "o", q.dtype, (B, H, dv)),
                               B, H, dk, dv, dt, _stream(stream))
    _check("jet_gdn_decode_step", st)
    return o


def jet_jetblock_decode_step(x, W1, W2, q, k, v, hist_in, hist_out, g, beta, S, o=None, taps=None, *,
                             stream=None):
    """Generator + conv + history shift + decode update for one new token per
    sequence. x [B,D], v [B,H,dv] raw, hist_in [B,3,H,dv] or None, hist_out
    [B,3,H,dv], S [B,H,dv,dk] float32 updated in place. Returns (o, taps)."""
    L = load_library()
    B, H, dk = q.shape
    dv = v.shape[-1]
    D = x.shape[-1]
    hidden, HW = W2.shape
    width = HW // H
    dt = _dt(q)
    if o is None:
        o = torch.empty((B, H, dv), device=q.device, dtype=q.dtype)
    if taps is None:
        taps = torch.empty((B, H, width), device=q.device, dtype=torch.float32)
    st = L.jet_jetblock_decode_step(
        _ptr(x, "x", q.dtype, (B, D)), _ptr(W1, "W1", q.dtype, (D, hidden)), _ptr(W2, "W2", q.dtype, (hidden, HW)),
        _ptr(q, "q"), _ptr(k, "k", q.dtype, q.shape), _ptr(v, "v", q.dtype, (B, H, dv)),
        _ptr(hist_in, "hist_in", q.dtype, (B, 3, H, dv)), _ptr(hist_out, "hist_out", q.dtype, (B, 3, H, dv)),
        _ptr(g, "g", torch.float32, (B, H)), _ptr(beta, "beta", torch.float32, (B, H)),
        _ptr(S, "S", torch.float32, (B, H, dv, dk)), _ptr(o, "o", q.dtype, (B, H, dv)),
        _ptr(taps, "taps", torch.float32, (B, H, width)),
        B, D, H, dk, dv, hidden, width, dt, _stream(stream))
    _check("jet_jetblock_decode_step", st)
    return o, taps


def jet_jetblock_decode_slots(x, W1, W2, q, k, v, g, beta, hist_pool, S_pool, slots, o=None, v_conv=None, taps=None,
                              *, stream=None):
    """One decode step for B sequences whose states and histories are pool
    entries: x [B,D], q,k [B,H,dk], v [B,H,dv] raw, g,beta [B,H] float32,
    hist_pool [N,3,H,dv] and S_pool [N,H,dv,dk] float32 updated in place at
    entries slots [B] (int32, distinct). Returns o [B,H,dv]."""
    L = load_library()
    B, H, dk = q.shape
    dv = v.shape[-1]
    D = x.shape[-1]
    hidden, HW = W2.shape
    width = HW // H
    N = S_pool.shape[0]
    if o is None:
        o = torch.empty((B, H, dv), device=q.device, dtype=q.dtype)
    if v_conv is None:
        v_conv = torch.empty((B, H, dv), device=q.device, dtype=q.dtype)
    st = L.jet_jetblock_decode_slots(
        _ptr(x, "x", q.dtype, (B, D)), _ptr(W1, "W1", q.dtype, (D, hidden)), _ptr(W2, "W2", q.dtype, (hidden, HW)),
        _ptr(q, "q"), _ptr(k, "k", q.dtype, q.shape), _ptr(v, "v", q.dtype, (B, H, dv)),
        _ptr(g, "g", torch.float32, (B, H)), _ptr(beta, "beta", torch.float32, (B, H)),
        _ptr(hist_pool, "hist_pool", q.dtype, (N, 3, H, dv)), _ptr(S_pool, "S_pool", torch.float32, (N, H, dv, dk)),
        _ptr(slots, "slots", torch.int32, (B,)), N, _ptr(o, "o", q.dtype, (B, H, dv)),
        _ptr(v_conv, "v_conv", q.dtype, (B, H, dv)), _ptr(taps, "taps", torch.float32, (B, H, width)),
        B, D, H, dk, dv, hidden, width, _dt(q), _stream(stream))
    _check("jet_jetblock_decode_slots", st)
    return o


def jet_conv_gdn_decode_step(q, k, v, hist_in, hist_out, taps, g, beta, S, o=None, *, stream=None):
    """Decode step with the conv of the new token fused in: v [B,H,dv] raw,
    taps [B,H,4] float32 from jet_kernel_gen, hist_in [B,3,H,dv] or None,
    hist_out [B,3,H,dv]; S updated in place. Returns o [B,H,dv]."""
    L = load_library()
    B, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    if o is None:
        o = torch.empty((B, H, dv), device=q.device, dtype=q.dtype)
    st = L.jet_conv_gdn_decode_step(
        _ptr(q, "q"), _ptr(k, "k", q.dtype, q.shape), _ptr(v, "v", q.dtype, (B, H, dv)),
        _ptr(hist_in, "hist_in", q.dtype, (B, 3, H, dv)), _ptr(hist_out, "hist_out", q.dtype, (B, 3, H, dv)),
        _ptr(taps, "taps", torch.float32, (B, H, 4)), _ptr(g, "g", torch.float32, (B, H)),
        _ptr(beta, "beta", torch.float32, (B, H)), _ptr(S, "S", torch.float32, (B, H, dv, dk)),
        _ptr(o, "o", q.dtype, (B, H, dv)), B, H, dk, dv, dt, _stream(stream))
    _check("jet_conv_gdn_decode_step", st)
    return o


# ---------------------------------------------------------------- softmax attention over a paged cache
# The decode step's calls take a few microseconds on the GPU. With outputs and
# workspace given, on the current device and stream, they go through _bind,
# which checks the arguments natively; anything else, every error, and every
# call where _bind cannot be loaded, through the checks here.
class _on:
    """Make device `index` current and issue on `stream` (default: the device's
    current stream) for the length of a call; what the call allocates belongs
    to that stream. Every tensor of the call has to be on the device."""

    __slots__ = ("_dev", "_stream", "_index")

    def __init__(self, index, stream):
        self._index, self._stream, self._dev = index, stream, None

    def __enter__(self):
        index, stream = self._index, self._stream
        if index != torch._C._cuda_getDevice():
            self._dev = torch.cuda.device(index)
            self._dev.__enter__()
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(index)
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        self._stream = torch.cuda.stream(torch.cuda.ExternalStream(raw) if raw else torch.cuda.default_stream(index))
        self._stream.__enter__()
        return raw

    def __exit__(self, *exc):
        if self._stream is not None:
            self._stream.__exit__(*exc)
        if self._dev is not None:
            self._dev.__exit__(*exc)
        return False


def _issue(index, stream, call):
    """call(raw stream) with GPU `index` current, on its current stream unless one is given."""
    if stream is None and torch._C._cuda_getDevice() == index:
        return call(torch._C._cuda_getCurrentRawStream(index))
    with _on(index, stream) as s:
        return call(s)


def _refuse(t, name, index, dtype, shape):
    """Raise what is wrong with an argument that has to be a tensor of this dtype and shape on GPU `index`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} has strides {t.stride()}: it must be contiguous, its last axis and its heads dense")


def _index(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _dense(t, name, index, dtype, shape):
    """Address of a contiguous tensor of this dtype and shape on GPU `index`."""
    try:
        if t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, index, dtype, shape)


def _scratch(t, name, index):
    """Address and bytes of a workspace."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.is_contiguous()):
        _refuse(t, name, index, None, None)
    return t.data_ptr(), t.numel() * t.element_size()


def _rows(t, name, index, dtype, shape):
    """[N, heads, d] with dense rows of heads: (address, elements between tokens)."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.shape == shape):
        _refuse(t, name, index, dtype, shape)
    N, H, d = shape
    sn, sh, sd = t.stride()
    if sd != 1 or (sh != d and H > 1):
        _refuse(t, name, index, dtype, shape)
    return t.data_ptr(), (sn if N > 1 else H * d)


def _kv_pools(k_pool, v_pool, index, dtype, Hk, d):
    """The pools' addresses, their common strides (page, head, row), pages and page size."""
    for t, name in ((k_pool, "k_pool"), (v_pool, "v_pool")):
        if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.dim() == 4):
            _refuse(t, name, index, dtype, None if isinstance(t, torch.Tensor) and t.dim() == 4 else ("pages", Hk, "page", d))
    shape, st = k_pool.shape, k_pool.stride()
    if shape[1] != Hk or shape[3] != d or v_pool.shape != shape:
        raise ValueError(f"the pools have shapes {tuple(shape)} and {tuple(v_pool.shape)}, expected [pages, {Hk}, page, {d}]")
    if st[3] != 1 or v_pool.stride() != st:
        raise ValueError("k_pool and v_pool must have the same strides and dense rows")
    if 1 in shape:                           # an axis of one entry has no stride that matters
        st = [st[i] if shape[i] > 1 else d for i in range(3)]
    return k_pool.data_ptr(), v_pool.data_ptr(), st[0], st[1], st[2], shape[0], shape[2]


_I32 = torch.int32


def _batch(cu_q, kv_lens, page_table, index):
    if not (isinstance(page_table, torch.Tensor) and page_table.get_device() == index and page_table.dtype is _I32
            and page_table.dim() == 2 and page_table.is_contiguous()):
        _refuse(page_table, "page_table", index, _I32, None if isinstance(page_table, torch.Tensor)
                and page_table.dim() == 2 else ("nseq", "max_pages"))
    nseq, max_pages = page_table.shape
    return (_dense(cu_q, "cu_q", index, _I32, (nseq + 1,)), _dense(kv_lens, "kv_lens", index, _I32, (nseq,)),
            page_table.data_ptr(), nseq, max_pages)


def jet_attn_rope_append(q, k, v, q_gamma, k_gamma, inv_freq, cu_q, kv_lens, page_table, k_pool, v_pool, q_out=None, *,
                         eps=1e-6, interleaved=False, stream=None):
    """Per-head RMSNorm of q [N,Hq,d] and k [N,Hk,d] (gammas [d] float32, or
    both None: no norm), rotation of their first 2 * len(inv_freq) elements by
    position * inv_freq (None: no rotation), and the append of k and
    v [N,Hk,d] to the pools [pages,Hk,page,d]. q, k, v may be slices of one
    projection's output. cu_q [nseq+1], kv_lens [nseq] (new tokens included)
    and page_table [nseq,max_pages] are int32 on the GPU. q_out may be q
    itself. Returns q_out [N,Hq,d]."""
    L = _lib or load_library()
    if _bind is not None and stream is None and q_out is not None:
        st = _bind.rope_append(L.at_jet_attn_rope_append, q, k, v, q_gamma, k_gamma, inv_freq, cu_q, kv_lens, page_table,
                               k_pool, v_pool, q_out, eps, interleaved)
        if st == 0:
            return q_out
        if st is not None:
            raise JetError("jet_attn_rope_append", st)
    index = _index(q, "q")
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q, k and v must be [N, heads, d]")
    dt, shape = q.dtype, q.shape
    N, Hq, d = shape
    Hk = k.shape[1]
    code, kv_shape = _dt(q), (N, Hk, d)
    qp, qs = _rows(q, "q", index, dt, shape)
    kp, ks = _rows(k, "k", index, dt, kv_shape)
    vp, vs = _rows(v, "v", index, dt, kv_shape)
    kpool, vpool, ps, hs, rs, n_pages, page = _kv_pools(k_pool, v_pool, index, dt, Hk, d)
    cu, kl, pt, nseq, max_pages = _batch(cu_q, kv_lens, page_table, index)
    gq = None if q_gamma is None else _dense(q_gamma, "q_gamma", index, torch.float32, (d,))
    gk = None if k_gamma is None else _dense(k_gamma, "k_gamma", index, torch.float32, (d,))
    rot, fr = 0, None
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        fr = _dense(inv_freq, "inv_freq", index, torch.float32, (rot // 2,))

    def call(s):
        out = torch.empty((N, Hq, d), device=q.device, dtype=dt) if q_out is None else q_out
        op, os_ = _rows(out, "q_out", index, dt, shape)
        st = L.jet_attn_rope_append(qp, qs, kp, ks, vp, vs, gq, gk, eps, fr, rot, 1 if interleaved else 0, op, os_, kpool,
                                    vpool, ps, hs, rs, cu, kl, pt, nseq, N, max_pages, n_pages, page, Hq, Hk, d, code, s)
        if st:
            raise JetError("jet_attn_rope_append", st)
        return out
    return _issue(index, stream, call)


def jet_attn_paged_workspace_size(nseq: int, N: int, Hq: int, Hk: int, d: int, dtype=torch.bfloat16) -> int:
    """Workspace bytes of jet_attn_paged for a batch of nseq sequences and N new tokens."""
    return int(load_library().jet_attn_paged_workspace_size(nseq, N, Hq, Hk, d,
                                                            JET_BF16 if dtype == torch.bfloat16 else JET_F32))


def jet_attn_paged(q, k_pool, v_pool, cu_q, kv_lens, page_table, max_new: int = 0, o=None, workspace=None, *,
                   window: int = 0, scale: float | None = None, stream=None):
    """Causal attention of the new tokens q [N,Hq,d] over the cached positions
    of their sequences (append theirs first): pools [pages,Hk,page,d], cu_q,
    kv_lens and page_table as in jet_attn_rope_append. window: positions a
    token sees, its own included (0: all). scale: 1/sqrt(d) by default.
    max_new: the largest number of new tokens of a sequence; it only chooses
    the kernel (0: by their average, slow for a long piece among many single
    tokens). In bf16 the softmax weights are rounded to bf16 before their
    product with V. Returns o [N,Hq,d]."""
    L = _lib or load_library()
    if _bind is not None and stream is None and workspace is not None and o is not None:
        st = _bind.attn_paged(L.at_jet_attn_paged, q, k_pool, v_pool, cu_q, kv_lens, page_table, max_new, o, workspace,
                              window, scale)
        if st == 0:
            return o
        if st is not None:
            raise JetError("jet_attn_paged", st)
    index = _index(q, "q")
    if q.dim() != 3 or not isinstance(k_pool, torch.Tensor) or k_pool.dim() != 4:
        raise ValueError("q must be [N, Hq, d] and the pools [pages, Hk, page, d]")
    dt, shape = q.dtype, q.shape
    N, Hq, d = shape
    code, Hk = _dt(q), k_pool.shape[1]
    qp, qs = _rows(q, "q", index, dt, shape)
    kpool, vpool, ps, hs, rs, n_pages, page = _kv_pools(k_pool, v_pool, index, dt, Hk, d)
    cu, kl, pt, nseq, max_pages = _batch(cu_q, kv_lens, page_table, index)

    def call(s):
        out = torch.empty((N, Hq, d), device=q.device, dtype=dt) if o is None else o
        ws = workspace
        if ws is None:
            ws = torch.empty(max(16, L.jet_attn_paged_workspace_size(nseq, N, Hq, Hk, d, code)), device=q.device,
                             dtype=torch.uint8)
        wp, wn = _scratch(ws, "workspace", index)
        st = L.jet_attn_paged(qp, qs, kpool, vpool, ps, hs, rs, cu, kl, pt, _dense(out, "o", index, dt, shape), wp, wn,
                              nseq, N, max_new, max_pages, n_pages, page, Hq, Hk, d, window,
                              d ** -0.5 if scale is None else scale, code, s)
        if st:
            raise JetError("jet_attn_paged", st)
        return out
    return _issue(index, stream, call)


# ---------------------------------------------------------------- cache entries
def _entries(pools, what="pools"):
    """Host arrays (addresses, entry bytes, entry strides) of pools with the
    same number of entries along their first axis, each entry dense."""
    if isinstance(pools, torch.Tensor) or len(pools) == 0:
        raise TypeError(f"{what} must be a non-empty list of tensors")
    index = _index(pools[0], f"{what}[0]")
    shape, dtype = pools[0].shape, pools[0].dtype
    entries = shape[0] if len(shape) else 0
    base, size, step = [], [], []
    for t in pools:
        if base and isinstance(t, torch.Tensor) and t.get_device() == index and t.shape == shape and t.dtype is dtype \
                and t.stride() == stride:        # laid out as the first one
            base.append(t.data_ptr())
            size.append(size[0])
            step.append(step[0])
            continue
        if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.dim() >= 2 and t.shape[0] == entries):
            _refuse(t, f"a tensor of {what}", index, None, (entries, "..."))
        es = t.element_size()
        if t.is_contiguous():
            per = t.numel() // max(1, entries)
        else:      # an entry's dimensions in any order, without gaps
            per = 1
            for st, sz in sorted((t.stride(j), t.shape[j]) for j in range(1, t.dim()) if t.shape[j] > 1):
                if st != per:
                    raise ValueError(f"the entries of {what} must be dense (strides {t.stride()})")
                per *= sz
        if not base:
            stride = t.stride()
        base.append(t.data_ptr())
        size.append(per * es)
        step.append(t.stride(0) * es if entries > 1 else per * es)
    return array("q", base), array("q", size), array("q", step), len(base), entries, index


def _host_ints(x, name):
    """Entry numbers as a host int32 array (a list, tuple or CPU tensor)."""
    if isinstance(x, torch.Tensor):
        if x.is_cuda:
            raise TypeError(f"{name} must be on the host: it is checked before the launch")
        x = x.tolist()
    return array("i", x)


def _at(a):
    """Address of a host array."""
    return a.buffer_info()[0] if len(a) else None


def jet_cache_copy(pools, src, dst, *, stream=None) -> None:
    """In every pool (tensors [entries, ...] with the same number of entries,
    each entry dense), entry dst[i] becomes a copy of entry src[i]. src and dst
    are host lists; a destination appears once and is no source."""
    L = _lib or load_library()
    if _bind is not None and stream is None:
        st = _bind.cache_copy(L.at_jet_cache_copy, pools, src, dst)
        if st == 0:
            return
        if st is not None:
            raise JetError("jet_cache_copy", st)
    base, size, step, n_pools, n_entries, index = _entries(pools)
    a, b = _host_ints(src, "src"), _host_ints(dst, "dst")
    if len(a) != len(b):
        raise ValueError(f"{len(a)} sources for {len(b)} destinations")
    st = _issue(index, stream, lambda s: L.jet_cache_copy(_at(base), _at(size), _at(step), n_pools, n_entries, _at(a),
                                                          _at(b), len(a), s))
    if st:
        raise JetError("jet_cache_copy", st)


def jet_cache_compact_workspace_size(n_pages: int) -> int:
    """Workspace bytes of jet_cache_compact."""
    return int(load_library().jet_cache_compact_workspace_size(n_pages))


def jet_cache_compact(pools, page_table, kv_lens, page_size: int, page_table_out=None, n_live=None, workspace=None, *,
                      stream=None):
    """Move the live pages (those that page_table [nseq,max_pages] names within
    kv_lens [nseq]) of the pools [pages, ...] to the lowest entries. Returns
    (page_table_out, n_live [1]): the rewritten tables (page_table itself may
    be given) and the number of live pages, on the GPU."""
    L = _lib or load_library()
    if _bind is not None and stream is None and workspace is not None:
        st = _bind.cache_compact(L.at_jet_cache_compact, pools, page_table, kv_lens, page_size, page_table_out, n_live,
                                 workspace)
        if st == 0:
            return page_table_out, n_live
        if st is not None:
            raise JetError("jet_cache_compact", st)
    base, size, step, n_pools, n_pages, index = _entries(pools)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [nseq, max_pages]")
    shape = page_table.shape
    nseq, max_pages = shape
    pt = _dense(page_table, "page_table", index, _I32, shape)
    kl = _dense(kv_lens, "kv_lens", index, _I32, (nseq,))

    def call(s):
        out = torch.empty_like(page_table) if page_table_out is None else page_table_out
        live = torch.empty(1, device=page_table.device, dtype=_I32) if n_live is None else n_live
        ws = workspace
        if ws is None:
            ws = torch.empty(max(16, L.jet_cache_compact_workspace_size(n_pages)), device=page_table.device,
                             dtype=torch.uint8)
        wp, wn = _scratch(ws, "workspace", index)
        st = L.jet_cache_compact(_at(base), _at(size), _at(step), n_pools, n_pages, page_size, pt, kl, nseq, max_pages,
                                 _dense(out, "page_table_out", index, _I32, shape),
                                 _dense(live, "n_live", index, _I32, (1,)), wp, wn, s)
        if st:
            raise JetError("jet_cache_compact", st)
        return out, live
    return _issue(index, stream, call)


def jet_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return int(load_library().jet_device_error(_stream(stream)))


def jet_status_string(status: int) -> str:
    return load_library().jet_status_string(status).decode()


def jet_launch_count() -> int:
    return int(load_library().jet_launch_count())


def jet_jetblock_layer_workspace_size(B: int, T: int, D: int, H: int, dk: int, dv: int) -> int:
    """Workspace bytes of jet_jetblock_layer (0: not a supported shape)."""
    return int(load_library().jet_jetblock_layer_workspace_size(B, T, D, H, dk, dv))


def jet_jetblock_layer(x, Wq, Wk, Wv, Wg, Wb, Wz, Wo, gamma, W1, W2, hist_in=None, hist_out=None, S0=None, S_out=None,
                       y=None, workspace=None, *, stream=None):
    """The JetBlock layer: x [B,T,D] bf16 -> y [B,T,D] (projections, mixer,
    per-head RMSNorm with gamma [dv] and SiLU output gate, output projection).
    Wq, Wk [D,H*dk]; Wv, Wz [D,H*dv]; Wg, Wb [D,H]; Wo [H*dv,D]; W1, W2 the
    generator's. S0 / S_out [B,H,dv,dk] float32 (may be the same tensor: with
    T = 1 the state advances in place); hist_in / hist_out [B,3,H,dv].
    Returns (y, S_out)."""
    L = load_library()
    B, T, D = x.shape
    H = Wg.shape[1]
    dk = Wq.shape[1] // H
    dv = Wv.shape[1] // H
    bf = torch.bfloat16
    if y is None:
        y = torch.empty((B, T, D), device=x.device, dtype=bf)
    if S_out is None:
        S_out = torch.empty((B, H, dv, dk), device=x.device, dtype=torch.float32)
    if workspace is None:
        workspace = torch.empty(max(16, jet_jetblock_layer_workspace_size(B, T, D, H, dk, dv)), device=x.device,
                                dtype=torch.uint8)
    st = L.jet_jetblock_layer(
        _ptr(x, "x", bf), _ptr(Wq, "Wq", bf, (D, H * dk)), _ptr(Wk, "Wk", bf, (D, H * dk)),
        _ptr(Wv, "Wv", bf, (D, H * dv)), _ptr(Wg, "Wg", bf, (D, H)), _ptr(Wb, "Wb", bf, (D, H)),
        _ptr(Wz, "Wz", bf, (D, H * dv)), _ptr(Wo, "Wo", bf, (H * dv, D)), _ptr(gamma, "gamma", torch.float32, (dv,)),
        _ptr(W1, "W1", bf), _ptr(W2, "W2", bf), _ptr(hist_in, "hist_in", bf, (B, 3, H, dv)),
        _ptr(hist_out, "hist_out", bf, (B, 3, H, dv)), _ptr(S0, "S0", torch.float32, (B, H, dv, dk)),
        _ptr(S_out, "S_out", torch.float32, (B, H, dv, dk)), _ptr(y, "y", bf, (B, T, D)), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), B, T, D, H, dk, dv, W1.shape[1], W2.shape[1] // H, JET_BF16,
        _stream(stream))
    _check("jet_jetblock_layer", st)
    return y, S_out
