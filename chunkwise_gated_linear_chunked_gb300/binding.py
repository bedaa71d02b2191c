"""Thin ctypes binding of libgla (``include/gla.h``): argument marshalling only.  The layer operators' usual calls
take a shorter way to the same C functions, through the ``_calls`` module, where it could be built.

Every step of the forward runs in libgla's CUDA kernels; torch supplies device memory and streams.  There is
no CPU fallback: if ``_build/libgla.so`` is missing the import fails loudly (run
``chunkwise_gated_linear_chunked_gb300.build.build()`` or ``__graft_entry__.build()`` first).
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import math
import os
import threading

import torch

from .build import LIB, calls_lib

GLA_OK, GLA_ERR_INVALID_ARG, GLA_ERR_UNSUPPORTED, GLA_ERR_ALIGNMENT, GLA_ERR_WORKSPACE, GLA_ERR_CUDA, \
    GLA_ERR_TIMEOUT, GLA_ERR_RANGE = range(8)
GLA_F32, GLA_BF16, GLA_BF16_OBF16, GLA_F16, GLA_BF16_GF32, GLA_F16_GF32, GLA_F16_OF16 = 0, 1, 2, 3, 4, 5, 6
GLA_HEAD_FIRST = 0x100   # OR-ed into the dtype code: [B, H, T, *] tensors
GLA_RES_F32 = 0x200      # OR-ed into the dtype code of the norms: fp32 residual stream

EXPORTS = ("gla_fwd", "gla_fwd_workspace_size", "gla_get_status", "gla_strerror", "gla_chunk_local_cumsum",
           "gla_profile_events", "gla_profile_launches", "gla_kernel_name", "gla_fwd_noalloc", "gla_bwd",
           "gla_bwd_workspace_size", "gla_ttt_linear_fwd", "gla_ttt_workspace_size", "gla_wy_fwd",
           "gla_wy_workspace_size", "gla_fwd_host", "gla_fwd_host_workspace_size", "gla_scan_fwd", "gla_scan_bwd",
           "gla_scan_step", "gla_scan_workspace_size", "gla_step", "gla_norm_fwd", "gla_norm_quant_fwd",
           "gla_norm_bwd", "gla_norm_bwd_workspace_size", "gla_scan_shared_workspace", "gla_delta_fwd",
           "gla_delta_fwd_workspace_size", "gla_delta_bwd", "gla_delta_bwd_workspace_size", "gla_delta_step",
           "gla_group_norm_fwd", "gla_group_norm_bwd", "gla_group_norm_workspace_size")

if not os.path.exists(LIB):
    raise ImportError(f"libgla.so not built ({LIB}); call chunkwise_gated_linear_chunked_gb300.build.build()")

_lib = ctypes.CDLL(LIB)
_p, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_lib.gla_fwd.argtypes = [_p, _p, _p, _p, _p, _f, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _p, _sz, _p]
_lib.gla_fwd.restype = _i
_lib.gla_fwd_workspace_size.argtypes = [_i] * 8
_lib.gla_fwd_workspace_size.restype = _sz
_lib.gla_fwd_host.argtypes = [_p, _p, _p, _p, _p, _f, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _p, _sz, _p]
_lib.gla_fwd_host.restype = _i
_lib.gla_fwd_host_workspace_size.argtypes = [_i] * 9
_lib.gla_fwd_host_workspace_size.restype = _sz
_lib.gla_get_status.argtypes = [_p, _p]
_lib.gla_get_status.restype = _i
_lib.gla_strerror.argtypes = [_i]
_lib.gla_strerror.restype = ctypes.c_char_p
_lib.gla_chunk_local_cumsum.argtypes = [_p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _p]
_lib.gla_chunk_local_cumsum.restype = _i
_lib.gla_profile_events.argtypes = [_p, _i, _p]
_lib.gla_profile_events.restype = _i
_lib.gla_profile_launches.argtypes = []
_lib.gla_profile_launches.restype = _i
_lib.gla_kernel_name.argtypes = [_i]
_lib.gla_kernel_name.restype = ctypes.c_char_p
_lib.gla_bwd.argtypes = [_p, _p, _p, _p, _p, _f, _p, _p, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _i,
                         _i, _p, _sz, _p]
_lib.gla_bwd.restype = _i
_lib.gla_bwd_workspace_size.argtypes = [_i] * 8
_lib.gla_bwd_workspace_size.restype = _sz
_lib.gla_ttt_linear_fwd.argtypes = [_p, _p, _p, _p, _p, _p, _f, _f, _p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i,
                                    _i, _p, _sz, _p]
_lib.gla_ttt_linear_fwd.restype = _i
_lib.gla_wy_fwd.argtypes = [_p, _p, _p, _p, _p, _p, _p, _p] + [_i] * 9 + [_p, _sz, _p]
_lib.gla_wy_fwd.restype = _i
_lib.gla_wy_workspace_size.argtypes = [_i, _i, _i, _i]
_lib.gla_wy_workspace_size.restype = _sz
_lib.gla_ttt_workspace_size.argtypes = []
_lib.gla_ttt_workspace_size.restype = _sz
_i64 = ctypes.c_int64
_lib.gla_scan_fwd.argtypes = [_p] * 6 + [_i] * 4 + [_i64] * 2 + [_i, _p, _sz, _p]
_lib.gla_scan_fwd.restype = _i
_lib.gla_scan_bwd.argtypes = [_p] * 9 + [_i] * 4 + [_i64] * 3 + [_i, _p, _sz, _p]
_lib.gla_scan_bwd.restype = _i
_lib.gla_scan_step.argtypes = [_p] * 6 + [_i] * 3 + [_i64] * 2 + [_i, _p, _sz, _p]
_lib.gla_scan_step.restype = _i
_lib.gla_scan_workspace_size.argtypes = []
_lib.gla_scan_workspace_size.restype = _sz
_lib.gla_scan_shared_workspace.argtypes = []
_lib.gla_scan_shared_workspace.restype = _p
_lib.gla_step.argtypes = [_p] * 5 + [_f] + [_p] * 3 + [_i] * 6 + [_p, _sz, _p]
_lib.gla_step.restype = _i
_lib.gla_norm_fwd.argtypes = [_p] * 6 + [_i64, _i, _f, _i, _p]
_lib.gla_norm_fwd.restype = _i
_lib.gla_norm_quant_fwd.argtypes = [_p] * 7 + [_i64, _i, _f, _i, _i, _p]
_lib.gla_norm_quant_fwd.restype = _i
_lib.gla_norm_bwd.argtypes = [_p] * 8 + [_i64, _i, _i, _p, _sz, _p]
_lib.gla_norm_bwd.restype = _i
_lib.gla_norm_bwd_workspace_size.argtypes = [_i64, _i]
_lib.gla_norm_bwd_workspace_size.restype = _sz
_lib.gla_delta_fwd.argtypes = [_p] * 6 + [_f] + [_p] * 3 + [_i] * 8 + [_p, _p, _sz, _p]
_lib.gla_delta_fwd.restype = _i
_lib.gla_delta_fwd_workspace_size.argtypes = [_i] * 9
_lib.gla_delta_fwd_workspace_size.restype = _sz
_lib.gla_delta_bwd.argtypes = [_p] * 6 + [_f] + [_p] * 9 + [_i] * 8 + [_p, _p, _sz, _p]
_lib.gla_delta_bwd.restype = _i
_lib.gla_delta_bwd_workspace_size.argtypes = [_i] * 9
_lib.gla_delta_bwd_workspace_size.restype = _sz
_lib.gla_delta_step.argtypes = [_p] * 6 + [_f] + [_p] * 3 + [_i] * 7 + [_p, _p]
_lib.gla_delta_step.restype = _i
_lib.gla_group_norm_fwd.argtypes = [_p] * 6 + [_i64, _i64, _i, _i, _f, _i, _i, _p, _sz, _p]
_lib.gla_group_norm_fwd.restype = _i
_lib.gla_group_norm_bwd.argtypes = [_p] * 9 + [_i64, _i64, _i, _i, _i, _i, _p, _sz, _p]
_lib.gla_group_norm_bwd.restype = _i
_lib.gla_group_norm_workspace_size.argtypes = [_i64, _i64, _i, _i, _i, _i]
_lib.gla_group_norm_workspace_size.restype = _sz


class _NoCalls:
    """Stands for the ``_calls`` module where it is missing (no host compiler, another torch than it was built for): every
    call is left to the checked functions."""

    def __getattr__(self, name):
        return lambda *args: None


def _load_calls():
    spec = importlib.util.spec_from_file_location("_calls", calls_lib())
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError:
        return _NoCalls()
    return module


_calls = _load_calls()


class GlaError(RuntimeError):
    def __init__(self, code: int, what: str = "gla_fwd"):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} (code {code})")


def lib():
    return _lib


def strerror(code: int) -> str:
    return _lib.gla_strerror(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


DTYPE_CODE = {(torch.float32, torch.float32): GLA_F32, (torch.bfloat16, torch.float32): GLA_BF16,
              (torch.bfloat16, torch.bfloat16): GLA_BF16_OBF16, (torch.float16, torch.float32): GLA_F16}

# 16-bit q, k, v with an fp32 g (o fp32)
GF32_CODE = {torch.bfloat16: GLA_BF16_GF32, torch.float16: GLA_F16_GF32}


def _dtype_code(q, g, out_dtype, what):
    """The dtype code of a call: q, k, v share one dtype; g has it too, or is fp32 beside 16-bit q, k, v."""
    if g.dtype == q.dtype:
        code = DTYPE_CODE.get((q.dtype, out_dtype)) if out_dtype is not None else \
            {torch.float32: GLA_F32, torch.bfloat16: GLA_BF16, torch.float16: GLA_F16}.get(q.dtype)
    elif g.dtype == torch.float32 and out_dtype in (None, torch.float32):
        code = GF32_CODE.get(q.dtype)
    else:
        code = None
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"{what} dtypes q {q.dtype}, g {g.dtype} -> {out_dtype}")
    return code


_ws_lock = threading.Lock()
_ws_cache: dict = {}


def workspace_size(B, T, H, K, V, N, chunk=64, dtype=GLA_BF16) -> int:
    return int(_lib.gla_fwd_workspace_size(B, T, H, K, V, N, chunk, dtype))


def get_workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-initialised, cached device workspace of at least ``nbytes`` (one per device and stream use)."""
    device = torch.device(device)
    key = (device.index if device.index is not None else torch.cuda.current_device())
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
            _ws_cache[key] = ws
        return ws


def fwd_into(q, k, v, g, o, scale, h0, ht, cu_seqlens, N, B, T, H, K, V, chunk, dtype, workspace,
             stream=None) -> int:
    """Raw call: tensors (or None) are passed as device pointers, sizes as given.  Returns the code."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return int(_lib.gla_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o), float(scale), _ptr(h0), _ptr(ht),
                            _ptr(cu_seqlens), int(N), int(B), int(T), int(H), int(K), int(V), int(chunk),
                            int(dtype), _ptr(workspace), nbytes, _stream_handle(stream)))


def host_workspace_size(B, T, H, K, V, N, chunk, dtype, head_groups) -> int:
    return int(_lib.gla_fwd_host_workspace_size(int(B), int(T), int(H), int(K), int(V), int(N), int(chunk),
                                                int(dtype), int(head_groups)))


def fwd_host_into(q, k, v, g, o, scale, h0, ht, cu_seqlens, N, B, T, H, K, V, chunk, dtype, head_groups, workspace,
                  stream=None) -> int:
    """Raw call of gla_fwd_host: q, k, v, g, o, h0, ht, cu_seqlens are HOST tensors (or None), the workspace a
    device tensor.  Returns the code."""
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("o", o), ("h0", h0), ("ht", ht),
                    ("cu_seqlens", cu_seqlens)):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise GlaError(GLA_ERR_INVALID_ARG, f"gla_fwd_host: {name} must be a contiguous host tensor")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return int(_lib.gla_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(o), float(scale), _ptr(h0), _ptr(ht),
                                 _ptr(cu_seqlens), int(N), int(B), int(T), int(H), int(K), int(V), int(chunk),
                                 int(dtype), int(head_groups), _ptr(workspace), nbytes, _stream_handle(stream)))


def gla_fwd(q, k, v, g, scale=None, initial_state=None, output_final_state=True, cu_seqlens=None,
            chunk=64, out_dtype=None, stream=None, workspace=None, head_first=False):
    """GLA forward on the GPU.

    q, k, g: [B, T, H, K]; v: [B, T, H, V] (cuda, contiguous, all fp32, all bf16 or all fp16), or
    [B, H, T, *] with head_first=True (with cu_seqlens: [1, H, T, *]).  initial_state: optional fp32 [N, H, K, V].
    cu_seqlens: optional int32 [N+1] cuda offsets (B == 1).  out_dtype: fp32 (default) or, for bf16 inputs,
    bf16.  Returns (o in the layout of the inputs, final_state or None).
    """
    if head_first:
        B, H, T, K = q.shape
    else:
        B, T, H, K = q.shape
    V = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    out_dtype = out_dtype or torch.float32
    code = _dtype_code(q, g, out_dtype, "gla_fwd")
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g)):
        if (t.dtype != q.dtype and t is not g) or not t.is_cuda or not t.is_contiguous():
            raise GlaError(GLA_ERR_INVALID_ARG, f"gla_fwd: {name} must be a contiguous cuda {q.dtype} tensor")
    o = torch.empty(*((B, H, T, V) if head_first else (B, T, H, V)), dtype=out_dtype, device=q.device)
    ht = torch.empty(N, H, K, V, dtype=torch.float32, device=q.device) if output_final_state else None
    h0 = initial_state
    if h0 is not None and (h0.dtype != torch.float32 or not h0.is_contiguous()):
        raise GlaError(GLA_ERR_INVALID_ARG, "gla_fwd: initial_state must be a contiguous fp32 tensor")
    if cu_seqlens is not None and cu_seqlens.dtype != torch.int32:
        raise GlaError(GLA_ERR_INVALID_ARG, "gla_fwd: cu_seqlens must be int32")
    if workspace is None:
        workspace = get_workspace(workspace_size(B, T, H, K, V, N, chunk, code), q.device)
    if head_first:
        code |= GLA_HEAD_FIRST
    rc = fwd_into(q, k, v, g, o, scale, h0, ht, cu_seqlens, N, B, T, H, K, V, chunk, code, workspace,
                  stream)
    if rc != GLA_OK:
        raise GlaError(rc)
    return o, ht


def bwd_workspace_size(B, T, H, K, V, N, chunk=64, dtype=GLA_BF16) -> int:
    return int(_lib.gla_bwd_workspace_size(B, T, H, K, V, N, chunk, dtype))


def bwd_into(q, k, v, g, do, scale, h0, dht, dq, dk, dv, dg, dh0, cu_seqlens, N, B, T, H, K, V, chunk, dtype,
             workspace, stream=None) -> int:
    """Raw backward call: tensors (or None) are passed as device pointers.  Returns the code."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return int(_lib.gla_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(do), float(scale), _ptr(h0), _ptr(dht),
                            _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dh0), _ptr(cu_seqlens), int(N), int(B),
                            int(T), int(H), int(K), int(V), int(chunk), int(dtype), _ptr(workspace), nbytes,
                            _stream_handle(stream)))


def gla_bwd(q, k, v, g, do, scale=None, initial_state=None, dht=None, cu_seqlens=None, chunk=64, stream=None,
            workspace=None, want_dh0=True, head_first=False):
    """GLA backward on the GPU for L = sum(o * do) + sum(ht * dht).

    q, k, g: [B, T, H, K]; v, do: [B, T, H, V] (cuda, contiguous, all fp32, bf16 or fp16), or [B, H, T, *]
    with head_first=True.  initial_state and dht: optional fp32 [N, H, K, V].  Returns fp32 (dq, dk, dv, dg,
    dh0 or None), in the layout of the inputs.
    """
    if head_first:
        B, H, T, K = q.shape
    else:
        B, T, H, K = q.shape
    V = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if scale is None:
        scale = K ** -0.5
    code = _dtype_code(q, g, None, "gla_bwd")
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("do", do)):
        if (t.dtype != q.dtype and t is not g) or not t.is_cuda or not t.is_contiguous():
            raise GlaError(GLA_ERR_INVALID_ARG, f"gla_bwd: {name} must be a contiguous cuda {q.dtype} tensor")
    for name, t in (("initial_state", initial_state), ("dht", dht)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
            raise GlaError(GLA_ERR_INVALID_ARG, f"gla_bwd: {name} must be a contiguous fp32 tensor")
    f32 = dict(dtype=torch.float32, device=q.device)
    shk, shv = ((B, H, T, K), (B, H, T, V)) if head_first else ((B, T, H, K), (B, T, H, V))
    dq, dk, dg = (torch.empty(*shk, **f32) for _ in range(3))
    dv = torch.empty(*shv, **f32)
    dh0 = torch.empty(N, H, K, V, **f32) if want_dh0 else None
    if workspace is None:
        workspace = get_workspace(bwd_workspace_size(B, T, H, K, V, N, chunk, code), q.device)
    if head_first:
        code |= GLA_HEAD_FIRST
    rc = bwd_into(q, k, v, g, do, scale, initial_state, dht, dq, dk, dv, dg, dh0, cu_seqlens, N, B, T, H, K, V,
                  chunk, code, workspace, stream)
    if rc != GLA_OK:
        raise GlaError(rc, "gla_bwd")
    return dq, dk, dv, dg, dh0


def ttt_linear_fwd(q, k, v, w, b, eta, scale=None, eps=1e-6, chunk=16, initial_state=None,
                   initial_state_bias=None, output_final_state=True, cu_seqlens=None, stream=None, workspace=None):
    """TTT-linear forward on the GPU.  q, k, v: [B, T, H, D] (cuda, contiguous, fp32 / bf16 / fp16); w, b:
    fp32 [H, D]; eta: fp32 [B, T, H] (or [..., 1]).  Returns fp32 (o [B, T, H, D], ht [N, H, D, D] or None,
    hbt [N, H, D] or None)."""
    B, T, H, D = q.shape
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if scale is None:
        scale = D ** -0.5
    code = {torch.float32: GLA_F32, torch.bfloat16: GLA_BF16, torch.float16: GLA_F16}.get(q.dtype)
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"gla_ttt_linear_fwd dtype {q.dtype}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != q.dtype or not t.is_cuda or not t.is_contiguous() or t.shape != q.shape:
            raise GlaError(GLA_ERR_INVALID_ARG, f"gla_ttt_linear_fwd: {name} must be a contiguous cuda tensor like q")
    f32 = lambda x: None if x is None else x.contiguous().float()
    w, b, eta = f32(w), f32(b), f32(eta)
    h0, hb0 = f32(initial_state), f32(initial_state_bias)
    o = torch.empty(B, T, H, D, dtype=torch.float32, device=q.device)
    ht = torch.empty(N, H, D, D, dtype=torch.float32, device=q.device) if output_final_state else None
    hbt = torch.empty(N, H, D, dtype=torch.float32, device=q.device) if output_final_state else None
    if workspace is None:
        workspace = get_workspace(int(_lib.gla_ttt_workspace_size()), q.device)
    nbytes = workspace.numel() * workspace.element_size()
    rc = int(_lib.gla_ttt_linear_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(b), _ptr(eta), float(scale),
                                     float(eps), _ptr(h0), _ptr(hb0), _ptr(o), _ptr(ht), _ptr(hbt), _ptr(cu_seqlens),
                                     N, B, T, H, D, int(chunk), code, _ptr(workspace), nbytes,
                                     _stream_handle(stream)))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_ttt_linear_fwd")
    return o, ht, hbt


def wy_into(k, v, beta, A, g, w, u, cu_seqlens, N, B, T, H, HV, K, V, chunk, dtype, workspace, stream=None) -> int:
    """Raw call of gla_wy_fwd: tensors (or None) are passed as device pointers, sizes as given.  Returns the
    code."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return int(_lib.gla_wy_fwd(_ptr(k), _ptr(v), _ptr(beta), _ptr(A), _ptr(g), _ptr(w), _ptr(u), _ptr(cu_seqlens),
                               int(N), int(B), int(T), int(H), int(HV), int(K), int(V), int(chunk), int(dtype),
                               _ptr(workspace), nbytes, _stream_handle(stream)))


def wy_fwd(k, v, beta, A, g=None, cu_seqlens=None, out_dtype=None, stream=None, workspace=None):
    """WY representation forward of the gated delta rule on the GPU: per chunk of BT = A.shape[-1] rows,
    u = A (v * beta) and w = A (k * beta * 2^g).  k: [B, T, H, K]; v: [B, T, HV, V]; beta: [B, T, HV];
    A: [B, T, HV, BT] (k, v, beta, A: one dtype, fp32 / bf16 / fp16, cuda, contiguous); g: fp32 [B, T, HV]
    (log2 units) or None.  Returns (w [B, T, HV, K], u [B, T, HV, V]) in fp32, or in bf16 when
    ``out_dtype=torch.bfloat16`` with bf16 inputs."""
    B, T, H, K = k.shape
    HV, V, BT = v.shape[2], v.shape[3], A.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    code = {torch.float32: GLA_F32, torch.bfloat16: GLA_BF16, torch.float16: GLA_F16}.get(k.dtype)
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"gla_wy_fwd dtype {k.dtype}")
    odt = torch.float32
    if out_dtype == torch.bfloat16:
        if code != GLA_BF16:
            raise GlaError(GLA_ERR_UNSUPPORTED, "gla_wy_fwd: bf16 outputs need bf16 inputs")
        code, odt = GLA_BF16_OBF16, torch.bfloat16
    for name, t in (("k", k), ("v", v), ("beta", beta), ("A", A)):
        if t.dtype != k.dtype or not t.is_cuda or not t.is_contiguous():
            raise GlaError(GLA_ERR_INVALID_ARG, f"gla_wy_fwd: {name} must be a contiguous cuda tensor of k's dtype")
    if g is not None:
        g = g.contiguous().float()
    w = torch.empty(B, T, HV, K, dtype=odt, device=k.device)
    u = torch.empty(B, T, HV, V, dtype=odt, device=k.device)
    if workspace is None:
        need = int(_lib.gla_wy_workspace_size(T, N, BT, int(cu_seqlens is not None)))
        workspace = get_workspace(max(need, 256), k.device)
    nbytes = workspace.numel() * workspace.element_size()
    rc = int(_lib.gla_wy_fwd(_ptr(k), _ptr(v), _ptr(beta), _ptr(A), _ptr(g), _ptr(w), _ptr(u), _ptr(cu_seqlens), N, B,
                             T, H, HV, K, V, int(BT), code, _ptr(workspace), nbytes, _stream_handle(stream)))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_wy_fwd")
    return w, u


# ---------------------------------------------------------------------------------------------------------
# Operators beside the chunkwise kernels: vector-state recurrence, one-token updates, residual norm
# ---------------------------------------------------------------------------------------------------------

# (x, gate, output) types of the recurrence -> dtype code
SCAN_CODE = {(torch.float32, torch.float32, torch.float32): GLA_F32,
             (torch.bfloat16, torch.bfloat16, torch.float32): GLA_BF16,
             (torch.bfloat16, torch.bfloat16, torch.bfloat16): GLA_BF16_OBF16,
             (torch.float16, torch.float16, torch.float32): GLA_F16,
             (torch.float16, torch.float16, torch.float16): GLA_F16_OF16,
             (torch.bfloat16, torch.float32, torch.float32): GLA_BF16_GF32,
             (torch.float16, torch.float32, torch.float32): GLA_F16_GF32}
_NORM_CODE = {torch.float32: GLA_F32, torch.bfloat16: GLA_BF16, torch.float16: GLA_F16}
_STATUS_BYTES = int(_lib.gla_scan_workspace_size())

_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle on a device, without a Stream object
_current_device = torch._C._cuda_getDevice
_shared_status: dict = {}   # by device: the address of the library's own status workspace


def _status_workspace(workspace, device: int):
    """(address, bytes) of a call's status workspace on the current device: the caller's, or the library's own, which
    calls on any stream share (they write it only to report an error)."""
    if workspace is not None:
        return workspace.data_ptr(), workspace.numel() * workspace.element_size()
    at = _shared_status.get(device)
    if at is None:
        at = _shared_status[device] = _lib.gla_scan_shared_workspace()
    return at, _STATUS_BYTES


def layer_status(device=None, stream=None) -> int:
    """What the kernels of ``scan_fwd``, ``scan_bwd``, ``scan_step`` and ``gla_step`` calls without a workspace of their
    own, and of ``delta_fwd``, ``delta_bwd`` and ``delta_step`` calls without a ``status`` of their own, have reported on a device (default: the current one) since the last look: GLA_OK, or the code of the first error,
    which this call clears.  Waits for ``stream`` (default: the current one); what runs on other streams may report
    later.  One word serves all streams; a call's own ``workspace`` (256 zeroed bytes) and ``get_status`` tell its errors
    apart."""
    with torch.cuda.device(device):
        at, _ = _status_workspace(None, torch.cuda.current_device())
        return int(_lib.gla_get_status(at, _stream_handle(stream)))


def _on_stream(fn):
    """Runs a call on its ``stream`` argument (or the current stream) of its first tensor's device: the outputs and
    the workspace are then allocated on the stream that the kernels run on.  The inputs are the caller's to order."""
    @functools.wraps(fn)
    def call(first, *args, stream, **kw):
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise GlaError(GLA_ERR_INVALID_ARG, f"{fn.__name__[1:-8]}: the first argument must be a cuda tensor")
        if stream is None and first.get_device() == _current_device():
            return fn(first, *args, **kw)
        with torch.cuda.stream(stream), torch.cuda.device(first.device):
            return fn(first, *args, **kw)
    return call


def _all_like(t, others):
    """Whether every tensor of ``others`` is contiguous and has t's dtype, shape and device, and t is contiguous."""
    dtype, shape, device = t.dtype, t.shape, t.get_device()
    for o in others:
        if o.dtype is not dtype or o.shape != shape or o.get_device() != device or not o.is_contiguous():
            return False
    return t.is_contiguous()


def _check(what, name, t, dtype, shape, device):
    """``t`` is a contiguous tensor of this dtype and shape on cuda device number ``device``."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: {name} must be a contiguous {dtype} tensor of shape "
                                            f"{tuple(shape)} on cuda:{device}")


def _row_stride(what, name, t, shape, device):
    """Elements between consecutive rows of a [..., D] tensor: the channels adjacent, the rows evenly spaced (a
    contiguous tensor, or a column range of one)."""
    if t.shape != shape or t.get_device() != device:
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: {name} must have shape {tuple(shape)} on cuda:{device}")
    D = shape[-1]
    if t.is_contiguous():
        return D
    # the innermost of the outer dimensions that has more than one row gives the spacing, and the others follow it
    rows, ld = 1, None
    for size, stride in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size > 1:
            ld = stride if ld is None else ld
            if stride != ld * rows:
                ld = -1
                break
        rows *= size
    ld = D if ld is None else ld
    if (D > 1 and t.stride(-1) != 1) or ld < D:
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: {name} must have adjacent channels and evenly spaced rows "
                                            f"(a contiguous tensor or a column range of one)")
    return ld


def _at(t):
    return None if t is None else t.data_ptr()


def _pack(what, shape, cu_seqlens, device):
    """(N, B, T, D) of a [B, T, D] recurrence, dense or packed."""
    if len(shape) != 3:
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: expected [B, T, D] tensors, got shape {tuple(shape)}")
    B, T, D = shape
    if cu_seqlens is None:
        return B, B, T, D
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or \
            cu_seqlens.get_device() != device or not cu_seqlens.is_contiguous():
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: cu_seqlens must be a contiguous int32 vector on cuda:{device}")
    return cu_seqlens.numel() - 1, B, T, D


def scan_fwd(x, g, initial_state=None, output_final_state=True, cu_seqlens=None, out_dtype=None, out=None,
             workspace=None, stream=None):
    """Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t on the GPU.

    x, g: [B, T, D], cuda, channels adjacent and rows evenly spaced (contiguous, or column ranges of one projection's
    output); both fp32, bf16 or fp16, or a 16-bit x with an fp32 g.  initial_state: fp32 [N, D] or None.
    cu_seqlens: int32 [N+1] cuda offsets (B == 1).  out_dtype: x's type (default; fp32 beside an fp32 g) or fp32.
    out: optional [B, T, D] tensor for h.  stream=: the stream to run on.  Returns (h, ht fp32 [N, D] or None).
    Offsets are checked on the device: a sequence whose offsets are bad is left out (its outputs are undefined) and
    reported, see ``layer_status``.
    """
    if out is None and workspace is None and stream is None:
        got = _calls.scan_fwd(x, g, initial_state, output_final_state, cu_seqlens, out_dtype)
        if got is not None:
            return got
    return _scan_fwd_checked(x, g, initial_state, output_final_state, cu_seqlens, out_dtype, out, workspace,
                             stream=stream)


@_on_stream
def _scan_fwd_checked(x, g, initial_state, output_final_state, cu_seqlens, out_dtype, out, workspace):
    shape, device = x.shape, x.get_device()
    N, B, T, D = _pack("gla_scan_fwd", shape, cu_seqlens, device)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else g.dtype
    code = SCAN_CODE.get((x.dtype, g.dtype, out_dtype))
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"gla_scan_fwd dtypes x {x.dtype}, g {g.dtype} -> {out_dtype}")
    ldx = _row_stride("gla_scan_fwd", "x", x, shape, device)
    ldg = _row_stride("gla_scan_fwd", "g", g, shape, device)
    if initial_state is not None:
        _check("gla_scan_fwd", "initial_state", initial_state, torch.float32, (N, D), device)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=device)
    else:
        _check("gla_scan_fwd", "out", out, out_dtype, shape, device)
    ht = torch.empty(N, D, dtype=torch.float32, device=device) if output_final_state else None
    rc = _lib.gla_scan_fwd(x.data_ptr(), g.data_ptr(), out.data_ptr(), _at(initial_state), _at(ht), _at(cu_seqlens),
                           N, B, T, D, ldx, ldg, code, *_status_workspace(workspace, device), _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_scan_fwd")
    return out, ht


def scan_bwd(g, h, dh, initial_state=None, dht=None, cu_seqlens=None, dx_dtype=None, want_dh0=True, dx=None,
             dg=None, workspace=None, stream=None):
    """Gradients of ``scan_fwd`` for L = sum(h * dh) + sum(ht * dht), from its gate g and its output h.

    g as for scan_fwd; h, dh: [B, T, D] contiguous, of the forward's out_dtype; initial_state, dht: fp32 [N, D] or
    None.  dx_dtype: x's type (default: g's).  dx, dg: optional tensors to write, which may be column ranges of one
    gradient.  Returns (dx, dg in g's type, dh0 fp32 [N, D] or None).  Bad offsets as for scan_fwd.
    """
    if dx is None and dg is None and workspace is None and stream is None:
        got = _calls.scan_bwd(g, h, dh, initial_state, dht, cu_seqlens, dx_dtype, want_dh0)
        if got is not None:
            return got
    return _scan_bwd_checked(g, h, dh, initial_state, dht, cu_seqlens, dx_dtype, want_dh0, dx, dg, workspace,
                             stream=stream)


@_on_stream
def _scan_bwd_checked(g, h, dh, initial_state, dht, cu_seqlens, dx_dtype, want_dh0, dx, dg, workspace):
    shape, device = g.shape, g.get_device()
    N, B, T, D = _pack("gla_scan_bwd", shape, cu_seqlens, device)
    if dx_dtype is None:
        dx_dtype = g.dtype if dx is None else dx.dtype
    code = SCAN_CODE.get((dx_dtype, g.dtype, h.dtype))
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"gla_scan_bwd dtypes dx {dx_dtype}, g {g.dtype}, h {h.dtype}")
    ldg = _row_stride("gla_scan_bwd", "g", g, shape, device)
    _check("gla_scan_bwd", "h", h, h.dtype, shape, device)
    _check("gla_scan_bwd", "dh", dh, h.dtype, shape, device)
    for name, t in (("initial_state", initial_state), ("dht", dht)):
        if t is not None:
            _check("gla_scan_bwd", name, t, torch.float32, (N, D), device)
    lddx = lddg = D
    if dx is None:
        dx = torch.empty(shape, dtype=dx_dtype, device=device)
    elif dx.dtype != dx_dtype:
        raise GlaError(GLA_ERR_INVALID_ARG, f"gla_scan_bwd: dx must be a {dx_dtype} tensor")
    else:
        lddx = _row_stride("gla_scan_bwd", "dx", dx, shape, device)
    if dg is None:
        dg = torch.empty(shape, dtype=g.dtype, device=device)
    elif dg.dtype != g.dtype:
        raise GlaError(GLA_ERR_INVALID_ARG, f"gla_scan_bwd: dg must be a {g.dtype} tensor")
    else:
        lddg = _row_stride("gla_scan_bwd", "dg", dg, shape, device)
    dh0 = torch.empty(N, D, dtype=torch.float32, device=device) if want_dh0 else None
    rc = _lib.gla_scan_bwd(g.data_ptr(), h.data_ptr(), dh.data_ptr(), _at(initial_state), _at(dht), dx.data_ptr(),
                           dg.data_ptr(), _at(dh0), _at(cu_seqlens), N, B, T, D, ldg, lddx, lddg, code,
                           *_status_workspace(workspace, device), _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_scan_bwd")
    return dx, dg, dh0


def _pool(what, state, state_out, slots, B, tail, device):
    """(pool rows, the pool to write) of a one-token update."""
    if state.dim() != 1 + len(tail) or (slots is None and state.shape[0] != B):
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: state must be [{'S' if slots is not None else B}, "
                                            f"{', '.join(map(str, tail))}]")
    S = state.shape[0]
    _check(what, "state", state, torch.float32, (S, *tail), device)
    if state_out is None:
        state_out = state
    elif not _all_like(state, (state_out,)):
        _check(what, "state_out", state_out, torch.float32, (S, *tail), device)
    if slots is not None:
        _check(what, "slots", slots, torch.int32, (B,), device)
    return S, state_out


def scan_step(x, g, state, slots=None, state_out=None, out_dtype=None, workspace=None, stream=None):
    """One token of ``scan_fwd``'s recurrence for each of B sequences.

    x, g: [B, D] (types and strides as for scan_fwd); state: fp32 [S, D] pool, updated in place (or written to
    state_out, of which only the addressed rows are written); slots: int32 [B] cuda, the pool row of each sequence
    (-1: idle, its h is zeros; any other slot outside the pool likewise, and reported, see ``layer_status``), or None
    when S == B.  Returns h [B, D].
    """
    if workspace is None and stream is None:
        got = _calls.scan_step(x, g, state, slots, state_out, out_dtype)
        if got is not None:
            return got
    return _scan_step_checked(x, g, state, slots, state_out, out_dtype, workspace, stream=stream)


@_on_stream
def _scan_step_checked(x, g, state, slots, state_out, out_dtype, workspace):
    if x.dim() != 2:
        raise GlaError(GLA_ERR_INVALID_ARG, f"gla_scan_step: x must be [B, D], got shape {tuple(x.shape)}")
    shape, device = x.shape, x.get_device()
    B, D = shape
    if out_dtype is None:
        out_dtype = g.dtype
    code = SCAN_CODE.get((x.dtype, g.dtype, out_dtype))
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"gla_scan_step dtypes x {x.dtype}, g {g.dtype} -> {out_dtype}")
    ldx = _row_stride("gla_scan_step", "x", x, shape, device)
    ldg = _row_stride("gla_scan_step", "g", g, shape, device)
    S, state_out = _pool("gla_scan_step", state, state_out, slots, B, (D,), device)
    h = torch.empty(shape, dtype=out_dtype, device=device)
    rc = _lib.gla_scan_step(x.data_ptr(), g.data_ptr(), h.data_ptr(), state.data_ptr(), state_out.data_ptr(),
                            _at(slots), B, S, D, ldx, ldg, code, *_status_workspace(workspace, device),
                            _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_scan_step")
    return h


def gla_step(q, k, v, g, state, scale=None, slots=None, state_out=None, out_dtype=None, workspace=None, stream=None):
    """One token of ``gla_fwd``'s recurrence for each of B sequences: S = diag(exp g) S + k^T v, o = scale q S.

    q, k, g: [B, H, K]; v: [B, H, V] (contiguous; types as for gla_fwd); state: fp32 [S, H, K, V] pool, updated in
    place (or written to state_out); slots as for scan_step.  out_dtype: fp32 (default) or q's type.
    Returns o [B, H, V].
    """
    if workspace is None and stream is None:
        got = _calls.gla_step(q, k, v, g, state, scale, slots, state_out, out_dtype)
        if got is not None:
            return got
    return _gla_step_checked(q, k, v, g, state, scale, slots, state_out, out_dtype, workspace, stream=stream)


@_on_stream
def _gla_step_checked(q, k, v, g, state, scale, slots, state_out, out_dtype, workspace):
    if q.dim() != 3 or v.dim() != 3:
        raise GlaError(GLA_ERR_INVALID_ARG, "gla_step: q, k, g must be [B, H, K] and v [B, H, V]")
    device = q.get_device()
    B, H, K = q.shape
    V = v.shape[-1]
    out_dtype = out_dtype or torch.float32
    code = SCAN_CODE.get((q.dtype, g.dtype, out_dtype))
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"gla_step dtypes q {q.dtype}, g {g.dtype} -> {out_dtype}")
    if not (V == K and _all_like(q, (k, v, g))):   # the usual call at once, else one by one
        _check("gla_step", "q", q, q.dtype, (B, H, K), device)
        _check("gla_step", "k", k, q.dtype, (B, H, K), device)
        _check("gla_step", "v", v, q.dtype, (B, H, V), device)
        _check("gla_step", "g", g, g.dtype, (B, H, K), device)
    S, state_out = _pool("gla_step", state, state_out, slots, B, (H, K, V), device)
    o = torch.empty(B, H, V, dtype=out_dtype, device=device)
    rc = _lib.gla_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), o.data_ptr(),
                       K ** -0.5 if scale is None else scale, state.data_ptr(), state_out.data_ptr(), _at(slots), B, S,
                       H, K, V, code, *_status_workspace(workspace, device), _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_step")
    return o


def _norm_args(what, x, residual, weight, stream_dtype):
    """(rows, D, dtype code) of a norm of x whose residual stream has this type."""
    code = _NORM_CODE.get(x.dtype)
    if code is None or stream_dtype not in (x.dtype, torch.float32):
        raise GlaError(GLA_ERR_UNSUPPORTED, f"{what} dtypes x {x.dtype}, residual {stream_dtype}")
    if x.dim() < 1 or not x.is_contiguous():
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: x must be a contiguous [..., D] tensor")
    D = x.shape[-1]
    if D == 0:
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: no columns")
    if residual is not None:
        _check(what, "residual", residual, stream_dtype, x.shape, x.get_device())
    if weight is not None:
        _check(what, "weight", weight, torch.float32, (D,), x.get_device())
    return x.numel() // D, D, code if stream_dtype == x.dtype else code | GLA_RES_F32


def norm_fwd(x, residual=None, weight=None, eps=1e-6, stream=None):
    """Residual addition and root-mean-square norm over the last dimension: s = x + residual, y = s rstd weight.

    x: contiguous [..., D] fp32 / bf16 / fp16; residual: like x, or fp32; weight: fp32 [D] or None.
    Returns (y in x's type, s in the residual's type (x itself without a residual), rstd fp32 [...]).
    """
    if stream is None:
        got = _calls.norm_fwd(x, residual, weight, eps)
        if got is not None:
            return got
    return _norm_fwd_checked(x, residual, weight, eps, stream=stream)


@_on_stream
def _norm_fwd_checked(x, residual, weight, eps):
    stream_dtype, device = x.dtype if residual is None else residual.dtype, x.get_device()
    rows, D, code = _norm_args("gla_norm_fwd", x, residual, weight, stream_dtype)
    y = torch.empty_like(x)
    s = None if residual is None else torch.empty_like(residual)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
    rc = _lib.gla_norm_fwd(x.data_ptr(), _at(residual), _at(weight), y.data_ptr(), _at(s), rstd.data_ptr(), rows, D,
                           eps, code, _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_norm_fwd")
    return y, x if s is None else s, rstd


def norm_quant_fwd(x, residual=None, weight=None, eps=1e-6, group=0, stream=None):
    """``norm_fwd`` with its output in 8 bits: y is q times its scale.  group: columns of one scale, 128, or 0 for
    one scale per row.  Returns (q float8_e4m3fn [..., D], scales fp32 [..., ceil(D / group)], s, rstd)."""
    if stream is None:
        got = _calls.norm_quant_fwd(x, residual, weight, eps, group)
        if got is not None:
            return got
    return _norm_quant_fwd_checked(x, residual, weight, eps, group, stream=stream)


@_on_stream
def _norm_quant_fwd_checked(x, residual, weight, eps, group):
    stream_dtype, device = x.dtype if residual is None else residual.dtype, x.get_device()
    rows, D, code = _norm_args("gla_norm_quant_fwd", x, residual, weight, stream_dtype)
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=device)
    groups = -(-D // group) if group > 0 else 1
    scales = torch.empty(*x.shape[:-1], groups, dtype=torch.float32, device=device)
    s = None if residual is None else torch.empty_like(residual)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
    rc = _lib.gla_norm_quant_fwd(x.data_ptr(), _at(residual), _at(weight), q.data_ptr(), scales.data_ptr(), _at(s),
                                 rstd.data_ptr(), rows, D, eps, group, code, _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_norm_quant_fwd")
    return q, scales, x if s is None else s, rstd


def norm_bwd(s, rstd, dy, weight=None, ds=None, want_dw=True, workspace=None, stream=None):
    """Gradients of ``norm_fwd`` from its s and rstd, for the gradients dy of y and ds of s (or None).

    Returns (the gradient of x in dy's type, the gradient of the residual in s's type, dw fp32 [D] or None).  The
    first two are one tensor when the types are the same.  ``want_dw=False`` skips dw (also None without a weight).
    workspace: one of the caller's, for one call at a time (default: memory of the call's own).
    """
    if workspace is None and stream is None:
        got = _calls.norm_bwd(s, rstd, dy, weight, ds, want_dw, None)
        if got is not None:
            return got
    return _norm_bwd_checked(s, rstd, dy, weight, ds, want_dw, workspace, stream=stream)


@_on_stream
def _norm_bwd_checked(s, rstd, dy, weight, ds, want_dw, workspace):
    rows, D, code = _norm_args("gla_norm_bwd", dy, s, weight, s.dtype)
    device = s.get_device()
    if ds is not None:
        _check("gla_norm_bwd", "ds", ds, s.dtype, s.shape, device)
    _check("gla_norm_bwd", "rstd", rstd, torch.float32, s.shape[:-1], device)
    dx = torch.empty_like(dy)
    dres = dx if s.dtype == dy.dtype else torch.empty_like(s)
    dw = torch.empty(D, dtype=torch.float32, device=device) if want_dw and weight is not None else None
    if workspace is None:
        # of this call alone: its two launches meet there, and another thread's may come between them on one stream
        workspace = torch.empty(int(_lib.gla_norm_bwd_workspace_size(rows, D)), dtype=torch.uint8, device=device)
    rc = _lib.gla_norm_bwd(s.data_ptr(), rstd.data_ptr(), _at(weight), dy.data_ptr(), _at(ds), dx.data_ptr(),
                           None if dres is dx else dres.data_ptr(), _at(dw), rows, D, code, workspace.data_ptr(),
                           workspace.numel(), _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_norm_bwd")
    return dx, dres, dw


# ---------------------------------------------------------------------------------------------------------
# Gated delta rule, and group norm with an activation
# ---------------------------------------------------------------------------------------------------------

# (input, output) types of the delta rule -> dtype code
DELTA_CODE = {(torch.float32, torch.float32): GLA_F32, (torch.bfloat16, torch.float32): GLA_BF16,
              (torch.bfloat16, torch.bfloat16): GLA_BF16_OBF16, (torch.float16, torch.float32): GLA_F16,
              (torch.float16, torch.float16): GLA_F16_OF16}
_ACTIVATION = {None: 0, "silu": 1}


def _status_of(what, status, device):
    """The address of a call's status word: the caller's 256 zeroed bytes, or the library's own."""
    if status is not None and (status.get_device() != device or not status.is_contiguous() or
                               status.numel() * status.element_size() < _STATUS_BYTES):
        raise GlaError(GLA_ERR_WORKSPACE, f"{what}: status must be {_STATUS_BYTES} contiguous bytes on cuda:{device}")
    return _status_workspace(status, device)[0]


def _scratch(what, workspace, nbytes, device):
    """(tensor, address, bytes) of a call's scratch: the caller's, or memory of the call's own."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: workspace must be a contiguous tensor on cuda:{device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _delta_shape(what, q, v, rank):
    """(leading sizes, H, HV, K, V) of q [..., H, K] and v [..., HV, V]."""
    if not isinstance(v, torch.Tensor) or q.dim() != rank or v.dim() != rank or q.shape[:-2] != v.shape[:-2]:
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: expected q, k [{'B, ' * (rank == 3) or 'B, T, '}H, K] and v [..., HV, V] "
                                            f"with the same leading sizes")
    (H, K), (HV, V) = q.shape[-2:], v.shape[-2:]
    if H < 1 or HV < 1 or HV % H:
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: {HV} value heads do not share {H} key heads evenly")
    return q.shape[:-2], H, HV, K, V


def _delta_inputs(what, q, k, v, g, beta, lead, HV, device):
    _check(what, "q", q, q.dtype, q.shape, device)
    _check(what, "k", k, q.dtype, q.shape, device)
    _check(what, "v", v, q.dtype, v.shape, device)
    _check(what, "g", g, torch.float32, (*lead, HV), device)
    _check(what, "beta", beta, torch.float32, (*lead, HV), device)


def _sequences(what, B, cu_seqlens, device):
    if cu_seqlens is None:
        return B
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or \
            cu_seqlens.get_device() != device or not cu_seqlens.is_contiguous():
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: cu_seqlens must be a contiguous int32 vector on cuda:{device}")
    return cu_seqlens.numel() - 1


def delta_fwd(q, k, v, g, beta, scale=None, initial_state=None, output_final_state=True, cu_seqlens=None, out_dtype=None,
              status=None, workspace=None, stream=None):
    """Gated delta rule on the GPU: S~ = exp(g_t) S, S = S~ + k_t^T beta_t (v_t - k_t S~), o_t = scale q_t S.

    q, k: [B, T, H, K]; v: [B, T, HV, V] (cuda, contiguous, all fp32, bf16 or fp16; HV a multiple of H, each key head
    serving HV / H value heads in a row; K, V up to 256); g, beta: fp32 [B, T, HV].  Keys are taken as they are: normalise
    them before (``norm_fwd`` with a weight of K^-0.5 gives unit length; an eps above 0 leaves keys of zero at zero).
    scale: K^-0.5 by default.  initial_state: fp32 [N, HV, K, V] or None.  cu_seqlens: int32 [N+1] cuda offsets (B == 1);
    rows outside all sequences keep what the allocator left in them.  out_dtype: q's type (default) or fp32.  Returns
    (o [B, T, HV, V], final state fp32 [N, HV, K, V] or None).  Bad offsets, and fp16 states that leave fp16's range, are
    reported on the device, see ``layer_status`` (or the call's own ``status``, 256 zeroed bytes).
    """
    if status is None and workspace is None and stream is None:
        got = _calls.delta_fwd(q, k, v, g, beta, scale, initial_state, output_final_state, cu_seqlens, out_dtype)
        if got is not None:
            return got
    return _delta_fwd_checked(q, k, v, g, beta, scale, initial_state, output_final_state, cu_seqlens, out_dtype, status,
                              workspace, stream=stream)


@_on_stream
def _delta_fwd_checked(q, k, v, g, beta, scale, initial_state, output_final_state, cu_seqlens, out_dtype, status, workspace):
    what, device = "gla_delta_fwd", q.get_device()
    lead, H, HV, K, V = _delta_shape(what, q, v, 4)
    code = DELTA_CODE.get((q.dtype, out_dtype or q.dtype))
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"{what} dtypes q {q.dtype} -> {out_dtype}")
    _delta_inputs(what, q, k, v, g, beta, lead, HV, device)
    (B, T), N = lead, _sequences(what, lead[0], cu_seqlens, device)
    if initial_state is not None:
        _check(what, "initial_state", initial_state, torch.float32, (N, HV, K, V), device)
    o = torch.empty(v.shape, dtype=out_dtype or q.dtype, device=device)
    ht = torch.empty(N, HV, K, V, dtype=torch.float32, device=device) if output_final_state else None
    need = _lib.gla_delta_fwd_workspace_size(N, B, T, H, HV, K, V, code, cu_seqlens is not None)
    workspace, at, nbytes = _scratch(what, workspace, need, device)
    rc = _lib.gla_delta_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), o.data_ptr(),
                            K ** -0.5 if scale is None else scale, _at(initial_state), _at(ht), _at(cu_seqlens), N, B, T,
                            H, HV, K, V, code, _status_of(what, status, device), at, nbytes, _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, what)
    return o, ht


def delta_bwd(q, k, v, g, beta, do, scale=None, initial_state=None, dht=None, cu_seqlens=None, want_dh0=True, status=None,
              workspace=None, stream=None):
    """Gradients of ``delta_fwd`` for L = sum(o * do) + sum(ht * dht); the states are computed again.

    The inputs as for delta_fwd; do: [B, T, HV, V] of q's type; dht: fp32 [N, HV, K, V] or None.  Returns (dq, dk, dv in
    q's type, dg, dbeta fp32 [B, T, HV], dh0 fp32 [N, HV, K, V] or None); rows outside all sequences are not written.
    """
    if status is None and workspace is None and stream is None:
        got = _calls.delta_bwd(q, k, v, g, beta, do, scale, initial_state, dht, cu_seqlens, want_dh0)
        if got is not None:
            return got
    return _delta_bwd_checked(q, k, v, g, beta, do, scale, initial_state, dht, cu_seqlens, want_dh0, status, workspace,
                              stream=stream)


@_on_stream
def _delta_bwd_checked(q, k, v, g, beta, do, scale, initial_state, dht, cu_seqlens, want_dh0, status, workspace):
    what, device = "gla_delta_bwd", q.get_device()
    lead, H, HV, K, V = _delta_shape(what, q, v, 4)
    code = _NORM_CODE.get(q.dtype)
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"{what} dtype {q.dtype}")
    _delta_inputs(what, q, k, v, g, beta, lead, HV, device)
    _check(what, "do", do, q.dtype, v.shape, device)
    (B, T), N = lead, _sequences(what, lead[0], cu_seqlens, device)
    for name, t in (("initial_state", initial_state), ("dht", dht)):
        if t is not None:
            _check(what, name, t, torch.float32, (N, HV, K, V), device)
    dq, dk, dv, dg, dbeta = (torch.empty_like(t) for t in (q, k, v, g, beta))
    dh0 = torch.empty(N, HV, K, V, dtype=torch.float32, device=device) if want_dh0 else None
    need = _lib.gla_delta_bwd_workspace_size(N, B, T, H, HV, K, V, code, cu_seqlens is not None)
    workspace, at, nbytes = _scratch(what, workspace, need, device)
    rc = _lib.gla_delta_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), do.data_ptr(),
                            K ** -0.5 if scale is None else scale, _at(initial_state), _at(dht), dq.data_ptr(),
                            dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), _at(dh0), _at(cu_seqlens), N, B,
                            T, H, HV, K, V, code, _status_of(what, status, device), at, nbytes, _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, what)
    return dq, dk, dv, dg, dbeta, dh0


def delta_step(q, k, v, g, beta, state, scale=None, slots=None, state_out=None, out_dtype=None, status=None, stream=None):
    """One token of ``delta_fwd``'s recurrence for each of B sequences, with the states in a pool.

    q, k: [B, H, K]; v: [B, HV, V] (types as for delta_fwd); g, beta: fp32 [B, HV]; state: fp32 [S, HV, K, V] pool,
    updated in place (or written to state_out, of which only the addressed rows are written); slots as for scan_step.
    out_dtype: q's type (default) or fp32.  Returns o [B, HV, V].
    """
    if status is None and stream is None:
        got = _calls.delta_step(q, k, v, g, beta, state, scale, slots, state_out, out_dtype)
        if got is not None:
            return got
    return _delta_step_checked(q, k, v, g, beta, state, scale, slots, state_out, out_dtype, status, stream=stream)


@_on_stream
def _delta_step_checked(q, k, v, g, beta, state, scale, slots, state_out, out_dtype, status):
    what, device = "gla_delta_step", q.get_device()
    lead, H, HV, K, V = _delta_shape(what, q, v, 3)
    code = DELTA_CODE.get((q.dtype, out_dtype or q.dtype))
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"{what} dtypes q {q.dtype} -> {out_dtype}")
    _delta_inputs(what, q, k, v, g, beta, lead, HV, device)
    B, = lead
    S, state_out = _pool(what, state, state_out, slots, B, (HV, K, V), device)
    o = torch.empty(v.shape, dtype=out_dtype or q.dtype, device=device)
    rc = _lib.gla_delta_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), o.data_ptr(),
                             K ** -0.5 if scale is None else scale, state.data_ptr(), state_out.data_ptr(), _at(slots), B,
                             S, H, HV, K, V, code, _status_of(what, status, device), _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, what)
    return o


def _group_norm_args(what, x, groups, weight, bias, activation):
    """(N, S, C, dtype code, activation code) of a group norm of x [N, ..., C]."""
    code = _NORM_CODE.get(x.dtype)
    if code is None:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"{what} dtype {x.dtype}")
    if activation not in _ACTIVATION:
        raise GlaError(GLA_ERR_UNSUPPORTED, f"{what}: activation {activation!r}")
    if x.dim() < 2 or not x.is_contiguous():
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: x must be a contiguous [N, ..., C] tensor")
    N, C = x.shape[0], x.shape[-1]
    S = math.prod(x.shape[1:-1])
    if groups < 1 or C < 1 or C % groups or S < 1:
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: {groups} groups of {C} channels at {S} positions")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _check(what, name, t, torch.float32, (C,), x.get_device())
    return N, S, C, code, _ACTIVATION[activation]


def group_norm_fwd(x, groups, weight=None, bias=None, activation=None, eps=1e-5, workspace=None, stream=None):
    """Group norm with an activation, channels last: y = act((x - mean) rstd weight + bias), mean and rstd over all
    positions and the channels of a group.

    x: contiguous [N, ..., C] fp32 / bf16 / fp16; a two-dimensional x [rows, C] has one position a row, as the heads of a
    mixing layer's output have (groups: the heads).  weight, bias: fp32 [C] or None; activation: None or "silu".
    Returns (y in x's type, mean, rstd fp32 [N, groups]).
    """
    if workspace is None and stream is None:
        got = _calls.group_norm_fwd(x, groups, weight, bias, activation, eps)
        if got is not None:
            return got
    return _group_norm_fwd_checked(x, groups, weight, bias, activation, eps, workspace, stream=stream)


@_on_stream
def _group_norm_fwd_checked(x, groups, weight, bias, activation, eps, workspace):
    what, device = "gla_group_norm_fwd", x.get_device()
    N, S, C, code, act = _group_norm_args(what, x, groups, weight, bias, activation)
    y = torch.empty_like(x)
    mean, rstd = (torch.empty(N, groups, dtype=torch.float32, device=device) for _ in range(2))
    workspace, at, nbytes = _scratch(what, workspace, _lib.gla_group_norm_workspace_size(N, S, C, groups, code, 0), device)
    rc = _lib.gla_group_norm_fwd(x.data_ptr(), _at(weight), _at(bias), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), N, S,
                                 C, groups, eps, act, code, at, nbytes, _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, what)
    return y, mean, rstd


def group_norm_bwd(x, mean, rstd, dy, weight=None, bias=None, activation=None, want_dw=True, workspace=None, stream=None):
    """Gradients of ``group_norm_fwd`` from its input and statistics, for the gradient dy of y.

    Returns (dx in x's type, dw fp32 [C] or None without a weight, db fp32 [C] or None without a bias);
    ``want_dw=False`` skips both.
    """
    if workspace is None and stream is None:
        got = _calls.group_norm_bwd(x, mean, rstd, dy, weight, bias, activation, want_dw)
        if got is not None:
            return got
    return _group_norm_bwd_checked(x, mean, rstd, dy, weight, bias, activation, want_dw, workspace, stream=stream)


@_on_stream
def _group_norm_bwd_checked(x, mean, rstd, dy, weight, bias, activation, want_dw, workspace):
    what, device = "gla_group_norm_bwd", x.get_device()
    if mean.dim() != 2:
        raise GlaError(GLA_ERR_INVALID_ARG, f"{what}: mean must be [N, groups]")
    groups = mean.shape[1]
    N, S, C, code, act = _group_norm_args(what, x, groups, weight, bias, activation)
    _check(what, "mean", mean, torch.float32, (N, groups), device)
    _check(what, "rstd", rstd, torch.float32, (N, groups), device)
    _check(what, "dy", dy, x.dtype, x.shape, device)
    dx = torch.empty_like(x)
    dw, db = (torch.empty(C, dtype=torch.float32, device=device) if want_dw and t is not None else None for t in (weight, bias))
    workspace, at, nbytes = _scratch(what, workspace, _lib.gla_group_norm_workspace_size(N, S, C, groups, code, 1), device)
    rc = _lib.gla_group_norm_bwd(x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _at(weight), _at(bias), dy.data_ptr(),
                                 dx.data_ptr(), _at(dw), _at(db), N, S, C, groups, act, code, at, nbytes,
                                 _raw_stream(device))
    if rc != GLA_OK:
        raise GlaError(rc, what)
    return dx, dw, db


def get_status(workspace, stream=None) -> int:
    return int(_lib.gla_get_status(_ptr(workspace), _stream_handle(stream)))


def chunk_local_cumsum(g, chunk=64, cu_seqlens=None, stream=None):
    B, T, H, K = g.shape
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    code = {torch.float32: GLA_F32, torch.bfloat16: GLA_BF16, torch.float16: GLA_F16}.get(g.dtype, GLA_BF16)
    G = torch.empty(B, T, H, K, dtype=torch.float32, device=g.device)
    rc = int(_lib.gla_chunk_local_cumsum(_ptr(g), _ptr(G), _ptr(cu_seqlens), N, B, T, H, K, chunk, code,
                                         _stream_handle(stream)))
    if rc != GLA_OK:
        raise GlaError(rc, "gla_chunk_local_cumsum")
    return G


class KernelTimer:
    """Arms gla_profile_events with CUDA events so each kernel launch of the next gla_fwd calls on this
    thread is bracketed by events on its stream.  ``results()`` (after a synchronize) gives
    [(kernel name, milliseconds)] for the last call."""

    def __init__(self, max_launches=16):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * max_launches)]
        for e in self.events:   # torch creates the CUDA event on first record: materialise the handles
            e.record()
        torch.cuda.synchronize()
        handles = [e.cuda_event for e in self.events]
        if not all(handles):
            raise RuntimeError("KernelTimer: could not create CUDA events")
        self._handles = (ctypes.c_void_p * len(self.events))(*handles)
        self._ids = (ctypes.c_int * max_launches)()

    def __enter__(self):
        _lib.gla_profile_events(self._handles, len(self.events), self._ids)
        return self

    def __exit__(self, *exc):
        _lib.gla_profile_events(None, 0, None)

    def results(self):
        n = int(_lib.gla_profile_launches())
        return [(_lib.gla_kernel_name(self._ids[i]).decode(), self.events[2 * i].elapsed_time(self.events[2 * i + 1]))
                for i in range(min(n, len(self.events) // 2))]
