"""Torch-tensor front end of the C ABI (argument marshalling only).

Every function checks dtypes, shapes and contiguity, passes ``data_ptr()``
values and the current CUDA stream to ``libckda.so`` and raises ``CKDAError``
on a non-zero status.  All arithmetic happens in the CUDA kernels.
"""
from __future__ import annotations

import functools
import math
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import CKDAError

_DT = {torch.float32: _lib.CKDA_F32, torch.bfloat16: _lib.CKDA_BF16}


def _stream_ptr(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def fwd_chunked(q, k, v, alpha, beta, S0=None, cu_seqlens=None, chunk: int = 64,
                out=None, S_final=None, return_final: bool = True, fp32core: bool = False,
                out_dtype=None, workspace=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked CKDA forward.  Shapes as in ``ckda_fwd_chunked`` (include/ckda.h).

    Fixed-length: q, k, alpha ``[B, T, H, dk]``; v ``[B, T, H, dv]``; beta ``[B, T, H]``.
    Packed: ``cu_seqlens`` int32 ``[N+1]`` and tensors with a leading 1 or without it.
    ``out_dtype`` (float32 or bfloat16) defaults to the dtype of ``out`` if given,
    else to the input dtype.  ``workspace`` is an optional uint8 CUDA tensor of at
    least ``workspace_bytes(...)`` bytes; without it one is taken from torch's
    caching allocator for the call.
    Returns ``(out, S_final)``; ``S_final`` is None when ``return_final`` is False.
    """
    dev = q.device
    B, T, H, dk, dv, N = _inputs_shape(q, k, v, alpha, beta, cu_seqlens)
    if S0 is not None:
        _need(S0, "S0", torch.float32, dev)
        if tuple(S0.shape) != (N, H, dk, dv):
            raise ValueError(f"S0 must be [{N}, {H}, {dk}, {dv}]")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if out is None:
        out = torch.empty(v.shape, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, dev)
        if out.shape != v.shape:
            raise ValueError("out must have v's shape")
    if return_final and S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if S_final is not None:
        _need(S_final, "S_final", torch.float32, dev)
    lib = _lib.load()
    with torch.cuda.device(dev):
        if fp32core:
            rc = lib.ckda_fwd_chunked_fp32core(
                _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(S0), _p(cu_seqlens), _p(out),
                _p(S_final), B, T, H, dk, dv, chunk, _DT[q.dtype], _DT[out_dtype],
                _stream_ptr(dev))
        else:
            need = workspace_bytes(B, T, H, dk, dv, chunk, q.dtype, out_dtype,
                                   cu_seqlens is not None)
            if workspace is None and need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            if workspace is not None:
                _need(workspace, "workspace", torch.uint8, dev)
            rc = lib.ckda_fwd_chunked(
                _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(S0), _p(cu_seqlens), _p(out),
                _p(S_final), B, T, H, dk, dv, chunk, _DT[q.dtype], _DT[out_dtype],
                _p(workspace), 0 if workspace is None else workspace.numel(), _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_fwd_chunked")
    return out, S_final


def fwd_chunked_static(q, k, v, alpha, beta, S0=None, cu_seqlens=None, chunk: int = 64,
                       out=None, S_final=None, return_final: bool = True, out_dtype=None):
    """``fwd_chunked`` through ``ckda_fwd_chunked_static``: no workspace is passed or
    allocated; the library's fixed device scratch (``CKDA_STATIC_SCRATCH_BYTES``)
    is used.  Calls that may run concurrently on one device race on that scratch."""
    dev = q.device
    B, T, H, dk, dv, N = _inputs_shape(q, k, v, alpha, beta, cu_seqlens)
    if S0 is not None:
        _need(S0, "S0", torch.float32, dev)
        if tuple(S0.shape) != (N, H, dk, dv):
            raise ValueError(f"S0 must be [{N}, {H}, {dk}, {dv}]")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if out is None:
        out = torch.empty(v.shape, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, dev)
        if out.shape != v.shape:
            raise ValueError("out must have v's shape")
    if return_final and S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if S_final is not None:
        _need(S_final, "S_final", torch.float32, dev)
    with torch.cuda.device(dev):
        rc = _lib.load().ckda_fwd_chunked_static(
            _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(S0), _p(cu_seqlens), _p(out),
            _p(S_final), B, T, H, dk, dv, chunk, _DT[q.dtype], _DT[out_dtype], _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_fwd_chunked_static")
    return out, S_final


def _inputs_shape(q, k, v, alpha, beta, cu_seqlens, pair_gates=False):
    """Checks the forward inputs; returns (B, T, H, dk, dv, N) as passed to the ABI.
    ``pair_gates``: alpha holds one decay per channel pair (last dim dk / 2)."""
    dev = q.device
    if q.dtype not in _DT:
        raise TypeError("q, k, v must be float32 or bfloat16")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, dev)
    _need(alpha, "alpha", torch.float32, dev)
    _need(beta, "beta", torch.float32, dev)
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError("q must be [B, T, H, dk]")
        B, T, H, dk = q.shape
        N = B
    else:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if q.dim() == 4:
            if q.shape[0] != 1:
                raise ValueError("packed inputs take a leading dimension of 1")
            T, H, dk = q.shape[1:]
        else:
            T, H, dk = q.shape
        N = cu_seqlens.numel() - 1
        B = N
    dv = v.shape[-1]
    a_shape = q.shape[:-1] + (dk // 2,) if pair_gates else q.shape
    if pair_gates and dk % 2:
        raise ValueError("the phase-decay gates pair the key channels: dk must be even")
    if k.shape != q.shape or alpha.shape != a_shape or v.shape[:-1] != q.shape[:-1]:
        raise ValueError("q, k, alpha must share a shape (alpha: last dim dk / 2 for paired "
                         "gates) and v must match it but for the last dim")
    if tuple(beta.shape) != tuple(q.shape[:-1]):
        raise ValueError("beta must have q's shape without the last dim")
    return B, T, H, dk, dv, N


def fwd_factors(q, k, v, alpha, beta, cu_seqlens=None, chunk: int = 64, workspace=None):
    """Phase 1 of the tensor-core forward: the S0-independent WY factors of every
    chunk, written to ``workspace`` (uint8 CUDA tensor; allocated if None).
    Returns the workspace, to be passed to ``fwd_carry`` with the same sizes."""
    B, T, H, dk, dv, N = _inputs_shape(q, k, v, alpha, beta, cu_seqlens)
    dev = q.device
    need = workspace_bytes(B, T, H, dk, dv, chunk, q.dtype, torch.float32, cu_seqlens is not None)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    with torch.cuda.device(dev):
        rc = _lib.load().ckda_fwd_factors(
            _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(cu_seqlens), B, T, H, dk, dv, chunk,
            _DT[q.dtype], _p(workspace), workspace.numel(), _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_fwd_factors")
    return workspace


def fwd_carry(workspace, v, B, T, H, dk, dv, S0=None, cu_seqlens=None, chunk: int = 64,
              dtype=torch.bfloat16, out=None, S_final=None, out_dtype=torch.float32,
              return_final: bool = True):
    """Phase 2: apply the factors in ``workspace`` from ``S0``.  ``v`` is the value
    tensor of the ``fwd_factors`` call (the carry reads it); sizes (B, T, H as in
    ``ckda_fwd_chunked``) and ``dtype`` must be those of that call.
    Returns ``(out, S_final)``."""
    dev = workspace.device
    _need(workspace, "workspace", torch.uint8, dev)
    _need(v, "v", dtype, dev)
    N = B
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    shape = (B, T, H, dv) if cu_seqlens is None else (T, H, dv)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, dev)
        if out.numel() != math.prod(shape):
            raise ValueError(f"out must hold {shape}")
    if S0 is not None:
        _need(S0, "S0", torch.float32, dev)
        if tuple(S0.shape) != (N, H, dk, dv):
            raise ValueError(f"S0 must be [{N}, {H}, {dk}, {dv}]")
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if return_final and S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if S_final is not None:
        _need(S_final, "S_final", torch.float32, dev)
    with torch.cuda.device(dev):
        rc = _lib.load().ckda_fwd_carry(
            _p(v), _p(S0), _p(cu_seqlens), _p(out), _p(S_final), B, T, H, dk, dv, chunk, _DT[dtype],
            _DT[out_dtype], _p(workspace), workspace.numel(), _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_fwd_carry")
    return out, S_final


def gdn2_fwd_chunked(q, k, v, alpha, b, w, S0=None, cu_seqlens=None, chunk: int = 64,
                     out=None, S_final=None, return_final: bool = True, out_dtype=None,
                     workspace=None):
    """Chunked Gated DeltaNet-2 forward (``ckda_gdn2_fwd_chunked``): CKDA with an
    erase gate ``b`` (fp32, shaped like ``k``) and a write gate ``w`` (fp32, shaped
    like ``v``) in place of beta.  Other arguments, the workspace and the result
    as in ``fwd_chunked``."""
    dev = q.device
    _need(b, "b", torch.float32, dev)
    _need(w, "w", torch.float32, dev)
    if b.shape != k.shape or w.shape != v.shape:
        raise ValueError("b must have k's shape and w v's shape")
    beta_like = b[..., 0]  # shape check only: [B, T, H] or [T, H]
    B, T, H, dk, dv, N = _inputs_shape(q, k, v, alpha, beta_like.contiguous(), cu_seqlens)
    if S0 is not None:
        _need(S0, "S0", torch.float32, dev)
        if tuple(S0.shape) != (N, H, dk, dv):
            raise ValueError(f"S0 must be [{N}, {H}, {dk}, {dv}]")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if out is None:
        out = torch.empty(v.shape, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, dev)
        if out.shape != v.shape:
            raise ValueError("out must have v's shape")
    if return_final and S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if S_final is not None:
        _need(S_final, "S_final", torch.float32, dev)
    need = workspace_bytes(B, T, H, dk, dv, chunk, q.dtype, out_dtype, cu_seqlens is not None)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    with torch.cuda.device(dev):
        rc = _lib.load().ckda_gdn2_fwd_chunked(
            _p(q), _p(k), _p(v), _p(alpha), _p(b), _p(w), _p(S0), _p(cu_seqlens), _p(out),
            _p(S_final), B, T, H, dk, dv, chunk, _DT[q.dtype], _DT[out_dtype], _p(workspace),
            0 if workspace is None else workspace.numel(), _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_gdn2_fwd_chunked")
    return out, S_final


def sfda_fwd_chunked(q, k, v, alpha, theta, beta, S0=None, cu_seqlens=None, chunk: int = 64,
                     out=None, S_final=None, return_final: bool = True, out_dtype=None,
                     workspace=None, fp32core: bool = False):
    """Chunked SFDA forward (``ckda_sfda_fwd_chunked``): the CKDA recurrence with
    Diag(alpha) replaced by phase-decay blocks ``alpha_p R(theta_p)`` on the key
    channel pairs ``(2p, 2p+1)``.  ``alpha`` and ``theta`` are fp32 shaped like
    ``k`` with the last dim halved; beta, the workspace and the other arguments
    as in ``fwd_chunked`` (``fp32core`` forces the fp32 CUDA-core kernel)."""
    dev = q.device
    B, T, H, dk, dv, N = _inputs_shape(q, k, v, alpha, beta, cu_seqlens, pair_gates=True)
    _need(theta, "theta", torch.float32, dev)
    if theta.shape != alpha.shape:
        raise ValueError("theta must have alpha's shape")
    if S0 is not None:
        _need(S0, "S0", torch.float32, dev)
        if tuple(S0.shape) != (N, H, dk, dv):
            raise ValueError(f"S0 must be [{N}, {H}, {dk}, {dv}]")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if out is None:
        out = torch.empty(v.shape, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, dev)
        if out.shape != v.shape:
            raise ValueError("out must have v's shape")
    if return_final and S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if S_final is not None:
        _need(S_final, "S_final", torch.float32, dev)
    lib = _lib.load()
    if fp32core:
        with torch.cuda.device(dev):
            rc = lib.ckda_sfda_fwd_chunked_fp32core(
                _p(q), _p(k), _p(v), _p(alpha), _p(theta), _p(beta), _p(S0), _p(cu_seqlens),
                _p(out), _p(S_final), B, T, H, dk, dv, chunk, _DT[q.dtype], _DT[out_dtype],
                _stream_ptr(dev))
        if rc != 0:
            raise CKDAError(rc, "ckda_sfda_fwd_chunked_fp32core")
        return out, S_final
    need = workspace_bytes(B, T, H, dk, dv, chunk, q.dtype, out_dtype, cu_seqlens is not None)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    with torch.cuda.device(dev):
        rc = lib.ckda_sfda_fwd_chunked(
            _p(q), _p(k), _p(v), _p(alpha), _p(theta), _p(beta), _p(S0), _p(cu_seqlens),
            _p(out), _p(S_final), B, T, H, dk, dv, chunk, _DT[q.dtype], _DT[out_dtype],
            _p(workspace), 0 if workspace is None else workspace.numel(), _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_sfda_fwd_chunked")
    return out, S_final


def scan_workspace_bytes(B, T, H, dk, dv, segments) -> int:
    """Scratch bytes ``fwd_chunked_scan`` needs for these sizes."""
    rc = _lib.load().ckda_fwd_chunked_scan_workspace_bytes(B, T, H, dk, dv, segments)
    if rc < 0:
        raise CKDAError(int(rc), "ckda_fwd_chunked_scan_workspace_bytes")
    return int(rc)


def fwd_chunked_scan(q, k, v, alpha, beta, segments: int, S0=None, chunk: int = 64, out=None,
                     S_final=None, return_final: bool = True, out_dtype=None, workspace=None):
    """``fwd_chunked`` for fixed-length batches as a chunk-parallel scan over
    ``segments`` segments of each sequence (``ckda_fwd_chunked_scan``): segment
    summaries [M | B] in parallel, a scan of the segment start states, then
    every segment's carry in parallel.  Same result up to rounding."""
    dev = q.device
    B, T, H, dk, dv, N = _inputs_shape(q, k, v, alpha, beta, None)
    if S0 is not None:
        _need(S0, "S0", torch.float32, dev)
        if tuple(S0.shape) != (N, H, dk, dv):
            raise ValueError(f"S0 must be [{N}, {H}, {dk}, {dv}]")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if out is None:
        out = torch.empty(v.shape, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, dev)
        if out.shape != v.shape:
            raise ValueError("out must have v's shape")
    if return_final and S_final is None:
        S_final = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if S_final is not None:
        _need(S_final, "S_final", torch.float32, dev)
        if tuple(S_final.shape) != (N, H, dk, dv):
            raise ValueError(f"S_final must be [{N}, {H}, {dk}, {dv}]")
    if workspace is None:
        workspace = torch.empty(max(1, scan_workspace_bytes(B, T, H, dk, dv, segments)),
                                dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    with torch.cuda.device(dev):
        rc = _lib.load().ckda_fwd_chunked_scan(
            _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(S0), _p(out), _p(S_final), B, T, H, dk,
            dv, chunk, _DT[q.dtype], _DT[out_dtype], segments, _p(workspace), workspace.numel(),
            _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_fwd_chunked_scan")
    return out, S_final


def bwd_workspace_bytes(B, T, H, dk, dv, varlen=False) -> int:
    """Scratch bytes ``bwd_chunked`` needs for these sizes."""
    rc = _lib.load().ckda_bwd_chunked_workspace_bytes(B, T, H, dk, dv, 1 if varlen else 0)
    if rc < 0:
        raise CKDAError(int(rc), "ckda_bwd_chunked_workspace_bytes")
    return int(rc)


def bwd_chunked(q, k, v, alpha, beta, dO, S0=None, dS_final=None, cu_seqlens=None,
                grads=None, want_dS0: bool = True, workspace=None):
    """Backward of ``fwd_chunked`` (``ckda_bwd_chunked``): the gradients of a scalar
    loss with respect to q, k, v, alpha, beta and S0, given ``dO`` (dL/dout, fp32 or
    bf16, shaped like v) and ``dS_final`` (dL/dS_final, fp32, or None = 0).

    Returns a dict of fp32 tensors ``dq, dk, dv, dalpha, dbeta`` (shaped like the
    inputs) and ``dS0`` (``[N, H, dk, dv]``, or None when ``want_dS0`` is false).
    ``grads`` may supply preallocated output tensors under the same names."""
    dev = q.device
    B, T, H, dk, dv, N = _inputs_shape(q, k, v, alpha, beta, cu_seqlens)
    if dO.dtype not in _DT:
        raise TypeError("dO must be float32 or bfloat16")
    _need(dO, "dO", dO.dtype, dev)
    if dO.shape != v.shape:
        raise ValueError("dO must have v's shape")
    if S0 is not None:
        _need(S0, "S0", torch.float32, dev)
        if tuple(S0.shape) != (N, H, dk, dv):
            raise ValueError(f"S0 must be [{N}, {H}, {dk}, {dv}]")
    if dS_final is not None:
        _need(dS_final, "dS_final", torch.float32, dev)
        if tuple(dS_final.shape) != (N, H, dk, dv):
            raise ValueError(f"dS_final must be [{N}, {H}, {dk}, {dv}]")
    want = {"dq": q.shape, "dk": k.shape, "dv": v.shape, "dalpha": alpha.shape,
            "dbeta": beta.shape}
    if want_dS0:
        want["dS0"] = (N, H, dk, dv)
    g = dict(grads or {})
    for name, shp in want.items():
        if g.get(name) is None:
            g[name] = torch.empty(shp, dtype=torch.float32, device=dev)
        _need(g[name], name, torch.float32, dev)
        if tuple(g[name].shape) != tuple(shp):
            raise ValueError(f"{name} must be {tuple(shp)}")
    if not want_dS0:
        g["dS0"] = None
    need = bwd_workspace_bytes(B, T, H, dk, dv, cu_seqlens is not None)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    with torch.cuda.device(dev):
        rc = _lib.load().ckda_bwd_chunked(
            _p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(S0), _p(cu_seqlens), _p(dO),
            _p(dS_final), _p(g["dq"]), _p(g["dk"]), _p(g["dv"]), _p(g["dalpha"]),
            _p(g["dbeta"]), _p(g["dS0"]), B, T, H, dk, dv, _DT[q.dtype], _DT[dO.dtype],
            _p(workspace), 0 if workspace is None else workspace.numel(), _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_bwd_chunked")
    return g


def workspace_bytes(B, T, H, dk, dv, chunk=64, dtype=torch.bfloat16, out_dtype=torch.float32,
                    varlen=False) -> int:
    """Scratch bytes ``fwd_chunked`` needs for these sizes (0 on the fp32 CUDA-core path)."""
    rc = _lib.load().ckda_fwd_chunked_workspace_bytes(B, T, H, dk, dv, chunk, _DT[dtype],
                                                      _DT[out_dtype], 1 if varlen else 0)
    if rc < 0:
        raise CKDAError(int(rc), "ckda_fwd_chunked_workspace_bytes")
    return int(rc)


def fwd_path(B, T, H, dk, dv, chunk=64, dtype=torch.bfloat16, out_dtype=torch.float32,
             varlen=False) -> str:
    """Which kernel ``fwd_chunked`` runs for these sizes: "tcgen05" or "fp32core"."""
    rc = _lib.load().ckda_fwd_chunked_path(B, T, H, dk, dv, chunk, _DT[dtype], _DT[out_dtype],
                                           1 if varlen else 0)
    if rc < 0:
        raise CKDAError(rc, "ckda_fwd_chunked_path")
    return "tcgen05" if rc == 1 else "fp32core"


def _decode_out(q, v, out, out_dtype, dev):
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    B, H, _ = q.shape
    if out is None:
        out = torch.empty((B, H, v.shape[-1]), dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, dev)
    return out, out_dtype


def _decode_checks(q, k, v, S, gates):
    dev = q.device
    if q.dtype not in _DT:
        raise TypeError("q, k, v must be float32 or bfloat16")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, dev)
    _need(S, "S", torch.float32, dev)
    B, H, dk = q.shape
    dv = v.shape[-1]
    if tuple(S.shape) != (B, H, dk, dv) or k.shape != q.shape or tuple(v.shape[:2]) != (B, H):
        raise ValueError("shape mismatch")
    for name, t, shape in gates:
        _need(t, name, torch.float32, dev)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {tuple(shape)}")
    return dev, B, H, dk, dv


def decode_step(q, k, v, alpha, beta, S, out=None, out_dtype=None) -> torch.Tensor:
    """One recurrent step, in place on ``S`` ``[B, H, dk, dv]`` (fp32).

    q, k, alpha ``[B, H, dk]``; v ``[B, H, dv]``; beta ``[B, H]``.  Returns ``out``
    (``out_dtype`` defaults to the dtype of ``out`` if given, else the input dtype).
    """
    B, H, dk = q.shape
    dev, B, H, dk, dv = _decode_checks(q, k, v, S, (("alpha", alpha, (B, H, dk)),
                                                    ("beta", beta, (B, H))))
    out, out_dtype = _decode_out(q, v, out, out_dtype, dev)
    with torch.cuda.device(dev):
        rc = _lib.load().ckda_decode_step(_p(q), _p(k), _p(v), _p(alpha), _p(beta), _p(S), _p(out),
                                          B, H, dk, dv, _DT[q.dtype], _DT[out_dtype],
                                          _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_decode_step")
    return out


def gdn2_decode_step(q, k, v, alpha, b, w, S, out=None, out_dtype=None) -> torch.Tensor:
    """One Gated DeltaNet-2 step in place on ``S`` (``ckda_gdn2_decode_step``):
    erase gate ``b`` ``[B, H, dk]`` and write gate ``w`` ``[B, H, dv]`` (fp32) in
    place of beta; otherwise as ``decode_step``."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev, B, H, dk, dv = _decode_checks(q, k, v, S, (("alpha", alpha, (B, H, dk)),
                                                    ("b", b, (B, H, dk)), ("w", w, (B, H, dv))))
    out, out_dtype = _decode_out(q, v, out, out_dtype, dev)
    with torch.cuda.device(dev):
        rc = _lib.load().ckda_gdn2_decode_step(_p(q), _p(k), _p(v), _p(alpha), _p(b), _p(w),
                                               _p(S), _p(out), B, H, dk, dv, _DT[q.dtype],
                                               _DT[out_dtype], _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_gdn2_decode_step")
    return out


def sfda_decode_step(q, k, v, alpha, theta, beta, S, out=None, out_dtype=None) -> torch.Tensor:
    """One SFDA step in place on ``S`` (``ckda_sfda_decode_step``): decays
    ``alpha`` and phases ``theta`` ``[B, H, dk / 2]`` (fp32) per channel pair,
    ``beta`` ``[B, H]``; otherwise as ``decode_step``."""
    B, H, dk = q.shape
    dev, B, H, dk, dv = _decode_checks(q, k, v, S, (("alpha", alpha, (B, H, dk // 2)),
                                                    ("theta", theta, (B, H, dk // 2)),
                                                    ("beta", beta, (B, H))))
    out, out_dtype = _decode_out(q, v, out, out_dtype, dev)
    with torch.cuda.device(dev):
        rc = _lib.load().ckda_sfda_decode_step(_p(q), _p(k), _p(v), _p(alpha), _p(theta),
                                               _p(beta), _p(S), _p(out), B, H, dk, dv,
                                               _DT[q.dtype], _DT[out_dtype], _stream_ptr(dev))
    if rc != 0:
        raise CKDAError(rc, "ckda_sfda_decode_step")
    return out


# ---- head-decay linear attention ------------------------------------------------

# A call's checks and its launch cost the host as much time as the smallest
# kernels take: the usual case is one pass over the tensors (``_check``, where
# that finds something, words the error), and the current device is set only
# when it is another one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_CF = torch.contiguous_format


def _plain(ix, dtype, *tensors):
    """Whether all are contiguous tensors of ``dtype`` on CUDA device ``ix``."""
    for t in tensors:
        if type(t) is not torch.Tensor or t.dtype is not dtype or t.get_device() != ix \
                or not t.is_contiguous():
            return False
    return ix >= 0


def _check(t, name, dtype, dev):
    if not (type(t) is torch.Tensor and t.dtype is dtype and t.device == dev
            and t.is_contiguous() and dev.type == "cuda"):
        _need(t, name, dtype, dev)


def _call(fn, dev, *args):
    """``fn(*args, stream)`` with ``dev`` as the current device."""
    ix = dev.index
    if ix != _current():
        with torch.cuda.device(dev):
            return fn(*args, _stream_ptr(dev))
    return fn(*args, _raw_stream(ix) if _raw_stream is not None else _stream_ptr(dev))


def _la_inputs(q, k, v, alpha, cu_seqlens):
    """Checks the inputs; returns (B, T, H, dk, dv, per_head) as passed to the ABI."""
    dev = q.device
    if q.dtype not in _DT:
        raise TypeError("q, k, v must be float32 or bfloat16")
    ix = q.get_device()
    if not (_plain(ix, q.dtype, q, k, v) and _plain(ix, torch.float32, alpha)):
        for name, t in (("q", q), ("k", k), ("v", v)):
            _check(t, name, q.dtype, dev)
        _check(alpha, "alpha", torch.float32, dev)
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError("q must be [B, T, H, dk]")
        B, T, H, dk = q.shape
    else:
        _check(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [N + 1]")
        if q.dim() == 4:
            if q.shape[0] != 1:
                raise ValueError("packed inputs take a leading dimension of 1")
        elif q.dim() != 3:
            raise ValueError("q must be [T, H, dk] or [1, T, H, dk]")
        T, H, dk = q.shape[-3:]
        B = cu_seqlens.numel() - 1
    if k.shape != q.shape or v.dim() != q.dim() or v.shape[:-1] != q.shape[:-1]:
        raise ValueError("q and k must share a shape and v must match it but for the last dim")
    per_head = alpha.dim() == 1
    if alpha.shape != ((H,) if per_head else q.shape[:-1]):
        raise ValueError("alpha must have q's shape without the last dim, or be [H]")
    return B, T, H, dk, v.shape[-1], per_head


def _la_state(t, name, shape, dev):
    if t is not None:
        _check(t, name, torch.float32, dev)
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}")


@functools.lru_cache(maxsize=1024)
def la_workspace_bytes(B, T, H, dk, dv, dtype=torch.bfloat16, varlen=False) -> int:
    """Scratch bytes ``la_fwd_chunked`` needs for these sizes."""
    rc = _lib.load().ckda_la_fwd_workspace_bytes(B, T, H, dk, dv, _DT[dtype], 1 if varlen else 0)
    if rc < 0:
        raise CKDAError(int(rc), "ckda_la_fwd_workspace_bytes")
    return int(rc)


def la_fwd_chunked(q, k, v, alpha, S0=None, cu_seqlens=None, out=None, S_final=None,
                   return_final: bool = True, out_dtype=None, workspace=None):
    """Chunked forward of head-decay linear attention (``ckda_la_fwd_chunked``):
    ``S_t = a_t S_{t-1} + k_t v_t^T``, ``o_t = S_t^T q_t``.

    q, k ``[B, T, H, dk]``, v ``[B, T, H, dv]``, alpha (fp32) ``[B, T, H]``, or ``[H]``
    for one decay per head; packed batches as in ``fwd_chunked``, and so the other
    arguments.  Returns ``(out, S_final)``."""
    dev = q.device
    B, T, H, dk, dv, per_head = _la_inputs(q, k, v, alpha, cu_seqlens)
    _la_state(S0, "S0", (B, H, dk, dv), dev)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else q.dtype
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if out is None:
        out = torch.empty_like(v, dtype=out_dtype, memory_format=_CF)
    else:
        _check(out, "out", out_dtype, dev)
        if out.shape != v.shape:
            raise ValueError("out must have v's shape")
    if return_final and S_final is None:
        S_final = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    else:
        _la_state(S_final, "S_final", (B, H, dk, dv), dev)
    need = la_workspace_bytes(B, T, H, dk, dv, q.dtype, cu_seqlens is not None)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8, dev)
    rc = _call(
        _lib.load().ckda_la_fwd_chunked, dev,
        q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), _p(S0), _p(cu_seqlens),
        out.data_ptr(), _p(S_final), B, T, H, dk, dv, 1 if per_head else 0, _DT[q.dtype], _DT[out_dtype], _p(workspace),
        0 if workspace is None else workspace.numel())
    if rc != 0:
        raise CKDAError(rc, "ckda_la_fwd_chunked")
    return out, S_final


@functools.lru_cache(maxsize=1024)
def la_bwd_workspace_bytes(B, T, H, dk, dv, alpha_per_head=False, dtype=torch.bfloat16,
                           varlen=False) -> int:
    """Scratch bytes ``la_bwd_chunked`` needs for these sizes."""
    rc = _lib.load().ckda_la_bwd_workspace_bytes(B, T, H, dk, dv, 1 if alpha_per_head else 0,
                                                 _DT[dtype], 1 if varlen else 0)
    if rc < 0:
        raise CKDAError(int(rc), "ckda_la_bwd_workspace_bytes")
    return int(rc)


def la_bwd_chunked(q, k, v, alpha, dO, S0=None, dS_final=None, cu_seqlens=None, grads=None,
                   want_dS0: bool = True, workspace=None):
    """Backward of ``la_fwd_chunked`` (``ckda_la_bwd_chunked``) given ``dO`` (dL/dout, shaped
    and typed like v) and ``dS_final`` (dL/dS_final, fp32, or None = 0).

    Returns a dict: ``dq, dk, dv`` shaped and typed like the inputs, ``dalpha`` (fp32, shaped
    like alpha) and ``dS0`` (fp32 ``[N, H, dk, dv]``, or None when ``want_dS0`` is false).
    ``grads`` may supply preallocated output tensors under the same names."""
    dev = q.device
    B, T, H, dk, dv, per_head = _la_inputs(q, k, v, alpha, cu_seqlens)
    _check(dO, "dO", q.dtype, dev)
    if dO.shape != v.shape:
        raise ValueError("dO must have v's shape")
    st = (B, H, dk, dv)
    _la_state(S0, "S0", st, dev)
    _la_state(dS_final, "dS_final", st, dev)
    want = [("dq", q.shape, q.dtype), ("dk", k.shape, q.dtype), ("dv", v.shape, q.dtype),
            ("dalpha", alpha.shape, torch.float32)]
    if want_dS0:
        want.append(("dS0", st, torch.float32))
    g = {}
    for name, shape, dtype in want:
        t = (grads or {}).get(name)
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _check(t, name, dtype, dev)
            if t.shape != shape:
                raise ValueError(f"{name} must be {list(shape)}")
        g[name] = t
    if not want_dS0:
        g["dS0"] = None
    need = la_bwd_workspace_bytes(B, T, H, dk, dv, per_head, q.dtype, cu_seqlens is not None)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8, dev)
    rc = _call(
        _lib.load().ckda_la_bwd_chunked, dev,
        _p(q), _p(k), _p(v), _p(alpha), _p(S0), _p(cu_seqlens), _p(dO), _p(dS_final),
        _p(g["dq"]), _p(g["dk"]), _p(g["dv"]), _p(g["dalpha"]), _p(g["dS0"]), B, T, H, dk, dv,
        1 if per_head else 0, _DT[q.dtype], _p(workspace),
        0 if workspace is None else workspace.numel())
    if rc != 0:
        raise CKDAError(rc, "ckda_la_bwd_chunked")
    return g


def la_decode_step(q, k, v, alpha, S, out=None, out_dtype=None) -> torch.Tensor:
    """One token of head-decay linear attention in place on ``S`` ``[B, H, dk, dv]``
    (``ckda_la_decode_step``): alpha (fp32) ``[B, H]``, or ``[H]`` for one decay per
    head; otherwise as ``decode_step``."""
    dev, dtype = q.device, q.dtype
    if dtype not in _DT:
        raise TypeError("q, k, v must be float32 or bfloat16")
    ix = q.get_device()
    if not (_plain(ix, dtype, q, k, v) and _plain(ix, torch.float32, S, alpha)):
        for name, t in (("q", q), ("k", k), ("v", v)):
            _check(t, name, dtype, dev)
        _check(S, "S", torch.float32, dev)
        _check(alpha, "alpha", torch.float32, dev)
    if S.dim() != 4 or q.shape != S.shape[:3] or k.shape != q.shape or \
            v.shape != S.shape[:2] + S.shape[3:]:
        raise ValueError("q, k must be [B, H, dk], v [B, H, dv] and S [B, H, dk, dv]")
    B, H, dk, dv = S.shape
    per_head = alpha.dim() == 1
    if alpha.shape != ((H,) if per_head else (B, H)):
        raise ValueError("alpha must be [B, H] or [H]")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else dtype
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if out is None:
        out = torch.empty_like(v, dtype=out_dtype, memory_format=_CF)
    else:
        _check(out, "out", out_dtype, dev)
        if out.shape != v.shape:
            raise ValueError("out must have v's shape")
    rc = _call(
        _lib.load().ckda_la_decode_step, dev,
        q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), S.data_ptr(), out.data_ptr(),
        B, H, dk, dv, 1 if per_head else 0, _DT[dtype], _DT[out_dtype])
    if rc != 0:
        raise CKDAError(rc, "ckda_la_decode_step")
    return out


# ---- norm of queries and keys, with the rotation ----------------------------------

_NORM = {"l2": _lib.CKDA_NORM_L2, "rms": _lib.CKDA_NORM_RMS}


def _token_stride(t, name):
    """Elements between the tokens of ``[..., H, d]``: the heads of a token lie together, the
    tokens at one distance (a view into a wider projection)."""
    H, d = t.shape[-2:]
    if t.is_contiguous() or t.numel() == 0:
        return H * d
    if t.dim() == 3 and t.stride(2) == 1 and (t.stride(1) == d or H == 1):
        return t.stride(0) if t.shape[0] > 1 else H * d
    if t.stride(-1) != 1 or (H > 1 and t.stride(-2) != d):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    step, span = None, None
    for n, s in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if n == 1:
            continue
        if step is None:
            step, span = s, s * n
        elif s != span:
            raise ValueError(f"the tokens of {name} must lie at one stride")
        else:
            span = s * n
    return H * d if step is None else step


def _qk_inputs(q, k, wq, wk, positions, inv_freq, norm):
    """Checks the inputs; returns (tokens, Hq, Hk, d, rot, q_stride, k_stride)."""
    for name, t in (("q", q), ("k", k)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    dev, ix = q.device, q.get_device()
    if q.dtype not in _DT:
        raise TypeError("q, k must be float32 or bfloat16")
    if k.dtype != q.dtype or k.get_device() != ix:
        raise ValueError("q and k must share a dtype and a device")
    qs, ks = q.shape, k.shape
    if len(qs) < 3 or len(ks) != len(qs) or ks[:-2] != qs[:-2] or ks[-1] != qs[-1]:
        raise ValueError("q and k must be [..., H, d] with the same tokens and d")
    if norm not in _NORM:
        raise ValueError("norm must be 'l2' or 'rms'")
    lead, (Hq, d), Hk = qs[:-2], qs[-2:], ks[-2]
    for name, w in (("wq", wq), ("wk", wk)):
        if w is not None:
            if not _plain(ix, torch.float32, w):
                _check(w, name, torch.float32, dev)
            if w.shape != (d,):
                raise ValueError(f"{name} must be [{d}]")
    rot = 0
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq come together")
    if positions is not None:
        if not (_plain(ix, torch.int32, positions) and _plain(ix, torch.float32, inv_freq)):
            _check(positions, "positions", torch.int32, dev)
            _check(inv_freq, "inv_freq", torch.float32, dev)
        if positions.shape != lead or inv_freq.dim() != 1:
            raise ValueError("positions must have the tokens' shape and inv_freq be [rot / 2]")
        rot = 2 * inv_freq.shape[0]
    return math.prod(lead), Hq, Hk, d, rot, _token_stride(q, "q"), _token_stride(k, "k")


def qk_norm_rope(q, k, wq=None, wk=None, positions=None, inv_freq=None, norm: str = "rms",
                 eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None,
                 out_dtype=None):
    """Norm of every head of q and k and the rotation by position in one pass
    (``ckda_qk_norm_rope``): the q and k that the recurrences of this package take.

    q ``[..., Hq, d]`` and k ``[..., Hk, d]`` share the tokens' shape; they may be views
    into one projection's output (the heads of a token contiguous, tokens at one stride).
    ``norm`` "rms" (unit mean square) or "l2" (unit length), ``wq``, ``wk`` fp32 ``[d]`` or
    None.  ``positions`` (int32, the tokens' shape) and ``inv_freq`` (fp32 ``[rot / 2]``)
    turn the first ``rot`` channels: pairs ``(p, p + rot / 2)``, or ``(2p, 2p + 1)`` when
    ``interleaved``; without them nothing is turned.  ``q_out`` and ``k_out`` may be q and k
    themselves if those are contiguous.  Returns ``(q_out, k_out)``, contiguous."""
    n, Hq, Hk, d, rot, qs, ks = _qk_inputs(q, k, wq, wk, positions, inv_freq, norm)
    dev = q.device
    if out_dtype is None:
        out_dtype = q_out.dtype if q_out is not None else q.dtype
    if out_dtype not in _DT:
        raise TypeError("out_dtype must be float32 or bfloat16")
    outs = []
    for name, t, x in (("q_out", q_out, q), ("k_out", k_out, k)):
        if t is None:
            t = torch.empty_like(x, dtype=out_dtype, memory_format=_CF)
        else:
            _check(t, name, out_dtype, dev)
            if t.shape != x.shape:
                raise ValueError(f"{name} must have {name[0]}'s shape")
        outs.append(t)
    rc = _call(
        _lib.load().ckda_qk_norm_rope, dev,
        q.data_ptr(), k.data_ptr(), _p(wq), _p(wk), _p(positions), _p(inv_freq),
        outs[0].data_ptr(), outs[1].data_ptr(), n, Hq, Hk, d, rot, 1 if interleaved else 0, _NORM[norm], eps, qs, ks, _DT[q.dtype],
        _DT[out_dtype])
    if rc != 0:
        raise CKDAError(rc, "ckda_qk_norm_rope")
    return outs[0], outs[1]


def qk_norm_rope_bwd(q, k, dq_out, dk_out, wq=None, wk=None, positions=None, inv_freq=None,
                     norm: str = "rms", eps: float = 1e-6, interleaved: bool = False,
                     workspace=None):
    """Backward of ``qk_norm_rope`` (``ckda_qk_norm_rope_bwd``) given ``dq_out`` and
    ``dk_out`` (contiguous, q's dtype); the other arguments are those of the forward.

    Returns a dict: ``dq``, ``dk`` (contiguous, q's dtype) and ``dwq``, ``dwk`` (fp32
    ``[d]``, each None without its weight)."""
    n, Hq, Hk, d, rot, qs, ks = _qk_inputs(q, k, wq, wk, positions, inv_freq, norm)
    dev = q.device
    plain = _plain(q.get_device(), q.dtype, dq_out, dk_out)
    for name, t, x in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if not plain:
            _check(t, name, q.dtype, dev)
        if t.shape != x.shape:
            raise ValueError(f"{name} must have {name[1]}'s shape")
    g = {"dq": torch.empty_like(q, memory_format=_CF), "dk": torch.empty_like(k, memory_format=_CF),
         "dwq": None if wq is None else torch.empty_like(wq),
         "dwk": None if wk is None else torch.empty_like(wk)}
    lib = _lib.load()
    if workspace is None and (wq is not None or wk is not None):
        need = lib.ckda_qk_norm_rope_bwd_workspace_bytes(d)
        if need < 0:
            raise CKDAError(int(need), "ckda_qk_norm_rope_bwd_workspace_bytes")
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8, dev)
    rc = _call(
        lib.ckda_qk_norm_rope_bwd, dev,
        _p(q), _p(k), _p(wq), _p(wk), _p(positions), _p(inv_freq), _p(dq_out), _p(dk_out),
        _p(g["dq"]), _p(g["dk"]), _p(g["dwq"]), _p(g["dwk"]), n, Hq, Hk, d, rot,
        1 if interleaved else 0, _NORM[norm], eps, qs, ks, _DT[q.dtype], _p(workspace),
        0 if workspace is None else workspace.numel())
    if rc != 0:
        raise CKDAError(rc, "ckda_qk_norm_rope_bwd")
    return g


def device_status(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device status word."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return _lib.load().ckda_device_status(_stream_ptr(dev))
