"""Chunkwise (gated) delta rule on AMD MI355X (gfx950).

The recurrence (Gated DeltaNet review thread, Table 1, rows "DeltaNet" and
"Gated DeltaNet"), per sequence and head:

    S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
    o_t = S_t q_t,   alpha_t = exp(g_t)

evaluated chunkwise in WY/UT form by hand-written HIP kernels in ``libdn.so``.
This module is a thin ctypes binding: it checks tensors, allocates outputs and
workspace with torch, and passes raw device pointers and the current HIP
stream to the C ABI declared in ``include/dn.h``.  Every step of the
computation runs in the library's kernels; there is no fallback.

States are stored transposed, ``h = S^T`` with shape ``[N, H, Dk, Dv]``.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

__all__ = ["chunk_fwd", "chunk_bwd", "chunk_bwd_noalloc", "bwd_workspace_bytes", "recurrent_step",
           "longhorn_eps", "longhorn_eps_bwd", "longhorn_fwd", "longhorn_bwd", "prologue", "prologue_bwd",
           "short_conv", "short_conv_bwd", "DeltaRule", "delta_rule", "ShortConv", "short_conv_fn",
           "ssm_fwd", "ssm_bwd", "ssm_step", "ssm_scan", "SsmScan", "conv_silu", "conv_silu_bwd", "conv_silu_step",
           "conv_silu_fn", "ConvSilu", "gated_norm", "gated_norm_bwd", "gated_norm_fn", "GatedNorm",
           "load_library", "LIB_PATH", "DnError"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdn.so")

DN_F32, DN_BF16 = 0, 1
DN_ZERO_TAIL = 0x100
_DTYPES = {torch.float32: DN_F32, torch.bfloat16: DN_BF16}


class DnError(RuntimeError):
    """A non-OK status returned by the library."""

    def __init__(self, fn: str, status: int, msg: str):
        super().__init__("%s: %s" % (fn, msg))
        self.status = status


class _Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("Dk", ctypes.c_int32), ("Dv", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class _SsmShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("G", ctypes.c_int32),
                ("Dk", ctypes.c_int32), ("Dv", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


_lib = None


def load_library():
    """Load libdn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libdn.so is not built (%s); run __graft_entry__.build() or "
                           "python chunkwise_delta_rule_wy_amd/build.py" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, S = ctypes.c_void_p, ctypes.POINTER(_Shape)
    lib.dn_status_str.argtypes = [ctypes.c_int]
    lib.dn_status_str.restype = ctypes.c_char_p
    lib.dn_chunk_fwd_workspace.argtypes = [S]
    lib.dn_chunk_fwd_workspace.restype = ctypes.c_size_t
    lib.dn_chunk_bwd_workspace.argtypes = [S]
    lib.dn_chunk_bwd_workspace.restype = ctypes.c_size_t
    lib.dn_chunk_fwd.argtypes = [S] + [P] * 9 + [P, ctypes.c_size_t, P]
    lib.dn_chunk_fwd.restype = ctypes.c_int
    lib.dn_chunk_bwd.argtypes = [S] + [P] * 7 + [P, P] + [P] * 6 + [P, ctypes.c_size_t, P]
    lib.dn_chunk_bwd.restype = ctypes.c_int
    lib.dn_chunk_bwd_events.argtypes = [S] + [P] * 7 + [P, P] + [P] * 6 + [P, ctypes.c_size_t, P, P]
    lib.dn_chunk_bwd_events.restype = ctypes.c_int
    lib.dn_chunk_fwd_save.argtypes = [S] + [P] * 9 + [P, ctypes.c_size_t, P]
    lib.dn_chunk_fwd_save.restype = ctypes.c_int
    lib.dn_chunk_bwd_saved.argtypes = [S] + [P] * 7 + [P, P] + [P] * 6 + [P, ctypes.c_size_t, P, P]
    lib.dn_chunk_bwd_saved.restype = ctypes.c_int
    lib.dn_chunk_bwd_prologue.argtypes = ([S] + [P] * 7 + [P, P] + [P, P, P, ctypes.c_float] + [P] * 6
                                          + [P, ctypes.c_size_t, P, P])
    lib.dn_chunk_bwd_prologue.restype = ctypes.c_int
    lib.dn_chunk_bwd_longhorn.argtypes = [S] + [P] * 7 + [P, P] + [P] + [P] * 6 + [P, ctypes.c_size_t, P, P]
    lib.dn_chunk_bwd_longhorn.restype = ctypes.c_int
    lib.dn_chunk_bwd_noalloc.argtypes = [S] + [P] * 7 + [P, P] + [P] * 6 + [P]
    lib.dn_chunk_bwd_noalloc.restype = ctypes.c_int
    lib.dn_recurrent_step.argtypes = [ctypes.c_int32] * 5 + [P] * 7 + [P]
    lib.dn_recurrent_step.restype = ctypes.c_int
    lib.dn_longhorn_eps.argtypes = [ctypes.c_int32] * 5 + [P] * 3 + [P]
    lib.dn_longhorn_eps.restype = ctypes.c_int
    lib.dn_longhorn_eps_bwd.argtypes = [ctypes.c_int32] * 5 + [P] * 5 + [P]
    lib.dn_longhorn_eps_bwd.restype = ctypes.c_int
    lib.dn_prologue.argtypes = [ctypes.c_int32] * 5 + [P] * 4 + [ctypes.c_float] + [P] * 4 + [P]
    lib.dn_prologue.restype = ctypes.c_int
    lib.dn_prologue_bwd.argtypes = [ctypes.c_int32] * 5 + [P] * 4 + [ctypes.c_float] + [P] * 8 + [P]
    lib.dn_prologue_bwd.restype = ctypes.c_int
    lib.dn_short_conv.argtypes = [ctypes.c_int32] * 7 + [P] * 4 + [P]
    lib.dn_short_conv.restype = ctypes.c_int
    lib.dn_short_conv_bwd.argtypes = [ctypes.c_int32] * 7 + [P] * 6 + [P]
    lib.dn_short_conv_bwd.restype = ctypes.c_int
    lib.dn_short_conv_l2.argtypes = [ctypes.c_int32] * 7 + [P] * 4 + [P]
    lib.dn_short_conv_l2.restype = ctypes.c_int
    lib.dn_short_conv_l2_bwd.argtypes = [ctypes.c_int32] * 7 + [P] * 6 + [P]
    lib.dn_short_conv_l2_bwd.restype = ctypes.c_int
    I, Z = ctypes.c_int32, ctypes.c_size_t
    SS = ctypes.POINTER(_SsmShape)
    lib.dn_ssm_fwd_workspace.argtypes = lib.dn_ssm_bwd_workspace.argtypes = [SS]
    lib.dn_ssm_fwd_workspace.restype = lib.dn_ssm_bwd_workspace.restype = Z
    lib.dn_ssm_fwd.argtypes = [SS] + [P] * 9 + [P, P] + [P, Z, P]
    lib.dn_ssm_bwd.argtypes = [SS] + [P] * 9 + [P, P] + [P] * 8 + [P, Z, P]
    lib.dn_ssm_step.argtypes = [I] * 6 + [P] * 9 + [P]
    lib.dn_conv_silu.argtypes = [I] * 7 + [P] * 7 + [P]
    lib.dn_conv_silu_bwd_workspace.argtypes = [I] * 5
    lib.dn_conv_silu_bwd_workspace.restype = Z
    lib.dn_conv_silu_bwd.argtypes = [I] * 7 + [P] * 11 + [P, Z, P]
    lib.dn_conv_silu_step.argtypes = [I] * 5 + [P] * 5 + [P]
    lib.dn_gated_norm.argtypes = [ctypes.c_int64, I, I, I] + [P] * 3 + [ctypes.c_float, I] + [P] + [P]
    lib.dn_gated_norm_bwd_workspace.argtypes = [ctypes.c_int64, I, I]
    lib.dn_gated_norm_bwd_workspace.restype = Z
    lib.dn_gated_norm_bwd.argtypes = ([ctypes.c_int64, I, I, I] + [P] * 3 + [ctypes.c_float, I] + [P] * 4
                                      + [P, Z, P])
    for name in ("ssm_fwd", "ssm_bwd", "ssm_step", "conv_silu", "conv_silu_bwd", "conv_silu_step", "gated_norm",
                 "gated_norm_bwd"):
        getattr(lib, "dn_" + name).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != 0:
        msg = load_library().dn_status_str(status).decode()
        raise DnError(fn, status, msg)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t, name, dtype, shape, dev):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _workspace(ws, dev, nbytes, name):
    """Check a caller's workspace: a contiguous uint8 tensor on the inputs'
    device holding at least nbytes."""
    if not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise TypeError("%s must be a contiguous uint8 tensor" % name)
    if ws.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, ws.device, dev))
    if ws.numel() < nbytes:
        raise ValueError("%s holds %d bytes, %d needed" % (name, ws.numel(), nbytes))
    return ws


def _shape(q, v, cu_seqlens, chunk):
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, Dk]")
    if q.dtype not in _DTYPES:
        raise TypeError("q, k, v must be float32 or bfloat16")
    if q.device.type != "cuda":
        raise ValueError("tensors must be on a GPU")
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    return _Shape(B, T, H, Dk, Dv, N, chunk, _DTYPES[q.dtype]), N


def chunk_fwd(q, k, v, beta, g=None, h0=None, cu_seqlens=None, output_final_state=True,
              chunk: int = 64, save_workspace: Optional[torch.Tensor] = None):
    """Chunkwise forward pass.

    q, k ``[B,T,H,Dk]``, v ``[B,T,H,Dv]`` (float32 or bfloat16, one dtype);
    beta, g ``[B,T,H]`` float32 (g None: no gate); h0 ``[N,H,Dk,Dv]`` float32
    or None; cu_seqlens int32 ``[N+1]`` on the device for packed sequences
    (then B == 1).  Returns ``(o, hT)`` (hT None unless output_final_state).
    ``save_workspace`` (uint8, at least ``bwd_workspace_bytes``; bfloat16
    inputs only): also store the chunk-start states there for
    ``chunk_bwd(..., saved=True)`` (``dn_chunk_fwd_save``).
    """
    lib = load_library()
    s, N = _shape(q, v, cu_seqlens, chunk)
    dev = q.device
    B, T, H, Dk, Dv = s.B, s.T, s.H, s.Dk, s.Dv
    _need(q, "q", q.dtype, (B, T, H, Dk), dev)
    _need(k, "k", q.dtype, (B, T, H, Dk), dev)
    _need(v, "v", q.dtype, (B, T, H, Dv), dev)
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    _need(g, "g", torch.float32, (B, T, H), dev)
    _need(h0, "h0", torch.float32, (N, H, Dk, Dv), dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    o = torch.empty((B, T, H, Dv), dtype=q.dtype, device=dev)
    hT = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=dev) if output_final_state else None
    if save_workspace is not None:
        _workspace(save_workspace, dev, lib.dn_chunk_bwd_workspace(ctypes.byref(s)), "save_workspace")
        _check("dn_chunk_fwd_save", lib.dn_chunk_fwd_save(
            ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
            _ptr(cu_seqlens), _ptr(o), _ptr(hT), _ptr(save_workspace), save_workspace.numel(),
            _stream(dev)))
        return o, hT
    wsb = lib.dn_chunk_fwd_workspace(ctypes.byref(s))
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    _check("dn_chunk_fwd", lib.dn_chunk_fwd(
        ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
        _ptr(cu_seqlens), _ptr(o), _ptr(hT), _ptr(ws), wsb, _stream(dev)))
    return o, hT


def chunk_bwd(q, k, v, beta, g, h0, dO, dhT=None, cu_seqlens=None, chunk: int = 64,
              workspace: Optional[torch.Tensor] = None, events=None, saved: bool = False,
              prologue_inputs=None, longhorn_beta: Optional[torch.Tensor] = None):
    """Backward pass of ``<dO, o> + <dhT, hT>``.

    Returns a dict of float32 gradients dq, dk, dv, dbeta, dg (None without a
    gate) and dh0.  ``workspace`` (uint8, at least ``bwd_workspace_bytes``)
    may be passed to avoid an allocation per call.  ``events``: four
    ``torch.cuda.Event(enable_timing=True)`` that the library records before
    its first kernel and after the recompute, the state-gradient sweep and the
    chunk-gradient kernel (``dn_chunk_bwd_events``); a None entry is not
    recorded.  ``saved``: skip the
    recompute and read the states that ``chunk_fwd(..., save_workspace=
    workspace)`` stored for these inputs (``dn_chunk_bwd_saved``).
    ``prologue_inputs`` = (q_in, k_in, x_in, gate_scale), with ``saved``: q, k,
    beta, g are ``prologue``'s outputs for these raw inputs, and the dict holds
    the gradients of the raw inputs instead: dq_in, dk_in, db_in, dx_in, with
    dv and dh0 (``dn_chunk_bwd_prologue``: the prologue's backward folded into
    the chunk-gradient kernel).  ``longhorn_beta`` (with ``saved``): beta is
    the Longhorn step size ``longhorn_eps(k, longhorn_beta)``; dbeta is then the
    gradient of ``longhorn_beta`` and dk includes the step size's key term
    (``dn_chunk_bwd_longhorn``).
    """
    lib = load_library()
    s, N = _shape(q, v, cu_seqlens, chunk)
    dev = q.device
    B, T, H, Dk, Dv = s.B, s.T, s.H, s.Dk, s.Dv
    _need(q, "q", q.dtype, (B, T, H, Dk), dev)
    _need(k, "k", q.dtype, (B, T, H, Dk), dev)
    _need(v, "v", q.dtype, (B, T, H, Dv), dev)
    _need(dO, "dO", q.dtype, (B, T, H, Dv), dev)
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    _need(g, "g", torch.float32, (B, T, H), dev)
    _need(h0, "h0", torch.float32, (N, H, Dk, Dv), dev)
    _need(dhT, "dhT", torch.float32, (N, H, Dk, Dv), dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    f32 = dict(dtype=torch.float32, device=dev)
    dq = torch.empty((B, T, H, Dk), **f32)
    dk = torch.empty((B, T, H, Dk), **f32)
    dv = torch.empty((B, T, H, Dv), **f32)
    dbeta = torch.empty((B, T, H), **f32)
    dg = torch.empty((B, T, H), **f32) if g is not None else None
    dh0 = torch.empty((N, H, Dk, Dv), **f32)
    wsb = lib.dn_chunk_bwd_workspace(ctypes.byref(s))
    if saved and workspace is None:
        raise ValueError("saved=True needs the workspace that chunk_fwd filled")
    if workspace is None:
        workspace = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    else:
        _workspace(workspace, dev, wsb, "workspace")
    ev = None
    if events is not None:
        if len(events) != 4:
            raise ValueError("events: four torch.cuda.Event objects (or None) expected")
        for e in events:
            if e is not None and e.cuda_event == 0:  # torch creates the event on its first record
                e.record(torch.cuda.current_stream(dev))
        ev = (ctypes.c_void_p * 4)(*[None if e is None else e.cuda_event for e in events])
    if longhorn_beta is not None:
        if not saved or prologue_inputs is not None:
            raise ValueError("longhorn_beta needs saved=True and no prologue_inputs")
        _need(longhorn_beta, "longhorn_beta", torch.float32, (B, T, H), dev)
        _check("dn_chunk_bwd_longhorn", lib.dn_chunk_bwd_longhorn(
            ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
            _ptr(cu_seqlens), _ptr(dO), _ptr(dhT), _ptr(longhorn_beta), _ptr(dq), _ptr(dk), _ptr(dv),
            _ptr(dbeta), _ptr(dg), _ptr(dh0), _ptr(workspace), workspace.numel(), _stream(dev), ev))
        return dict(dq=dq, dk=dk, dv=dv, dbeta=dbeta, dg=dg, dh0=dh0)
    if prologue_inputs is not None:
        if not saved:
            raise ValueError("prologue_inputs needs saved=True (the states dn_chunk_fwd_save kept)")
        q_in, k_in, x_in, gate_scale = prologue_inputs
        _need(q_in, "q_in", q.dtype, (B, T, H, Dk), dev)
        _need(k_in, "k_in", q.dtype, (B, T, H, Dk), dev)
        _need(x_in, "x_in", torch.float32, (B, T, H), dev)
        _check("dn_chunk_bwd_prologue", lib.dn_chunk_bwd_prologue(
            ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
            _ptr(cu_seqlens), _ptr(dO), _ptr(dhT), _ptr(q_in), _ptr(k_in), _ptr(x_in),
            float(gate_scale), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dg), _ptr(dh0),
            _ptr(workspace), workspace.numel(), _stream(dev), ev))
        return dict(dq_in=dq, dk_in=dk, dv=dv, db_in=dbeta, dx_in=dg, dh0=dh0)
    fn = lib.dn_chunk_bwd_saved if saved else lib.dn_chunk_bwd_events
    _check("dn_chunk_bwd_saved" if saved else "dn_chunk_bwd", fn(
        ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0),
        _ptr(cu_seqlens), _ptr(dO), _ptr(dhT), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta),
        _ptr(dg), _ptr(dh0), _ptr(workspace), workspace.numel(), _stream(dev), ev))
    return dict(dq=dq, dk=dk, dv=dv, dbeta=dbeta, dg=dg, dh0=dh0)


def chunk_bwd_noalloc(q, k, v, beta, g, h0, dO, dhT=None, cu_seqlens=None, out=None, chunk: int = 64):
    """``chunk_bwd`` (recomputing) through ``dn_chunk_bwd_noalloc``: the
    library's static scratch buffer replaces the workspace, so the call
    allocates no device memory of its own.  ``out``: optional dict of
    preallocated float32 gradients (dq, dk, dv, dbeta, dg, dh0) to write into;
    missing ones are allocated here.  Returns that dict."""
    lib = load_library()
    s, N = _shape(q, v, cu_seqlens, chunk)
    dev = q.device
    B, T, H, Dk, Dv = s.B, s.T, s.H, s.Dk, s.Dv
    _need(q, "q", q.dtype, (B, T, H, Dk), dev)
    _need(k, "k", q.dtype, (B, T, H, Dk), dev)
    _need(v, "v", q.dtype, (B, T, H, Dv), dev)
    _need(dO, "dO", q.dtype, (B, T, H, Dv), dev)
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    _need(g, "g", torch.float32, (B, T, H), dev)
    _need(h0, "h0", torch.float32, (N, H, Dk, Dv), dev)
    _need(dhT, "dhT", torch.float32, (N, H, Dk, Dv), dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    shapes = dict(dq=(B, T, H, Dk), dk=(B, T, H, Dk), dv=(B, T, H, Dv), dbeta=(B, T, H), dg=(B, T, H),
                  dh0=(N, H, Dk, Dv))
    res = dict(out) if out is not None else {}
    for name, shp in shapes.items():
        if name == "dg" and g is None:
            res[name] = None
        elif res.get(name) is None:
            res[name] = torch.empty(shp, dtype=torch.float32, device=dev)
        else:
            _need(res[name], name, torch.float32, shp, dev)
    _check("dn_chunk_bwd_noalloc", lib.dn_chunk_bwd_noalloc(
        ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(h0), _ptr(cu_seqlens),
        _ptr(dO), _ptr(dhT), _ptr(res["dq"]), _ptr(res["dk"]), _ptr(res["dv"]), _ptr(res["dbeta"]),
        _ptr(res["dg"]), _ptr(res["dh0"]), _stream(dev)))
    return res


def bwd_workspace_bytes(B, T, H, Dk, Dv, n_seqs=None, dtype=torch.bfloat16, chunk=64) -> int:
    s = _Shape(B, T, H, Dk, Dv, B if n_seqs is None else n_seqs, chunk, _DTYPES[dtype])
    return int(load_library().dn_chunk_bwd_workspace(ctypes.byref(s)))


def recurrent_step(q, k, v, beta, g, state):
    """One decode step.  q, k ``[B,H,Dk]``, v ``[B,H,Dv]``, beta/g ``[B,H]``
    float32 (g may be None), state ``[B,H,Dk,Dv]`` float32 updated in place.
    Returns o ``[B,H,Dv]``."""
    lib = load_library()
    if q.dim() != 3 or q.dtype not in _DTYPES or q.device.type != "cuda":
        raise ValueError("q must be a [B, H, Dk] float32/bfloat16 GPU tensor")
    dev = q.device
    B, H, Dk = q.shape
    Dv = v.shape[-1]
    _need(q, "q", q.dtype, (B, H, Dk), dev)
    _need(k, "k", q.dtype, (B, H, Dk), dev)
    _need(v, "v", q.dtype, (B, H, Dv), dev)
    _need(beta, "beta", torch.float32, (B, H), dev)
    _need(g, "g", torch.float32, (B, H), dev)
    _need(state, "state", torch.float32, (B, H, Dk, Dv), dev)
    o = torch.empty((B, H, Dv), dtype=q.dtype, device=dev)
    _check("dn_recurrent_step", lib.dn_recurrent_step(
        B, H, Dk, Dv, _DTYPES[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g),
        _ptr(state), _ptr(o), _stream(dev)))
    return o


def _key_rows(k, beta):
    """(B, T, H, Dk) of a key tensor [B,T,H,Dk] or a decode key [B,H,Dk]."""
    if k.dim() == 3:
        B, H, Dk = k.shape
        T = 1
    elif k.dim() == 4:
        B, T, H, Dk = k.shape
    else:
        raise ValueError("k must be [B,T,H,Dk] or [B,H,Dk]")
    if k.dtype not in _DTYPES or k.device.type != "cuda":
        raise ValueError("k must be a float32/bfloat16 GPU tensor")
    _need(k, "k", k.dtype, tuple(k.shape), k.device)
    _need(beta, "beta", torch.float32, tuple(k.shape[:-1]), k.device)
    return B, T, H, Dk


def longhorn_eps(k, beta):
    """Longhorn step size eps = beta / (1 + beta |k|^2) (``dn_longhorn_eps``),
    float32 with beta's shape; feed it to ``chunk_fwd`` / ``recurrent_step``
    as beta to run the Longhorn recurrence."""
    lib = load_library()
    B, T, H, Dk = _key_rows(k, beta)
    eps = torch.empty(beta.shape, dtype=torch.float32, device=k.device)
    _check("dn_longhorn_eps", lib.dn_longhorn_eps(
        B, T, H, Dk, _DTYPES[k.dtype], _ptr(k), _ptr(beta), _ptr(eps), _stream(k.device)))
    return eps


def longhorn_eps_bwd(k, beta, deps, dk):
    """Backward of ``longhorn_eps`` (``dn_longhorn_eps_bwd``): returns dbeta and
    adds the key term into ``dk`` (float32, updated in place)."""
    lib = load_library()
    B, T, H, Dk = _key_rows(k, beta)
    _need(deps, "deps", torch.float32, tuple(beta.shape), k.device)
    _need(dk, "dk", torch.float32, tuple(k.shape), k.device)
    dbeta = torch.empty(beta.shape, dtype=torch.float32, device=k.device)
    _check("dn_longhorn_eps_bwd", lib.dn_longhorn_eps_bwd(
        B, T, H, Dk, _DTYPES[k.dtype], _ptr(k), _ptr(beta), _ptr(deps), _ptr(dbeta), _ptr(dk),
        _stream(k.device)))
    return dbeta


def longhorn_fwd(q, k, v, beta, g=None, h0=None, cu_seqlens=None, output_final_state=True):
    """Forward pass of the Longhorn recurrence: ``longhorn_eps`` then
    ``chunk_fwd`` at beta := eps.  Returns (o, hT)."""
    return chunk_fwd(q, k, v, longhorn_eps(k, beta), g, h0, cu_seqlens, output_final_state)


def longhorn_bwd(q, k, v, beta, g, h0, dO, dhT=None, cu_seqlens=None, workspace=None):
    """Backward pass of the Longhorn recurrence: eps again (nothing is kept
    from the forward call), ``chunk_bwd`` at beta := eps, then
    ``longhorn_eps_bwd``.  Returns the gradient dict of ``chunk_bwd``."""
    eps = longhorn_eps(k, beta)
    gr = chunk_bwd(q, k, v, eps, g, h0, dO, dhT, cu_seqlens, workspace=workspace)
    gr["dbeta"] = longhorn_eps_bwd(k, beta, gr["dbeta"], gr["dk"])
    return gr


def prologue(q_in, k_in, b_in, x_in=None, gate_scale: float = 1.0):
    """Input prologue (``dn_prologue``): q, k L2-normalised per row (dtype of
    q_in), beta = sigmoid(b_in), g = -gate_scale * softplus(x_in) (None
    without x_in).  Returns (q, k, beta, g)."""
    lib = load_library()
    B, T, H, Dk = _key_rows(k_in, b_in)
    _need(q_in, "q_in", k_in.dtype, tuple(k_in.shape), k_in.device)
    _need(x_in, "x_in", torch.float32, tuple(b_in.shape), k_in.device)
    q = torch.empty_like(q_in)
    k = torch.empty_like(k_in)
    beta = torch.empty_like(b_in)
    g = torch.empty_like(x_in) if x_in is not None else None
    _check("dn_prologue", lib.dn_prologue(
        B, T, H, Dk, _DTYPES[k_in.dtype], _ptr(q_in), _ptr(k_in), _ptr(b_in), _ptr(x_in),
        float(gate_scale), _ptr(q), _ptr(k), _ptr(beta), _ptr(g), _stream(k_in.device)))
    return q, k, beta, g


def prologue_bwd(q_in, k_in, b_in, x_in, gate_scale, dq, dk, dbeta, dg=None):
    """Backward of ``prologue`` (``dn_prologue_bwd``): float32 gradients
    (dq_in, dk_in, db_in, dx_in) from those of q, k, beta, g."""
    lib = load_library()
    B, T, H, Dk = _key_rows(k_in, b_in)
    dev = k_in.device
    _need(q_in, "q_in", k_in.dtype, tuple(k_in.shape), dev)
    _need(x_in, "x_in", torch.float32, tuple(b_in.shape), dev)
    _need(dq, "dq", torch.float32, tuple(k_in.shape), dev)
    _need(dk, "dk", torch.float32, tuple(k_in.shape), dev)
    _need(dbeta, "dbeta", torch.float32, tuple(b_in.shape), dev)
    _need(dg, "dg", torch.float32, tuple(b_in.shape), dev)
    f32 = dict(dtype=torch.float32, device=dev)
    dq_in = torch.empty(k_in.shape, **f32)
    dk_in = torch.empty(k_in.shape, **f32)
    db_in = torch.empty(b_in.shape, **f32)
    dx_in = torch.empty(b_in.shape, **f32) if x_in is not None else None
    _check("dn_prologue_bwd", lib.dn_prologue_bwd(
        B, T, H, Dk, _DTYPES[k_in.dtype], _ptr(q_in), _ptr(k_in), _ptr(b_in), _ptr(x_in),
        float(gate_scale), _ptr(dq), _ptr(dk), _ptr(dbeta), _ptr(dg), _ptr(dq_in), _ptr(dk_in),
        _ptr(db_in), _ptr(dx_in), _stream(dev)))
    return dq_in, dk_in, db_in, dx_in


def _conv_dims(x, w, cu_seqlens):
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise ValueError("x must be a [B, T, H, D] tensor")
    if x.dtype not in _DTYPES:
        raise TypeError("x must be float32 or bfloat16")
    B, T, H, D = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 3 or tuple(w.shape[:2]) != (H, D):
        raise ValueError("w must be a [H, D, W] tensor")
    W = w.shape[2]
    _need(w, "w", torch.float32, (H, D, W), x.device)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    n_seqs = B
    if cu_seqlens is not None:
        n_seqs = cu_seqlens.numel() - 1
        _need(cu_seqlens, "cu_seqlens", torch.int32, (n_seqs + 1,), x.device)
    return B, T, H, D, W, n_seqs


def short_conv(x, w, cu_seqlens=None, l2norm: bool = False):
    """Depthwise causal short convolution (``dn_short_conv``): y[t] = sum_j
    w[:, :, j] x[t - (W - 1) + j] inside each sequence; x [B, T, H, D], w
    [H, D, W] float32.  With ``l2norm`` every (token, head) row of y is
    scaled to unit length in the same pass (``dn_short_conv_l2``).  Returns y
    (dtype of x)."""
    lib = load_library()
    B, T, H, D, W, n = _conv_dims(x, w, cu_seqlens)
    y = torch.empty_like(x)
    fn = "dn_short_conv_l2" if l2norm else "dn_short_conv"
    _check(fn, getattr(lib, fn)(
        B, T, H, D, W, n, _DTYPES[x.dtype], _ptr(x), _ptr(w), _ptr(cu_seqlens), _ptr(y), _stream(x.device)))
    return y


def short_conv_bwd(x, w, dy, cu_seqlens=None, l2norm: bool = False):
    """Backward of ``short_conv`` (``dn_short_conv_bwd``, or
    ``dn_short_conv_l2_bwd`` with ``l2norm``): float32 (dx, dw) from dy =
    dL/dy (float32, the shape of x)."""
    lib = load_library()
    B, T, H, D, W, n = _conv_dims(x, w, cu_seqlens)
    _need(dy, "dy", torch.float32, tuple(x.shape), x.device)
    dx = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    dw = torch.empty(w.shape, dtype=torch.float32, device=x.device)
    fn = "dn_short_conv_l2_bwd" if l2norm else "dn_short_conv_bwd"
    _check(fn, getattr(lib, fn)(
        B, T, H, D, W, n, _DTYPES[x.dtype], _ptr(x), _ptr(w), _ptr(cu_seqlens), _ptr(dy), _ptr(dx),
        _ptr(dw), _stream(x.device)))
    return dx, dw


class DeltaRule(torch.autograd.Function):
    """Autograd wrapper: forward by ``chunk_fwd``, backward by ``chunk_bwd``.
    Gradients are computed in float32 and cast to each input's dtype.  For
    bfloat16 inputs with ``save_states`` the forward pass keeps the bf16 chunk
    states (d_k d_v per chunk and head) and the backward pass skips their
    recompute; otherwise the backward pass recomputes them."""

    @staticmethod
    def forward(ctx, q, k, v, beta, g, h0, cu_seqlens, save_states=True):
        ws = None
        if save_states and q.dtype == torch.bfloat16:
            N = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
            ws = torch.empty(max(bwd_workspace_bytes(q.shape[0], q.shape[1], q.shape[2], q.shape[3],
                                                     v.shape[-1], N, q.dtype), 1),
                             dtype=torch.uint8, device=q.device)
        o, hT = chunk_fwd(q, k, v, beta, g, h0, cu_seqlens, output_final_state=True,
                          save_workspace=ws)
        ctx.save_for_backward(q, k, v, beta, g, h0, cu_seqlens)
        ctx.ws = ws
        return o, hT

    @staticmethod
    def backward(ctx, dO, dhT):
        q, k, v, beta, g, h0, cu = ctx.saved_tensors
        if dO is None:
            dO = torch.zeros(v.shape, dtype=q.dtype, device=q.device)
        ws, ctx.ws = ctx.ws, None
        gr = chunk_bwd(q, k, v, beta, g, h0, dO.to(q.dtype).contiguous(),
                       None if dhT is None else dhT.float().contiguous(), cu,
                       workspace=ws, saved=ws is not None)
        return (gr["dq"].to(q.dtype), gr["dk"].to(k.dtype), gr["dv"].to(v.dtype), gr["dbeta"],
                gr["dg"], None if h0 is None else gr["dh0"], None, None)


def delta_rule(q, k, v, beta, g=None, h0=None, cu_seqlens=None, save_states=True):
    """Differentiable chunkwise (gated) delta rule; returns (o, hT).
    ``save_states`` keeps the chunk states from the forward pass for the
    backward pass (bfloat16 inputs) instead of recomputing them."""
    return DeltaRule.apply(q, k, v, beta, g, h0, cu_seqlens, save_states)


class ShortConv(torch.autograd.Function):
    """Autograd wrapper of the depthwise causal short convolution: forward by
    ``short_conv``, backward by ``short_conv_bwd`` (dx cast to x's dtype, dw
    float32).  ``l2norm`` fuses the per-head L2 normalisation (q and k)."""

    @staticmethod
    def forward(ctx, x, w, cu_seqlens, l2norm=False):
        ctx.save_for_backward(x, w, cu_seqlens)
        ctx.l2norm = l2norm
        return short_conv(x, w, cu_seqlens, l2norm=l2norm)

    @staticmethod
    def backward(ctx, dy):
        x, w, cu = ctx.saved_tensors
        dx, dw = short_conv_bwd(x, w, dy.float().contiguous(), cu, l2norm=ctx.l2norm)
        return dx.to(x.dtype), dw, None, None


def short_conv_fn(x, w, cu_seqlens=None, l2norm=False):
    """Differentiable short convolution (optionally with the per-head L2
    normalisation fused in)."""
    return ShortConv.apply(x, w, cu_seqlens, l2norm)


# ------------------------------------------------- the state space mixer


# Single tokens are bound by what the host does before the launch: the calls
# below pass raw addresses, test a tensor in one expression (the slow path
# words the error) and ask for the device and its stream without their objects.

_MAX_SIZE = 2 ** 31 - 1  # the library's sizes are 32-bit


def _adr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _call(name, dev, *args):
    """Call a library function on ``dev``'s (a device or its index) current
    stream, with it as the current device (kernels start on the current device)."""
    fn = getattr(_lib or load_library(), name)
    i = dev if type(dev) is int else dev.index
    if torch._C._cuda_getDevice() == i:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if status:
        _check(name, status)


def _fits(t, dtype, shape, i):
    """Whether a tensor is a contiguous one of this type and shape on GPU i."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == i and t.is_contiguous()


def _is(t, name, dtype, shape, dev):
    """``_need`` with a quick way through for a tensor that is right."""
    if t is None or (isinstance(t, torch.Tensor) and _fits(t, dtype, shape, dev.index)):
        return
    _need(t, name, dtype, shape, dev)


def _gpu(t, name, dims, dtypes):
    """The device of a required tensor of these numbers of dimensions and types."""
    if not isinstance(t, torch.Tensor) or t.dim() not in dims:
        raise ValueError("%s must be a tensor of %s dimensions" % (name, " or ".join(str(d) for d in dims)))
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, " or ".join(str(d) for d in dtypes)))
    if t.device.type != "cuda":
        raise ValueError("tensors must be on a GPU")
    if any(n > _MAX_SIZE for n in t.shape):
        raise ValueError("%s has a size of 2^31 or more" % name)
    return t.device


def _given(**tensors):
    for name, t in tensors.items():
        if t is None:
            raise TypeError("%s is required" % name)


def _seqs(B, cu_seqlens, dev):
    """The number of sequences: B, or that of the packed offsets (B == 1)."""
    if cu_seqlens is None:
        return B
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-d tensor of at least two offsets")
    if B != 1:
        raise ValueError("packed sequences need a batch of one")
    _is(cu_seqlens, "cu_seqlens", torch.int32, (cu_seqlens.numel(),), dev)
    return cu_seqlens.numel() - 1


def _ssm_args(q, k, v, dt, A, dt_bias, skip, dtypes, dims):
    """(device, leading sizes, H, G, Dk, Dv) of a scan's inputs, checked."""
    dev = _gpu(v, "v", (dims,), dtypes)
    _gpu(q, "q", (dims,), (v.dtype,))
    lead, H, Dv, G, Dk = tuple(v.shape[:-2]), v.shape[-2], v.shape[-1], q.shape[-2], q.shape[-1]
    if G == 0 or H % G:
        raise ValueError("q has %d heads, which do not divide v's %d" % (G, H))
    _given(k=k, dt=dt, A=A)
    _is(q, "q", v.dtype, lead + (G, Dk), dev)
    _is(k, "k", v.dtype, lead + (G, Dk), dev)
    _is(v, "v", v.dtype, lead + (H, Dv), dev)
    _is(dt, "dt", torch.float32, lead + (H,), dev)
    _is(A, "A", torch.float32, (H,), dev)
    _is(dt_bias, "dt_bias", torch.float32, (H,), dev)
    _is(skip, "skip", torch.float32, (H,), dev)
    return dev, lead, H, G, Dk, Dv


def ssm_fwd(q, k, v, dt, A, dt_bias=None, skip=None, h0=None, cu_seqlens=None, output_final_state=True):
    """Forward pass of the selective state space scan (``dn_ssm_fwd``):

        s_t = softplus(dt_t + dt_bias),  S_t = exp(s_t A) S_{t-1} + s_t v_t k_t^T,
        o_t = S_t q_t + skip v_t.

    q, k ``[B,T,G,Dk]`` and v ``[B,T,H,Dv]`` bfloat16, G dividing H (head h
    reads group ``h // (H // G)``); dt ``[B,T,H]``, A, dt_bias, skip ``[H]``
    float32 (dt_bias, skip None: zero); h0 ``[N,H,Dk,Dv]`` float32 or None;
    cu_seqlens int32 ``[N+1]`` on the device for packed sequences (B == 1),
    from 0 to T; where it ends before T, the rows behind it are not used, and
    theirs in the results are zero.  Returns ``(o, hT)`` (hT None unless
    output_final_state)."""
    lib = load_library()
    dev, (B, T), H, G, Dk, Dv = _ssm_args(q, k, v, dt, A, dt_bias, skip, (torch.bfloat16,), 4)
    N = _seqs(B, cu_seqlens, dev)
    _is(h0, "h0", torch.float32, (N, H, Dk, Dv), dev)
    s = ctypes.byref(_SsmShape(B, T, H, G, Dk, Dv, N, DN_BF16 | DN_ZERO_TAIL))
    o = torch.empty_like(v)
    hT = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=dev) if output_final_state else None
    wsb = lib.dn_ssm_fwd_workspace(s)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
    _call("dn_ssm_fwd", dev, s, _adr(q), _adr(k), _adr(v), _adr(dt), _adr(A), _adr(dt_bias), _adr(skip), _adr(h0),
          _adr(cu_seqlens), _adr(o), _adr(hT), _adr(ws), wsb)
    return o, hT


def ssm_bwd(q, k, v, dt, A, dt_bias, skip, h0, dO, dhT=None, cu_seqlens=None):
    """Backward pass of ``<dO, o> + <dhT, hT>`` of ``ssm_fwd`` (``dn_ssm_bwd``;
    the states are recomputed).  Returns a dict: dq, dk, dv in bfloat16, ddt,
    dA, ddt_bias, dskip (None without the parameter) and dh0 in float32; rows
    behind the last packed sequence are zero."""
    lib = load_library()
    dev, (B, T), H, G, Dk, Dv = _ssm_args(q, k, v, dt, A, dt_bias, skip, (torch.bfloat16,), 4)
    N = _seqs(B, cu_seqlens, dev)
    _is(h0, "h0", torch.float32, (N, H, Dk, Dv), dev)
    _given(dO=dO)
    _is(dO, "dO", v.dtype, tuple(v.shape), dev)
    _is(dhT, "dhT", torch.float32, (N, H, Dk, Dv), dev)
    s = ctypes.byref(_SsmShape(B, T, H, G, Dk, Dv, N, DN_BF16 | DN_ZERO_TAIL))
    gr = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v), ddt=torch.empty_like(dt),
              dA=torch.empty_like(A), ddt_bias=None if dt_bias is None else torch.empty_like(dt_bias),
              dskip=None if skip is None else torch.empty_like(skip),
              dh0=torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=dev))
    wsb = lib.dn_ssm_bwd_workspace(s)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
    _call("dn_ssm_bwd", dev, s, _adr(q), _adr(k), _adr(v), _adr(dt), _adr(A), _adr(dt_bias), _adr(skip), _adr(h0),
          _adr(cu_seqlens), _adr(dO), _adr(dhT), *[_adr(g) for g in gr.values()], _adr(ws), wsb)
    return gr


def ssm_step(q, k, v, dt, A, dt_bias, skip, state):
    """One token of every sequence (``dn_ssm_step``): q, k ``[B,G,Dk]``, v
    ``[B,H,Dv]`` (float32 or bfloat16, one dtype), dt ``[B,H]`` float32, state
    ``[B,H,Dk,Dv]`` float32 updated in place.  Returns o ``[B,H,Dv]``."""
    try:  # the usual call in one expression; anything else goes through the checks that say what is wrong
        E, i, f32, qs, vs = v.dtype, v.get_device(), torch.float32, q.shape, v.shape
        H = vs[-2] if len(vs) == 3 else 0
        fits = (H and len(qs) == 3 and qs[0] == vs[0] <= _MAX_SIZE and qs[1] and H % qs[1] == 0 and E in _DTYPES and i >= 0
                and v.is_contiguous() and _fits(q, E, qs, i) and _fits(k, E, qs, i) and _fits(dt, f32, vs[:2], i)
                and _fits(A, f32, (H,), i) and (dt_bias is None or _fits(dt_bias, f32, (H,), i))
                and (skip is None or _fits(skip, f32, (H,), i))
                and _fits(state, f32, (vs[0], H, qs[2], vs[2]), i))
    except AttributeError:  # not a tensor
        fits = False
    if not fits:
        dev, (B,), H, G, Dk, Dv = _ssm_args(q, k, v, dt, A, dt_bias, skip, tuple(_DTYPES), 3)
        _given(state=state)
        _is(state, "state", torch.float32, (B, H, Dk, Dv), dev)
    o = torch.empty_like(v)
    _call("dn_ssm_step", i, vs[0], H, qs[1], qs[2], vs[2], _DTYPES[E], q.data_ptr(), k.data_ptr(), v.data_ptr(),
          dt.data_ptr(), A.data_ptr(), _adr(dt_bias), _adr(skip), state.data_ptr(), o.data_ptr())
    return o


def _conv_silu_args(x, w, bias, state, cu_seqlens, dims):
    """(device, leading sizes, H, D, W, sequences), checked; state may be None."""
    dev = _gpu(x, "x", (dims,), tuple(_DTYPES))
    lead, (H, D) = tuple(x.shape[:-2]), x.shape[-2:]
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w must be a [H, D, W] tensor")
    W = w.shape[2]
    N = _seqs(lead[0], cu_seqlens, dev)
    _is(x, "x", x.dtype, tuple(x.shape), dev)
    _is(w, "w", torch.float32, (H, D, W), dev)
    _is(bias, "bias", torch.float32, (H, D), dev)
    _is(state, "state", x.dtype, (N, max(W - 1, 0), H, D), dev)
    return dev, lead, H, D, W, N


def conv_silu(x, w, bias=None, s0=None, cu_seqlens=None):
    """Depthwise causal short convolution with bias and SiLU (``dn_conv_silu``):
    y = z sigmoid(z), z[t] = bias + sum_j w[:, :, j] x[t - (W - 1) + j], the
    inputs before a sequence's first token being s0 (zeros without it).  x
    ``[B,T,H,D]`` float32 or bfloat16, w ``[H,D,W]`` and bias ``[H,D]`` float32,
    s0 ``[N,W-1,H,D]`` in x's dtype, cu_seqlens as in ``ssm_fwd``.  Returns
    ``(y, sT)``, sT the last W - 1 inputs: the s0 of a continuation, or the
    state of ``conv_silu_step``."""
    dev, (B, T), H, D, W, N = _conv_silu_args(x, w, bias, s0, cu_seqlens, 4)
    y = torch.empty_like(x)
    sT = x.new_empty((N, max(W - 1, 0), H, D)) if s0 is None else torch.empty_like(s0)
    _call("dn_conv_silu", dev, B, T, H, D, W, N, _DTYPES[x.dtype] | DN_ZERO_TAIL, _adr(x), _adr(w), _adr(bias), _adr(s0),
          _adr(cu_seqlens), _adr(y), _adr(sT))
    return y, sT


def conv_silu_bwd(x, w, bias, s0, dy, dsT=None, cu_seqlens=None):
    """Backward of ``conv_silu`` (``dn_conv_silu_bwd``) from dy and dsT in x's
    dtype (dsT None: 0).  Returns a dict: dx and ds0 in x's dtype, dw and dbias
    (None without a bias) in float32."""
    dev, (B, T), H, D, W, N = _conv_silu_args(x, w, bias, s0, cu_seqlens, 4)
    _given(dy=dy)
    _is(dy, "dy", x.dtype, tuple(x.shape), dev)
    _is(dsT, "dsT", x.dtype, (N, max(W - 1, 0), H, D), dev)
    gr = dict(dx=torch.empty_like(x), dw=torch.empty_like(w), dbias=None if bias is None else torch.empty_like(bias),
              ds0=torch.empty((N, max(W - 1, 0), H, D), dtype=x.dtype, device=dev))
    wsb = load_library().dn_conv_silu_bwd_workspace(B, T, H, D, W)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
    _call("dn_conv_silu_bwd", dev, B, T, H, D, W, N, _DTYPES[x.dtype] | DN_ZERO_TAIL, _adr(x), _adr(w), _adr(bias), _adr(s0),
          _adr(cu_seqlens), _adr(dy), _adr(dsT), *[_adr(g) for g in gr.values()], _adr(ws), wsb)
    return gr


def conv_silu_step(x, w, bias, state):
    """One token of every sequence (``dn_conv_silu_step``): x ``[B,H,D]``, state
    ``[B,W-1,H,D]`` (x's dtype) holding the last W - 1 inputs, updated in
    place.  Returns y ``[B,H,D]``."""
    try:
        E, i, xs, ws = x.dtype, x.get_device(), x.shape, w.shape
        fits = (len(xs) == 3 and len(ws) == 3 and ws[:2] == xs[1:] and ws[2] and E in _DTYPES and i >= 0
                and xs.numel() <= _MAX_SIZE and x.is_contiguous() and _fits(w, torch.float32, ws, i)
                and (bias is None or _fits(bias, torch.float32, ws[:2], i))
                and _fits(state, E, (xs[0], ws[2] - 1, xs[1], xs[2]), i))
    except AttributeError:  # not a tensor
        fits = False
    if not fits:
        _given(state=state)
        _conv_silu_args(x, w, bias, state, None, 3)
    y = torch.empty_like(x)
    _call("dn_conv_silu_step", i, xs[0], xs[1], xs[2], ws[2], _DTYPES[E], x.data_ptr(), w.data_ptr(), _adr(bias),
          state.data_ptr(), y.data_ptr())
    return y


def _gated_norm_args(x, z, w):
    """(device, rows, D, weight rows), checked."""
    dev = _gpu(x, "x", tuple(range(1, 9)), tuple(_DTYPES))
    _given(z=z)
    D = x.shape[-1]
    if not isinstance(w, torch.Tensor) or w.dim() not in (1, 2):
        raise ValueError("w must be a [D] or [H, D] tensor")
    if w.dim() == 2 and (x.dim() < 2 or w.shape[0] != x.shape[-2]):
        raise ValueError("w has shape %s, expected one row for each of x's heads" % (tuple(w.shape),))
    R = 1 if w.dim() == 1 else w.shape[0]
    _is(x, "x", x.dtype, tuple(x.shape), dev)
    _is(z, "z", x.dtype, tuple(x.shape), dev)
    _is(w, "w", torch.float32, (D,) if w.dim() == 1 else (R, D), dev)
    return dev, x.numel() // D if D else 0, D, R


def gated_norm(x, z, w, eps: float = 1e-5, gate_first: bool = False):
    """Gated root-mean-square norm over the last dimension (``dn_gated_norm``):
    ``x / sqrt(mean(x^2) + eps) * w * silu(z)``, or with ``gate_first`` the norm
    of ``x silu(z)`` times w.  x, z ``[..., D]`` or ``[..., H, D]`` float32 or
    bfloat16; w float32 ``[D]``, or ``[H, D]`` for a weight per head.  Returns y
    in x's dtype."""
    try:
        E, i, xs, ws = x.dtype, x.get_device(), x.shape, w.shape
        R = ws[0] if len(ws) == 2 else 1
        fits = (len(xs) > 1 and 0 < xs[-1] <= _MAX_SIZE and ws == xs[-len(ws):] and 0 < len(ws) < 3 and E in _DTYPES
                and i >= 0 and x.is_contiguous() and _fits(z, E, xs, i) and _fits(w, torch.float32, ws, i))
    except AttributeError:  # not a tensor
        fits = False
    if not fits:
        _gated_norm_args(x, z, w)
    y = torch.empty_like(x)
    _call("dn_gated_norm", i, x.numel() // (xs[-1] or 1), xs[-1], R, _DTYPES[E], x.data_ptr(), z.data_ptr(), w.data_ptr(),
          eps, gate_first, y.data_ptr())
    return y


def gated_norm_bwd(x, z, w, dy, eps: float = 1e-5, gate_first: bool = False):
    """Backward of ``gated_norm`` (``dn_gated_norm_bwd``) from dy in x's dtype:
    ``(dx, dz, dw)``, dx and dz in x's dtype, dw float32."""
    dev, rows, D, R = _gated_norm_args(x, z, w)
    _given(dy=dy)
    _is(dy, "dy", x.dtype, tuple(x.shape), dev)
    dx, dz, dw = torch.empty_like(x), torch.empty_like(z), torch.empty_like(w)
    wsb = load_library().dn_gated_norm_bwd_workspace(rows, D, R)
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev) if wsb else None
    _call("dn_gated_norm_bwd", dev, rows, D, R, _DTYPES[x.dtype], _adr(x), _adr(z), _adr(w), float(eps), int(gate_first),
          _adr(dy), _adr(dx), _adr(dz), _adr(dw), _adr(ws), wsb)
    return dx, dz, dw


def _grad(t):
    """An incoming gradient as the kernels take it: autograd may hand on any
    view, also a contiguous slice that starts between 16-byte units."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class SsmScan(torch.autograd.Function):
    """Autograd wrapper: forward by ``ssm_fwd``, backward by ``ssm_bwd``."""

    @staticmethod
    def forward(ctx, q, k, v, dt, A, dt_bias, skip, h0, cu_seqlens):
        o, hT = ssm_fwd(q, k, v, dt, A, dt_bias, skip, h0, cu_seqlens)
        ctx.save_for_backward(q, k, v, dt, A, dt_bias, skip, h0, cu_seqlens)
        ctx.set_materialize_grads(False)
        return o, hT

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO, dhT):
        q, k, v, dt, A, dt_bias, skip, h0, cu = ctx.saved_tensors
        dO = torch.zeros_like(v) if dO is None else _grad(dO)
        gr = ssm_bwd(q, k, v, dt, A, dt_bias, skip, h0, dO, None if dhT is None else _grad(dhT), cu)
        return (gr["dq"], gr["dk"], gr["dv"], gr["ddt"], gr["dA"], gr["ddt_bias"], gr["dskip"],
                None if h0 is None else gr["dh0"], None)


def ssm_scan(q, k, v, dt, A, dt_bias=None, skip=None, h0=None, cu_seqlens=None):
    """Differentiable selective state space scan; returns (o, hT).  Rows behind the
    last packed sequence give zeros and get zero gradients."""
    return SsmScan.apply(q, k, v, dt, A, dt_bias, skip, h0, cu_seqlens)


class ConvSilu(torch.autograd.Function):
    """Autograd wrapper: forward by ``conv_silu``, backward by ``conv_silu_bwd``."""

    @staticmethod
    def forward(ctx, x, w, bias, s0, cu_seqlens):
        y, sT = conv_silu(x, w, bias, s0, cu_seqlens)
        ctx.save_for_backward(x, w, bias, s0, cu_seqlens)
        ctx.set_materialize_grads(False)
        return y, sT

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dsT):
        x, w, bias, s0, cu = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else _grad(dy)
        gr = conv_silu_bwd(x, w, bias, s0, dy, None if dsT is None else _grad(dsT), cu)
        return gr["dx"], gr["dw"], gr["dbias"], None if s0 is None else gr["ds0"], None


def conv_silu_fn(x, w, bias=None, s0=None, cu_seqlens=None):
    """Differentiable ``conv_silu``; returns (y, sT).  Rows behind the last packed
    sequence give zeros and get zero gradients."""
    return ConvSilu.apply(x, w, bias, s0, cu_seqlens)


class GatedNorm(torch.autograd.Function):
    """Autograd wrapper: forward by ``gated_norm``, backward by ``gated_norm_bwd``."""

    @staticmethod
    def forward(ctx, x, z, w, eps, gate_first):
        ctx.save_for_backward(x, z, w)
        ctx.eps, ctx.gate_first = eps, gate_first
        return gated_norm(x, z, w, eps, gate_first)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, z, w = ctx.saved_tensors
        return (*gated_norm_bwd(x, z, w, _grad(dy), ctx.eps, ctx.gate_first), None, None)


def gated_norm_fn(x, z, w, eps: float = 1e-5, gate_first: bool = False):
    """Differentiable ``gated_norm``."""
    return GatedNorm.apply(x, z, w, eps, gate_first)
