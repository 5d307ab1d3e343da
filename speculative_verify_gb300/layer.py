"""What a hybrid decoder layer runs between its weight reads: residual norm,
gated delta rule and gated feed-forward (the second half of
``include/specverify.h``).

Signatures and documentation; the argument checks, the outputs' allocation and
the calls are in ``csrc/layer_bind.cpp`` (native, as each call is only a few
microseconds of GPU time).  Tensors are torch CUDA tensors, all on one device,
each call is enqueued on ``stream`` (default: that device's current stream)
and returns at once, and outputs are allocated unless given.  A tensor may be a strided view where its
rows are equally far apart and dense inside.  Wrong types raise TypeError,
wrong shapes, strides or devices ValueError, and a refusal of the library
SpecVerifyError.  There are no gradients: a tensor that requires one raises
RuntimeError unless gradients are off (``torch.no_grad()``).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

from . import build as _build

ACTS = {"silu": 0, "gelu": 1}

_ext = None                             # the binding, loaded by the first call


def _load():
    """Load torch, the library and the binding on the first call."""
    global _ext
    import torch  # noqa: F401  (the binding uses its libraries)

    import speculative_verify_gb300 as root
    root.load()
    if not os.path.exists(_build.BIND_PATH):
        raise RuntimeError("%s is not built; run speculative_verify_gb300.build.build() or __graft_entry__.build()"
                           % _build.BIND_PATH)
    spec = importlib.util.spec_from_file_location("speculative_verify_gb300._layer", _build.BIND_PATH)
    ext = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ext)
    ext.set_error(root.SpecVerifyError)
    _ext = ext


class DeltaRows(ctypes.Structure):
    """sv_delta_rows of include/specverify.h."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("g", ctypes.c_void_p),
                ("beta", ctypes.c_void_p), ("ldq", ctypes.c_longlong), ("ldk", ctypes.c_longlong),
                ("ldv", ctypes.c_longlong), ("ldg", ctypes.c_longlong)]


class DeltaShape(ctypes.Structure):
    """sv_delta_shape of include/specverify.h."""
    _fields_ = [("Hk", ctypes.c_int), ("Hv", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
                ("scale", ctypes.c_float), ("flags", ctypes.c_int)]


def declare(lib) -> None:
    """The C signatures of this module's calls."""
    vp, ci, cl, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
    rows, shape = ctypes.POINTER(DeltaRows), ctypes.POINTER(DeltaShape)
    lib.rmsnorm_residual.argtypes = [vp, cl, vp, cl, vp, ci, ci, cf, ci, vp, cl, vp, cl, vp]
    lib.rmsnorm_residual.restype = ci
    lib.rmsnorm_residual_fp8.argtypes = [vp, cl, vp, cl, vp, ci, ci, cf, ci, ci, vp, cl, vp, cl, vp, cl, vp]
    lib.rmsnorm_residual_fp8.restype = ci
    lib.gated_delta_step.argtypes = [rows, ci, rows, ci, vp, ci, shape, vp, vp, ci, vp, cl, vp]
    lib.gated_delta_step.restype = ci
    lib.gated_delta_chunk_bytes.argtypes = [ci, ci, shape]
    lib.gated_delta_chunk_bytes.restype = sz
    lib.gated_delta_chunk.argtypes = [rows, ci, vp, ci, shape, vp, vp, ci, vp, cl, vp, sz, vp]
    lib.gated_delta_chunk.restype = ci
    lib.w4a16_gate_up.argtypes = [vp, vp, vp, ci, ci, ci, ci, vp, vp]
    lib.w4a16_gate_up.restype = ci


def rmsnorm(x, weight, residual=None, eps=1e-6, unit_offset=False, y=None, residual_out=None, stream=None):
    """(y, s): s = bf16(x + residual) (None without a residual), y = the
    root-mean-square norm of s times weight (or 1 + weight), bf16; see
    ``rmsnorm_residual`` in include/specverify.h.  residual_out=residual
    updates the residual stream in place."""
    if _ext is None:
        _load()
    return _ext.rmsnorm(x, weight, residual, eps, unit_offset, y, residual_out, stream)


def rmsnorm_fp8(x, weight, residual=None, eps=1e-6, unit_offset=False, group=128, y=None, scales=None,
                residual_out=None, stream=None):
    """(y8, scales, s): as :func:`rmsnorm` with y as float8_e4m3fn and fp32
    scales [T][ceil(D / 128)] (group=128) or [T][1] (group=0)."""
    if _ext is None:
        _load()
    return _ext.rmsnorm_fp8(x, weight, residual, eps, unit_offset, group, y, scales, residual_out, stream)


def gated_delta_step(q, k, v, g, beta, state, state_idx=None, prev=None, accept_len=None, commit=True, scale=None,
                     l2norm=False, o=None, stream=None):
    """Gated delta rule over decode or verify rows (``gated_delta_step`` in
    include/specverify.h); returns o [B][T][Hv][dv] bf16 and updates ``state``
    [slots][Hv][dv][dk] fp32 in place.

    q, k: [B][T][Hk][dk], v: [B][T][Hv][dv] bf16, g (log decay) and beta:
    [B][T][Hv] fp32.  commit=True keeps the rows (plain decode);
    commit=False leaves the state before them (drafts under verification).
    prev: (k, v, g, beta) of the last call's provisional rows, of which the
    first accept_len[b] + 1 (int32, from lmhead_verify; None: all) are
    replayed into the state first.  scale defaults to dk ** -0.5."""
    if _ext is None:
        _load()
    return _ext.gated_delta_step(q, k, v, g, beta, state, state_idx, prev, accept_len, commit, scale, l2norm, o,
                                 stream)


def gated_delta_chunk(q, k, v, g, beta, cu_seqlens, state, state_idx=None, zero_init=False, scale=None, l2norm=False,
                      o=None, workspace=None, stream=None):
    """Gated delta rule over whole prompts (``gated_delta_chunk`` in
    include/specverify.h); returns o [R][Hv][dv] bf16 and updates ``state``
    [slots][Hv][dv][dk] fp32 in place.

    q, k: [R][Hk][dk], v: [R][Hv][dv] bf16, g and beta: [R][Hv] fp32, the
    rows of all sequences one after another; cu_seqlens: int32 [B + 1] on the
    device.  zero_init starts every sequence from a zero state instead of its
    slot's.  workspace: a uint8 CUDA tensor of gated_delta_chunk_bytes, else
    one is allocated."""
    if _ext is None:
        _load()
    return _ext.gated_delta_chunk(q, k, v, g, beta, cu_seqlens, state, state_idx, zero_init, scale, l2norm, o,
                                  workspace, stream)


def w4a16_gate_up(x, Wq, scales, act="silu", h=None, stream=None):
    """h[T][F] (bf16) = act(x Wg^T) * (x Wu^T) from the fused int4 gate+up
    matrix: Wq [2F][K/8], scales [2F][K/128], the F gate rows first; act:
    "silu" or "gelu" (tanh form); 1 to 32 rows, all tensors contiguous.  Wq
    and scales must not be written by a kernel still in flight.  See
    ``w4a16_gate_up`` in include/specverify.h."""
    if _ext is None:
        _load()
    if act not in ACTS:
        raise ValueError("act must be one of %s" % sorted(ACTS))
    return _ext.w4a16_gate_up(x, Wq, scales, ACTS[act], h, stream)
