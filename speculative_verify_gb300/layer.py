"""What a hybrid decoder layer runs between its weight reads: residual norm,
gated delta rule or attention over a 4-bit cache, and gated feed-forward (the
second half of ``include/specverify.h``).

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


class Kv4Cache(ctypes.Structure):
    """sv_kv4_cache of include/specverify.h."""
    _fields_ = [("pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("ldt", ctypes.c_longlong),
                ("n_pages", ctypes.c_int), ("max_pages", ctypes.c_int), ("Hk", ctypes.c_int), ("d", ctypes.c_int),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


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
    cache = ctypes.POINTER(Kv4Cache)
    lib.rotary_embed.argtypes = [vp, cl, ci, vp, cl, ci, ci, ci, ci, vp, cl, ci, vp, vp, cf, ci, vp, cl, vp, cl, vp]
    lib.rotary_embed.restype = ci
    lib.kv4_page_bytes.argtypes = [ci, ci]
    lib.kv4_page_bytes.restype = sz
    lib.kv4_append.argtypes = [vp, cl, vp, cl, ci, vp, vp, ci, cache, vp]
    lib.kv4_append.restype = ci
    lib.kv4_gather.argtypes = [vp, cl, vp, cl, ci, vp, vp, ci, cache, vp]
    lib.kv4_gather.restype = ci
    lib.kv4_attention_bytes.argtypes = [ci, ci, ci, ci, cache]
    lib.kv4_attention_bytes.restype = sz
    lib.kv4_attention.argtypes = [vp, cl, ci, ci, vp, vp, ci, cache, cf, ci, ci, vp, cl, vp, sz, vp]
    lib.kv4_attention.restype = ci


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


def rotary(q, k, positions, inv_freq, axes=None, interleaved=False, factor=1.0, q_out=None, k_out=None, stream=None):
    """(q', k'): rotary positions into the first 2 * len(inv_freq) dimensions
    of every head (``rotary_embed`` in include/specverify.h).

    q, k: [T][H][d] or [B][T][H][d] bf16 (k may be None); positions: int32, one
    for each row, or [axes] of them (time, height, width); axes: int32
    [len(inv_freq)], the axis that each pair turns by (None: the first for
    all).  Pairs are (i, i + half), with interleaved=True (2i, 2i + 1).
    q_out=q and k_out=k rotate in place."""
    if _ext is None:
        _load()
    return _ext.rotary(q, k, positions, inv_freq, axes, interleaved, factor, q_out, k_out, stream)


KV4_PAGE = 32                           # tokens of a page


def kv4_cache(n_pages, Hk, d, device="cuda"):
    """Zeroed pages of a 4-bit cache: uint8 [n_pages][Hk][36 d], 32 tokens a
    page (the format is in include/specverify.h); d 64, 128 or 256."""
    import torch
    return torch.zeros(n_pages, Hk, 36 * d, dtype=torch.uint8, device=device)


def kv4_append(k, v, cache, page_table, seq_lens, cu_seqlens=None, k_scale=1.0, v_scale=1.0, stream=None):
    """Rows of keys and values into the 4-bit cache, in place.

    k, v: [B][T][Hk][d] bf16, or [R][Hk][d] with cu_seqlens (int32 [B + 1]);
    page_table: int32 [B][pages]; seq_lens: int32 [B], the tokens before these
    rows (negative: the sequence is left alone).  k_scale, v_scale: what the
    cache's values are multiples of, the same for every call on a cache."""
    if _ext is None:
        _load()
    return _ext.kv4_append(k, v, cache, page_table, seq_lens, cu_seqlens, k_scale, v_scale, stream)


def kv4_gather(cache, page_table, seq_lens, rows, cu_seqlens=None, k_scale=1.0, v_scale=1.0, k=None, v=None, stream=None):
    """(k, v): rows of the cache as bf16, [B][rows][Hk][d] from position
    seq_lens on, or [rows][Hk][d] with cu_seqlens (rows: their number in all;
    rows of no sequence are not written)."""
    if _ext is None:
        _load()
    return _ext.kv4_gather(cache, page_table, seq_lens, rows, cu_seqlens, k_scale, v_scale, k, v, stream)


def kv4_attention_bytes(q, cache, page_table, cu_seqlens=None):
    """Bytes of the workspace of such a kv4_attention call, from its tensors'
    shapes alone.  More rows do not always need more: with their number the cut
    of the work changes."""
    import speculative_verify_gb300 as root
    if q.dim() != (4 if cu_seqlens is None else 3) or cache.dim() != 3 or page_table.dim() != 2:
        raise ValueError("q must be [B][T][heads][d], or [R][heads][d] with cu_seqlens, cache [pages][Hk][36 d], "
                         "page_table [B][pages]")
    if cache.shape[2] != 36 * q.shape[-1] or (cu_seqlens is None and q.shape[0] != page_table.shape[0]):
        raise ValueError("q must have the cache's dimensions and as many sequences as page_table")
    c = Kv4Cache(None, None, page_table.shape[1], cache.shape[0], page_table.shape[1], cache.shape[1], q.shape[-1], 1.0, 1.0)
    n = root.load().kv4_attention_bytes(q.shape[:-2].numel(), page_table.shape[0], cu_seqlens is not None, q.shape[-2],
                                        ctypes.byref(c))
    if n == 0:
        raise ValueError("kv4_attention does not take these sizes")
    return n


def kv4_attention(q, cache, page_table, seq_lens, cu_seqlens=None, scale=None, window=0, sinks=0, k_scale=1.0,
                  v_scale=1.0, o=None, workspace=None, stream=None):
    """Causal attention of query rows over the 4-bit cache, which holds the
    rows' own tokens already (``kv4_attention`` in include/specverify.h);
    returns o, of q's shape.

    q: [B][T][Hq][d] bf16 (decode and verify rows), or [R][Hq][d] with
    cu_seqlens (prompts of uneven lengths); row t of sequence b sees the tokens
    up to seq_lens[b] + t, with a window only the last `window` of them and the
    first `sinks` of the sequence.  A sequence of negative length gives zeros.
    scale defaults to d ** -0.5.  workspace: a uint8 CUDA tensor of at least
    kv4_attention_bytes(q, cache, page_table, cu_seqlens), that no call which may
    overlap this one has, else one is allocated.  A call takes one kernel, by the
    query rows of a sequence on average: single rows are better not mixed with
    prompts of hundreds of rows in one."""
    if _ext is None:
        _load()
    return _ext.kv4_attention(q, cache, page_table, seq_lens, cu_seqlens, scale, window, sinks, k_scale, v_scale, o,
                              workspace, stream)
