"""What a hybrid decoder layer runs between its weight reads: residual norm,
gated delta rule and gated feed-forward (the second half of
``include/specverify.h``).

Argument marshalling only, as in the package's root: tensors are torch CUDA
tensors, each call is enqueued on ``stream`` (default: the current stream)
and returns at once, and outputs are allocated unless given.  A tensor may be
a strided view where its rows are equally far apart and dense inside.
"""
from __future__ import annotations

import ctypes

NORM_UNIT_OFFSET = 0x1
DELTA_L2NORM, DELTA_COMMIT, DELTA_ZERO_INIT = 0x1, 0x2, 0x4
ACTS = {"silu": 0, "gelu": 1}
FP8_GROUP = 128

torch = _lib = _bf16 = _f32 = _raw_stream = None        # set by the first call


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


def _init():
    """Load torch and the library on the first call; the calls below are short, so nothing is looked up twice."""
    global torch, _lib, _bf16, _f32, _raw_stream
    import torch as _torch

    import speculative_verify_gb300 as root
    torch, _lib = _torch, root.load()
    _bf16, _f32, _raw_stream = torch.bfloat16, torch.float32, torch._C._cuda_getCurrentRawStream


def _fail(fn, rc):
    import speculative_verify_gb300 as root
    raise root.SpecVerifyError(fn, rc)


def _raw(stream, t):
    """The stream's handle, or that of the current stream of t's device."""
    return _raw_stream(t.get_device()) if stream is None else stream.cuda_stream


def _rows2d(t, name, dtype, shape):
    """The row distance of a [T][D] CUDA tensor of that type with dense rows."""
    if t.dtype is not dtype or not t.is_cuda:
        raise TypeError("%s must be a 2-D %s CUDA tensor" % (name, dtype))
    if t.shape != shape:
        raise ValueError("%s must be [%d][%d]" % ((name,) + tuple(shape)))
    if t.is_contiguous():
        return shape[1]
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError("%s must have dense rows" % name)
    return ld if shape[0] > 1 else shape[1]


def _norm_args(x, weight, residual, residual_out):
    if _lib is None:
        _init()
    shape = x.shape
    if len(shape) != 2:
        raise TypeError("x must be a 2-D %s CUDA tensor" % _bf16)
    ldx = _rows2d(x, "x", _bf16, shape)
    if weight.dtype is not _bf16 or not weight.is_cuda or weight.shape != shape[1:] or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous bf16 CUDA tensor of %d entries" % shape[1])
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without a residual")
        return shape, ldx, None, 0, None, None, 0
    ldr = _rows2d(residual, "residual", _bf16, shape)
    if residual_out is None:
        residual_out = torch.empty(shape, dtype=_bf16, device=x.device)
        ldro = shape[1]
    else:
        ldro = _rows2d(residual_out, "residual_out", _bf16, shape)
    return shape, ldx, residual.data_ptr(), ldr, residual_out, residual_out.data_ptr(), ldro


def rmsnorm(x, weight, residual=None, eps=1e-6, unit_offset=False, y=None, residual_out=None, stream=None):
    """(y, s): s = bf16(x + residual) (None without a residual), y = the
    root-mean-square norm of s times weight (or 1 + weight), bf16; see
    ``rmsnorm_residual`` in include/specverify.h.  residual_out=residual
    updates the residual stream in place."""
    shape, ldx, rp, ldr, residual_out, rop, ldro = _norm_args(x, weight, residual, residual_out)
    T, D = shape
    if y is None:
        y = torch.empty(shape, dtype=_bf16, device=x.device)
        ldy = D
    else:
        ldy = _rows2d(y, "y", _bf16, shape)
    if T:
        rc = _lib.rmsnorm_residual(x.data_ptr(), ldx, rp, ldr, weight.data_ptr(), T, D, eps,
                                   NORM_UNIT_OFFSET if unit_offset else 0, rop, ldro, y.data_ptr(), ldy,
                                   _raw_stream(x.get_device()) if stream is None else stream.cuda_stream)
        if rc:
            _fail("rmsnorm_residual", rc)
    return y, residual_out


def rmsnorm_fp8(x, weight, residual=None, eps=1e-6, unit_offset=False, group=FP8_GROUP, y=None, scales=None,
                residual_out=None, stream=None):
    """(y8, scales, s): as :func:`rmsnorm` with y as float8_e4m3fn and fp32
    scales [T][ceil(D / 128)] (group=128) or [T][1] (group=0)."""
    shape, ldx, rp, ldr, residual_out, rop, ldro = _norm_args(x, weight, residual, residual_out)
    T, D = shape
    if group != FP8_GROUP and group != 0:
        raise ValueError("group must be 0 or %d" % FP8_GROUP)
    n = -(-D // group) if group else 1
    if y is None:
        y = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
        ldy = D
    else:
        ldy = _rows2d(y, "y", torch.float8_e4m3fn, shape)
    if scales is None:
        scales = torch.empty((T, n), dtype=_f32, device=x.device)
        lds = n
    else:
        lds = _rows2d(scales, "scales", _f32, (T, n))
    if T:
        rc = _lib.rmsnorm_residual_fp8(x.data_ptr(), ldx, rp, ldr, weight.data_ptr(), T, D, eps,
                                       NORM_UNIT_OFFSET if unit_offset else 0, group, rop, ldro, y.data_ptr(), ldy,
                                       scales.data_ptr(), lds, _raw(stream, x))
        if rc:
            _fail("rmsnorm_residual_fp8", rc)
    return y, scales, residual_out


def _row_stride(shape, stride, lead, name):
    """The distance between rows: the first `lead` dimensions number rows one
    after another, the others must be dense."""
    want = 1
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] > 1 and stride[d] != want:
            raise ValueError("the rows of %s must be dense" % name)
        want *= shape[d]
    ld, span = None, 1                  # span: rows that one step of dimension d passes over
    for d in range(lead - 1, -1, -1):
        if shape[d] > 1:
            if ld is None:
                ld, rest = divmod(stride[d], span)
                if rest:
                    raise ValueError("the rows of %s must be equally far apart" % name)
            elif stride[d] != ld * span:
                raise ValueError("the rows of %s must be equally far apart" % name)
        elif not shape[d]:
            return want                 # no rows
        span *= shape[d]
    return want if ld is None else ld


def _ld(t, shape, dtype, lead, name):
    """The row distance of t, a CUDA tensor of that shape and type."""
    if t.dtype is not dtype or not t.is_cuda:
        raise TypeError("%s must be a %d-D %s CUDA tensor" % (name, len(shape), dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s" % (name, "".join("[%d]" % n for n in shape)))
    stride = t.stride()
    if stride[-1] == 1:                 # the usual layouts at once
        if lead == 1:
            if shape[0] > 1 and (len(shape) == 2 or stride[1] == shape[2]):
                return stride[0]
        elif shape[1] > 1 and stride[0] == shape[1] * stride[1] and (len(shape) == 3 or stride[2] == shape[3]):
            return stride[1]
    return _row_stride(shape, stride, lead, name)


def _delta_rows(q, k, v, g, beta, rows, Hk, Hv, dk, dv):
    """sv_delta_rows of tensors whose first dimensions are `rows`; q may be None."""
    lead = len(rows)
    kshape, gshape = rows + (Hk, dk), rows + (Hv,)
    ldg = _ld(g, gshape, _f32, lead, "g")
    if _ld(beta, gshape, _f32, lead, "beta") != ldg:
        raise ValueError("g and beta must have the same row distance")
    ldk = _ld(k, kshape, _bf16, lead, "k")
    ldv = _ld(v, gshape + (dv,), _bf16, lead, "v")
    if q is None:
        return DeltaRows(None, k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), 0, ldk, ldv, ldg)
    return DeltaRows(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                     _ld(q, kshape, _bf16, lead, "q"), ldk, ldv, ldg)


def _i32(t, name, n=None):
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError("%s must be a contiguous int32 CUDA tensor" % name)
    if n is not None and t.numel() != n:
        raise ValueError("%s must have one entry per sequence" % name)
    return t.data_ptr()


def _delta_state(state, k):
    """(n_slots, Hv, dv) of a state pool [slots][Hv][dv][dk], after checking it."""
    shape = state.shape
    if state.dtype is not _f32 or not state.is_cuda or len(shape) != 4 or not state.is_contiguous():
        raise TypeError("state must be a contiguous float32 CUDA tensor [slots][Hv][dv][dk]")
    n_slots, Hv, dv, dk = shape
    if dk != k.shape[-1]:
        raise ValueError("state must be [slots][Hv][dv][dk]")
    return n_slots, Hv, dv


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
    if _lib is None:
        _init()
    if k.dim() != 4:
        raise TypeError("k must be [B][T][Hk][dk]")
    B, T, Hk, dk = k.shape
    n_slots, Hv, dv = _delta_state(state, k)
    rows = _delta_rows(q, k, v, g, beta, (B, T), Hk, Hv, dk, dv)
    P, prows = 0, None
    if prev is not None:
        pk, pv, pg, pbeta = prev
        if pk.dim() != 4:
            raise ValueError("prev must be rows of the same sequences")
        P = pk.shape[1]
        prows = _delta_rows(None, pk, pv, pg, pbeta, (B, P), Hk, Hv, dk, dv)
    ap = None
    if accept_len is not None:
        if prev is None:
            raise ValueError("accept_len needs prev")
        ap = _i32(accept_len, "accept_len", B)
    if o is None:
        o = torch.empty((B, T, Hv, dv), dtype=_bf16, device=k.device)
        ldo = Hv * dv
    else:
        ldo = _ld(o, (B, T, Hv, dv), _bf16, 2, "o")
    if B:
        rc = _lib.gated_delta_step(
            rows, T, prows, P, ap, B,
            DeltaShape(Hk, Hv, dk, dv, dk ** -0.5 if scale is None else scale,
                       (DELTA_L2NORM if l2norm else 0) | (DELTA_COMMIT if commit else 0)),
            state.data_ptr(), None if state_idx is None else _i32(state_idx, "state_idx", B), n_slots, o.data_ptr(),
            ldo, _raw(stream, k))
        if rc:
            _fail("gated_delta_step", rc)
    return o


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
    if _lib is None:
        _init()
    if k.dim() != 3:
        raise TypeError("k must be [R][Hk][dk]")
    R, Hk, dk = k.shape
    cu = _i32(cu_seqlens, "cu_seqlens")
    B = cu_seqlens.numel() - 1
    if B < 0:
        raise ValueError("cu_seqlens must have B + 1 entries")
    n_slots, Hv, dv = _delta_state(state, k)
    rows = _delta_rows(q, k, v, g, beta, (R,), Hk, Hv, dk, dv)
    shape = DeltaShape(Hk, Hv, dk, dv, dk ** -0.5 if scale is None else scale,
                       (DELTA_L2NORM if l2norm else 0) | (DELTA_ZERO_INIT if zero_init else 0))
    if o is None:
        o = torch.empty((R, Hv, dv), dtype=_bf16, device=k.device)
        ldo = Hv * dv
    else:
        ldo = _ld(o, (R, Hv, dv), _bf16, 1, "o")
    if not B:
        return o
    if workspace is None:
        need = max(_lib.gated_delta_chunk_bytes(R, B, shape), 16)
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=k.device)
        else:                       # its memory may be reused only after the work on `stream`
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=k.device)
    elif workspace.dtype is not torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 CUDA tensor")
    rc = _lib.gated_delta_chunk(rows, R, cu, B, shape, state.data_ptr(),
                                None if state_idx is None else _i32(state_idx, "state_idx", B), n_slots, o.data_ptr(),
                                ldo, workspace.data_ptr() or None, workspace.numel(), _raw(stream, k))
    if rc:
        _fail("gated_delta_chunk", rc)
    return o


def w4a16_gate_up(x, Wq, scales, act="silu", h=None, stream=None):
    """h[T][F] (bf16) = act(x Wg^T) * (x Wu^T) from the fused int4 gate+up
    matrix: Wq [2F][K/8], scales [2F][K/128], the F gate rows first; act:
    "silu" or "gelu" (tanh form).  See ``w4a16_gate_up`` in
    include/specverify.h."""
    if _lib is None:
        _init()
    T, K = x.shape
    N, words = Wq.shape
    for t, name in ((x, "x"), (scales, "scales")):
        if t.dtype is not _bf16 and t.dtype not in (torch.int16, torch.uint16):
            raise TypeError("%s must hold bf16 values (bfloat16, or int16/uint16 raw bits)" % name)
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a contiguous CUDA tensor" % name)
    if Wq.dtype is not torch.int32 and Wq.dtype is not torch.uint32:
        raise TypeError("Wq must be int32/uint32 packed nibble words")
    if not Wq.is_cuda or not Wq.is_contiguous():
        raise ValueError("Wq must be a contiguous CUDA tensor")
    if act not in ACTS:
        raise ValueError("act must be one of %s" % sorted(ACTS))
    if N % 2 or words * 8 != K or scales.shape != (N, K // 128):
        raise ValueError("shape mismatch: x %s, Wq %s, scales %s" % (tuple(x.shape), tuple(Wq.shape),
                                                                      tuple(scales.shape)))
    if h is None:
        h = torch.empty((T, N // 2), dtype=_bf16, device=x.device)
    elif h.dtype is not _bf16 or not h.is_cuda or not h.is_contiguous() or h.shape != (T, N // 2):
        raise ValueError("h must be a contiguous bf16 CUDA tensor [T][F]")
    rc = _lib.w4a16_gate_up(x.data_ptr(), Wq.data_ptr(), scales.data_ptr(), T, K, N // 2, ACTS[act], h.data_ptr(),
                            _raw(stream, x))
    if rc:
        _fail("w4a16_gate_up", rc)
    return h
