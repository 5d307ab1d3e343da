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

torch = None                            # set, with the library, by the first call
_lib = None


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
    global torch, _lib
    import torch as _torch

    import speculative_verify_gb300 as root
    torch, _lib = _torch, root.load()


def _fail(fn, rc):
    import speculative_verify_gb300 as root
    raise root.SpecVerifyError(fn, rc)


def _raw(stream, t):
    """The stream's handle, or that of the current stream of t's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else stream.cuda_stream


def _rows2d(t, name, dtype, T, D):
    """The row distance of a [T][D] CUDA tensor of `dtype` with dense rows."""
    if t.dtype is not dtype or not t.is_cuda or t.dim() != 2:
        raise TypeError("%s must be a 2-D %s CUDA tensor" % (name, dtype))
    if tuple(t.shape) != (T, D):
        raise ValueError("%s must be [%d][%d]" % (name, T, D))
    ld, one = t.stride()
    if one != 1 and D > 1 and T:
        raise ValueError("%s must have dense rows" % name)
    return ld if ld > D else D if T < 2 else ld


def _norm_args(x, weight, residual, residual_out):
    if _lib is None:
        _init()
    bf = torch.bfloat16
    if x.dim() != 2:
        raise TypeError("x must be a 2-D %s CUDA tensor" % bf)
    T, D = x.shape
    ldx = _rows2d(x, "x", bf, T, D)
    if weight.dtype is not bf or not weight.is_cuda or weight.dim() != 1 or weight.shape[0] != D or \
            not weight.is_contiguous():
        raise ValueError("weight must be a contiguous bf16 CUDA tensor of %d entries" % D)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without a residual")
        return T, D, ldx, None, 0, None, 0
    ldr = _rows2d(residual, "residual", bf, T, D)
    if residual_out is None:
        residual_out = x.new_empty((T, D))
        ldro = D
    else:
        ldro = _rows2d(residual_out, "residual_out", bf, T, D)
    return T, D, ldx, residual.data_ptr(), ldr, residual_out, ldro


def rmsnorm(x, weight, residual=None, eps=1e-6, unit_offset=False, y=None, residual_out=None, stream=None):
    """(y, s): s = bf16(x + residual) (None without a residual), y = the
    root-mean-square norm of s times weight (or 1 + weight), bf16; see
    ``rmsnorm_residual`` in include/specverify.h.  residual_out=residual
    updates the residual stream in place."""
    T, D, ldx, rp, ldr, residual_out, ldro = _norm_args(x, weight, residual, residual_out)
    if y is None:
        y = x.new_empty((T, D))
        ldy = D
    else:
        ldy = _rows2d(y, "y", torch.bfloat16, T, D)
    if T:
        rc = _lib.rmsnorm_residual(x.data_ptr(), ldx, rp, ldr, weight.data_ptr(), T, D, eps,
                                   NORM_UNIT_OFFSET if unit_offset else 0,
                                   None if rp is None else residual_out.data_ptr(), ldro, y.data_ptr(), ldy,
                                   _raw(stream, x))
        if rc:
            _fail("rmsnorm_residual", rc)
    return y, residual_out


def rmsnorm_fp8(x, weight, residual=None, eps=1e-6, unit_offset=False, group=FP8_GROUP, y=None, scales=None,
                residual_out=None, stream=None):
    """(y8, scales, s): as :func:`rmsnorm` with y as float8_e4m3fn and fp32
    scales [T][ceil(D / 128)] (group=128) or [T][1] (group=0)."""
    T, D, ldx, rp, ldr, residual_out, ldro = _norm_args(x, weight, residual, residual_out)
    if group != FP8_GROUP and group != 0:
        raise ValueError("group must be 0 or %d" % FP8_GROUP)
    n = -(-D // group) if group else 1
    if y is None:
        y = x.new_empty((T, D), dtype=torch.float8_e4m3fn)
        ldy = D
    else:
        ldy = _rows2d(y, "y", torch.float8_e4m3fn, T, D)
    if scales is None:
        scales = x.new_empty((T, n), dtype=torch.float32)
        lds = n
    else:
        lds = _rows2d(scales, "scales", torch.float32, T, n)
    if T:
        rc = _lib.rmsnorm_residual_fp8(x.data_ptr(), ldx, rp, ldr, weight.data_ptr(), T, D, eps,
                                       NORM_UNIT_OFFSET if unit_offset else 0, group,
                                       None if rp is None else residual_out.data_ptr(), ldro, y.data_ptr(), ldy,
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
    if t.dtype is not dtype or not t.is_cuda or t.dim() != len(shape):
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
    lead, bf = len(rows), torch.bfloat16
    kshape, gshape = rows + (Hk, dk), rows + (Hv,)
    ldg = _ld(g, gshape, torch.float32, lead, "g")
    if _ld(beta, gshape, torch.float32, lead, "beta") != ldg:
        raise ValueError("g and beta must have the same row distance")
    return DeltaRows(None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                     0 if q is None else _ld(q, kshape, bf, lead, "q"), _ld(k, kshape, bf, lead, "k"),
                     _ld(v, gshape + (dv,), bf, lead, "v"), ldg)


def _i32(t, name, n=None):
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError("%s must be a contiguous int32 CUDA tensor" % name)
    if n is not None and t.numel() != n:
        raise ValueError("%s must have one entry per sequence" % name)
    return t.data_ptr()


def _delta_state(state, k):
    """(n_slots, Hv, dv) of a state pool [slots][Hv][dv][dk], after checking it."""
    if state.dtype is not torch.float32 or not state.is_cuda or state.dim() != 4 or not state.is_contiguous():
        raise TypeError("state must be a contiguous float32 CUDA tensor [slots][Hv][dv][dk]")
    n_slots, Hv, dv, dk = state.shape
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
        o = k.new_empty((B, T, Hv, dv))
        ldo = Hv * dv
    else:
        ldo = _ld(o, (B, T, Hv, dv), torch.bfloat16, 2, "o")
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
        o = k.new_empty((R, Hv, dv))
        ldo = Hv * dv
    else:
        ldo = _ld(o, (R, Hv, dv), torch.bfloat16, 1, "o")
    if not B:
        return o
    if workspace is None:
        need = max(_lib.gated_delta_chunk_bytes(R, B, shape), 16)
        if stream is None:
            workspace = k.new_empty(need, dtype=torch.uint8)
        else:                       # its memory may be reused only after the work on `stream`
            with torch.cuda.stream(stream):
                workspace = k.new_empty(need, dtype=torch.uint8)
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
    import speculative_verify_gb300 as root
    root._bits16(x, "x"), root._words(Wq, "Wq"), root._bits16(scales, "scales")
    T, K = x.shape
    if act not in ACTS:
        raise ValueError("act must be one of %s" % sorted(ACTS))
    N, words = Wq.shape
    if N % 2 or words * 8 != K or scales.shape != (N, K // 128):
        raise ValueError("shape mismatch: x %s, Wq %s, scales %s" % (tuple(x.shape), tuple(Wq.shape),
                                                                      tuple(scales.shape)))
    if h is None:
        h = x.new_empty((T, N // 2), dtype=torch.bfloat16)
    else:
        root._bits16(h, "h")
        if h.shape != (T, N // 2):
            raise ValueError("h must be [T][F]")
    rc = _lib.w4a16_gate_up(x.data_ptr(), Wq.data_ptr(), scales.data_ptr(), T, K, N // 2, ACTS[act], h.data_ptr(),
                            _raw(stream, x))
    if rc:
        _fail("w4a16_gate_up", rc)
    return h
