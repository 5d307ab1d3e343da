"""The layer operators' C ABI without a GPU: exported names and bindings, the
workspace sizes, and every documented refusal before a CUDA call."""
import ctypes

import pytest

import speculative_verify_gb300 as sv
from speculative_verify_gb300 import build as svbuild
from speculative_verify_gb300.layer import DeltaRows, DeltaShape

NAMES = ("rmsnorm_residual", "rmsnorm_residual_fp8", "gated_delta_step", "gated_delta_chunk_bytes",
         "gated_delta_chunk", "w4a16_gate_up")
NULL, SHAPE, ALIGN = -1, -2, -3
L2NORM, COMMIT, ZERO_INIT = 1, 2, 4
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    svbuild.build()
    return sv.load()


def _has_gpu():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


# Addresses that are never dereferenced: each call has to fail its checks
# before any CUDA call.
nogpu = pytest.mark.skipif(_has_gpu(), reason="fake-pointer checks run only where no GPU exists")
A, M8, M2, M1 = 0x10000, 0x10008, 0x10002, 0x10001


def test_header_and_binding_names(lib):
    assert set(NAMES) <= set(sv.header_symbols())
    for name in NAMES:
        assert hasattr(lib, name), name
    for name in ("rmsnorm", "rmsnorm_fp8", "gated_delta_step", "gated_delta_chunk", "w4a16_gate_up"):
        assert callable(getattr(sv, name))
        assert getattr(sv, name).__doc__


@nogpu
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(weight=None), NULL), (dict(y=None), NULL),
    (dict(residual=A), NULL),                   # a residual without a place for the sum
    (dict(residual_out=A), NULL),               # a place for the sum without a residual
    (dict(T=-1), SHAPE), (dict(D=0), SHAPE), (dict(D=65537, ldx=65537, ldy=65537), SHAPE),
    (dict(ldx=511), SHAPE), (dict(ldy=511), SHAPE),
    (dict(residual=A, residual_out=A, ldr=511), SHAPE), (dict(residual=A, residual_out=A, ldro=511), SHAPE),
    (dict(eps=-1e-6), SHAPE), (dict(eps=NAN), SHAPE), (dict(flags=2), SHAPE),
    (dict(x=M1), ALIGN), (dict(weight=M1), ALIGN), (dict(y=M1), ALIGN),
    (dict(T=0, x=None, y=None), 0),             # no rows: nothing to do
])
def test_rmsnorm_refusals(lib, kw, code):
    a = dict(x=A, ldx=512, residual=None, ldr=512, weight=A, T=4, D=512, eps=1e-6, flags=0, residual_out=None,
             ldro=512, y=A, ldy=512)
    a.update(kw)
    assert lib.rmsnorm_residual(*a.values(), None) == code


@nogpu
@pytest.mark.parametrize("kw,code", [
    (dict(group=64), SHAPE), (dict(group=-1), SHAPE), (dict(lds=3), SHAPE), (dict(group=0, lds=0), SHAPE),
    (dict(scales=None), NULL), (dict(y=None), NULL), (dict(scales=M2), ALIGN), (dict(eps=NAN), SHAPE),
    (dict(T=0, scales=None), 0),
])
def test_rmsnorm_fp8_refusals(lib, kw, code):
    a = dict(x=A, ldx=512, residual=None, ldr=512, weight=A, T=4, D=512, eps=1e-6, flags=0, group=128,
             residual_out=None, ldro=512, y=A, ldy=512, scales=A, lds=4)
    a.update(kw)
    assert lib.rmsnorm_residual_fp8(*a.values(), None) == code


def rows(**kw):
    a = dict(q=A, k=A, v=A, g=A, beta=A, ldq=10240, ldk=10240, ldv=10240, ldg=48)
    a.update(kw)
    return DeltaRows(*a.values())


def shape(**kw):
    a = dict(Hk=16, Hv=48, dk=128, dv=128, scale=0.088, flags=0)
    a.update(kw)
    return DeltaShape(*a.values())


SHAPES = [(dict(Hk=0), SHAPE), (dict(Hv=47), SHAPE), (dict(dk=96), SHAPE), (dict(dv=32), SHAPE),
          (dict(scale=NAN), SHAPE), (dict(flags=8), SHAPE)]
ROWS = [(dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(g=None), NULL),
        (dict(beta=None), NULL), (dict(ldq=2047), SHAPE), (dict(ldk=2040), SHAPE), (dict(ldv=6136), SHAPE),
        (dict(ldg=47), SHAPE), (dict(q=M8), ALIGN), (dict(k=M8), ALIGN), (dict(v=M8), ALIGN), (dict(g=M2), ALIGN),
        (dict(beta=M2), ALIGN), (dict(ldk=10241), ALIGN), (dict(ldv=10244), ALIGN)]


@nogpu
@pytest.mark.parametrize("kw,code", [
    (dict(rows=None), NULL), (dict(shape=None), NULL), (dict(prev=None), NULL), (dict(state=None), NULL),
    (dict(o=None), NULL), (dict(T=-1), SHAPE), (dict(T=33), SHAPE), (dict(prev_T=33), SHAPE), (dict(prev_T=-1), SHAPE),
    (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(n_slots=0), SHAPE),
    (dict(idx=None, n_slots=3), SHAPE),         # fewer slots than sequences and no table
    (dict(ldo=6136), SHAPE), (dict(ldo=6148), ALIGN), (dict(o=M8), ALIGN), (dict(state=M8), ALIGN),
    (dict(idx=M2), ALIGN), (dict(accept=M2), ALIGN), (dict(shape=shape(flags=ZERO_INIT)), SHAPE),
    (dict(B=0), 0), (dict(T=0, prev_T=0, rows=None, prev=None, o=None), 0),
] + [(dict(shape=shape(**k)), c) for k, c in SHAPES] + [(dict(rows=rows(**k)), c) for k, c in ROWS]
    + [(dict(prev=rows(**k)), c) for k, c in ROWS if "q" not in k and "ldq" not in k])
def test_gated_delta_step_refusals(lib, kw, code):
    a = dict(rows=rows(), T=4, prev=rows(q=None, ldq=0), prev_T=4, accept=A, B=4, shape=shape(), state=A, idx=A,
             n_slots=8, o=A, ldo=6144)
    a.update(kw)
    assert lib.gated_delta_step(*a.values(), None) == code


@nogpu
@pytest.mark.parametrize("kw,code", [
    (dict(rows=None), NULL), (dict(shape=None), NULL), (dict(state=None), NULL), (dict(o=None), NULL),
    (dict(cu=None), NULL), (dict(ws=None), NULL), (dict(R=-1), SHAPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE),
    (dict(n_slots=0), SHAPE), (dict(idx=None, n_slots=1), SHAPE), (dict(ldo=6136), SHAPE), (dict(ldo=6148), ALIGN),
    (dict(cu=M2), ALIGN), (dict(ws=M8), ALIGN), (dict(state=M8), ALIGN), (dict(ws_bytes=15), SHAPE),
    (dict(shape=shape(flags=COMMIT)), SHAPE), (dict(B=0), 0),
] + [(dict(shape=shape(**k)), c) for k, c in SHAPES] + [(dict(rows=rows(**k)), c) for k, c in ROWS])
def test_gated_delta_chunk_refusals(lib, kw, code):
    a = dict(rows=rows(), R=1000, cu=A, B=2, shape=shape(flags=L2NORM), state=A, idx=A, n_slots=4, o=A, ldo=6144, ws=A)
    a["ws_bytes"] = 1 << 40
    a.update(kw)
    assert lib.gated_delta_chunk(*a.values(), None) == code


def test_gated_delta_chunk_bytes(lib):
    size = lib.gated_delta_chunk_bytes
    assert size(-1, 1, shape()) == 0 and size(1, -1, shape()) == 0 and size(100, 1, shape(dk=100)) == 0
    assert size(0, 0, shape()) > 0
    # what a call with more rows or sequences needs holds one with fewer
    for R in (1, 63, 64, 65, 4096, 1 << 20):
        assert size(R, 1, shape()) <= size(R + 64, 1, shape())
    big = size(64 << 16, 8, shape())
    assert big >= 48 * 65536 * 64 * 64 * 2      # a 64-row block of each head holds more than one 64 x 64 matrix
    if not _has_gpu():
        assert lib.gated_delta_chunk(rows(), 64 << 16, A, 8, shape(), A, None, 8, A, 6144, A, big - 1, None) == SHAPE


@nogpu
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(Wq=None), NULL), (dict(scales=None), NULL), (dict(h=None), NULL),
    (dict(T=0), SHAPE), (dict(T=33), SHAPE), (dict(K=0), SHAPE), (dict(K=192), SHAPE), (dict(F=0), SHAPE),
    (dict(F=(1 << 30) + 1), SHAPE), (dict(act=2), SHAPE), (dict(act=-1), SHAPE),
    (dict(x=M8), ALIGN), (dict(Wq=M8), ALIGN), (dict(scales=M8), ALIGN), (dict(h=M8), ALIGN),
])
def test_gate_up_refusals(lib, kw, code):
    a = dict(x=A, Wq=A, scales=A, T=4, K=512, F=333, act=0, h=A)
    a.update(kw)
    assert lib.w4a16_gate_up(*a.values(), None) == code
