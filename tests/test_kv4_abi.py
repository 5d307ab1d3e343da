"""The attention layers' C ABI without a GPU: exported names and bindings,
workspace and page sizes, and every documented refusal before a CUDA call."""
import ctypes

import pytest

import speculative_verify_gb300 as sv
from speculative_verify_gb300 import build as svbuild
from speculative_verify_gb300.layer import Kv4Cache

NAMES = ("rotary_embed", "kv4_page_bytes", "kv4_append", "kv4_gather", "kv4_attention_bytes", "kv4_attention")
OK, NULL, SHAPE, ALIGN = 0, -1, -2, -3
NAN, INF = float("nan"), float("inf")


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
    for name in ("rotary", "kv4_cache", "kv4_append", "kv4_gather", "kv4_attention"):
        assert callable(getattr(sv, name))
        assert getattr(sv, name).__doc__


def test_page_bytes(lib):
    for d in (64, 128, 256):
        assert lib.kv4_page_bytes(3, d) == 3 * (2 * 32 * d // 2 + 2 * 32 * d // 16)
    for Hk, d in ((0, 64), (1, 96), (1, 0), (65536, 64), (-1, 128)):
        assert lib.kv4_page_bytes(Hk, d) == 0


@nogpu
@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(q_out=None), NULL), (dict(k_out=None), NULL),
    (dict(positions=None), NULL), (dict(inv_freq=None), NULL),
    (dict(rows=-1), SHAPE), (dict(Hq=-1), SHAPE), (dict(Hk=-1), SHAPE), (dict(Hq=0, Hk=0), SHAPE), (dict(Hq=65536), SHAPE),
    (dict(d=8), SHAPE), (dict(d=68), SHAPE), (dict(d=1032, ldq=8256, ldk=8256, ldqo=8256, ldko=8256), SHAPE),
    (dict(rot=0), SHAPE), (dict(rot=24), SHAPE), (dict(rot=80), SHAPE), (dict(n_axes=0), SHAPE), (dict(n_axes=17), SHAPE),
    (dict(n_axes=2, ldp=9), SHAPE), (dict(flags=2), SHAPE), (dict(factor=NAN), SHAPE), (dict(factor=INF), SHAPE),
    (dict(ldq=504), SHAPE), (dict(ldk=120), SHAPE), (dict(ldqo=504), SHAPE), (dict(ldko=120), SHAPE),
    (dict(ldq=513), ALIGN), (dict(ldk=132), ALIGN), (dict(ldqo=516), ALIGN), (dict(ldko=129), ALIGN),
    (dict(q=M8), ALIGN), (dict(k=M8), ALIGN), (dict(q_out=M8), ALIGN), (dict(k_out=M8), ALIGN),
    (dict(positions=M2), ALIGN), (dict(axes=M2), ALIGN), (dict(inv_freq=M1), ALIGN),
    (dict(rows=0, q=None, k=None, positions=None), OK),
])
def test_rotary_refusals(lib, kw, code):
    a = dict(q=A, ldq=512, Hq=8, k=A, ldk=128, Hk=2, rows=10, d=64, rot=64, positions=A, ldp=10, n_axes=1, axes=None,
             inv_freq=A, factor=1.0, flags=0, q_out=A, ldqo=512, k_out=A, ldko=128)
    a.update(kw)
    assert lib.rotary_embed(*a.values(), None) == code


@nogpu
def test_sizes_past_the_index_range_are_refused(lib):
    """Rows whose count rounds up past 31 bits, query heads beyond any memory, a scale that leaves fp32 with k_scale."""
    assert lib.rotary_embed(A, 16, 1, None, 0, 0, (1 << 30) + 1, 16, 16, A, (1 << 30) + 1, 1, None, A, 1.0, 0, A, 16, None, 0,
                            None) == SHAPE

    def attention(R, Hq, scale=1.0, **kw):
        c = cache_of(kw)
        assert (lib.kv4_attention_bytes(R, 4, 0, Hq, ctypes.byref(c)) == 0) == (scale == 1.0)
        return lib.kv4_attention(A, Hq * 64, R, Hq, None, A, 4, ctypes.byref(c), scale, 0, 0, A, Hq * 64, A, 1 << 60, None)

    assert attention(1 << 29, 64, Hk=64) == SHAPE
    assert attention(8, 8, scale=1e38, k_scale=1e3) == SHAPE
    assert attention(8, 8, scale=-3.4e38) == SHAPE


def cache_of(kw):
    c = dict(pages=A, page_table=A, ldt=8, n_pages=20, max_pages=8, Hk=2, d=64, k_scale=1.0, v_scale=1.0)
    c.update({n: kw.pop(n) for n in list(kw) if n in c})
    return Kv4Cache(**c)


CACHE = [
    (dict(pages=None), NULL), (dict(page_table=None), NULL), (dict(lens=None), NULL),
    (dict(d=96), SHAPE), (dict(d=0), SHAPE), (dict(Hk=0), SHAPE), (dict(Hk=65536), SHAPE), (dict(n_pages=-1), SHAPE),
    (dict(max_pages=-1), SHAPE), (dict(max_pages=(1 << 24) + 1, ldt=1 << 25), SHAPE), (dict(ldt=7), SHAPE),
    (dict(k_scale=0.0), SHAPE), (dict(k_scale=-1.0), SHAPE), (dict(v_scale=NAN), SHAPE), (dict(v_scale=INF), SHAPE),
    (dict(v_scale=1e-31), SHAPE),
    (dict(R=-1), SHAPE), (dict(B=-1), SHAPE), (dict(R=7), SHAPE), (dict(R=(1 << 29) + 4), SHAPE), (dict(B=0), SHAPE),
    (dict(pages=M8), ALIGN), (dict(page_table=M2), ALIGN), (dict(lens=M2), ALIGN), (dict(cu=M1), ALIGN),
    (dict(R=0), OK), (dict(R=0, B=0), OK), (dict(B=0, cu=A), OK),
]


@nogpu
@pytest.mark.parametrize("fn", ["kv4_append", "kv4_gather"])
@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(ldk=120), SHAPE), (dict(ldv=120), SHAPE),
    (dict(ldk=132), ALIGN), (dict(ldv=130), ALIGN), (dict(k=M8), ALIGN), (dict(v=M8), ALIGN),
])
def test_row_refusals(lib, fn, kw, code):
    kw = dict(kw)
    c = cache_of(kw)
    a = dict(k=A, ldk=128, v=A, ldv=128, R=8, cu=None, lens=A, B=4)
    a.update(kw)
    assert getattr(lib, fn)(*a.values(), ctypes.byref(c), None) == code


@nogpu
@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(q=None), NULL), (dict(o=None), NULL), (dict(ws=None), NULL), (dict(Hq=0), SHAPE), (dict(Hq=7), SHAPE),
    (dict(ldq=504), SHAPE), (dict(ldo=504), SHAPE), (dict(scale=NAN), SHAPE), (dict(scale=INF), SHAPE),
    (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(window=(1 << 30) + 1), SHAPE), (dict(sinks=(1 << 30) + 1), SHAPE),
    (dict(ws_bytes=64), SHAPE), (dict(R=1 << 29, Hq=8, B=1), SHAPE),
    (dict(ldq=516), ALIGN), (dict(ldo=513), ALIGN), (dict(q=M8), ALIGN), (dict(o=M8), ALIGN), (dict(ws=M8), ALIGN),
])
def test_attention_refusals(lib, kw, code):
    kw = dict(kw)
    c = cache_of(kw)
    a = dict(q=A, ldq=512, R=8, Hq=8, cu=None, lens=A, B=4)
    b = dict(scale=0.125, window=0, sinks=0, o=A, ldo=512, ws=A, ws_bytes=1 << 40)
    for n in kw:
        (a if n in a else b)[n] = kw[n]
    assert lib.kv4_attention(*a.values(), ctypes.byref(c), *b.values(), None) == code


def test_no_cache(lib):
    assert lib.kv4_append(A, 128, A, 128, 8, None, A, 4, None, None) == NULL
    assert lib.kv4_attention(A, 512, 8, 8, None, A, 4, None, 1.0, 0, 0, A, 512, A, 1 << 40, None) == NULL
    assert lib.kv4_attention_bytes(8, 4, 0, 8, None) == 0


def test_workspace_bytes(lib):
    """0 for invalid sizes; never more than two tiles of sums a block and a little, however long the cache."""
    def need(R, B, ragged, Hq, **kw):
        return lib.kv4_attention_bytes(R, B, ragged, Hq, ctypes.byref(cache_of(kw)))

    assert need(8, 4, 0, 7) == 0 and need(8, 4, 0, 8, d=96) == 0 and need(-1, 4, 0, 8) == 0 and need(8, 4, 0, 0) == 0
    for d in (64, 128, 256):
        for R, B, Hq, pages in ((1, 1, 8, 8), (8, 4, 48, 1 << 24), (1 << 20, 4, 8, 1 << 12), (1 << 29, 1 << 20, 2, 1 << 24)):
            for ragged in (0, 1):
                n = need(R, B, ragged, Hq, d=d, max_pages=pages, ldt=pages)
                assert 16 <= n <= 512 << 20
