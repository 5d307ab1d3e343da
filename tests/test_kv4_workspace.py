"""The size of the attention's workspace, without a GPU."""
import ctypes

import pytest

import speculative_verify_gb300 as sv
from speculative_verify_gb300 import build as svbuild
from test_kv4_abi import cache_of


@pytest.fixture(scope="module")
def lib():
    svbuild.build()
    return sv.load()


def need(lib, R, B, ragged, Hq, **kw):
    return lib.kv4_attention_bytes(R, B, ragged, Hq, ctypes.byref(cache_of(kw)))


@pytest.mark.parametrize("ragged", [0, 1])
def test_no_size_for_what_the_call_refuses(lib, ragged):
    """The limits of a call's rows, sequences and heads are those of its workspace."""
    assert need(lib, 1 << 20, 1 << 20, ragged, 2) > 0
    assert need(lib, 1 << 21, 1 << 21, ragged, 2) == 0 and need(lib, 0, 1 << 21, ragged, 2) == 0
    assert need(lib, 8, 8, ragged, 65535, Hk=65535) > 0 and need(lib, 8, 8, ragged, 65536, Hk=65536) == 0
    assert need(lib, 1 << 29, 8, ragged, 2) > 0 and need(lib, (1 << 29) + 8, 8, ragged, 2) == 0
    assert need(lib, 8, 8, ragged, 2, n_pages=-1) == 0
    assert (need(lib, 9, 8, ragged, 2) > 0) == bool(ragged) and (need(lib, 9, 0, ragged, 2) > 0) == bool(ragged)


def test_size_from_tensors(lib):
    """kv4_attention_bytes of Python: the C call's answer for the tensors' shapes, errors for those that do not fit."""
    torch = pytest.importorskip("torch")

    def e(*s):
        return torch.empty(*s, device="meta")

    for d in (64, 128, 256):
        for B, T, Hq, Hk, pages in ((1, 1, 8, 8, 3), (4, 9, 24, 4, 70), (2, 300, 6, 2, 1000), (3, 0, 4, 2, 5)):
            cache, table = e(20, Hk, 36 * d), e(B, pages)
            kw = dict(Hk=Hk, d=d, max_pages=pages, ldt=pages)
            assert sv.kv4_attention_bytes(e(B, T, Hq, d), cache, table) == need(lib, B * T, B, 0, Hq, **kw)
            assert sv.kv4_attention_bytes(e(B * T + 1, Hq, d), cache, table, e(B + 1)) == need(lib, B * T + 1, B, 1, Hq, **kw)
    q, cache, table = e(2, 3, 4, 64), e(9, 2, 36 * 64), e(2, 5)
    for a in ((q[0], cache, table), (q, cache, table, e(3)), (q, cache[0], table), (q, cache, table[0]), (q, cache, e(3, 5)),
              (e(2, 3, 4, 128), cache, table), (e(2, 3, 5, 64), cache, table), (e(2, 3, 4, 96), e(9, 2, 36 * 96), table)):
        with pytest.raises(ValueError):
            sv.kv4_attention_bytes(*a)
