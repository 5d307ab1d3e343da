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
