"""Sizes at which a layer operator's counts would leave 32 bits, without a GPU."""
import pytest

import speculative_verify_gb300 as sv
from speculative_verify_gb300 import build as svbuild
from speculative_verify_gb300.layer import DeltaRows, DeltaShape

SHAPE = -2
A = 0x10000                             # never dereferenced: the call fails its checks, or at the device


def _has_gpu():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


pytestmark = pytest.mark.skipif(_has_gpu(), reason="fake-pointer checks run only where no GPU exists")


@pytest.fixture(scope="module")
def lib():
    svbuild.build()
    return sv.load()


def chunk(lib, R, B, Hv):
    rows = DeltaRows(A, A, A, A, A, 64, 64, Hv * 64, Hv)
    shape = DeltaShape(1, Hv, 64, 64, 0.125, 0)
    return lib.gated_delta_chunk(rows, R, A, B, shape, A, A, 1, A, Hv * 64, A, 1 << 62, None)


def test_chunk_counts_fit_32_bits(lib):
    """Blocks and the places of every sequence's start and end, times the value heads: beyond 2^31 - 1 refused."""
    for R, B in ((1000, 65535), (1 << 27, 1), (1 << 20, 30000), (65, 65535)):
        most = (2 ** 31 - 1) // (R // 64 + B + 2 * B)
        assert chunk(lib, R, B, min(most, 65535)) not in (0, SHAPE)     # (only the device is missing)
        if most < 65535:
            assert chunk(lib, R, B, most + 1) == SHAPE
