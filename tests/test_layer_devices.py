"""The device of a layer operator's call, without a GPU: tensors that have a
device but no memory, and where the current device matters a fake CUDA runtime
that says which one was made current."""
import os
import shutil
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="tensors without memory are used only where no GPU exists")

RUNTIME = """
#include <stdio.h>
static int current = 0;
int cudaGetDeviceCount(int *n) { *n = 2; return 0; }
int cudaGetDevice(int *d) { *d = current; return 0; }
int cudaSetDevice(int d) { current = d; printf("current %d\\n", d); fflush(stdout); return 0; }
int cudaDeviceGetStreamPriorityRange(int *least, int *greatest) { *least = 0; *greatest = -5; return 0; }
"""

CALLS = """
import sys
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
torch.cuda.is_available = lambda: False
import speculative_verify_gb300 as sv
with FakeTensorMode():
    e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda:1")
    f = torch.float32
    x, w, W, sc = e(4, 256), e(256), e(64, 32, t=torch.int32), e(64, 2)
    step = (e(2, 3, 1, 64), e(2, 3, 1, 64), e(2, 3, 2, 64), e(2, 3, 2, t=f), e(2, 3, 2, t=f))
    rows = (e(6, 1, 64), e(6, 1, 64), e(6, 2, 64), e(6, 2, t=f), e(6, 2, t=f))
    state, cu = e(2, 2, 64, 64, t=f), e(3, t=torch.int32)
    y, y8, ys, h = e(4, 256), e(4, 256, t=torch.float8_e4m3fn), e(4, 2, t=f), e(4, 32)
    o, oc, ws = e(2, 3, 2, 64), e(6, 2, 64), e(1 << 20, t=torch.uint8)
for call in (lambda: sv.rmsnorm(x, w, y=y), lambda: sv.rmsnorm_fp8(x, w, y=y8, scales=ys),
             lambda: sv.gated_delta_step(*step, state, o=o),
             lambda: sv.gated_delta_chunk(*rows, cu, state, o=oc, workspace=ws), lambda: sv.w4a16_gate_up(x, W, sc, h=h)):
    print("call", flush=True)
    try:
        call()
    except sv.SpecVerifyError:          # (no memory behind the tensors)
        pass
"""


@pytest.fixture(scope="module")
def sv():
    import speculative_verify_gb300 as m
    from speculative_verify_gb300 import build
    build.build()
    return m


def test_call_runs_on_its_tensors_device(sv, tmp_path):
    """With device 0 current, a call on tensors of device 1 makes that one current, and then device 0 again."""
    if not shutil.which("gcc"):
        pytest.skip("no C compiler")
    (tmp_path / "runtime.c").write_text(RUNTIME)
    fake = tmp_path / "runtime.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(fake), str(tmp_path / "runtime.c")], check=True)
    env = dict(os.environ, LD_PRELOAD=str(fake), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CALLS], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["call", "current", "1", "current", "0"] * 5
