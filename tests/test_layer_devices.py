"""The device of a layer operator's call, without a GPU: calls on tensors that
have a device but no memory, in a process whose CUDA runtime is a fake with two
devices that says which one was made current (this file, run as a program)."""
import os
import shutil
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUNTIME = r"""
#include <stdio.h>
static int current = 0;
int cudaGetDeviceCount(int *n) { *n = 2; return 0; }
int cudaGetDevice(int *d) { *d = current; return 0; }
int cudaSetDevice(int d) { current = d; printf("current %d\n", d); fflush(stdout); return 0; }
int cudaDeviceGetStreamPriorityRange(int *least, int *greatest) { *least = 0; *greatest = -5; return 0; }
"""

PREV = ("k", "v", "g", "beta")
# every operator's arguments; the first is the one that the call goes by
ARGS = {
    "rmsnorm": ("x", "weight", "residual", "y", "residual_out"),
    "rmsnorm_fp8": ("x", "weight", "residual", "y", "residual_out", "scales"),
    "gated_delta_step": ("k", "q", "v", "g", "beta", "state", "state_idx", "accept_len", "o",
                         *("prev %d" % i for i in range(4))),
    "gated_delta_chunk": ("k", "q", "v", "g", "beta", "cu_seqlens", "state", "state_idx", "o", "workspace"),
    "w4a16_gate_up": ("x", "Wq", "scales", "h"),
}


def tensors(device):
    """{operator: {argument: tensor}} on that device."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        def e(*s, t=torch.bfloat16):
            return torch.empty(*s, dtype=t, device=device)

        f, i = torch.float32, torch.int32
        norm = dict(x=e(4, 256), weight=e(256), residual=e(4, 256), y=e(4, 256), residual_out=e(4, 256))
        step = dict(q=e(2, 3, 1, 64), k=e(2, 3, 1, 64), v=e(2, 3, 2, 64), g=e(2, 3, 2, t=f), beta=e(2, 3, 2, t=f),
                    state=e(2, 2, 64, 64, t=f), state_idx=e(2, t=i), accept_len=e(2, t=i), o=e(2, 3, 2, 64))
        chunk = dict(q=e(6, 1, 64), k=e(6, 1, 64), v=e(6, 2, 64), g=e(6, 2, t=f), beta=e(6, 2, t=f), cu_seqlens=e(3, t=i),
                     state=e(2, 2, 64, 64, t=f), state_idx=e(2, t=i), o=e(6, 2, 64), workspace=e(1 << 20, t=torch.uint8))
        return {"rmsnorm": norm, "rmsnorm_fp8": dict(norm, y=e(4, 256, t=torch.float8_e4m3fn), scales=e(4, 2, t=f)),
                "gated_delta_step": dict(step, prev=[step[n] for n in PREV]), "gated_delta_chunk": chunk,
                "w4a16_gate_up": dict(x=e(4, 256), Wq=e(64, 32, t=i), scales=e(64, 2), h=e(4, 32))}


def program():
    torch.cuda.is_available = lambda: False     # (else tensors without memory touch the device)
    import speculative_verify_gb300 as sv

    def call(op, args):
        try:
            getattr(sv, op)(**args)
        except Exception as e:
            print(type(e).__name__, str(e)[:60].replace("\n", " "), flush=True)

    one, other = tensors("cuda:1"), tensors("cuda:0")
    for op, names in ARGS.items():
        print("= %s %s" % (op, names[0]), flush=True)
        call(op, one[op])
        for name in names[1:]:
            print("= %s %s" % (op, name), flush=True)
            args = dict(one[op])
            if name.startswith("prev"):
                args["prev"] = list(args["prev"])
                args["prev"][int(name[-1])] = other[op]["prev"][int(name[-1])]
            else:
                args[name] = other[op][name]
            call(op, args)


if __name__ == "__main__":
    program()


@pytest.fixture(scope="module")
def said(tmp_path_factory):
    """{(operator, argument on the other device, or the call's own one): what the call printed}."""
    if torch.cuda.is_available() or not shutil.which("gcc"):
        pytest.skip("runs where there is no GPU, and a C compiler")
    from speculative_verify_gb300 import build
    build.build()
    d = tmp_path_factory.mktemp("runtime")
    (d / "runtime.c").write_text(RUNTIME)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(d / "runtime.so"), str(d / "runtime.c")], check=True)
    env = dict(os.environ, LD_PRELOAD=str(d / "runtime.so"), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = {}
    for line in r.stdout.splitlines():
        if line.startswith("= "):
            lines = out[tuple(line[2:].split(" ", 1))] = []
        else:
            lines.append(line)
    return out


@pytest.mark.parametrize("op", ARGS)
def test_call_runs_on_its_tensors_device(said, op):
    """With device 0 current, a call on tensors of device 1 makes that one current, and then device 0 again."""
    lines = said[op, ARGS[op][0]]
    assert lines[:2] == ["current 1", "current 0"] and lines[2].startswith("SpecVerifyError")   # (no memory behind them)
    assert len(lines) == 3


@pytest.mark.parametrize("op,name", [(op, name) for op, names in ARGS.items() for name in names[1:]])
def test_tensors_of_two_devices_are_refused(said, op, name):
    lines = said[op, name]
    assert lines[-1].startswith("ValueError") and "device" in lines[-1], lines
