"""The device of an attention layer's call, without a GPU, as
test_layer_devices.py has it for the calls before: calls on tensors that have a
device but no memory, with a fake CUDA runtime of two devices; and the
binding's refusals of shapes, types and gradients on such tensors."""
import os
import shutil
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if __name__ == "__main__":
    sys.path.insert(0, os.path.join(ROOT, "tests"))

from test_layer_devices import RUNTIME  # noqa: E402

ARGS = {
    "rotary": ("q", "k", "positions", "inv_freq", "axes", "q_out", "k_out"),
    "kv4_append": ("k", "v", "cache", "page_table", "seq_lens", "cu_seqlens"),
    "kv4_gather": ("cache", "page_table", "seq_lens", "cu_seqlens", "k", "v"),
    "kv4_attention": ("q", "cache", "page_table", "seq_lens", "cu_seqlens", "o", "workspace"),
}


def tensors(device):
    """{operator: {argument: tensor}} on that device."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        def e(*s, t=torch.bfloat16):
            return torch.empty(*s, dtype=t, device=device)

        i = torch.int32
        cache = dict(cache=e(9, 2, 36 * 64, t=torch.uint8), page_table=e(3, 4, t=i), seq_lens=e(3, t=i), cu_seqlens=e(4, t=i))
        return {"rotary": dict(q=e(6, 4, 64), k=e(6, 2, 64), positions=e(2, 6, t=i), inv_freq=e(32, t=torch.float32),
                               axes=e(32, t=i), q_out=e(6, 4, 64), k_out=e(6, 2, 64)),
                "kv4_append": dict(cache, k=e(6, 2, 64), v=e(6, 2, 64)),
                "kv4_gather": dict(cache, rows=6, k=e(6, 2, 64), v=e(6, 2, 64)),
                "kv4_attention": dict(cache, q=e(6, 4, 64), o=e(6, 4, 64), workspace=e(1 << 24, t=torch.uint8))}


def wrong():
    """{operator: [(what, changed arguments, the error)]}, on device 1."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        def e(*s, t=torch.bfloat16, grad=False):
            x = torch.empty(*s, dtype=t, device="cuda:1")
            return x.requires_grad_() if grad else x

        i, u8, f = torch.int32, torch.uint8, torch.float32
        kv = [("gradient", dict(k=e(6, 2, 64, grad=True)), "RuntimeError"), ("type of k", dict(k=e(6, 2, 64, t=f)), "TypeError"),
              ("heads", dict(k=e(6, 3, 64)), "ValueError"), ("dimensions", dict(v=e(6, 2, 128)), "ValueError"),
              ("rows", dict(v=e(5, 2, 64)), "ValueError"), ("batched with cu_seqlens", dict(k=e(3, 2, 2, 64)), "ValueError"),
              ("rows that are not dense", dict(k=e(6, 64, 2).transpose(1, 2)), "ValueError")]
        cache = [("type of cache", dict(cache=e(9, 2, 36 * 64, t=torch.int8)), "TypeError"),
                 ("bytes of a page", dict(cache=e(9, 2, 36 * 64 + 1, t=u8)), "ValueError"),
                 ("cache of two dimensions", dict(cache=e(9, 36 * 64, t=u8)), "TypeError"),
                 ("cache that is not contiguous", dict(cache=e(2, 9, 36 * 64, t=u8).transpose(0, 1)), "TypeError"),
                 ("table", dict(page_table=e(3, t=i)), "TypeError"), ("type of table", dict(page_table=e(3, 4, t=torch.int64)), "TypeError"),
                 ("lengths", dict(seq_lens=e(2, t=i)), "ValueError"), ("type of lengths", dict(seq_lens=e(3, t=torch.int64)), "TypeError"),
                 ("cu_seqlens", dict(cu_seqlens=e(3, t=i)), "ValueError"), ("scale", dict(k_scale="x"), "TypeError")]
        return {"rotary": [("gradient", dict(q=e(6, 4, 64, grad=True)), "RuntimeError"), ("type", dict(q=e(6, 4, 64, t=f)), "TypeError"),
                           ("rows of k", dict(k=e(5, 2, 64)), "ValueError"), ("dimensions of k", dict(k=e(6, 2, 32)), "ValueError"),
                           ("positions", dict(positions=e(2, 5, t=i)), "ValueError"), ("type of positions", dict(positions=e(6, t=f)), "TypeError"),
                           ("axes", dict(axes=e(31, t=i)), "ValueError"), ("frequencies", dict(inv_freq=e(2, 16, t=f)), "ValueError"),
                           ("q_out", dict(q_out=e(6, 2, 64)), "ValueError"), ("k_out without k", dict(k=None), "ValueError"),
                           ("two dimensions", dict(q=e(6, 256)), "ValueError")],
                "kv4_append": kv + cache, "kv4_gather": kv[1:3] + cache + [("negative rows", dict(rows=-1), "ValueError")],
                "kv4_attention": cache + [("gradient", dict(q=e(6, 4, 64, grad=True)), "RuntimeError"),
                                          ("heads", dict(q=e(6, 5, 64), o=None), "ValueError"),
                                          ("dimensions", dict(q=e(6, 4, 128), o=None), "ValueError"),
                                          ("o", dict(o=e(6, 2, 64)), "ValueError"), ("window", dict(window=-1), "ValueError"),
                                          ("sinks", dict(sinks=(1 << 30) + 1), "ValueError"),
                                          ("type of workspace", dict(workspace=e(1 << 20, t=f)), "TypeError"),
                                          ("batched with cu_seqlens", dict(q=e(3, 2, 4, 64), o=None), "ValueError")]}


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
            call(op, dict(one[op], **{name: other[op][name]}))
    for op, cases in wrong().items():
        for what, changed, _ in cases:
            print("= %s wrong %s" % (op, what), flush=True)
            call(op, dict(one[op], **changed))


if __name__ == "__main__":
    program()


@pytest.fixture(scope="module")
def said(tmp_path_factory):
    """{(operator, what): what the call printed}."""
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


def test_wrong_arguments_are_refused(said):
    for op, cases in wrong().items():
        for what, _, error in cases:
            lines = said[op, "wrong " + what]
            assert lines[-1].startswith(error), (op, what, lines)
