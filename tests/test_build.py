"""What build() compiles, with the compilers replaced by a recorder of their
commands."""
import os

import pytest

from speculative_verify_gb300 import build as b


@pytest.fixture
def ran(tmp_path, monkeypatch):
    """build()'s commands; its outputs are empty files in a folder of their own."""
    cmds = []

    def run(batch, verbose):
        for cmd in batch:
            cmds.append(cmd)
            open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "_nvcc", lambda: "nvcc")
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / "libspecverify.so"))
    monkeypatch.setattr(b, "BIND_PATH", str(tmp_path / "_layer.so"))
    monkeypatch.setattr(b, "BIND_FOR", str(tmp_path / "_layer.so.for"))
    return cmds


def built(path, cmds):
    return sum(os.path.basename(path) in os.path.basename(c[c.index("-o") + 1]) for c in cmds)


def without_torch(monkeypatch):
    find = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_library_without_torch(ran, monkeypatch):
    """The C library needs nvcc only; the binding waits until there is a torch."""
    with monkeypatch.context() as m:
        without_torch(m)
        assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
        assert ran and all(c[0] == "nvcc" for c in ran) and not os.path.exists(b.BIND_PATH)
        ran.clear()
        b.build()
        assert not ran                          # nothing is older than its sources
    pytest.importorskip("torch")
    b.build()
    assert os.path.exists(b.BIND_PATH) and not any(c[0] == "nvcc" for c in ran)


def test_both_are_built_once(ran):
    pytest.importorskip("torch")
    b.build()
    assert built(b.LIB_PATH, ran) == 1 and built(b.BIND_PATH, ran) == 1
    ran.clear()
    b.build()
    assert not ran
    os.utime(b.LIB_PATH, (1, 1))
    b.build()
    assert built(b.LIB_PATH, ran) == 1 and built(b.BIND_PATH, ran) == 0
    assert not [f for f in os.listdir(b.BUILD_DIR) if f.endswith(".tmp") or f.endswith(".o")]


def test_binding_is_rebuilt_for_another_torch(ran, tmp_path, monkeypatch):
    """The binding uses torch's C++ internals: another torch or Python needs another one, the library does not."""
    root = tmp_path / "torch"
    root.mkdir()
    monkeypatch.setattr(b, "_torch_root", lambda: str(root))
    (root / "version.py").write_text("__version__ = '1'\n")
    b.build()
    ran.clear()
    b.build()
    assert not ran
    (root / "version.py").write_text("__version__ = '2'\n")
    b.build()
    assert built(b.BIND_PATH, ran) == 1 and built(b.LIB_PATH, ran) == 0
    ran.clear()
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-399")
    b.build()
    assert built(b.BIND_PATH, ran) == 1 and built(b.LIB_PATH, ran) == 0
