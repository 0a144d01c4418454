"""The build of the binding's C++ part."""
import importlib.util
import os
import subprocess
import sys
import time
import types

import pytest

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """A library directory of its own with an up-to-date library in it, and no compiler that runs in earnest."""
    lib = tmp_path / "_lib"
    lib.mkdir()
    monkeypatch.setattr(build, "LIB_DIR", str(lib))
    monkeypatch.setattr(build, "LIB_PATH", str(lib / "libattn_fwd.so"))
    monkeypatch.setattr(build, "LIB_PATH_DEBUG", str(lib / "libattn_fwd_debug.so"))
    (lib / "libattn_fwd.so").write_bytes(b"")
    return tmp_path


def _fake_torch(path, monkeypatch, cuda, version="2.9.1+cu130"):
    for d in ("lib", "include"):
        (path / "torch" / d).mkdir(parents=True)
    (path / "torch" / "__init__.py").write_text("")
    (path / "torch" / "version.py").write_text(f"from typing import Optional\n__version__ = '{version}'\ndebug = False\n")
    for n in ("libc10.so", "libtorch.so", "libtorch_cpu.so", "libtorch_python.so") + (("libc10_cuda.so",) if cuda else ()):
        (path / "torch" / "lib" / n).write_bytes(b"")
    spec = types.SimpleNamespace(submodule_search_locations=[str(path / "torch")])
    real = importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else real(name, *a))


def test_a_torch_without_cuda_needs_no_binding(sandbox, monkeypatch):
    """The C library builds beside it as it does without any torch."""
    _fake_torch(sandbox, monkeypatch, cuda=False)
    monkeypatch.setattr(build.subprocess, "Popen", lambda *a, **k: pytest.fail("a compiler was started"))
    assert build.build() == build.LIB_PATH
    assert build.up_to_date()


def _compiler(monkeypatch):
    """In place of the host compiler: writes its arguments to what it is to make. Returns the runs."""
    runs = []

    class Run:
        returncode = 0

        def __init__(self, cmd, **kw):
            runs.append(cmd)
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write(" ".join(cmd))

        def poll(self):
            return 0

        def wait(self):
            return 0

    monkeypatch.setattr(build.subprocess, "Popen", Run)
    return runs


def test_a_binding_is_for_one_torch_and_one_python(sandbox, monkeypatch):
    """After a change of either the built one is neither up to date nor loaded, whatever the files' times."""
    _fake_torch(sandbox / "a", monkeypatch, cuda=True)
    runs = _compiler(monkeypatch)
    assert not build.up_to_date()
    build.build()
    assert len(runs) == 1 and build.up_to_date()
    build.build()
    assert len(runs) == 1
    _fake_torch(sandbox / "b", monkeypatch, cuda=True, version="2.11.0+cu130")
    assert not build.up_to_date()
    monkeypatch.setattr(attn, "_binding", None)
    with pytest.raises(RuntimeError, match="binding not built"):
        attn._load_binding()
    build.build()
    assert len(runs) == 2 and build.up_to_date()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: ".cpython-399-x.so")
    assert not build.up_to_date()
    build.build()
    assert len(runs) == 3 and build.up_to_date()


def test_the_built_binding_is_found_and_loads():
    """With the torch that is here, beside a library that is built."""
    build.build()
    assert hasattr(attn._load_binding(), "fwd_paged")
    assert os.path.exists(build.binding_path()) and "torch" in sys.modules


def test_no_compilation_is_left_behind_when_the_library_fails(sandbox, monkeypatch):
    """The host compiler runs beside nvcc: where that fails, it is ended and waited for, and its file removed."""
    _fake_torch(sandbox, monkeypatch, cuda=True)
    (sandbox / "_lib" / "libattn_fwd.so").unlink()
    started = []

    def popen(cmd, **kw):
        to = cmd[cmd.index("-o") + 1]
        run = real([sys.executable, "-c", "import sys, time; open(sys.argv[1], 'w').close(); time.sleep(60)", to], **kw)
        while not os.path.exists(to) and run.poll() is None:
            time.sleep(0.01)
        started.append((run, to))
        return run

    def fails(cmd, **kw):
        raise subprocess.CalledProcessError(1, cmd)

    real = subprocess.Popen
    monkeypatch.setattr(build.subprocess, "Popen", popen)
    monkeypatch.setattr(build.subprocess, "run", fails)
    try:
        with pytest.raises(subprocess.CalledProcessError):
            build.build()
        (run, to), = started
        assert run.returncode is not None, "still running"
        assert not os.path.exists(to)
    finally:
        for run, _ in started:
            run.kill()
            run.wait()


def test_a_failed_binding_leaves_no_file(sandbox, monkeypatch):
    _fake_torch(sandbox, monkeypatch, cuda=True)
    real = subprocess.Popen
    monkeypatch.setattr(build.subprocess, "Popen", lambda cmd, **kw: real(
        [sys.executable, "-c", "import sys; open(sys.argv[1], 'w').close(); sys.exit(3)", cmd[cmd.index("-o") + 1]], **kw))
    with pytest.raises(subprocess.CalledProcessError):
        build.build()
    assert os.listdir(sandbox / "_lib") == ["libattn_fwd.so"]
