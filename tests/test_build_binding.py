"""The build of the binding's C++ part."""
import types

import pytest

from bf16_forward_attention_gb300 import build


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """A library directory of its own with an up-to-date library in it, and no compiler that runs in earnest."""
    lib = tmp_path / "_lib"
    lib.mkdir()
    monkeypatch.setattr(build, "LIB_DIR", str(lib))
    monkeypatch.setattr(build, "LIB_PATH", str(lib / "libattn_fwd.so"))
    monkeypatch.setattr(build, "LIB_PATH_DEBUG", str(lib / "libattn_fwd_debug.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(lib / "attn_binding.so"))
    (lib / "libattn_fwd.so").write_bytes(b"")
    return tmp_path


def _fake_torch(path, monkeypatch, cuda):
    for d in ("lib", "include"):
        (path / "torch" / d).mkdir(parents=True)
    (path / "torch" / "__init__.py").write_text("")
    for n in ("libc10.so", "libtorch.so", "libtorch_cpu.so", "libtorch_python.so") + (("libc10_cuda.so",) if cuda else ()):
        (path / "torch" / "lib" / n).write_bytes(b"")
    spec = types.SimpleNamespace(submodule_search_locations=[str(path / "torch")])
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec)


def test_a_torch_without_cuda_needs_no_binding(sandbox, monkeypatch):
    """The C library builds beside it as it does without any torch."""
    _fake_torch(sandbox, monkeypatch, cuda=False)
    monkeypatch.setattr(build.subprocess, "Popen", lambda *a, **k: pytest.fail("a compiler was started"))
    assert build.build() == build.LIB_PATH
    assert build.up_to_date()
