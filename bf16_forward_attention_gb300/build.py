"""Builds the CUDA library in-tree: ``_lib/libattn_fwd.so`` for sm_103a.

    python -m bf16_forward_attention_gb300.build [--force] [--debug]

``--debug`` builds ``_lib/libattn_fwd_debug.so`` with -DATTN_DEBUG=1 instead: the
same kernels with bounds and protocol checks that report through the device
status word (see include/attn_fwd.h).

One translation unit per group of kernels with their launcher (the forward ones,
the backward ones, a batch on a shared prefix, norms with rotation, attention
over a paged cache, its eviction) and the host-buffer pipeline, compiled at once,
one -gencode; the CUDA runtime is linked statically and the driver's tensor-map
encoder is looked up at run time, so the library loads (and reports
ATTN_ERR_NO_DEVICE) on a machine without a GPU. Beside it the host compiler builds
``_lib/attn_binding-*.so``, the C++ part of the Python binding, against the installed
torch, whose version and Python's are in its name; the library itself knows nothing of torch.
"""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import signal
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libattn_fwd.so")
LIB_PATH_DEBUG = os.path.join(LIB_DIR, "libattn_fwd_debug.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("attn_fwd.cu", "attn_bwd.cu", "attn_prefix.cu", "attn_rope.cu",
                                            "attn_paged.cu", "attn_evict.cu", "attn_host.cu")]
GENCODE = "arch=compute_103a,code=sm_103a"


def _deps():
    deps = list(SOURCES)
    for d in (CSRC, INCLUDE):
        deps += [os.path.join(d, f) for f in os.listdir(d) if f.endswith((".cuh", ".h", ".cu"))]
    return deps


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found (set CUDA_HOME or put nvcc on PATH)")


def lib_path(debug: bool = False) -> str:
    return LIB_PATH_DEBUG if debug else LIB_PATH


def _newer(path: str, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _library_up_to_date(debug: bool = False) -> bool:
    return _newer(lib_path(debug), _deps())


def _torch_dir():
    """Where torch is installed; None without it, or where it is one without CUDA, which has no tensors that
    the binding takes (the library can be used from C all the same)."""
    spec = importlib.util.find_spec("torch")
    if not spec or not spec.submodule_search_locations:
        return None
    path = spec.submodule_search_locations[0]
    return path if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def binding_path() -> str:
    """The C++ part of the binding for the torch and the Python that are here: it holds to the layout of their
    objects, so that one built for others is never taken for it. "" where there is no torch for it."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return ""
    with open(os.path.join(torch_dir, "version.py")) as f:
        version = re.search(r"__version__ *= *['\"]([^'\"]+)", f.read())
    name = f"attn_binding-torch{version.group(1) if version else ''}{sysconfig.get_config_var('EXT_SUFFIX')}"
    return os.path.join(LIB_DIR, name)


def _binding_up_to_date() -> bool:
    path = binding_path()
    return not path or _newer(path, [BINDING_SOURCE, os.path.join(INCLUDE, "attn_fwd.h")])


def up_to_date(debug: bool = False) -> bool:
    return _library_up_to_date(debug) and (debug or _binding_up_to_date())


def _binding_build(force: bool):
    """A running compilation of the binding's C++ part (no kernels) against the installed torch and
    Python, its command, where its output is and where that belongs; None if the binding is newer
    than its sources, or there is no torch for it."""
    torch_dir = _torch_dir()
    if torch_dir is None or (not force and _binding_up_to_date()):
        return None
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    path = binding_path()
    tmp = path + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-std=c++17", "-O2", "-fPIC", "-shared", "-o", tmp, BINDING_SOURCE]
    for d in (INCLUDE, os.path.join(torch_dir, "include"),
              os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], cuda):
        cmd += ["-I", d]
    cmd += ["-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    return subprocess.Popen(cmd, start_new_session=True), cmd, tmp, path  # a group: the compiler has children


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile the library (release, or the debug flavour) if any source is newer
    than it, and beside the release one the binding. Returns the library's path."""
    path = lib_path(debug)
    os.makedirs(LIB_DIR, exist_ok=True)
    binding = None if debug else _binding_build(force)
    try:
        if force or not _library_up_to_date(debug):
            tmp = path + f".tmp{os.getpid()}"
            cmd = [nvcc_path(), "-gencode", GENCODE, "-O3", "-lineinfo", "-std=c++17",
                   "--threads", "0", "-Xcompiler", "-fPIC", "-shared", "-I", INCLUDE, "-o", tmp] + SOURCES
            if debug:
                cmd.insert(1, "-DATTN_DEBUG=1")
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
            os.replace(tmp, path)
        if binding:
            run, cmd, tmp, to = binding
            if run.wait() != 0:
                raise subprocess.CalledProcessError(run.returncode, cmd)
            os.replace(tmp, to)
    finally:
        if binding:  # nothing of it is left, however the library's compilation ended
            run, _, tmp, _ = binding
            if run.poll() is None:
                os.killpg(run.pid, signal.SIGTERM)
                run.wait()
            if os.path.exists(tmp):
                os.remove(tmp)
    return path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
