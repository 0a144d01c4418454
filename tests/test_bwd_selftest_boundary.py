"""attn_bwd_timeout_selftest without a GPU: it takes attn_bwd's refusals, and a limit of 1 ns to 2 s
and a kernel of its own."""
import ctypes
import shutil

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build


@pytest.fixture(scope="module")
def lib():
    if not build.up_to_date():
        if shutil.which("nvcc") is None:
            pytest.skip("library not built and nvcc not available")
        build.build()
    return attn.load_library()


A = 1 << 30  # fake, aligned addresses, far apart: never dereferenced on these paths


@pytest.mark.parametrize("kw,status", [
    (dict(ns=0), attn.ATTN_ERR_INVALID_ARG), (dict(ns=2_000_000_001), attn.ATTN_ERR_INVALID_ARG),
    (dict(kernel=2), attn.ATTN_ERR_INVALID_ARG), (dict(kernel=-1), attn.ATTN_ERR_INVALID_ARG),
    (dict(flags=2), attn.ATTN_ERR_UNSUPPORTED), (dict(d=64), attn.ATTN_ERR_UNSUPPORTED),
    (dict(ws=0), attn.ATTN_ERR_INVALID_ARG), (dict(dq=A), attn.ATTN_ERR_ALIASING),
    (dict(), attn.ATTN_ERR_NO_DEVICE),
])
def test_refusals(lib, kw, status):
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    a = dict(ns=20_000_000, kernel=0, flags=0, d=128, ws=10 * A, dq=7 * A)
    a.update(kw)
    assert lib.attn_bwd_timeout_selftest(A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, a["dq"], 8 * A, 9 * A, 0, 1, 4, 2, 300,
                                         200, a["d"], ctypes.c_float(0.1), 0, a["flags"], a["ws"], 1 << 29, 0,
                                         a["ns"], a["kernel"]) == status
