"""attn_fwd_prefix without a GPU: bad arguments are refused on the host before any
launch, and workspace sizes cannot overflow."""
import ctypes
import math
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
INVALID, UNSUPPORTED = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
MISALIGNED, ALIASING, LARGE = attn.ATTN_ERR_MISALIGNED, attn.ATTN_ERR_ALIASING, attn.ATTN_ERR_TOO_LARGE


def _call(lib, q=A, kp=2 * A, vp=3 * A, k=4 * A, v=5 * A, n=6 * A, o=7 * A, l=8 * A, layout=1, B=4, Hq=8, Hkv=2,
          Sq=1, Sp=1000, cap=64, d=128, scale=0.1, mode=0, flags=0, ws=9 * A, ws_bytes=1 << 29):
    return lib.attn_fwd_prefix(q, kp, vp, k, v, n, o, l, layout, B, Hq, Hkv, Sq, Sp, cap, d, ctypes.c_float(scale),
                               mode, flags, ws, ws_bytes, 0)


@pytest.mark.parametrize("kw,status", [
    *[({x: 0}, INVALID) for x in ("q", "kp", "vp", "k", "v", "n", "o", "l", "ws")],
    (dict(B=0), INVALID), (dict(Hq=7), INVALID), (dict(Hkv=0), INVALID), (dict(Sq=0), INVALID),
    (dict(Sp=-1), INVALID), (dict(cap=0), INVALID), (dict(scale=math.nan), INVALID), (dict(ws_bytes=64), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(layout=-1), UNSUPPORTED), (dict(mode=3), UNSUPPORTED),
    (dict(flags=2), UNSUPPORTED), (dict(q=A + 8), MISALIGNED), (dict(kp=2 * A + 4), MISALIGNED),
    (dict(n=6 * A + 2), MISALIGNED), (dict(l=8 * A + 1), MISALIGNED), (dict(ws=9 * A + 8), MISALIGNED),
    (dict(o=A), ALIASING), (dict(o=2 * A), ALIASING), (dict(l=6 * A), ALIASING), (dict(ws=5 * A), ALIASING),
    (dict(l=7 * A), ALIASING), (dict(B=1 << 31), LARGE), (dict(cap=1 << 31), LARGE),
    (dict(B=1 << 24, Sq=1 << 10), LARGE), (dict(Hkv=1 << 12, Hq=1 << 12, Sp=1 << 30), LARGE),
])
def test_refusals(lib, kw, status):
    assert _call(lib, **kw) == status


def test_good_arguments_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    assert _call(lib) == attn.ATTN_ERR_NO_DEVICE
    assert _call(lib, Sp=0, kp=0, vp=0) == attn.ATTN_ERR_NO_DEVICE


def test_workspace_sizes(lib):
    # At least the packed queries, one part of the prefix and one of the own keys.
    assert attn.prefix_workspace_bytes(4, 8, 2, 1, 1000, 64) >= 4 * 8 * 256 + 2 * 2 * 256 * 520
    assert attn.prefix_workspace_bytes(4, 8, 2, 1, 0, 64) >= 2 * 256 * 520
    for args in [(0, 8, 2, 1, 10, 10), (1, 7, 2, 1, 10, 10), (1, 8, 2, 1, -1, 10), (1, 8, 2, 1, 10, 0)]:
        with pytest.raises(attn.AttnError) as e:
            attn.prefix_workspace_bytes(*args)
        assert e.value.status == INVALID
    with pytest.raises(attn.AttnError) as e:
        attn.prefix_workspace_bytes(1 << 28, 64, 1, 1, 10, 10)
    assert e.value.status == LARGE


@pytest.mark.parametrize("change,exc", [
    (dict(layout="sbhd"), ValueError), (dict(rounding="up"), ValueError), (dict(), TypeError),  # not on a GPU
])
def test_python_refusals(change, exc):
    q, k = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 8, 2, 128, dtype=torch.bfloat16)
    p = torch.zeros(5, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(exc):
        attn.attn_fwd_prefix(q, p, p, k, k, torch.zeros(2, dtype=torch.int32), **{"layout": "bshd", **change})
