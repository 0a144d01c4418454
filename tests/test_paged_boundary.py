"""attn_fwd_paged without a GPU: bad arguments are refused on the host before any launch, and
workspace sizes cannot overflow."""
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


A = 1 << 32  # fake, aligned addresses, far apart: never dereferenced on these paths
INVALID, UNSUPPORTED = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
MISALIGNED, ALIASING, LARGE = attn.ATTN_ERR_MISALIGNED, attn.ATTN_ERR_ALIASING, attn.ATTN_ERR_TOO_LARGE


def _call(lib, q=A, kp=2 * A, vp=3 * A, table=4 * A, n=5 * A, o=6 * A, l=7 * A, mass=8 * A, layout=1, B=4, Hq=8,
          Hkv=2, Sq=1, n_pages=100, page=16, stride=16 * 2 * 128, max_pages=20, d=128, scale=0.1, mode=0, flags=0,
          ws=9 * A, ws_bytes=1 << 31):
    return lib.attn_fwd_paged(q, kp, vp, table, n, o, l, mass, layout, B, Hq, Hkv, Sq, n_pages, page, stride, max_pages,
                              d, ctypes.c_float(scale), mode, flags, ws, ws_bytes, 0)


@pytest.mark.parametrize("kw,status", [
    *[({x: 0}, INVALID) for x in ("q", "kp", "vp", "table", "n", "o", "l", "ws")],
    (dict(B=0), INVALID), (dict(Hq=7), INVALID), (dict(Hkv=0), INVALID), (dict(Sq=0), INVALID),
    (dict(n_pages=0), INVALID), (dict(page=0), INVALID), (dict(max_pages=0), INVALID), (dict(scale=math.inf), INVALID),
    (dict(ws_bytes=64), INVALID), (dict(stride=16 * 2 * 128 - 128), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(layout=-1), UNSUPPORTED), (dict(mode=3), UNSUPPORTED),
    (dict(flags=2), UNSUPPORTED), (dict(flags=4), UNSUPPORTED), (dict(q=A + 8), MISALIGNED),
    (dict(kp=2 * A + 4), MISALIGNED), (dict(n=5 * A + 2), MISALIGNED), (dict(l=7 * A + 1), MISALIGNED),
    (dict(mass=8 * A + 2), MISALIGNED), (dict(table=4 * A + 1), MISALIGNED), (dict(ws=9 * A + 8), MISALIGNED),
    (dict(stride=16 * 2 * 128 + 64), MISALIGNED),
    (dict(o=A), ALIASING), (dict(o=2 * A), ALIASING), (dict(l=5 * A), ALIASING), (dict(ws=3 * A), ALIASING),
    (dict(l=6 * A), ALIASING), (dict(mass=4 * A), ALIASING), (dict(mass=9 * A), ALIASING), (dict(o=8 * A), ALIASING),
    (dict(B=1 << 31), LARGE), (dict(max_pages=1 << 27), LARGE), (dict(page=1 << 31), LARGE),
    (dict(Sq=1 << 29), LARGE), (dict(n_pages=1 << 27), LARGE), (dict(Hq=1 << 21, Hkv=1 << 21), LARGE),
    (dict(B=1 << 30, max_pages=(1 << 27) - 5), LARGE),
])
def test_refusals(lib, kw, status):
    assert _call(lib, **kw) == status


def test_good_arguments_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    assert _call(lib) == attn.ATTN_ERR_NO_DEVICE
    assert _call(lib, mass=0) == attn.ATTN_ERR_NO_DEVICE
    assert _call(lib, n_pages=1, stride=128) == attn.ATTN_ERR_NO_DEVICE   # one page: its stride is not looked at


def test_workspace_sizes(lib):
    # At least a partial row per run; with a mass, a logit per row and slot.
    assert attn.paged_workspace_bytes(4, 8, 2, 1, 16, 20) >= 8 * 520
    more = attn.paged_workspace_bytes(4, 8, 2, 1, 16, 20, with_mass=True) - attn.paged_workspace_bytes(4, 8, 2, 1, 16, 20)
    assert more >= 4 * 2 * 4 * 320 * 4
    for args in [(0, 8, 2, 1, 16, 10), (1, 7, 2, 1, 16, 10), (1, 8, 2, 0, 16, 10), (1, 8, 2, 1, 0, 10), (1, 8, 2, 1, 1, 0)]:
        with pytest.raises(attn.AttnError) as e:
            attn.paged_workspace_bytes(*args)
        assert e.value.status == INVALID
    for args in [(1, 8, 2, 1, 1 << 20, 1 << 12), (1 << 30, 8, 8, 1, 1 << 10, 1 << 20)]:
        with pytest.raises(attn.AttnError) as e:
            attn.paged_workspace_bytes(*args)
        assert e.value.status == LARGE
    with pytest.raises(attn.AttnError) as e:
        attn.paged_workspace_bytes(1 << 16, 64, 64, 1, 1 << 10, 1 << 17, with_mass=True)
    assert e.value.status == LARGE


@pytest.mark.parametrize("change,exc", [
    (dict(layout="sbhd"), ValueError), (dict(rounding="up"), ValueError), (dict(), TypeError),  # not on a GPU
])
def test_python_refusals(change, exc):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(exc):
        attn.attn_fwd_paged(bf(2, 1, 4, 128), bf(8, 16, 2, 128), bf(8, 16, 2, 128),
                            torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                            **{"layout": "bshd", **change})


@pytest.mark.parametrize("kw,ns,status", [
    (dict(Hq=40), 0, INVALID), (dict(Hq=40), 2_000_000_001, INVALID), (dict(Hq=32), 20_000_000, UNSUPPORTED),
    (dict(Hq=40, d=64), 20_000_000, UNSUPPORTED), (dict(Hq=40, o=A), 20_000_000, ALIASING),
    (dict(Hq=40), 20_000_000, attn.ATTN_ERR_NO_DEVICE),
])
def test_selftest_refusals(lib, kw, ns, status):
    """It takes attn_fwd_paged's refusals, a limit of 1 ns to 2 s, and only more than 16 rows."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    a = dict(o=6 * A, Hq=8, d=128)
    a.update(kw)
    assert lib.attn_fwd_paged_timeout_selftest(A, 2 * A, 3 * A, 4 * A, 5 * A, a["o"], 7 * A, 8 * A, 1, 4, a["Hq"], 2, 1,
                                               100, 16, 16 * 2 * 128, 20, a["d"], ctypes.c_float(0.1), 0, 0, 9 * A,
                                               1 << 31, 0, ns) == status
