"""attn_cache_evict without a GPU: bad arguments are refused on the host before any launch."""
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


def _call(lib, kp=A, vp=2 * A, table=3 * A, n=4 * A, mass=5 * A, mass_out=6 * A, n_out=7 * A, layout=1, B=4, Hkv=2,
          n_pages=100, page=16, stride=16 * 2 * 128, max_pages=20, d=128, budget=64, recent=8, ws=8 * A, ws_bytes=1 << 24):
    return lib.attn_cache_evict(kp, vp, table, n, mass, mass_out, n_out, layout, B, Hkv, n_pages, page, stride,
                                max_pages, d, budget, recent, ws, ws_bytes, 0)


@pytest.mark.parametrize("kw,status", [
    *[({x: 0}, INVALID) for x in ("kp", "vp", "table", "n", "mass", "mass_out", "n_out", "ws")],
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(n_pages=0), INVALID), (dict(page=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(budget=0), INVALID), (dict(recent=-1), INVALID), (dict(recent=65), INVALID),
    (dict(ws_bytes=64), INVALID), (dict(stride=128), INVALID), (dict(d=64), UNSUPPORTED), (dict(layout=2), UNSUPPORTED),
    (dict(kp=A + 8), MISALIGNED), (dict(mass=5 * A + 2), MISALIGNED), (dict(n_out=7 * A + 1), MISALIGNED),
    (dict(ws=8 * A + 8), MISALIGNED), (dict(stride=16 * 2 * 128 + 8), MISALIGNED),
    (dict(vp=A), ALIASING), (dict(vp=A + 256), ALIASING), (dict(mass=A), ALIASING), (dict(table=2 * A), ALIASING),
    (dict(mass_out=5 * A + 64), ALIASING), (dict(mass_out=4 * A), ALIASING), (dict(n_out=3 * A), ALIASING),
    (dict(n_out=6 * A), ALIASING), (dict(ws=5 * A), ALIASING), (dict(ws=7 * A), ALIASING), (dict(n_out=4 * A + 4), ALIASING),
    (dict(B=1 << 28), LARGE), (dict(max_pages=1 << 27), LARGE), (dict(n_pages=1 << 28), LARGE),
    (dict(budget=1 << 31), LARGE), (dict(page=1 << 32), LARGE),
])
def test_refusals(lib, kw, status):
    assert _call(lib, **kw) == status


def test_good_arguments_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    assert _call(lib) == attn.ATTN_ERR_NO_DEVICE
    assert _call(lib, mass_out=5 * A, n_out=4 * A) == attn.ATTN_ERR_NO_DEVICE          # in place
    assert _call(lib, vp=A + 16 * 2 * 256, stride=2 * 16 * 2 * 128) == attn.ATTN_ERR_NO_DEVICE
    assert _call(lib, budget=10 ** 6, recent=10 ** 6) == attn.ATTN_ERR_NO_DEVICE       # a budget beyond the table


def test_workspace_sizes(lib):
    n = attn.evict_workspace_bytes(4, 2, 100, 16, 20, 64)
    assert n >= 400 + 64 + 2 * 4 * 2 * 64 * 4
    assert attn.evict_workspace_bytes(4, 2, 100, 16, 20, 10 ** 6) == attn.evict_workspace_bytes(4, 2, 100, 16, 20, 320)
    for args, status in (((0, 2, 100, 16, 20, 64), INVALID), ((4, 2, 100, 16, 20, 0), INVALID),
                         ((1 << 28, 2, 100, 16, 20, 64), LARGE), ((4, 2, 100, 16, 1 << 27, 64), LARGE)):
        with pytest.raises(attn.AttnError) as e:
            attn.evict_workspace_bytes(*args)
        assert e.value.status == status


def test_python_refusals():
    bf = torch.zeros(8, 16, 2, 128, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_cache_evict(bf, bf, i(2, 4), i(2), torch.zeros(2, 2, 64), 8, layout="sbhd")
    with pytest.raises(TypeError):
        attn.attn_cache_evict(bf, bf, i(2, 4), i(2), torch.zeros(2, 2, 64), 8, layout="bshd")  # not on a GPU
