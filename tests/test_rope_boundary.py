"""The norm-and-rotation calls without a GPU: bad arguments are refused on the host before any
launch."""
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
OK = attn.ATTN_ERR_NO_DEVICE  # good arguments get as far as the device


def _at(x):
    return None if x is None else (ctypes.c_int64 * 3)(*x)


def _fwd(lib, q=A, k=2 * A, wq=3 * A, wk=4 * A, cos=5 * A, sin=6 * A, pos=7 * A, qo=8 * A, ko=9 * A, B=2, S=64, Hq=8,
         Hkv=2, d=128, max_pos=100, rot=128, eps=1e-6, mode=0, flags=0, q_at="", k_at="", qo_at="", ko_at=""):
    dense = lambda H: (S * H * 128, H * 128, 128)
    q_at, qo_at = (dense(Hq) if x == "" else x for x in (q_at, qo_at))
    k_at, ko_at = (dense(Hkv) if x == "" else x for x in (k_at, ko_at))
    return lib.attn_qk_norm_rope(q, k, wq, wk, cos, sin, pos, qo, ko, _at(q_at), _at(k_at), _at(qo_at), _at(ko_at), B,
                                 S, Hq, Hkv, d, max_pos, rot, ctypes.c_float(eps), mode, flags, 0)


BAD = [
    *[({x: 0}, INVALID) for x in ("q", "k", "wq", "wk", "cos", "sin", "pos")],
    (dict(q_at=None), INVALID), (dict(B=0), INVALID), (dict(S=0), INVALID), (dict(Hq=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(max_pos=0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=-1e-9), INVALID),
    (dict(d=64), UNSUPPORTED), (dict(rot=0), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=144), UNSUPPORTED),
    (dict(flags=1), UNSUPPORTED), (dict(mode=3), UNSUPPORTED),
    (dict(B=1 << 16, S=1 << 16), LARGE), (dict(Hq=(1 << 20) + 1), LARGE), (dict(max_pos=1 << 31), LARGE),
    (dict(q_at=((1 << 40) - 8, (1 << 40) - 8, 128), S=1 << 20), LARGE), (dict(q_at=(1 << 40, 1024, 128)), INVALID),
    (dict(q_at=(65536, -1024, 128)), INVALID),
    (dict(q=A + 8), MISALIGNED), (dict(cos=5 * A + 8), MISALIGNED), (dict(wq=3 * A + 2), MISALIGNED),
    (dict(pos=7 * A + 2), MISALIGNED), (dict(k_at=(64 * 260, 260, 128)), MISALIGNED),
]


@pytest.mark.parametrize("kw,status", BAD + [
    (dict(qo=0), INVALID), (dict(ko=0), INVALID), (dict(ko_at=None), INVALID),
    (dict(qo=2 * A), ALIASING), (dict(qo=7 * A), ALIASING), (dict(ko=A + 4096), ALIASING), (dict(ko=8 * A), ALIASING),
    (dict(qo=A + 16), ALIASING), (dict(qo_at=(0, 1024, 128)), ALIASING), (dict(ko_at=(64 * 256, 256, 64)), ALIASING),
    (dict(qo=A, qo_at=(64 * 1024, 2048, 128)), ALIASING),
])
def test_forward_refusals(lib, kw, status):
    assert _fwd(lib, **kw) == status


def test_good_arguments_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    assert _fwd(lib) == OK
    assert _fwd(lib, qo=A, ko=2 * A) == OK                      # in place
    one = (64 * 1536, 1536, 128)                                # columns of one projection's output
    assert _fwd(lib, k=A + 2048, q_at=one, k_at=one) == OK
    assert _fwd(lib, k=A + 2048, q_at=one, k_at=one, qo=A, ko=A + 2048, qo_at=one, ko_at=one) == OK
    assert _fwd(lib, q_at=(0, 1024, 128)) == OK                 # a batch that shares its queries
    assert _fwd(lib, B=1, S=1, Hkv=1, k_at=(3, 5, 7)) == OK     # one row: no stride is looked at
    assert _paged(lib) == OK
    assert _paged(lib, vp=11 * A + 64 * 2 * 256, stride=2 * 64 * 2 * 128, kp=11 * A) == OK
    assert _bwd(lib) == OK
    assert _bwd(lib, dq=A, dk=2 * A) == OK


def _paged(lib, kp=11 * A, vp=12 * A, n=32, page=64, stride=64 * 2 * 128, layout=1, v=10 * A, slots=13 * A, qo=8 * A,
           Hkv=2, pos=7 * A):
    B, S, Hq = 2, 64, 8
    q_at, k_at = _at((S * Hq * 128, Hq * 128, 128)), _at((S * Hkv * 128, Hkv * 128, 128))
    return lib.attn_qk_norm_rope_paged(A, 2 * A, v, 3 * A, 4 * A, 5 * A, 6 * A, pos, slots, qo, kp, vp, q_at, k_at,
                                       k_at, q_at, layout, B, S, Hq, Hkv, n, page, stride, 128, 100, 128,
                                       ctypes.c_float(1e-6), 0, 0, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(kp=0), INVALID), (dict(vp=0), INVALID), (dict(v=0), INVALID), (dict(slots=0), INVALID),
    (dict(n=0), INVALID), (dict(page=0), INVALID), (dict(stride=64 * 2 * 128 - 128), INVALID),
    (dict(layout=2), UNSUPPORTED), (dict(kp=11 * A + 8), MISALIGNED), (dict(stride=64 * 2 * 128 + 8), MISALIGNED),
    (dict(slots=13 * A + 1), MISALIGNED),
    (dict(n=1 << 26), LARGE), (dict(page=1 << 31), LARGE), (dict(stride=1 << 40), LARGE),
    (dict(vp=11 * A), ALIASING), (dict(vp=11 * A + 256), ALIASING), (dict(kp=10 * A), ALIASING),
    (dict(kp=13 * A), ALIASING), (dict(qo=12 * A), ALIASING), (dict(qo=10 * A), ALIASING), (dict(kp=A), ALIASING),
    (dict(kp=3 * A), ALIASING),
])
def test_paged_refusals(lib, kw, status):
    assert _paged(lib, **kw) == status


def _bwd(lib, gq=A, gk=2 * A, q=14 * A, k=15 * A, dq=8 * A, dk=9 * A, dwq=16 * A, dwk=17 * A, ws=18 * A,
         ws_bytes=1 << 24, gq_at="", dk_at="", S=64, Hq=8):
    B, Hkv = 2, 2
    dense = lambda H: (S * H * 128, H * 128, 128)
    q_at, k_at = _at(dense(Hq)), _at(dense(Hkv))
    gq_at, dk_at = (y if x == "" else _at(x) for x, y in ((gq_at, q_at), (dk_at, k_at)))
    return lib.attn_qk_norm_rope_bwd(gq, gk, q, k, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A, dq, dk, dwq, dwk, gq_at, k_at,
                                     q_at, k_at, q_at, dk_at, B, S, Hq, Hkv, 128, 100, 128, ctypes.c_float(1e-6), 0,
                                     0, ws, ws_bytes, 0)


@pytest.mark.parametrize("kw,status", [
    *[({x: 0}, INVALID) for x in ("gq", "gk", "q", "k", "dq", "dk", "dwq", "dwk", "ws")],
    (dict(ws_bytes=1000), INVALID), (dict(gq_at=None), INVALID),
    (dict(dwq=16 * A + 2), MISALIGNED), (dict(ws=18 * A + 4), MISALIGNED), (dict(gq=A + 2), MISALIGNED),
    (dict(dq=14 * A), ALIASING), (dict(dk=15 * A), ALIASING), (dict(dk=A), ALIASING), (dict(dq=9 * A), ALIASING),
    (dict(dwq=17 * A), ALIASING), (dict(dwk=3 * A), ALIASING), (dict(ws=8 * A), ALIASING), (dict(ws=7 * A), ALIASING),
    (dict(dk_at=(0, 256, 128)), ALIASING),
])
def test_backward_refusals(lib, kw, status):
    assert _bwd(lib, **kw) == status


def test_workspace_sizes(lib):
    assert attn.qk_norm_rope_bwd_workspace_bytes(1, 1, 1, 1) == 1024
    assert attn.qk_norm_rope_bwd_workspace_bytes(8, 8192, 32, 8) >= 1024
    for args, status in (((0, 1, 1, 1), INVALID), ((1, 1, 0, 1), INVALID), ((1, 1, 1, 1, 64), UNSUPPORTED),
                         ((1 << 20, 1 << 20, 1, 1), LARGE), ((1, 1, 1 << 21, 1), LARGE)):
        with pytest.raises(attn.AttnError) as e:
            attn.qk_norm_rope_bwd_workspace_bytes(*args)
        assert e.value.status == status


@pytest.mark.parametrize("change,exc", [
    (dict(layout="sbhd"), ValueError), (dict(rounding="up"), ValueError), (dict(), TypeError),  # not on a GPU
])
def test_python_refusals(change, exc):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q, k, w, t = bf(5, 4, 128), bf(5, 2, 128), bf(128), torch.zeros(9, 64)
    at = torch.zeros(5, dtype=torch.int32)
    kw = {"layout": "bshd", **change}
    with pytest.raises(exc):
        attn.attn_qk_norm_rope(q, k, w, w, t, t, at, **kw)
    with pytest.raises(exc):
        attn.attn_qk_norm_rope_bwd(q, k, q, k, w, w, t, t, at, **kw)
    with pytest.raises(exc):
        attn.attn_qk_norm_rope_paged(q, k, k, w, w, t, t, at, at, bf(3, 4, 2, 128), bf(3, 4, 2, 128), **kw)


def test_arguments_of_the_wrong_type():
    """Errors of the compiled binding arrive as Python's own, before any tensor is looked at."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    q, k, w, t, at = bf(5, 4, 128), bf(5, 2, 128), bf(128), torch.zeros(9, 64), torch.zeros(5, dtype=torch.int32)
    for eps in ("small", None, [1e-6]):
        with pytest.raises(TypeError):
            attn.attn_qk_norm_rope(q, k, w, w, t, t, at, eps=eps)
    for bad in (None, 3, "q", q.numpy if hasattr(q, "numpy") else object()):
        with pytest.raises(TypeError):
            attn.attn_qk_norm_rope(bad, k, w, w, t, t, at)
    with pytest.raises((TypeError, ValueError)):
        attn.attn_fwd_paged(bf(1, 1, 2, 128), None, None, None, None)
    with pytest.raises((TypeError, ValueError)):
        attn.attn_cache_evict(bf(3, 2, 4, 128), bf(3, 2, 4, 128), None, None, None, "all")
