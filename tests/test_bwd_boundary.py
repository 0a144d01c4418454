"""attn_fwd_lse, attn_bwd and their packed forms without a GPU: bad arguments are
refused on the host before any launch, and workspace sizes cannot overflow. The
gradient formulas that the GPU tests use are checked against autograd."""
import ctypes
import math
import shutil

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _grad


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


def _lse(lib, q=A, k=2 * A, v=3 * A, o=4 * A, l=5 * A, layout=0, B=1, Hq=4, Hkv=2, Sq=300, Sk=200, d=128,
         scale=0.1, mode=0, flags=0):
    return lib.attn_fwd_lse(q, k, v, o, l, layout, B, Hq, Hkv, Sq, Sk, d, ctypes.c_float(scale), mode, flags, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(l=0), INVALID), (dict(q=0), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(scale=math.nan), INVALID), (dict(d=64), UNSUPPORTED), (dict(flags=2), UNSUPPORTED),
    (dict(flags=4), UNSUPPORTED), (dict(mode=3), UNSUPPORTED), (dict(l=5 * A + 2), MISALIGNED),
    (dict(l=4 * A + 1024), ALIASING), (dict(l=A), ALIASING), (dict(o=2 * A), ALIASING),
    (dict(Sq=1 << 31), LARGE),
])
def test_lse_refusals(lib, kw, status):
    assert _lse(lib, **kw) == status


def _bwd(lib, do=A, q=2 * A, k=3 * A, v=4 * A, o=5 * A, l=6 * A, dq=7 * A, dk=8 * A, dv=9 * A, layout=0, B=1,
         Hq=4, Hkv=2, Sq=300, Sk=200, d=128, scale=0.1, mode=0, flags=0, ws=10 * A, ws_bytes=1 << 29):
    return lib.attn_bwd(do, q, k, v, o, l, dq, dk, dv, layout, B, Hq, Hkv, Sq, Sk, d, ctypes.c_float(scale), mode,
                        flags, ws, ws_bytes, 0)


@pytest.mark.parametrize("kw,status", [
    *[({n: 0}, INVALID) for n in ("do", "q", "k", "v", "o", "l", "dq", "dk", "dv", "ws")],
    (dict(B=0), INVALID), (dict(Hq=5), INVALID), (dict(Hkv=0), INVALID), (dict(Sq=0), INVALID),
    (dict(Sk=-1), INVALID), (dict(scale=math.inf), INVALID), (dict(ws_bytes=100), INVALID),
    (dict(d=256), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(mode=-1), UNSUPPORTED),
    (dict(flags=2), UNSUPPORTED), (dict(dq=7 * A + 8), MISALIGNED), (dict(ws=10 * A + 4), MISALIGNED),
    (dict(l=6 * A + 2), MISALIGNED), (dict(dq=A), ALIASING), (dict(dk=8 * A, dv=8 * A + 1024), ALIASING),
    (dict(ws=6 * A), ALIASING), (dict(dv=5 * A), ALIASING), (dict(dq=8 * A), ALIASING),
    (dict(Sq=1 << 31), LARGE), (dict(B=1 << 20, Hq=1 << 12, Hkv=1 << 12), LARGE),
    (dict(Hq=1 << 20, Hkv=1 << 20, Sq=1 << 20), LARGE),
])
def test_bwd_refusals(lib, kw, status):
    assert _bwd(lib, **kw) == status


def _varlen(lib, do=A, q=2 * A, k=3 * A, v=4 * A, o=5 * A, l=6 * A, dq=7 * A, dk=8 * A, dv=9 * A, cq=11 * A,
            ck=12 * A, B=3, Hq=4, Hkv=2, tq=300, tk=200, mq=100, mk=100, d=128, scale=0.1, mode=0, flags=0,
            ws=10 * A, ws_bytes=1 << 29):
    return lib.attn_bwd_varlen(do, q, k, v, o, l, dq, dk, dv, cq, ck, B, Hq, Hkv, tq, tk, mq, mk, d,
                               ctypes.c_float(scale), mode, flags, ws, ws_bytes, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(cq=0), INVALID), (dict(ck=0), INVALID), (dict(mq=0), INVALID), (dict(mq=301), INVALID),
    (dict(mk=201), INVALID), (dict(tq=0), INVALID), (dict(ws_bytes=0), INVALID), (dict(cq=11 * A + 1), MISALIGNED),
    (dict(dq=11 * A), ALIASING), (dict(ws=12 * A), ALIASING), (dict(tk=1 << 31), LARGE),
    (dict(B=1 << 30), LARGE),
])
def test_bwd_varlen_refusals(lib, kw, status):
    assert _varlen(lib, **kw) == status


def test_good_arguments_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake")
    none = attn.ATTN_ERR_NO_DEVICE
    assert _lse(lib) == none and _bwd(lib) == none and _varlen(lib) == none


def test_workspace_sizes(lib):
    assert attn.bwd_workspace_bytes(1, 2, 2, 128, 128) >= 2 * 1024
    for args in [(1, 3, 2, 8, 8), (0, 2, 2, 8, 8), (1, 2, 2, 8, 0)]:
        with pytest.raises(attn.AttnError) as e:
            attn.bwd_workspace_bytes(*args)
        assert e.value.status == INVALID
    with pytest.raises(attn.AttnError) as e:
        attn.bwd_workspace_bytes(1 << 30, 1 << 10, 1 << 10, 1 << 10, 1 << 10)
    assert e.value.status == LARGE
    # Large but allowed sizes: positive, and at least the statistics' bytes.
    n = attn.bwd_workspace_bytes(1, 8, 8, 1 << 20, 1 << 20)
    assert n >= 8 * (1 << 20) * 8
    assert attn.bwd_varlen_workspace_bytes(5, 4, 2, 1000, 900, 300, 300) >= 4 * (1000 // 128 + 6) * 1024


@pytest.mark.parametrize("Sq,Sk,causal,g", [(5, 7, False, 1), (6, 6, True, 2), (9, 4, True, 1), (1, 1, False, 3)])
def test_reference_against_autograd(Sq, Sk, causal, g):
    gen = torch.Generator().manual_seed(Sq * 10 + Sk)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    q, k, v, do = r(Sq, 2 * g, 128), r(Sk, 2, 128), r(Sk, 2, 128), r(Sq, 2 * g, 128)
    got, _ = _grad.sequence(q, k, v, do, 0.1, causal)
    q, k, v = (t.requires_grad_() for t in (q, k, v))
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(g, 1)) * 0.1
    s = s.masked_fill(~_grad.visible(Sq, Sk, causal), -math.inf)
    rows = torch.isfinite(s).any(-1)[0]          # rows that see a key
    o = torch.einsum("hij,jhd->ihd", torch.softmax(s[:, rows], -1), v.repeat_interleave(g, 1))
    o.backward(do[rows])
    for n, t in (("dq", q), ("dk", k), ("dv", v)):
        assert torch.allclose(got[n], t.grad, rtol=1e-10, atol=1e-12), n
    assert (got["dq"][~rows] == 0).all()


@pytest.mark.parametrize("make,exc", [
    (lambda q, l: attn.attn_fwd_lse(q.float(), q, q), TypeError),
    (lambda q, l: attn.attn_fwd_lse(q, q, q), TypeError),                 # not on a GPU
    (lambda q, l: attn.attn_bwd(q, q, q, q, q, l), TypeError),
    (lambda q, l: attn.attn_fwd_lse(q, q, q, layout="hsbd"), ValueError),
    (lambda q, l: attn.attn_bwd(q, q, q, q, q, l, rounding="up"), ValueError),
    (lambda q, l: attn.attn_bwd_varlen(q[0], q[0], q[0], q[0], q[0], l, None, None, 1, 1), TypeError),
])
def test_python_refusals(make, exc):
    q = torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(exc):
        make(q, torch.zeros(1, 2, 8))
