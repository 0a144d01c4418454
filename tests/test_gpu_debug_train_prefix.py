"""The debug flavour of the library on the training and shared-prefix calls: its checks stay silent
and the results equal the release build's bit for bit."""
import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _libraries():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    build.build(debug=True)
    attn.load_library(debug=False)
    attn.load_library(debug=True)


def _same_in_both(monkeypatch, fn):
    got = []
    for debug in ("0", "1"):
        monkeypatch.setenv("ATTN_FWD_DEBUG", debug)
        assert attn.load_library().attn_fwd_debug_build() == int(debug)
        got.append(fn())
        torch.cuda.synchronize()
        assert attn.attn_fwd_last_error() == attn.ATTN_OK
    for a, b in zip(*got):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("layout,B,Hq,Hkv,Sq,Sk", [
    ("bshd", 2, 6, 2, 300, 517),      # tiles shared between CTAs
    ("bhsd", 4, 16, 16, 600, 640),    # several items a CTA
    ("bshd", 2, 96, 96, 500, 77),     # forward: the persistent form
    ("bhsd", 1, 1, 1, 1, 1),
    ("bshd", 1, 1, 1, 34000, 33000),  # several accumulators
])
def test_training(monkeypatch, layout, B, Hq, Hkv, Sq, Sk, causal):
    r = _rand(Sq + Sk)
    sh = lambda H, S: (B, S, H, 128) if layout == "bshd" else (B, H, S, 128)
    q, k, v, do = r(*sh(Hq, Sq)), r(*sh(Hkv, Sk)), r(*sh(Hkv, Sk)), r(*sh(Hq, Sq))

    def step():
        out, lse = attn.attn_fwd_lse(q, k, v, layout=layout, causal=causal)
        return (out, lse, *attn.attn_bwd(do, q, k, v, out, lse, layout=layout, causal=causal))

    if causal and Sq > Sk:  # rows without keys: NaN outputs, whose bits are one pattern
        assert torch.isnan(step()[0]).any()
    _same_in_both(monkeypatch, step)


@pytest.mark.parametrize("causal", [False, True])
def test_packed_training(monkeypatch, causal):
    r = _rand(3)
    cu = torch.tensor([0, 130, 130, 700, 1500], dtype=torch.int32, device="cuda")
    q, k, v, do = r(1500, 6, 128), r(1500, 3, 128), r(1500, 3, 128), r(1500, 6, 128)

    def step():
        out, lse = attn.attn_fwd_varlen_lse(q, k, v, cu, cu, 800, causal=causal)
        return (out, lse, *attn.attn_bwd_varlen(do, q, k, v, out, lse, cu, cu, 800, 800, causal=causal))

    _same_in_both(monkeypatch, step)


@pytest.mark.parametrize("layout,B,Sq,Hq,Hkv,Sp,cap", [
    ("bshd", 3, 1, 8, 2, 300, 64),       # few rows: two launches
    ("bhsd", 40, 2, 14, 2, 900, 333),    # the fused kernel takes the prefix
    ("bshd", 4, 5, 28, 4, 0, 500),       # no prefix, two blocks of rows
    ("bhsd", 1, 1, 304, 304, 0, 20000),  # long parts
    ("bshd", 1, 1, 1, 1, 1, 1),
])
def test_prefix(monkeypatch, layout, B, Sq, Hq, Hkv, Sp, cap):
    r = _rand(Sp + cap)
    bshd = layout == "bshd"
    q = r(B, Sq, Hq, 128) if bshd else r(B, Hq, Sq, 128)
    k, v = ((r(B, cap, Hkv, 128), r(B, cap, Hkv, 128)) if bshd else (r(B, Hkv, cap, 128), r(B, Hkv, cap, 128)))
    kp = vp = None
    if Sp:
        kp, vp = (r(Sp, Hkv, 128), r(Sp, Hkv, 128)) if bshd else (r(Hkv, Sp, 128), r(Hkv, Sp, 128))
    n = torch.tensor([max(1, cap - 13 * b) for b in range(B)], dtype=torch.int32, device="cuda")
    for causal in (False, True):
        _same_in_both(monkeypatch, lambda: attn.attn_fwd_prefix(q, kp, vp, k, v, n, causal=causal, layout=layout))
