"""Backward pass with more tiles than SMs: each CTA takes over further items, of several streamed
tiles each, with the barriers' phases, the rings and the record of non-finite elements carried from
one to the next."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _grad

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


def _inputs(B, Sq, Sk, Hq, Hkv, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    return [r(B, Sq, Hq, 128), r(B, Sk, Hkv, 128), r(B, Sk, Hkv, 128), r(B, Sq, Hq, 128)]


def _several_items_a_cta(B, Sq, Sk, Hq, Hkv):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = lambda n: (n + 127) // 128
    assert B * Hq * tiles(Sq) > 2 * sms and B * Hkv * tiles(Sk) > 2 * sms
    # No tile is shared: the workspace holds the row statistics alone.
    assert attn.bwd_workspace_bytes(B, Hq, Hkv, Sq, Sk) == B * Hq * tiles(Sq) * 1024


def _run(q, k, v, do, **kw):
    out, lse = attn.attn_fwd_lse(q, k, v, layout="bshd", **kw)
    grads = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd", **kw)
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    return grads


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hkv", [
    (4, 640, 640, 16, 16),
    (4, 600, 700, 32, 16),   # ragged, grouped
    (5, 900, 650, 12, 12),   # the mask leaves rows without keys
])
def test_gradients(B, Sq, Sk, Hq, Hkv, causal):
    _several_items_a_cta(B, Sq, Sk, Hq, Hkv)
    t = _inputs(B, Sq, Sk, Hq, Hkv, seed=Sq + Sk)
    grads = _run(*(x.cuda() for x in t), causal=causal)
    for b in range(B):
        want, bound = _grad.sequence(*(x[b] for x in t), SCALE, causal)
        for n, g in zip(("dq", "dk", "dv"), grads):
            _grad.check(f"{n}[{b}]", g[b], want[n], bound[n])


@pytest.mark.parametrize("causal", [False, True])
def test_packed(causal):
    B, S, H = 20, 400, 6
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert B * H * 4 > 2 * sms
    lens = [S - 7 * b for b in range(B)]
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    n = int(cu[-1])
    t = [x[0] for x in _inputs(1, n, n, H, H, seed=71)]
    q, k, v, do = (x.cuda() for x in t)
    c = cu.cuda()
    out, lse = attn.attn_fwd_varlen_lse(q, k, v, c, c, S, causal=causal)
    grads = attn.attn_bwd_varlen(do, q, k, v, out, lse, c, c, S, S, causal=causal)
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    for b in range(B):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        want, bound = _grad.sequence(*(x[rows] for x in t), SCALE, causal)
        for name, g in zip(("dq", "dk", "dv"), grads):
            _grad.check(f"{name} of sequence {b}", g[rows], want[name], bound[name])


@pytest.mark.parametrize("where", ["k", "do"])
def test_non_finite_values_stay_with_their_head(where):
    """Causal: NaN and infinities in every third head, in masked tiles (where they are taken out and
    recorded) and elsewhere. The other heads' gradients keep their bits, and the record of one item does
    not reach the next: rows and keys that see none of the values stay finite."""
    B, S, H = 4, 640, 16
    _several_items_a_cta(B, S, S, H, H)
    t = [x.cuda() for x in _inputs(B, S, S, H, H, seed=72)]
    clean = _run(*t, causal=True)
    hit = torch.zeros(B, H, dtype=torch.bool, device="cuda")
    hit.view(-1)[::3] = True
    at, col = 300, 17                     # the third tile: masked for its own rows, whole for later ones
    x = t[1] if where == "k" else t[3]
    x[:, at, :, col] = torch.where(hit, torch.tensor(math.nan, dtype=x.dtype, device="cuda"), x[:, at, :, col])
    dq, dk, dv = _run(*t, causal=True)
    for g, c in zip((dq, dk, dv), clean):
        g, c = g.transpose(1, 2)[~hit], c.transpose(1, 2)[~hit]
        assert torch.equal(g.view(torch.int16), c.view(torch.int16))
    dq, dk, dv = (g.transpose(1, 2)[hit] for g in (dq, dk, dv))   # (heads, S, 128)
    cq, ck, cv = (g.transpose(1, 2)[hit] for g in clean)
    if where == "k":                      # the rows that see the key have a NaN logit, and all keys see such a row
        assert torch.isnan(dq[:, at:]).all()
        assert torch.equal(dq[:, :at].view(torch.int16), cq[:, :at].view(torch.int16))
        assert torch.isnan(dk).all() and torch.isnan(dv).all()
    else:
        rest = [r for r in range(S) if r != at]
        assert torch.isnan(dq[:, at]).all()
        assert torch.equal(dq[:, rest].view(torch.int16), cq[:, rest].view(torch.int16))
        assert torch.isnan(dk[:, :at + 1]).all() and torch.isnan(dv[:, :at + 1, col]).all()
        others = [c for c in range(128) if c != col]
        assert torch.isfinite(dv[:, :, others]).all()
        assert torch.equal(dk[:, at + 1:].view(torch.int16), ck[:, at + 1:].view(torch.int16))
        assert torch.equal(dv[:, at + 1:].view(torch.int16), cv[:, at + 1:].view(torch.int16))
