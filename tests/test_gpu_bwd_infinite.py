"""Backward pass of rows whose logits are infinite: the definition makes their gradients, and
those of the keys that they see, NaN; the others keep their bits."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


def _step(q, k, v, do, cu=None, **kw):
    if cu is None:
        out, lse = attn.attn_fwd_lse(q, k, v, layout="bshd", **kw)
        grads = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd", **kw)
    else:
        out, lse = attn.attn_fwd_varlen_lse(q, k, v, *cu, 200, **kw)
        grads = attn.attn_bwd_varlen(do, q, k, v, out, lse, *cu, 200, 200, **kw)
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    return out, lse, grads


def _inputs(Sq, Sk, H=1, seed=51):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    return [r(1, Sq, H, 128), r(1, Sk, H, 128), r(1, Sk, H, 128), r(1, Sq, H, 128)]


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("packed", [False, True])
def test_a_row_of_one_key(packed):
    """Causal: row 0 sees key 0 alone and its logit is -Inf. A softmax over -Inf alone is NaN."""
    S = 200
    q, k, v, do = _inputs(S, S)
    q[0, 0, 0, 5], k[0, 0, 0, 5] = 1.0, -1.0
    t = [x.cuda() for x in (q, k, v, do)]
    cu = None
    if packed:  # a second sequence, whose first row is like that as well
        t = [torch.cat([x[0], x[0, :70]]) for x in t]
        cu = [torch.tensor([0, S, S + 70], dtype=torch.int32, device="cuda")] * 2
    row = lambda x, i: x[i] if packed else x[0, i]
    clean = _step(*t, cu, causal=True)[2]
    rows = [0, S] if packed else [0]
    for i in rows:
        row(t[0], i)[0, 5] = math.inf
    out, lse, grads = _step(*t, cu, causal=True)
    n = out.shape[0 if packed else 1]
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[rows] = False
    for i in rows:
        assert torch.isnan(row(out, i)).all()
        assert (lse[:, i] if packed else lse[0, :, i]).item() == -math.inf
        for name, g in zip(("dq", "dk", "dv"), grads):
            assert torch.isnan(row(g, i)).all(), name
    for name, g, c in zip(("dq", "dk", "dv"), grads, clean):
        g, c = (g, c) if packed else (g[0], c[0])
        assert _same(g[keep], c[keep]), name


@pytest.mark.parametrize("Sq,Sk,causal", [(150, 130, False), (4000, 60, False), (50, 4000, False), (300, 300, True)])
def test_every_logit_of_a_row(Sq, Sk, causal):
    """One row's visible logits are all -Inf (its query is infinite in a column where every key is
    negative); tiles shared between CTAs among the sizes."""
    at = Sq // 2
    q, k, v, do = _inputs(Sq, Sk)
    k[0, :, 0, 9] = -k[0, :, 0, 9].abs() - 0.25
    t = [x.cuda() for x in (q, k, v, do)]
    clean = _step(*t, causal=causal)[2]
    t[0][0, at, 0, 9] = math.inf
    out, lse, (dq, dk, dv) = _step(*t, causal=causal)
    assert lse[0, 0, at].item() == -math.inf and torch.isnan(out[0, at]).all()
    keys = torch.arange(Sk, device="cuda") <= (at if causal else Sk)
    assert torch.isnan(dq[0, at]).all()
    assert torch.isnan(dk[0, keys]).all() and torch.isnan(dv[0, keys]).all()
    others = torch.arange(Sq, device="cuda") != at
    assert _same(dq[0, others], clean[0][0, others])
    assert torch.isfinite(dk[0, ~keys]).all() and _same(dk[0, ~keys], clean[1][0, ~keys])
    assert _same(dv[0, ~keys], clean[2][0, ~keys])


def test_rows_without_keys_stay_out():
    """Sq > Sk under the mask: rows that see no key have lse -Inf too, whatever they hold."""
    Sq, Sk = 300, 130
    q, k, v, do = (x.cuda() for x in _inputs(Sq, Sk))
    clean = _step(q, k, v, do, causal=True)[2]
    q[0, :Sq - Sk, 0, 3] = math.inf
    dq, dk, dv = _step(q, k, v, do, causal=True)[2]
    assert (dq[0, :Sq - Sk] == 0).all()
    for a, b in zip((dq, dk, dv), clean):
        assert _same(a, b)
