"""Packed batches whose offsets are far out of range: the sequences beside them are computed, the
others left as they were, and the status reports them."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _grad

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)
LO, HI = -(1 << 31), (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


@pytest.mark.parametrize("which", ["q", "k", "both"])
@pytest.mark.parametrize("causal", [False, True])
def test_far_offsets(which, causal):
    g = torch.Generator().manual_seed(31)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    n, H = 400, 2
    q, k, v, do = r(n, H, 128), r(n, H, 128), r(n, H, 128), r(n, H, 128)
    Q, K, V, DO = (t.cuda() for t in (q, k, v, do))
    # Sequences 1 to 3 are invalid: to 2^31 - 1, from there to -2^31 (one token, where sums wrap), and from there.
    far = torch.tensor([0, 100, HI, LO, 300, 400], dtype=torch.int32).cuda()
    near = torch.tensor([0, 100, 150, 200, 300, 400], dtype=torch.int32).cuda()
    cu_q, cu_k = (far if which != "k" else near), (far if which != "q" else near)

    def reported():
        torch.cuda.synchronize()
        assert attn.attn_fwd_last_error() == attn.ATTN_ERR_SEQLENS
        assert attn.attn_fwd_last_error() == attn.ATTN_OK

    out, lse = torch.full_like(Q, 9.0), torch.full((H, n), 9.0, device="cuda")
    attn.attn_fwd_varlen(Q, K, V, cu_q, cu_k, 100, causal=causal, out=out)
    reported()
    assert (out[100:300] == 9.0).all()
    attn.attn_fwd_varlen_lse(Q, K, V, cu_q, cu_k, 100, causal=causal, out=out, lse=lse)
    reported()
    assert (out[100:300] == 9.0).all() and (lse[:, 100:300] == 9.0).all()
    grads = [torch.full_like(Q, 9.0) for _ in range(3)]
    attn.attn_bwd_varlen(DO, Q, K, V, out, lse, cu_q, cu_k, 100, 100, causal=causal, dq=grads[0], dk=grads[1],
                         dv=grads[2])
    reported()
    for x in grads:
        assert (x[100:300] == 9.0).all()
    for s in (slice(0, 100), slice(300, 400)):
        want, bound = _grad.sequence(q[s], k[s], v[s], do[s], SCALE, causal)
        assert ((lse[:, s].cpu().double() - want["lse"]).abs() <= 1e-4).all()
        for name, x in zip(("dq", "dk", "dv"), grads):
            _grad.check(name, x[s], want[name], bound[name])
