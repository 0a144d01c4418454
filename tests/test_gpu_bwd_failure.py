"""The backward kernels' bounded waits, without a fault: a launch in which one signal is waited for
once more than it is sent (20 ms limit) stops by itself, reports ATTN_ERR_TIMEOUT once, stores no
result of its own, and leaves the context and the next call as they should be."""
import ctypes
import math
import time

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


# One item a CTA; masked tiles and their check; many items, of which a CTA has claimed another when
# it gives up; items of more than one accumulator's tiles.
@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("B,H,Sq,Sk,causal", [(1, 2, 256, 256, False), (1, 2, 300, 300, True), (4, 16, 640, 640, True),
                                              (4, 16, 640, 640, False), (1, 1, 33100, 33100, True)])
def test_withheld_signal_times_out_cleanly(B, H, Sq, Sk, causal, kernel):
    g = torch.Generator(device="cuda").manual_seed(Sq)
    r = lambda s: torch.randn(B, H, s, 128, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v, do = r(Sq), r(Sk), r(Sk), r(Sq)
    out, lse = attn.attn_fwd_lse(q, k, v, causal=causal)
    want = attn.attn_bwd(do, q, k, v, out, lse, causal=causal)
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
    ws = torch.zeros(attn.bwd_workspace_bytes(B, H, H, Sq, Sk), dtype=torch.uint8, device="cuda")
    t0 = time.time()
    st = attn.load_library().attn_bwd_timeout_selftest(
        *(x.data_ptr() for x in (do, q, k, v, out, lse, *grads)), 0, B, H, H, Sq, Sk, 128, ctypes.c_float(SCALE), 0,
        attn.ATTN_FLAG_CAUSAL if causal else 0, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream,
        20_000_000, kernel)
    assert st == attn.ATTN_OK
    torch.cuda.synchronize()
    assert time.time() - t0 < 10.0
    assert attn.attn_fwd_last_error() == attn.ATTN_ERR_TIMEOUT
    assert attn.attn_fwd_last_error() == attn.ATTN_OK  # reading clears it
    # (Where tiles are shared, or sums added up in the workspace, the join rounds what lies there.)
    if ws.numel() == B * H * ((Sq + 127) // 128) * 1024:
        assert all((x == 7.0).all() for x in (grads[:1] if kernel == 0 else grads[1:]))
    again = attn.attn_bwd(do, q, k, v, out, lse, causal=causal, workspace=ws)
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    for a, b in zip(again, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
