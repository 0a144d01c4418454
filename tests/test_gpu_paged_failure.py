"""The paged attention's bounded waits, without a fault: a launch whose runs never hear of their first
products (20 ms limit) stops by itself, reports ATTN_ERR_TIMEOUT once, stores no result, and leaves the
context and the next call as they should be."""
import ctypes
import time

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


# One item; items cut between CTAs; many items a CTA; 20, 35 and 80 rows.
@pytest.mark.parametrize("B,Sq,Hq,Hkv,per,lens", [(1, 5, 4, 1, 4, [60]), (2, 5, 28, 4, 100, [1600, 900]),
                                                  (60, 20, 4, 1, 3, None)])
def test_withheld_signal_times_out_cleanly(B, Sq, Hq, Hkv, per, lens):
    page = 16
    lens = lens or [1 + i % (page * per) for i in range(B)]
    t = [torch.tensor(x, dtype=torch.int32).cuda() if isinstance(x, list) else x.cuda()
         for x in _paged.inputs("bshd", B, Sq, Hq, Hkv, page, per, lens, seed=80)]
    q, kp, vp, table, n = t
    want = attn.attn_fwd_paged(*t, layout="bshd")
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    out, lse = torch.full_like(q, 7.0), torch.full((B, Hq, Sq), 7.0, device="cuda")
    ws = torch.zeros(attn.paged_workspace_bytes(B, Hq, Hkv, Sq, page, per), dtype=torch.uint8, device="cuda")
    t0 = time.time()
    st = attn.load_library().attn_fwd_paged_timeout_selftest(
        *(x.data_ptr() for x in (q, kp, vp, table, n, out, lse)), None, 1, B, Hq, Hkv, Sq, kp.shape[0], page,
        kp.stride(0), per, 128, ctypes.c_float(_paged.SCALE), 0, 0, ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream, 20_000_000)
    assert st == attn.ATTN_OK
    torch.cuda.synchronize()
    assert time.time() - t0 < 10.0
    assert attn.attn_fwd_last_error() == attn.ATTN_ERR_TIMEOUT
    assert attn.attn_fwd_last_error() == attn.ATTN_OK  # reading clears it
    assert (out == 7.0).all() and (lse == 7.0).all()
    again = attn.attn_fwd_paged(*t, layout="bshd", workspace=ws)
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    for a, b in zip(again, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
