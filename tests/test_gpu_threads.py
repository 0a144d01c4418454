"""Calls of the compiled binding from several threads at once. What goes wrong in a thread (an error that is
raised, or one that is not) fails the test."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _paged
import _rope

pytestmark = pytest.mark.gpu

THREADS, TIMES = 4, 25


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


def _case():
    t = _paged.inputs("bshd", 4, 1, 8, 2, 16, 20, [320, 1, 77, 200], seed=90)
    q, kp, vp, table, _ = (x.cuda() if torch.is_tensor(x) else x for x in t)
    lens = torch.tensor(t[4], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(91)
    x, y = (torch.randn(33, h, 128, generator=g).to(torch.bfloat16).cuda() for h in (8, 2))
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    cos, sin = (z.cuda() for z in _rope.table(40, 128))
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    mass = torch.rand(4, 2, 320, generator=g).cuda()

    def paged(q=q):
        return attn.attn_fwd_paged(q, kp, vp, table, lens, layout="bshd")

    def rope(x=x):
        return (*attn.attn_qk_norm_rope(x, y, w, w, cos, sin, pos),
                *attn.attn_qk_norm_rope_bwd(x, y, x, y, w, w, cos, sin, pos))

    def evict(mass=mass):  # nothing is over the budget: the pages stay
        return attn.attn_cache_evict(kp, vp, table, lens, mass, 320, layout="bshd")

    return [(paged, q[:1]), (rope, x[:1]), (evict, mass[:1])]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_from_threads(which):
    call, bad = _case()[which]
    want = call()
    torch.cuda.synchronize()

    def work(_):
        s = torch.cuda.Stream()
        done = 0
        with torch.cuda.stream(s):
            for _ in range(TIMES):
                got = call()
                with pytest.raises(ValueError):
                    call(bad)
                s.synchronize()
                assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))
                done += 1
        return done

    with ThreadPoolExecutor(THREADS) as pool:
        assert [f.result() for f in [pool.submit(work, i) for i in range(THREADS)]] == [TIMES] * THREADS
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
