"""The debug flavour of the library on the norm, rotation and paged-cache calls: its checks stay silent and
the results equal the release build's bit for bit."""
import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _paged
import _rope

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


@pytest.mark.parametrize("rot,inter", [(128, False), (64, False), (96, True)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (333, 9, 2), (3000, 16, 16)])
def test_norms_and_rotation(monkeypatch, T, Hq, Hkv, rot, inter):
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, wq, wk = r(T, Hq, 128), r(T, Hkv, 128), r(128), r(128)
    cos, sin = (t.cuda() for t in _rope.table(T, rot))
    pos = torch.randperm(T, generator=g, device="cuda").to(torch.int32)
    slots = torch.randperm(T + 7, generator=g, device="cuda")[:T].to(torch.int32)

    def step():
        pages = [torch.zeros(T + 7, 1, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        y = attn.attn_qk_norm_rope(q, k, wq, wk, cos, sin, pos, interleaved=inter)
        p = attn.attn_qk_norm_rope_paged(q, k, k, wq, wk, cos, sin, pos, slots, *pages, interleaved=inter, layout="bshd")
        return (*y, p, *pages, *attn.attn_qk_norm_rope_bwd(q, k, q, k, wq, wk, cos, sin, pos, interleaved=inter))

    _same_in_both(monkeypatch, step)


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("layout,B,Sq,Hq,Hkv,page,per,lens", [
    ("bshd", 1, 1, 1, 1, 1, 1, [1]),
    ("bhsd", 3, 1, 8, 2, 16, 200, [3200, 0, 77]),
    ("bshd", 2, 5, 28, 4, 20, 60, [1200, 5]),
    ("bhsd", 2, 3, 4, 1, 7, 40, [280, 2]),
    ("bshd", 1, 100, 2, 1, 16, 30, [480]),
])
def test_paged(monkeypatch, layout, B, Sq, Hq, Hkv, page, per, lens, with_mass):
    t = [torch.tensor(x, dtype=torch.int32).cuda() if isinstance(x, list) else x.cuda()
         for x in _paged.inputs(layout, B, Sq, Hq, Hkv, page, per, lens, seed=70)]

    def step():
        mass = torch.zeros(B, Hkv, page * per, device="cuda") if with_mass else None
        got = attn.attn_fwd_paged(*t, causal=True, layout=layout, mass=mass)
        return (*got, mass) if with_mass else got

    _same_in_both(monkeypatch, step)


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
def test_evict(monkeypatch, layout):
    B, Hkv, page, per = 4, 3, 16, 150
    g = torch.Generator().manual_seed(71)
    kp, vp = (t.cuda() for t in _paged.pages_of(layout, B * per, page, Hkv, g))
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).cuda()
    mass = torch.rand(B, Hkv, page * per, generator=g).cuda()
    n = torch.tensor([2400, 0, 700, 699], dtype=torch.int32).cuda()

    def step():
        k, v = kp.clone(), vp.clone()
        return (k, v, *attn.attn_cache_evict(k, v, table, n, mass, 699, recent=100, layout=layout))

    _same_in_both(monkeypatch, step)
