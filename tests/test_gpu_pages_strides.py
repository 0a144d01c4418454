"""Pages whose dimensions of one entry have strides of any value: such a stride says nothing, and each page
is contiguous all the same."""
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


def _ok():
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK


def _forms(n, page, Hkv, layout):
    """Pairs of page tensors of one shape, all with the same contents: as they come, and views that differ in
    strides of dimensions of one entry, pages apart or not."""
    shape = (n, page, Hkv, 128) if layout == "bshd" else (n, Hkv, page, 128)
    g = torch.Generator().manual_seed(n + page)
    kv = torch.randn(2, *shape, generator=g).to(torch.bfloat16).cuda()
    def apart():
        return kv[0].clone(), kv[1].clone()

    def halves():
        both = torch.stack((kv[0], kv[1]), 1)
        return both[:, 0], both[:, 1]

    def other(t):
        return t.as_strided(t.shape, [s if m > 1 else 8 for s, m in zip(t.stride(), t.shape)], t.storage_offset())

    for make in (apart, halves):  # each with memory of its own: the calls write to it
        yield make()
        k, v = make()
        yield other(k), other(v)
        k, v = make()
        yield k, other(v)


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("n,page,Hkv", [(5, 16, 1), (5, 1, 2), (1, 16, 2), (1, 1, 1), (4, 1, 1)])
def test_strides_of_one_entry(layout, n, page, Hkv):
    g = torch.Generator().manual_seed(3)
    q = torch.randn(*((1, 1, 2, 128) if layout == "bshd" else (1, 2, 1, 128)), generator=g).to(torch.bfloat16).cuda()
    table = torch.randperm(n, generator=g).to(torch.int32)[None].cuda()
    lens = torch.tensor([n * page], dtype=torch.int32).cuda()
    new_k, new_v = (torch.randn(1, Hkv, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    turn = [torch.ones(2, 64, device="cuda"), torch.zeros(2, 64, device="cuda")]
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([n * page - 1], dtype=torch.int32, device="cuda")
    mass = torch.rand(1, Hkv, n * page, generator=g).cuda()
    budget = max(1, n * page // 2)
    first = None
    for k, v in _forms(n, page, Hkv, layout):
        attn.attn_qk_norm_rope_paged(new_k, new_k, new_v, w, w, *turn, at, slot, k, v, layout=layout)
        out, lse = attn.attn_fwd_paged(q, k, v, table, lens, layout=layout)
        left, masses = attn.attn_cache_evict(k, v, table, lens, mass, budget, layout=layout)
        _ok()
        got = [t.contiguous().clone() for t in (out, lse, left, masses, k, v)]
        first = first or got
        for a, b in zip(got, first):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_pages_that_are_not_contiguous_are_refused():
    kv = torch.zeros(4, 16, 2, 256, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for k, v in ((kv[..., :128], kv[..., 128:]), (kv[:, ::2, :, :128].contiguous()[:, ::2], kv[:, :4, :, :128].contiguous()),
                 (kv[:, :, :, :128].contiguous(), kv.view(4, 2, 16, 2, 128)[:, 0])):
        with pytest.raises(ValueError):
            attn.attn_fwd_paged(q, k, v, table, lens, layout="bshd")
