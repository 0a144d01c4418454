"""attn_fwd_paged against attention over the gathered keys in 64 bits."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _paged
from _parity import assert_parity, bits_of, compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


def _ok(status=attn.ATTN_OK):
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == status


def _cuda(t):
    return [torch.tensor(x, dtype=torch.int32).cuda() if isinstance(x, list) else x.cuda() for x in t]


def _check(t, layout, causal, got, lse, mode="rtne", scale=_paged.SCALE, mass=None, base=0.0, only=slice(None)):
    want, want_lse, want_mass, bound = _paged.exact(*t, layout, causal, scale)
    if layout == "bshd":
        want = want.transpose(1, 2).contiguous()
    # Rows of few keys reach magnitudes where one unit in the last place is above the
    # absolute bound: the bound is then on the error beyond the rounding's own.
    assert_parity(compare(bits_of(got[only]), want[only].numpy(), mode), excess=True)
    want_lse, lse = want_lse[only], lse[only].cpu().double()
    seen = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(lse), seen)
    assert ((lse - want_lse).abs()[seen] <= 1e-4 + 1e-6 * want_lse.abs()[seen]).all()
    if mass is not None:
        full = want_mass + base
        # Adding to what was there rounds once more.
        over = (mass.cpu().double() - full).abs() - (bound + 2.0 ** -23 * full.abs())
        assert over[only].max() <= 0, float(over[only].max())


CASES = [
    # layout, B, Sq, Hq, Hkv, page, max_pages, lens, causal
    ("bshd", 1, 1, 1, 1, 1, 1, [1], False),
    ("bshd", 3, 1, 8, 2, 16, 20, [0, 1, 320], False),            # no key, one key, a full table
    ("bhsd", 3, 1, 8, 2, 16, 5, [17, 16, 15], True),
    ("bshd", 2, 5, 28, 4, 20, 17, [333, 5], True),               # 35 rows per kv head: two blocks
    ("bhsd", 2, 5, 28, 4, 33, 11, [200, 3], True),               # fewer keys than new tokens
    ("bhsd", 4, 3, 6, 1, 1, 20, [3, 20, 11, 0], False),          # pages of one key, 18 rows
    ("bshd", 5, 1, 7, 7, 7, 100, [700, 1, 300, 257, 31], False),
    ("bhsd", 2, 1, 40, 2, 64, 32, [2000, 999], False),           # long: several parts; 20 rows
    ("bshd", 70, 1, 16, 2, 5, 4, None, False),                   # many short sequences
    ("bshd", 300, 1, 2, 1, 16, 2, None, False),                  # more sequences than threads of a block
    ("bshd", 1, 9, 4, 4, 256, 3, [650], True),
    ("bhsd", 1, 1, 1, 1, 128, 80, [10000], False),               # one row over every CTA
    ("bshd", 9, 2, 4, 2, 48, 20, [900, 1, 2, 3, 4, 5, 6, 7, 8], True),  # a long one among short ones
    ("bshd", 2, 32, 2, 2, 16, 9, [140, 33], True),               # 32 rows
    ("bhsd", 2, 70, 1, 1, 16, 9, [140, 69], True),               # 70 rows, more new tokens than keys
    ("bshd", 3, 17, 1, 1, 16, 70, [1100, 1, 0], False),          # 17 rows, long, one key, none
    ("bhsd", 2, 9, 14, 2, 10, 150, [1500, 640], True),           # 63 rows, several parts
    ("bshd", 1, 128, 1, 1, 32, 40, [1280], True),                # 128 rows over many CTAs
    ("bhsd", 1, 129, 1, 1, 32, 10, [300], True),                 # two blocks
    ("bshd", 2, 301, 2, 2, 16, 40, [590, 301], True),            # 301 rows: three blocks
    ("bshd", 40, 6, 8, 2, 16, 8, None, True),                    # 24 rows, many short sequences
    ("bhsd", 2, 20, 4, 1, 48, 11, [528, 100], False),            # 80 rows
]


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("layout,B,Sq,Hq,Hkv,page,max_pages,lens,causal", CASES)
def test_parity(layout, B, Sq, Hq, Hkv, page, max_pages, lens, causal, with_mass):
    lens = lens or [i % (page * max_pages + 1) for i in range(B)]
    t = _paged.inputs(layout, B, Sq, Hq, Hkv, page, max_pages, lens, seed=B * 100 + page)
    mass = torch.full((B, Hkv, page * max_pages), 0.25, device="cuda") if with_mass else None
    out, lse = attn.attn_fwd_paged(*_cuda(t), causal=causal, layout=layout, mass=mass)
    _ok()
    _check(t, layout, causal, out, lse, mass=mass, base=0.25)
    if with_mass:
        for b, n in enumerate(lens):
            assert (mass[b, :, n:] == 0.25).all()


@pytest.mark.parametrize("mode", ["rtne", "rtna", "rtz"])
@pytest.mark.parametrize("scale", [0.3, -0.1, 0.0])
def test_modes_and_scales(mode, scale):
    t = _paged.inputs("bshd", 2, 2, 4, 2, 16, 6, [90, 33], seed=41)
    mass = torch.zeros(2, 2, 96, device="cuda")
    out, lse = attn.attn_fwd_paged(*_cuda(t), layout="bshd", rounding=mode, scale=scale, causal=True, mass=mass)
    _ok()
    _check(t, "bshd", True, out, lse, mode, scale, mass)


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
def test_pages_that_are_shared_or_lie_apart(layout):
    """Sequences that list the same pages, and pages that are halves of one tensor."""
    B, Hq, Hkv, page, n = 3, 4, 2, 16, 9
    g = torch.Generator().manual_seed(42)
    kp, vp = _paged.pages_of(layout, n, page, Hkv, g)
    q = torch.randn(*((B, 1, Hq, 128) if layout == "bshd" else (B, Hq, 1, 128)), generator=g).to(torch.bfloat16)
    table = torch.tensor([[4, 4, 8], [4, 0, 2], [4, 0, 2]], dtype=torch.int32)
    t = (q, kp, vp, table, [48, 40, 33])
    one = torch.stack((kp, vp), 1).cuda()
    out, lse = attn.attn_fwd_paged(q.cuda(), one[:, 0], one[:, 1], *_cuda(t[3:]), layout=layout)
    _ok()
    _check(t, layout, False, out, lse)


def test_equals_the_contiguous_cache():
    """The shared-prefix call without a prefix reads the same keys from contiguous caches: both
    within one unit in the last place of the exact value, so within two of each other."""
    lens = [700, 1, 63, 400]
    t = _paged.inputs("bshd", 4, 2, 8, 2, 24, 30, lens, seed=43)
    out, lse = attn.attn_fwd_paged(*_cuda(t), layout="bshd", causal=True)
    k, v = (torch.zeros(4, 720, 2, 128, dtype=torch.bfloat16) for _ in range(2))
    for b, n in enumerate(lens):
        k[b, :n], v[b, :n] = (_paged.rows(p, t[3], b, n, "bshd") for p in t[1:3])
    o2, l2 = attn.attn_fwd_prefix(t[0].cuda(), None, None, k.cuda(), v.cuda(), *_cuda([lens]), layout="bshd", causal=True)
    _ok()
    seen = torch.isfinite(l2)
    assert torch.equal(seen, torch.isfinite(lse)) and (lse - l2)[seen].abs().max() <= 2e-5
    a, b = out.float(), o2.float()
    ok = torch.isfinite(b)
    assert torch.equal(ok, torch.isfinite(a))
    assert ((a - b).abs() <= 2 ** -7 * b.abs() + 1e-3)[ok].all()


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("which", [1, 2])
@pytest.mark.parametrize("g", [3, 7, 13, 26])  # 15, 35, 65 and 130 rows a key/value head
def test_non_finite_values_at_hidden_keys(which, value, g):
    """A drafted token's own key or value that earlier tokens do not see reaches only the tokens
    that see it, and only their masses."""
    Sq, n, page = 5, 37, 8
    t = list(_paged.inputs("bshd", 2, Sq, 2 * g, 2, page, 8, [n, n], seed=44))
    masses = [torch.zeros(2, 2, 64, device="cuda") for _ in range(2)]
    clean, _ = attn.attn_fwd_paged(*_cuda(t), layout="bshd", causal=True, mass=masses[0])
    j = n - 2                                 # the last but one new token's slot
    t[which] = t[which].clone()
    t[which][t[3][0, j // page].long(), j % page, 1, 5] = value
    out, _ = attn.attn_fwd_paged(*_cuda(t), layout="bshd", causal=True, mass=masses[1])
    _ok()
    sees = torch.arange(Sq) + n - Sq >= j     # tokens 3 and 4
    hit = torch.zeros(2, Sq, 2 * g, 128, dtype=torch.bool)
    if which == 2:
        hit[0, sees, g:, 5] = True
    elif value != value:
        hit[0, sees, g:] = True
    else:                                     # an infinite key: +Inf logits make the row NaN
        pos = sees[:, None] & (t[0][0, :, g:, 5].float() > 0)
        hit[0, :, g:][pos] = True
    out = out.cpu()
    assert torch.isinf(out[hit]).all() if which == 2 and value == math.inf else torch.isnan(out[hit]).all()
    assert torch.isfinite(out[~hit]).all()
    hidden = torch.ones(2, Sq, dtype=torch.bool)
    hidden[0, sees] = False
    a, b = out[hidden].float(), clean.cpu()[hidden].float()
    assert ((a - b).abs() <= 2 ** -7 * b.abs() + 1e-6).all()
    # Masses: the other sequence's and the other head's are the same bits; with a value at a key
    # the weights do not change at all.
    assert torch.equal(masses[0][1], masses[1][1]) and torch.equal(masses[0][0, 0], masses[1][0, 0])
    if which == 2:
        assert torch.equal(masses[0], masses[1])
    else:
        assert torch.isnan(masses[1][0, 1, :n - 1]).all() and (masses[1][0, 1, n:] == 0).all()


def test_rows_of_minus_infinity():
    """Logits that are all -Inf: the row is NaN with lse -Inf, as in attn_fwd, and adds no mass."""
    t = list(_paged.inputs("bhsd", 1, 1, 2, 1, 4, 2, [5], seed=45))
    t[0][0, 0], t[0][0, 1] = 1.0, 1.0
    t[0][0, 0, 0, 3] = -math.inf
    kp = t[1]
    kp[...] = 1.0
    mass = torch.zeros(1, 1, 8, device="cuda")
    out, lse = attn.attn_fwd_paged(*_cuda(t), mass=mass)
    _ok()
    assert torch.isnan(out[0, 0]).all() and lse[0, 0, 0] == -math.inf
    assert torch.isfinite(out[0, 1]).all()
    assert ((mass[0, 0, :5] - 0.2).abs() <= 1e-5).all() and (mass[0, 0, 5:] == 0).all()


def test_bad_lengths_and_pages_are_reported():
    lens = [30, 33, -1, 0, 32, 17]
    good = [30, 0, 0, 0, 32, 17]
    t = list(_paged.inputs("bshd", 6, 1, 4, 2, 8, 4, good, seed=46))
    q, kp, vp, table, _ = t
    for bad in ("length", "page"):
        out, lse = torch.full((6, 1, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((6, 4, 1), 9.0, device="cuda")
        mass = torch.full((6, 2, 32), 0.5, device="cuda")
        tab = table.clone()
        if bad == "page":
            tab[4, 1], tab[5, 2] = kp.shape[0], -1     # one past the last page; a negative number
        attn.attn_fwd_paged(q.cuda(), kp.cuda(), vp.cuda(), *_cuda([tab, lens if bad == "length" else good]),
                            layout="bshd", out=out, lse=lse, mass=mass)
        _ok(attn.ATTN_ERR_SEQLENS if bad == "length" else attn.ATTN_ERR_INDEX)
        _ok()
        left = [1, 2] if bad == "length" else [4, 5]
        assert (out[left] == 9.0).all() and (lse[left] == 9.0).all() and (mass[left] == 0.5).all()
        rest = [b for b in range(6) if b not in left]
        _check(t, "bshd", False, out, lse, mass=mass, base=0.5, only=rest)


def test_a_bad_page_of_a_long_sequence():
    """The page is read by one of many CTAs: none of the sequence's rows is written."""
    t = list(_paged.inputs("bhsd", 2, 1, 8, 2, 16, 500, [8000, 7000], seed=47))
    out, lse = torch.full((2, 8, 1, 128), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, 8, 1), 9.0, device="cuda")
    mass = torch.zeros(2, 2, 8000, device="cuda")
    t[3] = t[3].clone()
    t[3][1, 300] = -1
    attn.attn_fwd_paged(*_cuda(t), out=out, lse=lse, mass=mass)
    _ok(attn.ATTN_ERR_INDEX)
    assert (out[1] == 9.0).all() and (lse[1] == 9.0).all() and (mass[1] == 0).all()
    first = [t[0][:1], t[1], t[2], t[3][:1], [8000]]
    _check(first, "bhsd", False, out[:1], lse[:1], mass=mass[:1])


def test_bits_repeat_and_replay_in_a_graph():
    t = _cuda(_paged.inputs("bhsd", 6, 2, 8, 2, 16, 40, [640] * 6, seed=48))
    n = t[4]
    n.copy_(torch.tensor([300, 5, 77, 2, 640, 299], dtype=torch.int32))

    def step():
        mass = torch.zeros(6, 2, 640, device="cuda")
        return (*attn.attn_fwd_paged(*t, causal=True, mass=mass), mass)

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    n.copy_(torch.tensor([299, 640, 70, 3, 0, 300], dtype=torch.int32))   # lengths move on between replays
    graph.replay()
    _ok()
    fresh = step()
    _ok()
    for x, y in ((first, again), (held, fresh)):
        for a, b in zip(x, y):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_given_workspace_is_kept_to():
    t = _cuda(_paged.inputs("bshd", 3, 1, 8, 2, 16, 21, [333, 0, 9], seed=49))
    for with_mass in (False, True):
        masses = [torch.zeros(3, 2, 336, device="cuda") if with_mass else None for _ in range(2)]
        want = attn.attn_fwd_paged(*t, layout="bshd", mass=masses[0])
        need = attn.paged_workspace_bytes(3, 8, 2, 1, 16, 21, with_mass=with_mass)
        ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
        got = attn.attn_fwd_paged(*t, layout="bshd", workspace=ws[:need], mass=masses[1])
        _ok()
        assert (ws[need:] == 0x7F).all()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert not with_mass or torch.equal(*masses)
        with pytest.raises(attn.AttnError) as e:
            attn.attn_fwd_paged(*t, layout="bshd", workspace=ws[:need - 16], mass=masses[0])
        assert e.value.status == attn.ATTN_ERR_INVALID_ARG


def test_long_parts_keep_the_contract():
    """Items that a CTA has whole, a warp's share of them far over 4096 keys: the sums are added to
    nearest (rows of up to 16 always, more than that where the cache is long)."""
    for Hq, seed in ((320, 50), (320 * 20, 51)):
        B, Hkv, page, n = 1, 320, 256, 20000 if Hq == 320 else 17000
        max_pages = -(-n // page)
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
        q, kp, vp = r(B, Hq, 1, 128), r(max_pages, Hkv, page, 128), r(max_pages, Hkv, page, 128)
        table = torch.arange(max_pages, dtype=torch.int32, device="cuda")[None]
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        out, lse = attn.attn_fwd_paged(q, kp, vp, table, lens)
        _ok()
        k, v = (t.transpose(0, 1).reshape(Hkv, -1, 128)[:, :n] for t in (kp, vp))
        some = torch.arange(0, Hkv, 16, device="cuda")
        rows = q.view(Hkv, Hq // Hkv, 128)[some]
        s = torch.einsum("hgd,hjd->hgj", rows.double(), k[some].double()) * _paged.SCALE
        want = torch.einsum("hgj,hjd->hgd", torch.softmax(s, -1), v[some].double())
        got = out.view(Hkv, Hq // Hkv, 128)[some].contiguous()
        assert_parity(compare(bits_of(got), want.cpu().numpy(), "rtne"))


def test_offsets_beyond_32_bits():
    """Keys whose byte and element offsets in the pages pass 2^32."""
    page, Hkv = 64, 8
    n = (1 << 33) // (page * Hkv * 256) + 40
    kp, vp = (torch.zeros(n, page, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(52)
    table = torch.randperm(20, generator=g)[:16].view(2, 8).to(torch.int32) + n - 20
    small = _paged.pages_of("bshd", n - (n - 20), page, Hkv, g)
    kp[n - 20:], vp[n - 20:] = small[0].cuda(), small[1].cuda()
    q = torch.randn(2, 1, 16, 128, generator=g).to(torch.bfloat16)
    lens = [500, 77]
    out, lse = attn.attn_fwd_paged(q.cuda(), kp, vp, *_cuda([table, lens]), layout="bshd")
    _ok()
    _check((q, small[0], small[1], table - (n - 20), lens), "bshd", False, out, lse)
