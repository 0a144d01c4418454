"""attn_cache_evict against the definition, value for value."""
import math

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


def _ok(status=attn.ATTN_OK):
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == status


def _kept(mass, n, budget, recent):
    """The places that stay of n keys, ascending."""
    if n <= budget:
        return list(range(n))
    old = n - recent
    key = lambda i: (0 if math.isnan(mass[i]) else 1, -mass[i] if not math.isnan(mass[i]) else 0.0, i)
    return sorted(sorted(range(old), key=key)[:budget - recent]) + list(range(old, n))


def _want(kp, vp, table, lens, mass, budget, recent, layout, leave=()):
    """(k_pages, v_pages, masses, lengths) afterwards; sequences in `leave` as they are."""
    kp, vp, out = kp.clone(), vp.clone(), mass.clone()
    page = kp.shape[1 if layout == "bshd" else 2]
    left = list(lens)
    for b, n in enumerate(lens):
        if b in leave:
            continue
        out[b, :, max(0, n):] = 0
        left[b] = min(n, budget)
        for h in range(mass.shape[1]):
            src = torch.tensor(_kept(mass[b, h].tolist(), n, budget, recent), dtype=torch.long)
            d = torch.arange(len(src))
            out[b, h] = 0
            out[b, h, d] = mass[b, h, src]
            for t in (kp, vp):
                f, g = table[b, src // page].long(), table[b, d // page].long()
                if layout == "bshd":
                    t[g, d % page, h] = t[f, src % page, h].clone()
                else:
                    t[g, h, d % page] = t[f, h, src % page].clone()
    return kp, vp, out, left


def _same(a, b):
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))


def _pages(layout, n, page, Hkv, seed):
    return _paged.pages_of(layout, n, page, Hkv, torch.Generator().manual_seed(seed))


def _run(kp, vp, table, lens, mass, budget, recent, layout, **kw):
    k, v = kp.cuda(), vp.cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    got_n, got_m = attn.attn_cache_evict(k, v, table.cuda(), n, mass.cuda(), budget, recent=recent, layout=layout, **kw)
    return k, v, got_m, got_n


def _masses(kind, B, H, cap, g):
    if kind == "ties":                        # many equal values, some at the border
        return torch.randint(0, 3, (B, H, cap), generator=g).float()
    if kind == "all equal":
        return torch.full((B, H, cap), 0.5)
    if kind == "close":                       # equal in the upper digits
        return 1 + torch.randint(0, 1 << 12, (B, H, cap), generator=g).float() * 2.0 ** -23
    if kind == "special":
        m = torch.randn(B, H, cap, generator=g)
        pick = torch.randint(0, 8, (B, H, cap), generator=g)
        for i, x in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0)):
            m[pick == i] = x
        return m
    return torch.exp(2 * torch.randn(B, H, cap, generator=g) - 4)


@pytest.mark.parametrize("kind", ["skewed", "ties", "all equal", "close", "special"])
@pytest.mark.parametrize("layout,B,Hkv,page,max_pages,lens,budget,recent", [
    ("bshd", 3, 2, 16, 10, [160, 100, 0], 64, 8),
    ("bhsd", 3, 3, 1, 40, [40, 1, 2], 1, 0),                 # a budget of one
    ("bshd", 2, 1, 7, 30, [210, 51], 50, 50),                # only the latest stay
    ("bhsd", 2, 2, 33, 20, [660, 659], 659, 1),              # one key goes; nothing goes
    ("bshd", 1, 2, 64, 32, [2048], 1500, 0),                 # several rounds
    ("bhsd", 1, 1, 16, 400, [6400], 3000, 100),
    ("bshd", 4, 1, 5, 4, [20, 20, 20, 20], 21, 3),           # a budget beyond the table
    ("bhsd", 40, 2, 8, 3, None, 9, 4),
])
def test_evict(layout, B, Hkv, page, max_pages, lens, budget, recent, kind):
    cap = page * max_pages
    lens = lens or [i % (cap + 1) for i in range(B)]
    g = torch.Generator().manual_seed(B * 1000 + page)
    kp, vp = _pages(layout, B * max_pages + 2, page, Hkv, seed=B + page)
    table = torch.randperm(B * max_pages + 2, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32)
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = -9                        # not looked at
    mass = _masses(kind, B, Hkv, cap, g)
    k, v, m, n = _run(kp, vp, table, lens, mass, budget, recent, layout)
    _ok()
    wk, wv, wm, wn = _want(kp, vp, table, lens, mass, budget, recent, layout)
    assert n.tolist() == wn
    ok = torch.isnan(wm)
    assert torch.equal(torch.isnan(m.cpu()), ok) and torch.equal(m.cpu()[~ok], wm[~ok])
    assert _same(k, wk) and _same(v, wv)


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
def test_in_place_and_halves_of_one_tensor(layout):
    B, Hkv, page, max_pages, budget, recent = 3, 2, 16, 20, 100, 20
    lens = [320, 99, 200]
    g = torch.Generator().manual_seed(5)
    kp, vp = _pages(layout, B * max_pages, page, Hkv, seed=6)
    table = torch.randperm(B * max_pages, generator=g).view(B, max_pages).to(torch.int32)
    mass = _masses("skewed", B, Hkv, page * max_pages, g)
    wk, wv, wm, wn = _want(kp, vp, table, lens, mass, budget, recent, layout)
    one = torch.stack((kp, vp), 1).cuda()
    n, m = torch.tensor(lens, dtype=torch.int32).cuda(), mass.cuda()
    got = attn.attn_cache_evict(one[:, 0], one[:, 1], table.cuda(), n, m, budget, recent=recent, layout=layout,
                                mass_out=m, seqlens_out=n)
    _ok()
    assert got[0] is n and got[1] is m and n.tolist() == wn and torch.equal(m.cpu(), wm)
    assert _same(one[:, 0].contiguous(), wk) and _same(one[:, 1].contiguous(), wv)
    # Once more: nothing is over its budget any more.
    before = one.clone()
    attn.attn_cache_evict(one[:, 0], one[:, 1], table.cuda(), n, m, budget, recent=recent, layout=layout, mass_out=m,
                          seqlens_out=n)
    _ok()
    assert n.tolist() == wn and torch.equal(m.cpu(), wm) and _same(one, before)


@pytest.mark.parametrize("what", ["twice in one", "in two", "page", "negative page", "length", "negative length"])
def test_refused_sequences_stay_as_they_were(what):
    B, Hkv, page, max_pages, budget, recent = 4, 2, 8, 6, 20, 4
    lens = [48, 40, 10, 33]
    g = torch.Generator().manual_seed(7)
    n_pages = B * max_pages
    kp, vp = _pages("bshd", n_pages, page, Hkv, seed=8)
    table = torch.randperm(n_pages, generator=g).view(B, max_pages).to(torch.int32)
    mass = _masses("skewed", B, Hkv, page * max_pages, g)
    leave, status = [1], attn.ATTN_ERR_INDEX
    if what == "twice in one":
        table[1, 4] = table[1, 0]
    elif what == "in two":                    # sequence 2 is short and stays as it is anyway
        table[2, 1] = table[1, 3]
        table[3, 0] = table[0, 5]
        leave = [0, 1, 3]
    elif what == "page":
        table[1, 2] = n_pages
    elif what == "negative page":
        table[1, 4] = -1
    else:
        lens[1], status = (49 if what == "length" else -1), attn.ATTN_ERR_SEQLENS
    out = torch.full(mass.shape, 9.0, device="cuda")
    n_out = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    k, v, m, n = _run(kp, vp, table, lens, mass, budget, recent, "bshd", mass_out=out, seqlens_out=n_out)
    _ok(status)
    _ok()
    wk, wv, wm, wn = _want(kp, vp, table, lens, mass, budget, recent, "bshd", leave)
    rest = [b for b in range(B) if b not in leave]
    assert (m[leave] == 9.0).all() and (n[leave] == 77).all()
    assert torch.equal(m.cpu()[rest], wm[rest]) and [n.tolist()[b] for b in rest] == [wn[b] for b in rest]
    assert _same(k, wk) and _same(v, wv)


def test_many_keys_of_one_head():
    """A long cache: several digits' histograms over many keys, many rounds of moves."""
    page, max_pages, budget, recent = 128, 1600, 150000, 1000
    n = page * max_pages - 3
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn(max_pages, 1, page, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = torch.randperm(max_pages, generator=g, device="cuda").to(torch.int32)[None]
    mass = torch.rand(1, 1, page * max_pages, generator=g, device="cuda")
    order = torch.sort(mass[0, 0, :n - recent], descending=True, stable=True).indices[:budget - recent].sort().values
    src = torch.cat((order, torch.arange(n - recent, n, device="cuda")))
    rows = lambda t, j: t[table[0, j // page].long(), 0, j % page]
    want = [rows(t, src) for t in (k, v)]
    lens, m = attn.attn_cache_evict(k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda"), mass, budget,
                                    recent=recent)
    _ok()
    d = torch.arange(budget, device="cuda")
    assert lens.tolist() == [budget] and torch.equal(m[0, 0, :budget], mass[0, 0, src]) and (m[0, 0, budget:] == 0).all()
    for t, w in zip((k, v), want):
        assert _same(rows(t, d), w)


def test_bits_repeat_and_replay_in_a_graph():
    B, Hkv, page, max_pages = 5, 2, 16, 30
    g = torch.Generator().manual_seed(10)
    kp, vp = (t.cuda() for t in _pages("bhsd", B * max_pages, page, Hkv, seed=11))
    table = torch.randperm(B * max_pages, generator=g).view(B, max_pages).to(torch.int32).cuda()
    mass = _masses("ties", B, Hkv, page * max_pages, g).cuda()
    n = torch.tensor([480, 5, 300, 101, 100], dtype=torch.int32, device="cuda")

    def step():
        k, v = kp.clone(), vp.clone()
        return (k, v, *attn.attn_cache_evict(k, v, table, n, mass, 100, recent=10))

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    n.copy_(torch.tensor([99, 480, 250, 0, 333], dtype=torch.int32))
    graph.replay()
    graph.replay()
    _ok()
    fresh = step()
    _ok()
    for x, y in ((first, again), (held, fresh)):
        for a, b in zip(x, y):
            assert _same(a, b)


def test_given_workspace_is_kept_to():
    B, Hkv, page, max_pages = 3, 2, 16, 9
    kp, vp = _pages("bshd", B * max_pages, page, Hkv, seed=12)
    table = torch.arange(B * max_pages).view(B, max_pages).to(torch.int32)
    mass = _masses("skewed", B, Hkv, page * max_pages, torch.Generator().manual_seed(13))
    args = (kp, vp, table, [144, 20, 90], mass, 40, 8, "bshd")
    want = _run(*args)
    need = attn.evict_workspace_bytes(B, Hkv, B * max_pages, page, max_pages, 40)
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    got = _run(*args, workspace=ws[:need])
    _ok()
    assert (ws[need:] == 0x7F).all()
    for a, b in zip(got, want):
        assert _same(a, b)
    with pytest.raises(attn.AttnError) as e:
        _run(*args, workspace=ws[:need - 16])
    assert e.value.status == attn.ATTN_ERR_INVALID_ARG


def test_offsets_beyond_32_bits():
    page, Hkv, max_pages = 64, 8, 4
    n = (1 << 33) // (page * Hkv * 256) + 8
    k, v = (torch.zeros(n, Hkv, page, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kp, vp = _pages("bhsd", 8, page, Hkv, seed=14)
    k[n - 8:], v[n - 8:] = kp.cuda(), vp.cuda()
    g = torch.Generator().manual_seed(15)
    table = torch.randperm(8, generator=g).view(2, 4).to(torch.int32)
    mass = _masses("skewed", 2, Hkv, page * max_pages, g)
    lens = [256, 130]
    got = attn.attn_cache_evict(k, v, (table + n - 8).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), mass.cuda(),
                                100, recent=30)
    _ok()
    wk, wv, wm, wn = _want(kp, vp, table, lens, mass, 100, 30, "bhsd")
    assert got[0].tolist() == wn and torch.equal(got[1].cpu(), wm) and _same(k[n - 8:], wk) and _same(v[n - 8:], wv)
