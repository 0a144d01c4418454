"""The calls around a paged cache and around a training step together, as a user runs them: prompts
written to the cache, tokens sampled one by one against it with their keys' weights accumulated,
the cache cut to a budget on the way, and sampling going on; and a training step whose queries and keys are
normed and rotated. Every call's result is compared with its definition in 64 bits, on the
inputs that the calls before it really left."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _grad
import _paged
import _rope
from _parity import assert_parity, bits_of, compare

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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
def test_sampling_with_a_budget(layout):
    B, Hq, Hkv, page, per, rot = 3, 8, 2, 8, 12, 64
    prompt, steps, budget, recent = [50, 9, 31], 30, 40, 10
    g = torch.Generator().manual_seed(60)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    wq, wk = r(128), r(128)
    cos, sin = _rope.table(200, rot)
    W = [t.cuda() for t in (wq, wk, cos, sin)]
    kp, vp = (t.cuda() for t in _paged.pages_of(layout, B * per, page, Hkv, fill=math.nan))
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32)
    T = table.cuda()
    slot = lambda b, j: int(table[b, j // page]) * page + j % page
    mass = torch.zeros(B, Hkv, page * per, device="cuda")
    kw = {"layout": layout, "interleaved": True}

    # ---- the prompts, packed, into the cache.
    q, k, v = r(sum(prompt), Hq, 128), r(sum(prompt), Hkv, 128), r(sum(prompt), Hkv, 128)
    pos = torch.cat([torch.arange(n) for n in prompt]).to(torch.int32)
    slots = torch.tensor([slot(b, j) for b, n in enumerate(prompt) for j in range(n)], dtype=torch.int32)
    q_out = attn.attn_qk_norm_rope_paged(q.cuda(), k.cuda(), v.cuda(), *W, pos.cuda(), slots.cuda(), kp, vp, **kw)
    _ok()
    _rope.check("q", q_out, *_rope.forward(q, wq, cos, sin, pos, True))
    at = 0
    for b, n in enumerate(prompt):
        rows = _paged.rows(kp.cpu(), table, b, n, layout)
        _rope.check("k", rows, *_rope.forward(k[at:at + n], wk, cos, sin, pos[at:at + n], True))
        assert torch.equal(_paged.rows(vp.cpu(), table, b, n, layout), v[at:at + n])
        at += n

    # ---- tokens, one a sequence and step. Positions go on where lengths may have been cut.
    lens, seen = list(prompt), list(prompt)
    want_mass = torch.zeros(B, Hkv, page * per, dtype=torch.float64)
    bound = torch.zeros_like(want_mass)
    workspace = torch.empty(max(attn.paged_workspace_bytes(B, Hq, Hkv, 1, page, per, with_mass=True),
                                attn.evict_workspace_bytes(B, Hkv, B * per, page, per, budget)),
                            dtype=torch.uint8, device="cuda")
    for step in range(steps):
        q, k, v = r(B, 1, Hq, 128), r(B, 1, Hkv, 128), r(B, 1, Hkv, 128)
        form = (lambda t: t) if layout == "bshd" else (lambda t: t.transpose(1, 2).contiguous())
        back = (lambda t: t) if layout == "bshd" else (lambda t: t.transpose(1, 2))
        pos = torch.tensor(seen, dtype=torch.int32)[:, None]
        q_out = attn.attn_qk_norm_rope_paged(*(form(t).cuda() for t in (q, k, v)), *W, pos.cuda(),
                                             _i32([[slot(b, lens[b])] for b in range(B)]), kp, vp, **kw)
        lens, seen = [n + 1 for n in lens], [n + 1 for n in seen]
        out, lse = attn.attn_fwd_paged(q_out, kp, vp, T, _i32(lens), layout=layout, mass=mass, workspace=workspace)
        _ok()
        _rope.check("q", back(q_out)[:, 0], *_rope.forward(q[:, 0], wq, cos, sin, pos[:, 0], True))
        o, l, m, e = _paged.exact(q_out.cpu(), kp.cpu(), vp.cpu(), table, lens, layout, False)
        got = out if layout == "bhsd" else out.transpose(1, 2)
        assert_parity(compare(bits_of(got), o.numpy(), "rtne"), excess=True)
        assert (lse.cpu().double() - l).abs().max() <= 1e-4
        want_mass += m
        bound += e + 2.0 ** -23 * want_mass
        assert ((mass.cpu().double() - want_mass).abs() <= bound).all()
        if step % 12 == 11:                  # cut to the budget
            keys = [[_paged.rows(t.cpu(), table, b, lens[b], layout) for b in range(B)] for t in (kp, vp)]
            before = mass.cpu()
            new = _i32(lens)
            attn.attn_cache_evict(kp, vp, T, new, mass, budget, recent=recent, layout=layout, mass_out=mass,
                                  seqlens_out=new, workspace=workspace)
            _ok()
            assert new.tolist() == [min(n, budget) for n in lens]
            moved, moved_bound = torch.zeros_like(want_mass), torch.zeros_like(bound)
            for b, n in enumerate(lens):
                for h in range(Hkv):
                    old = n - recent
                    first = torch.sort(before[b, h, :max(old, 0)], descending=True, stable=True).indices
                    src = (torch.cat((first[:budget - recent].sort().values, torch.arange(old, n))) if n > budget
                           else torch.arange(n))
                    m = len(src)
                    for t, was in zip((kp, vp), keys):
                        assert torch.equal(_paged.rows(t.cpu(), table, b, m, layout)[:, h], was[b][src, h])
                    assert torch.equal(mass[b, h, :m].cpu(), before[b, h, src]) and (mass[b, h, m:] == 0).all()
                    moved[b, h, :m], moved_bound[b, h, :m] = want_mass[b, h, src], bound[b, h, src]
            want_mass, bound = moved, moved_bound
            lens = new.tolist()
    assert max(lens) > budget and seen[1] == prompt[1] + steps


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
def test_a_training_step(layout):
    """Norms and rotation, attention, its gradients, and theirs: queries, keys and values are columns
    of one projection's output, and their gradients columns of its gradient."""
    B, S, Hq, Hkv = 2, 130, 4, 2
    g = torch.Generator().manual_seed(61)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    x, wq, wk, do = r(B, S, Hq + 2 * Hkv, 128), r(128), r(128), r(B, S, Hq, 128)
    cos, sin = _rope.table(S, 128)
    pos = torch.arange(S, dtype=torch.int32).repeat(B, 1)
    form = (lambda t: t) if layout == "bshd" else (lambda t: t.transpose(1, 2))
    fused, grads = x.cuda(), torch.full_like(x, 9.0).cuda()
    q, k, v = (form(t) for t in fused.split((Hq, Hkv, Hkv), 2))
    gq, gk, gv = (form(t) for t in grads.split((Hq, Hkv, Hkv), 2))
    W = [t.cuda() for t in (wq, wk, cos, sin, pos)]
    qr, kr = attn.attn_qk_norm_rope(q, k, *W, layout=layout)
    vc, doc = v.contiguous(), form(do.cuda()).contiguous()
    out, lse = attn.attn_fwd_lse(qr, kr, vc, causal=True, layout=layout)
    dqr, dkr, dv = attn.attn_bwd(doc, qr, kr, vc, out, lse, causal=True, layout=layout)
    gv.copy_(dv)
    _, _, dwq, dwk = attn.attn_qk_norm_rope_bwd(dqr, dkr, q, k, *W, layout=layout, dq=gq, dk=gk)
    _ok()
    tokens = lambda t: form(t).reshape(B * S, -1, 128).cpu()
    flat = pos.flatten()
    for name, y, w, src in (("q", qr, wq, q), ("k", kr, wk, k)):
        _rope.check(name, tokens(y), *_rope.forward(tokens(src), w, cos, sin, flat, False))
    for b in range(B):
        want, bound = _grad.sequence(*(form(t)[b].cpu() for t in (qr, kr, vc, doc)), _paged.SCALE, True)
        for name, t in (("dq", dqr), ("dk", dkr), ("dv", dv)):
            _grad.check(name, form(t)[b], want[name], bound[name])
    for name, dy, y, w, src, dx, dw in (("dq", dqr, qr, wq, q, gq, dwq), ("dk", dkr, kr, wk, k, gk, dwk)):
        want, mag, wdw, mag_w = _rope.backward(tokens(dy), tokens(src), w, cos, sin, flat, False)
        _rope.check(name, tokens(dx), want, mag)
        _rope.check_weight(name + "_weight", dw, wdw, mag_w)
    # The whole step's gradient with respect to the projection's output, against differences in 64 bits
    # along a direction: what the roundings on the way leave is 2^-8 a step of each element.
    d = torch.randn(x.shape, generator=g, dtype=torch.float64)

    def loss(t):
        q, k, v = t.split((Hq, Hkv, Hkv), 2)
        q, k = (_rope.forward(a.reshape(B * S, -1, 128), w, cos, sin, flat, False)[0].view(B, S, -1, 128)
                for a, w in ((q, wq), (k, wk)))
        s = torch.einsum("bihd,bjhd->bhij", q, k.repeat_interleave(Hq // Hkv, 2)) * _paged.SCALE
        p = torch.softmax(s.masked_fill(~torch.ones(S, S, dtype=torch.bool).tril(), -math.inf), -1)
        return (torch.einsum("bhij,bjhd->bihd", p, v.repeat_interleave(Hq // Hkv, 2)) * do.double()).sum()

    h = 1e-5
    slope = float((loss(x.double() + h * d) - loss(x.double() - h * d)) / (2 * h))
    got = grads.cpu().double()
    # Roundings of P, dS, O, dq, dk, q and k in turn: below 8 independent ones of 2^-8 / sqrt(3) * |g d| each.
    noise = 2.0 ** -8 / math.sqrt(3) * float((got * d).norm()) * math.sqrt(8)
    assert abs(slope - float((got * d).sum())) <= 6 * noise


def _paged_case(seed, B=4, Hq=8, Hkv=2, Sq=1, page=16, per=20):
    lens = [page * per, 3, 0, 200][:B]
    t = _paged.inputs("bshd", B, Sq, Hq, Hkv, page, per, lens, seed=seed)
    return [torch.tensor(x, dtype=torch.int32).cuda() if isinstance(x, list) else x.cuda() for x in t]


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("Sq", [1, 6])
def test_two_graphs_share_a_workspace(Sq):
    """Two captured calls of different sizes with one workspace, replayed in turn, and an eager call
    between them: each overwrites what it uses before it reads it."""
    a, b = _paged_case(62, Sq=Sq), _paged_case(63, B=2, Hq=24, Hkv=3, Sq=Sq, page=7, per=60)
    need = max(attn.paged_workspace_bytes(4, 8, 2, Sq, 16, 20, with_mass=True),
               attn.paged_workspace_bytes(2, 24, 3, Sq, 7, 60, with_mass=True))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    masses = [torch.zeros(4, 2, 320, device="cuda"), torch.zeros(2, 3, 420, device="cuda")]

    def call(t, i):
        masses[i].zero_()
        return (*attn.attn_fwd_paged(*t, causal=True, layout="bshd", mass=masses[i], workspace=ws), masses[i])

    want = [[x.clone() for x in call(t, i)] for i, t in enumerate((a, b))]
    graphs, held = [], []
    for i, t in enumerate((a, b)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(call(t, i))
        graphs.append(g)
    for order in ((0, 1, 0), (1, 1, 0, 1)):
        for i in order:
            graphs[i].replay()
            _ok()
            assert all(_same(x, y) for x, y in zip(held[i], want[i]))
            eager = call((b, a)[i], 1 - i)
            _ok()
            assert all(_same(x, y) for x, y in zip(eager, want[1 - i]))


def test_calls_at_once_on_two_streams():
    """Independent calls on two streams, each with results and workspace of its own."""
    cases = [_paged_case(64), _paged_case(65, B=2, Hq=24, Hkv=3, Sq=6, page=7, per=60)]
    want = [attn.attn_fwd_paged(*t, layout="bshd") for t in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(attn.attn_fwd_paged(*cases[i], layout="bshd"))
    _ok()
    for i in range(2):
        for res in got[i]:
            assert all(_same(x, y) for x, y in zip(res, want[i]))


def test_calls_from_threads():
    """The binding's checks and calls from several threads at once."""
    import threading

    t = _paged_case(66)
    want = attn.attn_fwd_paged(*t, layout="bshd")
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(25):
                res = attn.attn_fwd_paged(*t, layout="bshd")
                with pytest.raises(ValueError):
                    attn.attn_fwd_paged(t[0][:1], *t[1:], layout="bshd")
                s.synchronize()
                if not all(_same(x, y) for x, y in zip(res, want)):
                    bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    _ok()
    assert not bad
