"""attn_fwd_lse and attn_bwd (dense and packed) against their definition in 64 bits."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _grad

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


def _ok():
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK


def _rand(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def _inputs(layout, B, Hq, Hkv, Sq, Sk, seed):
    g = torch.Generator().manual_seed(seed)
    qs, ks = ((B, Sq, Hq, 128), (B, Sk, Hkv, 128)) if layout == "bshd" else ((B, Hq, Sq, 128), (B, Hkv, Sk, 128))
    return _rand(g, *qs), _rand(g, *ks), _rand(g, *ks), _rand(g, *qs)


def _major(t, layout):
    """(B, S, H, d) view."""
    return t if layout == "bshd" else t.transpose(1, 2)


def _run(q, k, v, do, layout, **kw):
    cu = [t.cuda() for t in (q, k, v, do)]
    rounding = kw.pop("rounding", "rtne")
    out, lse = attn.attn_fwd_lse(*cu[:3], layout=layout, **kw)
    grads = attn.attn_bwd(cu[3], *cu[:3], out, lse, layout=layout, rounding=rounding, **kw)
    _ok()
    return out, lse, grads


def _check(q, k, v, do, layout, out, lse, grads, causal=False, scale=SCALE, u_mode=_grad.U, norm=6e-3):
    for b in range(q.shape[0]):
        want, bound = _grad.sequence(*(_major(t, layout)[b] for t in (q, k, v, do)), scale, causal)
        # lse: fp32; its error is that of one logit's sum, the exponentials' (2^-22 each)
        # and the logarithm's.
        seen = torch.isfinite(want["lse"])
        got = lse[b].cpu().double()
        assert torch.equal(torch.isfinite(got), seen)
        assert (got[~seen] == -math.inf).all()
        assert ((got - want["lse"]).abs()[seen] <= 1e-4 + 1e-6 * want["lse"].abs()[seen]).all()
        for n, g in zip(("dq", "dk", "dv"), grads):
            _grad.check(f"{n}[{b}]", _major(g, layout)[b], want[n], bound[n], u_mode, norm)


@pytest.mark.parametrize("layout,B,Hq,Hkv,Sq,Sk,causal", [
    ("bhsd", 1, 1, 1, 128, 128, False),
    ("bhsd", 1, 2, 2, 256, 256, False),
    ("bshd", 2, 3, 3, 300, 421, False),      # ragged, unequal
    ("bshd", 1, 2, 2, 300, 300, True),
    ("bhsd", 2, 2, 2, 129, 700, True),       # Sq < Sk: every row sees the early keys
    ("bshd", 1, 2, 1, 700, 200, True),       # Sq > Sk: the first 500 rows see no key
    ("bshd", 1, 6, 2, 257, 257, True),       # three query heads per key/value head
    ("bhsd", 1, 7, 1, 100, 333, False),
    ("bshd", 2, 2, 2, 1, 1, False),          # one query, one key
    ("bhsd", 1, 2, 1, 1, 1000, True),        # one query
    ("bshd", 1, 2, 2, 1000, 1, False),       # one key
    ("bshd", 1, 2, 2, 1000, 77, False),      # few keys
    ("bhsd", 1, 1, 1, 4000, 60, False),      # query tiles shared by several CTAs
    ("bhsd", 1, 1, 1, 50, 4000, False),      # key tiles shared by several CTAs
    ("bshd", 1, 2, 1, 1500, 1500, True),     # both shared, causal
    ("bshd", 3, 8, 8, 640, 640, False),      # more tiles than SMs
    ("bshd", 1, 2, 1, 1100, 1100, True),     # nine tiles
    ("bhsd", 1, 1, 1, 1000, 1290, False),
    ("bhsd", 1, 2, 2, 1030, 900, True),      # rows without keys
])
def test_gradients(layout, B, Hq, Hkv, Sq, Sk, causal):
    t = _inputs(layout, B, Hq, Hkv, Sq, Sk, seed=Sq * 7 + Sk + Hq)
    out, lse, grads = _run(*t, layout, causal=causal)
    # One key: dS = P (dP - D) is 0 up to fp32 rounding, so dq and dk are noise of
    # the size the bound allows; there is no relative error to speak of.
    _check(*t, layout, out, lse, grads, causal, norm=math.inf if Sk == 1 else 6e-3)
    ref = attn.attn_fwd_ex(*(x.cuda() for x in t[:3]), layout=layout, causal=causal)
    if not (causal and Sq > Sk):
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))


def test_splits_are_reached():
    """The shapes above that share a tile's range between CTAs do so (their workspace holds
    more than the row statistics)."""
    stats = lambda B, H, Sq: B * H * ((Sq + 127) // 128) * 1024
    assert attn.bwd_workspace_bytes(1, 1, 1, 4000, 60) > stats(1, 1, 4000)
    assert attn.bwd_workspace_bytes(1, 1, 1, 50, 4000) > stats(1, 1, 50)
    assert attn.bwd_workspace_bytes(3, 8, 8, 640, 640) == stats(3, 8, 640)


@pytest.mark.parametrize("rounding,u", [("rtne", 2.0 ** -8), ("rtna", 2.0 ** -8), ("rtz", 2.0 ** -7)])
def test_rounding_modes(rounding, u):
    t = _inputs("bshd", 1, 2, 2, 200, 150, seed=3)
    out, lse, grads = _run(*t, "bshd", rounding=rounding)
    _check(*t, "bshd", out, lse, grads, u_mode=u, norm=6e-3 if rounding != "rtz" else 1.2e-2)


def test_rtz_and_rtna_round_the_same_sums():
    t = _inputs("bshd", 1, 2, 2, 200, 150, seed=4)
    z = _run(*t, "bshd", rounding="rtz")[2]
    a = _run(*t, "bshd", rounding="rtna")[2]
    for x, y in zip(z, a):  # toward zero is at most one step below nearest, in magnitude
        step = y.view(torch.int16).int() - x.view(torch.int16).int()
        assert ((step == 0) | (step == 1)).all()
        assert (step == 1).any()


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_scales(scale):
    t = _inputs("bhsd", 1, 2, 1, 150, 260, seed=5)
    out, lse, grads = _run(*t, "bhsd", scale=scale, causal=True)
    if scale == 0.0:
        assert all((g == 0).all() for g in grads[:2])
        want, bound = _grad.sequence(*(_major(x, "bhsd")[0] for x in t), 0.0, True)
        _grad.check("dv", _major(grads[2], "bhsd")[0], want["dv"], bound["dv"])
    else:
        _check(*t, "bhsd", out, lse, grads, True, scale)


def test_gradient_against_differences():
    """<gradient, direction> against the central difference of L = sum(dout * O) in 64 bits,
    within what the gradient's element bounds allow (the difference itself is off by
    h^2 times a third derivative, under 1e-6 of it here)."""
    t = _inputs("bshd", 1, 2, 1, 70, 90, seed=6)
    out, lse, grads = _run(*t, "bshd", causal=True)
    q, k, v, do = (x[0].double() for x in t)
    want, bound = _grad.sequence(*(x[0] for x in t), SCALE, True)
    g = torch.Generator().manual_seed(7)
    loss = lambda q, k, v: (_grad.sequence(q, k, v, do, SCALE, True)[0]["out"] * do).sum()
    args = [q, k, v]
    for i, n in enumerate(("dq", "dk", "dv")):
        u = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        h = 1e-4
        plus, minus = ([a + s * h * u if j == i else a for j, a in enumerate(args)] for s in (1, -1))
        diff = (loss(*plus) - loss(*minus)) / (2 * h)
        got = grads[i][0].cpu().double()
        tol = ((bound[n] + _grad.U * (want[n].abs() + bound[n])) * u.abs()).sum()
        assert (got * u).sum().sub(diff).abs() <= tol + 1e-6 * diff.abs()
        assert (want[n] * u).sum().sub(diff).abs() <= 1e-6 * (want[n].norm() * u.norm())


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (6, 2)])
@pytest.mark.parametrize("lq,lk", [
    ([130, 0, 1, 257, 40, 128], [200, 50, 1, 257, 0, 300]),
    ([1100, 0, 130, 700, 257, 128], [1100, 300, 129, 1025, 0, 90]),   # several tiles a sequence
])
def test_packed(causal, Hq, Hkv, lq, lk):
    """Ragged sequences, one without queries, one without keys, and tokens behind the last
    sequence: they hold NaN, take no part, and their gradients stay as they were."""
    extra = 37
    g = torch.Generator().manual_seed(11)
    nq, nk = sum(lq) + extra, sum(lk) + extra
    q, do = _rand(g, nq, Hq, 128), _rand(g, nq, Hq, 128)
    k, v = _rand(g, nk, Hkv, 128), _rand(g, nk, Hkv, 128)
    for t in (q, do, k, v):
        t[-extra:] = math.nan
    cuq = torch.tensor([0] + torch.tensor(lq).cumsum(0).tolist(), dtype=torch.int32)
    cuk = torch.tensor([0] + torch.tensor(lk).cumsum(0).tolist(), dtype=torch.int32)
    Q, K, V, DO, CQ, CK = (t.cuda() for t in (q, k, v, do, cuq, cuk))
    out = torch.full_like(Q, math.nan)
    lse = torch.full((Hq, nq), 5.0, device="cuda")
    attn.attn_fwd_varlen_lse(Q, K, V, CQ, CK, max(lq), causal=causal, out=out, lse=lse)
    assert torch.equal(lse[:, -extra:], torch.full_like(lse[:, -extra:], 5.0))
    grads = [torch.full_like(x, 9.0) for x in (Q, K, V)]
    attn.attn_bwd_varlen(DO, Q, K, V, out, lse, CQ, CK, max(lq), max(lk), causal=causal, dq=grads[0],
                         dk=grads[1], dv=grads[2])
    _ok()
    assert all((x[-extra:] == 9.0).all() for x in grads)
    for b in range(len(lq)):
        a, z, c, w = cuq[b], cuq[b + 1], cuk[b], cuk[b + 1]
        got = [grads[0][a:z], grads[1][c:w], grads[2][c:w]]
        if lq[b] == 0 or lk[b] == 0:
            assert all((x == 0).all() for x in got)
            assert (lse[:, a:z] == -math.inf).all()
            continue
        want, bound = _grad.sequence(q[a:z], k[c:w], v[c:w], do[a:z], SCALE, causal)
        seen = torch.isfinite(want["lse"])
        assert ((lse[:, a:z].cpu().double() - want["lse"]).abs()[seen] <= 1e-4).all()
        assert (lse[:, a:z].cpu()[~seen] == -math.inf).all()
        for n, x in zip(("dq", "dk", "dv"), got):
            _grad.check(f"{n} of sequence {b}", x, want[n], bound[n], norm=math.inf if lk[b] == 1 else 6e-3)


def test_packed_equals_dense():
    """Sequences of one length, packed, against the same batch as a dense call: the same
    tiles and sums, so the same bits."""
    B, S, Hq, Hkv = 20, 256, 8, 8   # more tiles than SMs either way: no tile is shared
    q, k, v, do = (x.cuda() for x in _inputs("bshd", B, Hq, Hkv, S, S, seed=12))
    out, lse = attn.attn_fwd_lse(q, k, v, layout="bshd", causal=True)
    dense = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd", causal=True)
    flat = [x.flatten(0, 1) for x in (do, q, k, v, out)]
    cu = torch.arange(0, (B + 1) * S, S, dtype=torch.int32, device="cuda")
    packed = attn.attn_bwd_varlen(*flat, lse.transpose(0, 1).flatten(1).contiguous(), cu, cu, S, S, causal=True)
    _ok()
    for a, b in zip(dense, packed):
        assert torch.equal(a.flatten(0, 1).view(torch.int16), b.view(torch.int16))


def test_packed_bad_offsets_are_reported():
    """A sequence whose offsets are invalid is left alone and reported; the others are right."""
    g = torch.Generator().manual_seed(13)
    n, H = 300, 2
    q, k, v, do = (_rand(g, n, H, 128) for _ in range(4))
    good = torch.tensor([0, 100, 200, 300], dtype=torch.int32).cuda()
    bad = torch.tensor([0, 100, 90, 300], dtype=torch.int32).cuda()   # sequence 1: -10 keys; 2: 210 > max
    Q, K, V, DO = (t.cuda() for t in (q, k, v, do))
    out, lse = attn.attn_fwd_varlen_lse(Q, K, V, good, good, 100)
    _ok()
    grads = [torch.full_like(Q, 9.0) for _ in range(3)]
    attn.attn_bwd_varlen(DO, Q, K, V, out, lse, good, bad, 100, 100, dq=grads[0], dk=grads[1], dv=grads[2])
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_ERR_SEQLENS
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    assert (grads[0][100:] == 9.0).all()
    want, bound = _grad.sequence(q[:100], k[:100], v[:100], do[:100], SCALE, False)
    for name, x in zip(("dq", "dk", "dv"), grads):
        _grad.check(name, x[:100], want[name], bound[name])


def test_rows_that_see_no_key_take_no_part():
    """Causal, more queries than keys: NaN and infinities in the rows that see no key reach
    nothing, and their dq is 0."""
    layout, Sq, Sk = "bshd", 450, 190
    t = list(_inputs(layout, 1, 2, 2, Sq, Sk, seed=14))
    clean = _run(*t, layout, causal=True)
    blind = Sq - Sk
    q, do = t[0].clone(), t[3].clone()
    q[:, :blind:3] = math.inf
    q[:, 1:blind:3] = math.nan
    do[:, :blind:2] = math.nan
    do[:, 1:blind:2] = -math.inf
    out, lse, grads = _run(q, t[1], t[2], do, layout, causal=True)
    assert torch.equal(lse[:, :, blind:], clean[1][:, :, blind:])
    assert (grads[0][:, :blind] == 0).all()
    for a, b in zip(grads, clean[2]):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("where", ["q", "k", "v", "do"])
@pytest.mark.parametrize("at", [3, 130, 200])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_non_finite_values_reach_only_the_pairs_that_see_them(where, at, value):
    """Causal, one non-finite element: gradients that no visible pair carries it to keep
    their bits, and every element that the definition makes non-finite is non-finite."""
    layout, S = "bshd", 260
    t = list(_inputs(layout, 1, 1, 1, S, S, seed=15))
    clean = _run(*t, layout, causal=True)[2]
    i = "qkv".index(where) if where != "do" else 3
    col = 17
    t[i] = t[i].clone()
    t[i][0, at, 0, col] = value
    got = _run(*t, layout, causal=True)[2]
    q, k, v, do = (x[0, :, 0].double() for x in t)
    seen = _grad.visible(S, S, True)
    # Pairs that carry the value. NaN in a logit (q or k; an infinite element makes
    # logits of both signs, so the row's largest is +Inf) makes the row's every P NaN.
    rows = torch.zeros(S, dtype=torch.bool)
    if where == "q":
        rows[at] = True
    elif where == "k":
        s = torch.where(seen, q @ k.T, torch.full((S, S), -math.inf, dtype=torch.float64))
        rows = seen[:, at] & ((s[:, at] == math.inf) | torch.isnan(s[:, at]))
    elif where == "v":
        rows = seen[:, at].clone()      # dP and D
    else:
        rows[at] = True
    keys = (seen & rows[:, None]).any(0)
    bad = dict(dq=rows[:, None].expand(S, 128).clone(), dk=keys[:, None].expand(S, 128).clone(),
               dv=keys[:, None].expand(S, 128).clone())
    if where == "v":
        bad["dv"][:] = False            # dV = P^T dO holds no V
    if where == "do":
        bad["dv"][:] = False
        bad["dv"][keys, col] = True
    if where == "k":
        bad["dq"][seen[:, at], col] = True   # dS K, also where the pair's weight is 0
    for n, g, c in zip(("dq", "dk", "dv"), got, clean):
        g, c = g[0, :, 0].cpu(), c[0, :, 0].cpu()
        assert (~torch.isfinite(g[bad[n]])).all(), n
        assert torch.isfinite(g[~bad[n]]).all(), n
        if not (where == "k" and value == math.inf):  # (there -Inf logits change the rest)
            # Untouched rows keep their bits; the others differ only where they are bad.
            same = ~bad[n].any(1)
            if where in ("q", "do") or n == "dq":
                assert torch.equal(g[same].view(torch.int16), c[same].view(torch.int16)), n


def test_runs_are_bit_identical_and_replay_in_a_graph():
    q, k, v, do = (x.cuda() for x in _inputs("bshd", 1, 4, 2, 900, 900, seed=16))
    out, lse = attn.attn_fwd_lse(q, k, v, layout="bshd", causal=True)
    first = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd", causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd", causal=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, l2 = attn.attn_fwd_lse(q, k, v, layout="bshd", causal=True)
        held = attn.attn_bwd(do, q, k, v, o2, l2, layout="bshd", causal=True)
    do2 = torch.randn_like(do.float()).to(torch.bfloat16)
    do.copy_(do2)
    graph.replay()
    _ok()
    fresh = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd", causal=True)
    _ok()
    for a, b in zip(first, again):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    for a, b in zip(held, fresh):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_given_outputs_and_workspace():
    q, k, v, do = (x.cuda() for x in _inputs("bhsd", 1, 2, 2, 200, 300, seed=17))
    out, lse = attn.attn_fwd_lse(q, k, v)
    want = attn.attn_bwd(do, q, k, v, out, lse)
    need = attn.bwd_workspace_bytes(1, 2, 2, 200, 300)
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    got = attn.attn_bwd(do, q, k, v, out, lse, dq=torch.empty_like(q), dk=torch.empty_like(k),
                        dv=torch.empty_like(v), workspace=ws[:need])
    _ok()
    assert (ws[need:] == 0x7F).all()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    with pytest.raises(attn.AttnError) as e:
        attn.attn_bwd(do, q, k, v, out, lse, workspace=ws[:need - 16])
    assert e.value.status == attn.ATTN_ERR_INVALID_ARG
