"""attn_qk_norm_rope, its paged form and its gradients against their definition in 64 bits."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _rope

pytestmark = pytest.mark.gpu

ROPE_KW = [dict(rot=128, interleaved=False), dict(rot=128, interleaved=True), dict(rot=64, interleaved=False),
           dict(rot=16, interleaved=True), dict(rot=96, interleaved=False), dict(rot=112, interleaved=False)]


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


def _ok(status=attn.ATTN_OK):
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == status


def _case(T, Hq, Hkv, rot, seed, max_pos=None, scale=1.0):
    """q, k (T, H, 128), weights, cos, sin, positions on the CPU."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: (scale * torch.randn(*s, generator=g)).to(torch.bfloat16)
    max_pos = max_pos or T + 3
    q, k = r(T, Hq, 128), r(T, Hkv, 128)
    w = [(1 + 0.3 * torch.randn(128, generator=g)).to(torch.bfloat16) for _ in range(2)]
    pos = torch.randint(0, max_pos, (T,), generator=g).to(torch.int32)
    return q, k, *w, *_rope.table(max_pos, rot), pos


def _cuda(ts):
    return [t.cuda() for t in ts]


def _check_forward(c, got, inter, mode="rtne", eps=1e-6):
    q, k, wq, wk, cos, sin, pos = c
    for name, x, w, y in (("q", q, wq, got[0]), ("k", k, wk, got[1])):
        _rope.check(name, y, *_rope.forward(x, w, cos, sin, pos, inter, eps), mode)


@pytest.mark.parametrize("kw", ROPE_KW)
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (5, 8, 2), (37, 9, 3), (130, 17, 1), (3, 1, 40)])
def test_forward(T, Hq, Hkv, kw):
    c = _case(T, Hq, Hkv, kw["rot"], seed=T + Hq)
    got = attn.attn_qk_norm_rope(*_cuda(c), interleaved=kw["interleaved"])
    _ok()
    _check_forward(c, got, kw["interleaved"])


@pytest.mark.parametrize("mode", ["rtne", "rtna", "rtz"])
@pytest.mark.parametrize("scale,eps", [(1.0, 1e-6), (1e-3, 1e-2), (1e4, 0.0)])
def test_modes_and_scales(mode, scale, eps):
    c = _case(70, 6, 2, 128, seed=5, scale=scale)
    got = attn.attn_qk_norm_rope(*_cuda(c), rounding=mode, eps=eps)
    _ok()
    _check_forward(c, got, False, mode, eps)


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("S", [1, 19])
def test_layouts_and_views(layout, S):
    """4-D tensors of both layouts, and queries and keys as columns of one projection's output,
    read and written in place: the same bits as packed rows."""
    B, Hq, Hkv = 3, 6, 2
    c = _case(B * S, Hq, Hkv, 128, seed=6)
    packed = attn.attn_qk_norm_rope(*_cuda(c))
    q, k, wq, wk, cos, sin, pos = _cuda(c)
    pos = pos.view(B, S)
    four = [t.view(B, S, -1, 128) if layout == "bshd" else t.view(B, S, -1, 128).transpose(1, 2).contiguous()
            for t in (q, k)]
    got = attn.attn_qk_norm_rope(*four, wq, wk, cos, sin, pos, layout=layout)
    fused = torch.full((B, S, Hq + 2 * Hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    views = list(fused.split((Hq, Hkv, Hkv), 2)[:2])
    if layout == "bhsd":
        views = [t.transpose(1, 2) for t in views]
    for t, x in zip(views, four):
        t.copy_(x)
    strided = attn.attn_qk_norm_rope(*views, wq, wk, cos, sin, pos, layout=layout)
    same = attn.attn_qk_norm_rope(*views, wq, wk, cos, sin, pos, layout=layout, q_out=views[0], k_out=views[1])
    _ok()
    assert (fused[:, :, Hq + Hkv:] == 7.0).all()
    for i in range(2):
        want = packed[i].view(B, S, -1, 128)
        for t in (got[i], strided[i], same[i]):
            t = t if layout == "bshd" else t.transpose(1, 2)
            assert torch.equal(t.contiguous().view(torch.int16), want.view(torch.int16))


def test_special_values():
    """A NaN reaches its whole row and no other; an infinite element makes its pair NaN and the
    others 0; a row of zeros stays 0; values whose squares overflow fp32 give 0, as the formula in
    fp32 does."""
    c = _case(8, 2, 1, 64, seed=7)
    q = c[0]
    q[1, 0, 3], q[2, 1, 100], q[3, 0] = math.nan, math.inf, 0.0
    q[4, 1] = 3e38
    got, _ = attn.attn_qk_norm_rope(*_cuda(c))
    _ok()
    got = got.cpu()
    assert torch.isnan(got[1, 0]).all() and torch.isnan(got[2, 1, 100])
    assert (got[2, 1, :100] == 0).all() and (got[2, 1, 101:] == 0).all()
    assert (got[3, 0] == 0).all() and (got[4, 1] == 0).all()
    clean = torch.ones(8, 2, dtype=torch.bool)
    for t, h in ((1, 0), (2, 1), (3, 0), (4, 1)):
        clean[t, h] = False
    want, mag = _rope.forward(torch.where(clean[..., None], q, 1.0), c[2], c[4], c[5], c[6], False)
    _rope.check("q", got[clean], want[clean], mag[clean])


def test_bad_positions_are_reported():
    c = _case(6, 4, 2, 128, seed=8, max_pos=10)
    c[6][1], c[6][4] = 10, -1
    d = _cuda(c)
    q_out, k_out = torch.full_like(d[0], 9.0), torch.full_like(d[1], 9.0)
    attn.attn_qk_norm_rope(*d, q_out=q_out, k_out=k_out)
    _ok(attn.ATTN_ERR_INDEX)
    _ok()
    bad, good = [1, 4], [0, 2, 3, 5]
    assert (q_out[bad] == 9.0).all() and (k_out[bad] == 9.0).all()
    part = [t[good] if i in (0, 1, 6) else t for i, t in enumerate(c)]
    _check_forward(part, (q_out[good], k_out[good]), False)
    # Backward: their gradients are not written and the weights' sums do without them.
    g = torch.Generator().manual_seed(9)
    dq, dk = (torch.randn(t.shape, generator=g).to(torch.bfloat16) for t in c[:2])
    gq, gk = torch.full_like(d[0], 9.0), torch.full_like(d[1], 9.0)
    got = attn.attn_qk_norm_rope_bwd(dq.cuda(), dk.cuda(), *d, dq=gq, dk=gk)
    _ok(attn.ATTN_ERR_INDEX)
    assert (gq[bad] == 9.0).all() and (gk[bad] == 9.0).all()
    _check_backward(part, (dq[good], dk[good]), (gq[good], gk[good], *got[2:]), False)


# ---------------------------------------------------------------- backward

def _check_backward(c, dys, got, inter, mode="rtne", eps=1e-6):
    q, k, wq, wk, cos, sin, pos = c
    for i, (x, w) in enumerate(((q, wq), (k, wk))):
        dx, mag, dw, mag_w = _rope.backward(dys[i], x, w, cos, sin, pos, inter, eps)
        _rope.check("d" + "qk"[i], got[i], dx, mag, mode)
        _rope.check_weight("dw_" + "qk"[i], got[2 + i], dw, mag_w)


def _grads_of(c, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(t.shape, generator=g).to(torch.bfloat16) for t in c[:2]]


@pytest.mark.parametrize("kw", ROPE_KW)
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (5, 8, 2), (37, 9, 3), (700, 17, 1), (3, 1, 40)])
def test_backward(T, Hq, Hkv, kw):
    c = _case(T, Hq, Hkv, kw["rot"], seed=T + Hq)
    dys = _grads_of(c, T)
    got = attn.attn_qk_norm_rope_bwd(*_cuda(dys), *_cuda(c), interleaved=kw["interleaved"])
    _ok()
    _check_backward(c, dys, got, kw["interleaved"])


@pytest.mark.parametrize("mode", ["rtne", "rtna", "rtz"])
@pytest.mark.parametrize("scale,eps", [(1e-3, 1e-2), (1e3, 0.0)])
def test_backward_modes_and_scales(mode, scale, eps):
    c = _case(70, 6, 2, 64, seed=15, scale=scale)
    dys = _grads_of(c, 3)
    got = attn.attn_qk_norm_rope_bwd(*_cuda(dys), *_cuda(c), rounding=mode, eps=eps)
    _ok()
    _check_backward(c, dys, got, False, mode, eps)


@pytest.mark.parametrize("inter", [False, True])
def test_backward_against_differences(inter):
    """The kernel's gradients along a direction against differences of the formula in 64 bits.
    The quotient's own error: h^2 times a third derivative of the order of the sum, 1e-8; the
    gradients' roundings (2^-8 each, independent) leave 2^-8 |dx| |v| / sqrt(n) * a few."""
    c = _case(20, 3, 2, 64, seed=16)
    dys = _grads_of(c, 4)
    got = attn.attn_qk_norm_rope_bwd(*_cuda(dys), *_cuda(c), interleaved=inter)
    _ok()
    q, k, wq, wk, cos, sin, pos = c
    g = torch.Generator().manual_seed(17)
    h = 1e-4
    for i, (x, w) in enumerate(((q, wq), (k, wk))):
        f = lambda x, w: (_rope.forward(x, w, cos, sin, pos, inter)[0] * dys[i].double()).sum()
        v, vw = (torch.randn(t.shape, generator=g, dtype=torch.float64) for t in (x, w))
        x, w = x.double(), w.double()
        dx, dw = got[i].cpu().double(), got[2 + i].cpu().double()
        rounding = 2.0 ** -8 * float((dx * v).norm())       # one standard deviation is under 0.6 of it
        assert abs(float((f(x + h * v, w) - f(x - h * v, w)) / (2 * h) - (dx * v).sum())) <= 5 * rounding + 1e-6 * float(dx.norm())
        assert abs(float((f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h) - (dw * vw).sum())) <= 1e-5 * float(dw.norm()) * 12


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
def test_backward_layouts_and_views(layout):
    """4-D tensors, gradients into columns of one tensor, and in place of what came in."""
    B, S, Hq, Hkv = 2, 23, 6, 2
    c = _case(B * S, Hq, Hkv, 128, seed=18)
    dys = _grads_of(c, 5)
    packed = attn.attn_qk_norm_rope_bwd(*_cuda(dys), *_cuda(c))
    q, k, wq, wk, cos, sin, pos = _cuda(c)
    form = lambda t: (t.view(B, S, -1, 128) if layout == "bshd"
                      else t.view(B, S, -1, 128).transpose(1, 2).contiguous())
    dq, dk, q, k = (form(t) for t in (*_cuda(dys), q, k))
    fused = torch.full((B, S, Hq + 2 * Hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    views = list(fused.split((Hq, Hkv, Hkv), 2)[:2])
    if layout == "bhsd":
        views = [t.transpose(1, 2) for t in views]
    rest = (q, k, wq, wk, cos, sin, pos.view(B, S))
    runs = [attn.attn_qk_norm_rope_bwd(dq, dk, *rest, layout=layout),
            attn.attn_qk_norm_rope_bwd(dq, dk, *rest, layout=layout, dq=views[0], dk=views[1]),
            attn.attn_qk_norm_rope_bwd(dq, dk, *rest, layout=layout, dq=dq, dk=dk)]
    _ok()
    assert (fused[:, :, Hq + Hkv:] == 7.0).all()
    for got in runs:
        for i in range(4):
            t = got[i] if i > 1 or layout == "bshd" else got[i].transpose(1, 2)
            assert torch.equal(t.contiguous().view(-1).view(torch.int16), packed[i].view(-1).view(torch.int16))


# ---------------------------------------------------------------- the paged form

def _pages(layout, n, page, Hkv, fill=7.0):
    shape = (n, page, Hkv, 128) if layout == "bshd" else (n, Hkv, page, 128)
    return [torch.full(shape, fill, dtype=torch.bfloat16, device="cuda") for _ in range(2)]


def _slot_rows(pages, slots, page, layout):
    p, i = slots // page, slots % page
    return pages[p, i] if layout == "bshd" else pages[p, :, i]


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("T,Hq,Hkv,page,rot,inter", [
    (1, 1, 1, 1, 128, False), (64, 8, 2, 16, 128, False), (41, 14, 9, 5, 64, True), (300, 4, 1, 33, 96, False),
])
def test_paged(layout, T, Hq, Hkv, page, rot, inter):
    c = _case(T, Hq, Hkv, rot, seed=T + page)
    g = torch.Generator().manual_seed(T)
    v = torch.randn(T, Hkv, 128, generator=g).to(torch.bfloat16)
    n = T // page + 3
    slots = torch.randperm(n * page, generator=g)[:T].to(torch.int32)
    if T > 3:
        slots[T // 2] = -1                                   # padding
    kp, vp = _pages(layout, n, page, Hkv)
    q, k, wq, wk, cos, sin, pos = _cuda(c)
    q_out = attn.attn_qk_norm_rope_paged(q, k, v.cuda(), wq, wk, cos, sin, pos, slots.cuda(), kp, vp,
                                         interleaved=inter, layout=layout)
    _ok()
    kept = slots >= 0
    at = slots[kept].long()
    rows = _slot_rows(kp.cpu(), at, page, layout)
    _rope.check("q", q_out, *_rope.forward(c[0], c[2], c[4], c[5], c[6], inter))
    want, mag = _rope.forward(c[1], c[3], c[4], c[5], c[6], inter)
    _rope.check("k", rows, want[kept], mag[kept])
    assert torch.equal(_slot_rows(vp.cpu(), at, page, layout).view(torch.int16), v[kept].view(torch.int16))
    for pages in (kp, vp):                                   # nothing else was written
        flat = (pages if layout == "bshd" else pages.transpose(1, 2)).reshape(-1, Hkv * 128).cpu()
        other = torch.ones(n * page, dtype=torch.bool)
        other[at] = False
        assert (flat[other] == 7.0).all()


def test_pages_of_one_tensor_and_columns_of_one_projection():
    """Keys and values as halves of one tensor's pages, q, k and v as columns of one projection's
    output: the same bits."""
    B, S, Hq, Hkv, page, n = 3, 4, 6, 2, 8, 5
    c = _case(B * S, Hq, Hkv, 128, seed=20)
    q, k, wq, wk, cos, sin, pos = _cuda(c)
    fused = torch.randn(B, S, Hq + 2 * Hkv, 128, device="cuda").to(torch.bfloat16)
    fused[:, :, :Hq], fused[:, :, Hq:Hq + Hkv] = q.view(B, S, Hq, 128), k.view(B, S, Hkv, 128)
    slots = torch.randperm(n * page)[:B * S].to(torch.int32).cuda().view(B, S)
    one = torch.full((n, 2, page, Hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    apart = _pages("bshd", n, page, Hkv)
    args = (wq, wk, cos, sin, pos.view(B, S), slots)
    views = fused.split((Hq, Hkv, Hkv), 2)
    a = attn.attn_qk_norm_rope_paged(*views, *args, one[:, 0], one[:, 1], layout="bshd")
    b = attn.attn_qk_norm_rope_paged(*(t.contiguous() for t in views), *args, *apart, layout="bshd")
    _ok()
    for x, y in ((a, b), (one[:, 0], apart[0]), (one[:, 1], apart[1])):
        assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))


def test_bad_slots_are_reported():
    c = _case(5, 4, 2, 128, seed=21)
    q, k, wq, wk, cos, sin, pos = _cuda(c)
    kp, vp = _pages("bhsd", 3, 4, 2)
    slots = torch.tensor([0, 12, -2, 11, -1], dtype=torch.int32).cuda()
    q_out = torch.full_like(q, 9.0)
    attn.attn_qk_norm_rope_paged(q, k, k, wq, wk, cos, sin, pos, slots, kp, vp, q_out=q_out)
    _ok(attn.ATTN_ERR_INDEX)
    assert (q_out[1:3] == 9.0).all() and not (q_out[[0, 3, 4]] == 9.0).any()
    assert (kp == 7.0).sum() == (12 - 2) * 2 * 128 and torch.equal(vp[0, :, 0], k[0]) and torch.equal(vp[2, :, 3], k[3])


def test_offsets_beyond_32_bits():
    """Tokens and pages whose byte and element offsets pass 2^32."""
    T, Hq, Hkv, page = 70000, 256, 2, 16
    n = (1 << 33) // (page * Hkv * 256) + 2
    q = torch.zeros(T, Hq, 128, dtype=torch.bfloat16, device="cuda")
    assert q.numel() > 1 << 31
    c = _case(T, 1, Hkv, 128, seed=22, max_pos=100)
    _, k, wq, wk, cos, sin, pos = _cuda(c)
    at = torch.tensor([0, T // 2, T - 1])
    q[at.cuda()] = torch.randn(3, Hq, 128, device="cuda").to(torch.bfloat16)
    shape = (n, page, Hkv, 128)
    kp, vp = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = (n * page - 1 - torch.arange(T, dtype=torch.int32)).cuda()
    q_out = attn.attn_qk_norm_rope_paged(q, k, k, wq, wk, cos, sin, pos, slots, kp, vp, layout="bshd")
    _ok()
    part = lambda t: t[at.to(t.device)].cpu()
    _rope.check("q", part(q_out), *_rope.forward(part(q), c[2], c[4], c[5], part(c[6]), False))
    want, mag = _rope.forward(c[1], c[3], c[4], c[5], c[6], False)
    rows = kp.view(-1, Hkv, 128)[slots.long()]
    _rope.check("k", rows, want, mag)
    assert torch.equal(vp.view(-1, Hkv, 128)[slots.long()], k)
    del q_out, kp, vp
    dq, dk, _, _ = attn.attn_qk_norm_rope_bwd(q, k, q, k, wq, wk, cos, sin, pos)
    _ok()
    dx, mag, _, _ = _rope.backward(part(q), part(q), c[2], c[4], c[5], part(c[6]), False)
    _rope.check("dq", part(dq), dx, mag)


# ---------------------------------------------------------------- streams, graphs, workspaces

def test_bits_repeat_and_replay_in_a_graph():
    c = _case(200, 9, 3, 128, seed=23)
    d, dys = _cuda(c), _cuda(_grads_of(c, 6))
    kp, vp = _pages("bhsd", 30, 8, 3)
    slots = torch.randperm(240)[:200].to(torch.int32).cuda()

    def step():
        y = attn.attn_qk_norm_rope(*d)
        q_out = attn.attn_qk_norm_rope_paged(d[0], d[1], d[1], *d[2:], slots, kp, vp)
        return (*y, q_out, kp.clone(), vp.clone(), *attn.attn_qk_norm_rope_bwd(*dys, *d))

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    d[0].copy_(d[0].flip(0))
    d[6].copy_(d[6].flip(0))
    graph.replay()
    _ok()
    fresh = step()
    _ok()
    for a, b in zip(first, again):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    for a, b in zip(held, fresh):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_given_workspace_is_kept_to():
    c = _case(500, 5, 2, 128, seed=24)
    d, dys = _cuda(c), _cuda(_grads_of(c, 7))
    want = attn.attn_qk_norm_rope_bwd(*dys, *d)
    need = attn.qk_norm_rope_bwd_workspace_bytes(1, 500, 5, 2)
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    got = attn.attn_qk_norm_rope_bwd(*dys, *d, workspace=ws[:need])
    _ok()
    assert (ws[need:] == 0x7F).all()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    with pytest.raises(attn.AttnError) as e:
        attn.attn_qk_norm_rope_bwd(*dys, *d, workspace=ws[:need - 16])
    assert e.value.status == attn.ATTN_ERR_INVALID_ARG
