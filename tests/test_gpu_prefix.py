"""attn_fwd_prefix against attention over the concatenated keys in 64 bits."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

from _parity import assert_parity, bits_of, compare

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


def _inputs(layout, B, Sq, Hq, Hkv, Sp, cap, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    if layout == "bshd":
        return r(B, Sq, Hq, 128), r(Sp, Hkv, 128), r(Sp, Hkv, 128), r(B, cap, Hkv, 128), r(B, cap, Hkv, 128)
    return r(B, Hq, Sq, 128), r(Hkv, Sp, 128), r(Hkv, Sp, 128), r(B, Hkv, cap, 128), r(B, Hkv, cap, 128)


def _exact(q, kp, vp, k, v, lens, layout, causal, scale=SCALE):
    """(out, lse) in 64 bits, heads first, from the keys each row sees."""
    if layout == "bshd":
        q, k, v = (t.transpose(1, 2) for t in (q, k, v))
        kp, vp = (t.transpose(0, 1) for t in (kp, vp))
    q, kp, vp, k, v = (t.double() for t in (q, kp, vp, k, v))
    B, Hq, Sq, d = q.shape
    g = Hq // k.shape[1]
    out, lse = torch.empty(B, Hq, Sq, d, dtype=torch.float64), torch.empty(B, Hq, Sq, dtype=torch.float64)
    for b, n in enumerate(lens):
        for i in range(Sq):
            m = max(0, min(n, i + n - Sq + 1)) if causal else n
            for h in range(Hq):
                keys = torch.cat([kp[h // g], k[b, h // g, :m]])
                vals = torch.cat([vp[h // g], v[b, h // g, :m]])
                s = keys @ q[b, h, i] * scale
                w = torch.exp(s - s.max()) if len(s) else s
                out[b, h, i] = (w @ vals) / w.sum()
                lse[b, h, i] = torch.logsumexp(s, 0)
    return out, lse


def _check(t, lens, layout, causal, got, lse, mode="rtne", scale=SCALE, excess=True):
    want, want_lse = _exact(*t, lens, layout, causal, scale)
    if layout == "bshd":
        want = want.transpose(1, 2).contiguous()
    # Rows of few keys reach magnitudes where one unit in the last place is above the
    # absolute bound: the bound is then on the error beyond the rounding's own.
    assert_parity(compare(bits_of(got), want.numpy(), mode), excess=excess)
    seen = torch.isfinite(want_lse)
    lse = lse.cpu().double()
    assert torch.equal(torch.isfinite(lse), seen)
    assert ((lse - want_lse).abs()[seen] <= 1e-4 + 1e-6 * want_lse.abs()[seen]).all()


def _run(t, lens, layout, **kw):
    c = [x.cuda() for x in t]
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    got = attn.attn_fwd_prefix(*c, n, layout=layout, **kw)
    _ok()
    return got


@pytest.mark.parametrize("layout,B,Sq,Hq,Hkv,Sp,cap,lens,causal", [
    ("bshd", 1, 1, 1, 1, 1, 1, [1], False),
    ("bshd", 3, 1, 8, 2, 300, 64, [0, 1, 64], False),         # a sequence without own keys
    ("bhsd", 3, 1, 8, 2, 129, 50, [17, 16, 15], True),
    ("bshd", 2, 5, 28, 4, 500, 333, [333, 5], True),          # 35 rows per kv head: two blocks
    ("bhsd", 2, 5, 28, 4, 500, 333, [200, 3], True),          # fewer own keys than new tokens
    ("bhsd", 4, 3, 6, 1, 70, 20, [3, 20, 11, 0], False),      # 18 rows
    ("bshd", 5, 1, 7, 7, 1000, 700, [700, 1, 300, 257, 31], False),  # one head a group
    ("bhsd", 2, 1, 40, 2, 64, 2000, [2000, 999], False),      # long own keys: several parts
    ("bshd", 70, 1, 16, 2, 200, 16, None, False),             # more than 256 packed rows
    ("bshd", 1, 9, 4, 4, 2500, 40, [40], True),
    ("bhsd", 5, 1, 12, 2, 3001, 30, [0, 30, 7, 1, 22], False),  # 30 packed rows: one block of 32
    ("bshd", 16, 1, 2, 2, 5000, 8, None, True),               # 16 packed rows, many prefix parts
    ("bhsd", 9, 2, 4, 2, 900, 33, None, True),                # 36 packed rows: the fused kernel
])
def test_parity(layout, B, Sq, Hq, Hkv, Sp, cap, lens, causal):
    t = _inputs(layout, B, Sq, Hq, Hkv, Sp, cap, seed=B * 100 + Sp + cap)
    lens = lens or [i % (cap + 1) for i in range(B)]
    # Slots past a sequence's length hold NaN: they are not read.
    for x in t[3:]:
        for b, n in enumerate(lens):
            (x[b, n:] if layout == "bshd" else x[b, :, n:]).fill_(math.nan)
    out, lse = _run(t, lens, layout, causal=causal)
    _check(t, lens, layout, causal, out, lse)


@pytest.mark.parametrize("mode", ["rtne", "rtna", "rtz"])
@pytest.mark.parametrize("scale", [0.3, -0.1, 0.0])
def test_modes_and_scales(mode, scale):
    t = _inputs("bshd", 2, 2, 4, 2, 150, 90, seed=41)
    out, lse = _run(t, [90, 33], "bshd", rounding=mode, scale=scale, causal=True)
    _check(t, [90, 33], "bshd", True, out, lse, mode, scale)


def test_without_a_prefix():
    t = _inputs("bshd", 3, 2, 6, 3, 0, 100, seed=42)
    lens = [100, 0, 1]
    c = [x.cuda() for x in t]
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = attn.attn_fwd_prefix(c[0], None, None, c[3], c[4], n, layout="bshd", causal=True)
    _ok()
    # Sequence 1 has no key, and sequence 2's first new token sees none: NaN and -Inf.
    assert torch.isnan(out[1]).all() and (lse[1] == -math.inf).all()
    assert torch.isnan(out[2, 0]).all() and (lse[2, :, 0] == -math.inf).all()
    _check(t, lens, "bshd", True, out, lse)


def test_packed_batch_equals_one_sequence():
    """The shared-prefix call against attn_fwd_lse over each sequence's whole keys: both
    within one unit in the last place of the exact value, so within two of each other."""
    B, Hq, Hkv, Sp, cap = 4, 8, 2, 400, 100
    t = _inputs("bshd", B, 1, Hq, Hkv, Sp, cap, seed=43)
    lens = [100, 7, 55, 1]
    out, lse = _run(t, lens, "bshd")
    q, kp, vp, k, v = (x.cuda() for x in t)
    for b, n in enumerate(lens):
        keys, vals = torch.cat([kp, k[b, :n]])[None].contiguous(), torch.cat([vp, v[b, :n]])[None].contiguous()
        o, l = attn.attn_fwd_lse(q[b:b + 1], keys, vals, layout="bshd")
        _ok()
        assert (l[0] - lse[b]).abs().max() <= 2e-5
        assert ((o[0].float() - out[b].float()).abs() <= 2 ** -7 * o[0].float().abs() + 1e-3).all()


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("which", [3, 4])
def test_non_finite_values_at_hidden_keys(which, value):
    """A drafted token's own key or value that earlier tokens do not see reaches only
    the tokens that see it."""
    Sq, n = 5, 37
    t = list(_inputs("bshd", 2, Sq, 6, 2, 100, 64, seed=44))
    clean, clean_lse = _run(t, [n, n], "bshd", causal=True)
    t[which] = t[which].clone()
    j = n - 2                                 # the last but one new token's slot
    t[which][0, j, 1, 5] = value
    out, lse = _run(t, [n, n], "bshd", causal=True)
    sees = torch.arange(Sq) + n - Sq >= j     # tokens 3 and 4
    hit = torch.zeros(2, Sq, 6, 128, dtype=torch.bool)
    if which == 4:
        hit[0, sees, 3:, 5] = True
    elif value != value:
        hit[0, sees, 3:] = True
    else:                                     # an infinite key: +Inf logits make the row NaN
        pos = sees[:, None] & (t[0][0, :, 3:, 5].float() > 0)
        hit[0, :, 3:][pos] = True
    out = out.cpu()
    assert (~torch.isfinite(out[hit])).all()
    assert torch.isfinite(out[~hit]).all()
    hidden = torch.ones(2, Sq, dtype=torch.bool)
    hidden[0, sees] = False
    a, b = out[hidden].float(), clean.cpu()[hidden].float()
    assert ((a - b).abs() <= 2 ** -7 * b.abs() + 1e-6).all()


def test_bad_lengths_are_reported():
    t = _inputs("bshd", 4, 1, 4, 2, 100, 30, seed=45)
    c = [x.cuda() for x in t]
    out = torch.full_like(c[0], 9.0)
    lse = torch.full((4, 4, 1), 9.0, device="cuda")
    n = torch.tensor([30, 31, -1, 0], dtype=torch.int32).cuda()
    attn.attn_fwd_prefix(*c, n, layout="bshd", out=out, lse=lse)
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_ERR_SEQLENS
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    assert (out[1:3] == 9.0).all() and (lse[1:3] == 9.0).all()
    good = [x[[0, 3]] if i in (0, 3, 4) else x for i, x in enumerate(t)]
    _check(good, [30, 0], "bshd", False, out[[0, 3]], lse[[0, 3]])


def test_bits_repeat_and_replay_in_a_graph():
    t = [x.cuda() for x in _inputs("bhsd", 6, 2, 8, 2, 700, 300, seed=46)]
    n = torch.tensor([300, 5, 77, 2, 150, 299], dtype=torch.int32).cuda()
    first = attn.attn_fwd_prefix(*t, n, causal=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = attn.attn_fwd_prefix(*t, n, causal=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = attn.attn_fwd_prefix(*t, n, causal=True)
    n.copy_(torch.tensor([299, 6, 70, 3, 0, 300], dtype=torch.int32))   # lengths move on between replays
    graph.replay()
    _ok()
    fresh = attn.attn_fwd_prefix(*t, n, causal=True)
    _ok()
    for a, b in zip(first, again):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    for a, b in zip(held, fresh):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_given_workspace_is_kept_to():
    t = [x.cuda() for x in _inputs("bshd", 3, 1, 8, 2, 333, 64, seed=47)]
    n = torch.tensor([64, 0, 9], dtype=torch.int32).cuda()
    want = attn.attn_fwd_prefix(*t, n, layout="bshd")
    need = attn.prefix_workspace_bytes(3, 8, 2, 1, 333, 64)
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    got = attn.attn_fwd_prefix(*t, n, layout="bshd", workspace=ws[:need])
    _ok()
    assert (ws[need:] == 0x7F).all()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
