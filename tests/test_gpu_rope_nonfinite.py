"""NaN and infinities in the rows, weights and gradients of the norms with rotation: they reach exactly
the results whose formula has them. A column that is not rotated (at or after rotary_dim) has none of
its neighbour in it, and the neighbour none of it."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _rope

pytestmark = pytest.mark.gpu

T, HQ, HKV = 5, 2, 1
FORMS = [(128, False), (128, True), (64, False), (64, True), (96, False), (96, True), (16, False), (16, True),
         (112, True)]
VALUES = [math.nan, math.inf, -math.inf]


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


def _ok():
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK


def _case(rot, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    w = [(1 + 0.3 * torch.randn(128, generator=g)).to(torch.bfloat16) for _ in range(2)]
    pos = torch.tensor([3, 0, 8, 1, 6], dtype=torch.int32)  # the second: cos 1, sin 0
    return [r(T, HQ, 128), r(T, HKV, 128), *w, *_rope.table(9, rot), pos], [r(T, HQ, 128), r(T, HKV, 128)]


def _columns(rot):
    """Both columns of a pair in either form, the last rotated one, and, past them, an even one, an odd
    one and the last."""
    return sorted({0, 1, rot // 2, rot - 1} | ({rot, rot + 3, 127} if rot < 128 else set()))


def _same(name, got, want, mag, u):
    """The same kinds everywhere, and where the formula is finite its value within the bounds of _rope."""
    got = got.cpu().double()
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(kind(got), kind(want)), (name, kind.__name__, (kind(got) != kind(want)).nonzero()[:8].tolist())
    fin = torch.isfinite(want)
    e = _rope.FP32 * mag[fin]
    over = (got[fin] - want[fin]).abs() - (e + u * (want[fin].abs() + e))
    assert over.numel() == 0 or over.max() <= 1e-30, (name, float(over.max()))


def _forward(c, inter):
    got = attn.attn_qk_norm_rope(*(t.cuda() for t in c), interleaved=inter)
    kp, vp = (torch.zeros(T, HKV, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    d = [t.cuda() for t in c]
    q_out = attn.attn_qk_norm_rope_paged(d[0], d[1], d[1], *d[2:], torch.arange(T, dtype=torch.int32).cuda(), kp, vp,
                                         interleaved=inter)
    _ok()
    for i, n in enumerate("qk"):
        want, mag = _rope.forward(c[i], c[2 + i], c[4], c[5], c[6], inter)
        _same(n, got[i], want, mag, 2.0 ** -8)
        _same(n + " paged", (q_out, kp[:, :, 0])[i], want, mag, 2.0 ** -8)


def _backward(c, dys, inter):
    got = attn.attn_qk_norm_rope_bwd(*(t.cuda() for t in (*dys, *c)), interleaved=inter)
    _ok()
    for i, n in enumerate("qk"):
        dx, mag, dw, mag_w = _rope.backward(dys[i], c[i], c[2 + i], c[4], c[5], c[6], inter)
        _same("d" + n, got[i], dx, mag, 2.0 ** -8)
        _same("dw " + n, got[2 + i], dw, mag_w, 0.0)


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("rot,inter", FORMS)
def test_in_a_row(rot, inter, value):
    for col in _columns(rot):
        c, dys = _case(rot, seed=col)
        c[0][2, 1, col] = c[1][1, 0, col] = value
        _forward(c, inter)
        _backward(c, dys, inter)


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("rot,inter", FORMS)
def test_in_a_weight(rot, inter, value):
    for col in _columns(rot):
        c, dys = _case(rot, seed=200 + col)
        c[2][col] = c[3][127 - col] = value
        _forward(c, inter)
        _backward(c, dys, inter)


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("rot,inter", FORMS)
def test_in_a_gradient(rot, inter, value):
    for col in _columns(rot):
        c, dys = _case(rot, seed=400 + col)
        dys[0][2, 1, col] = dys[1][1, 0, col] = value
        _backward(c, dys, inter)


@pytest.mark.parametrize("rot,inter", FORMS)
def test_a_root_that_overflows(rot, inter):
    """Without eps, squares that are 0 in fp32 make r infinite: a column that is not rotated is x r w by
    itself, an infinity of the sign of x w."""
    c, _ = _case(rot, seed=600)
    c[0][3, 0] = (1e-30 * torch.randn(128, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16)
    got, _ = attn.attn_qk_norm_rope(*(t.cuda() for t in c), interleaved=inter, eps=0.0)
    _ok()
    want = math.inf * torch.sign(c[0][3, 0, rot:].float() * c[2][rot:].float().sign())
    assert torch.equal(got[3, 0, rot:].cpu().float(), want)


@pytest.mark.parametrize("rot,inter", [f for f in FORMS if f[0] < 128])
def test_signed_zeros(rot, inter):
    """A zero in a column that is not rotated keeps its sign, times the weight's, beside values and zeros of
    either sign."""
    c, _ = _case(rot, seed=700)
    signs = torch.tensor([1.0, -1.0, -1.0, 1.0]).repeat(32).to(torch.bfloat16)
    c[0][2, 1, rot:] = 0.0 * signs[rot:]
    c[0][3, 0, rot + 1::2] = -0.0
    c[2][rot + 3::4] *= -1
    d = [t.cuda() for t in c]
    got, _ = attn.attn_qk_norm_rope(*d, interleaved=inter)
    _ok()
    want = torch.signbit(c[0]) ^ torch.signbit(c[2])
    assert torch.equal(torch.signbit(got.cpu())[..., rot:], want[..., rot:])
