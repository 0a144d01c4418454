"""Backward pass over long streamed ranges: sums of more tiles than one tensor-memory
accumulator takes (256 tiles of 128), with and without the mask, packed, and shared between CTAs."""
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


def _rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _exact(q, k, v, do, causal, rows=1024, bounds=True):
    """(S, H, d) tensors of one sequence on the GPU: gradients and their error bounds in 64 bits, a
    block of query rows at a time."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    Sq, Hq, _ = q.shape
    Sk, Hkv, _ = k.shape
    want = dict(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    bound = {n: torch.zeros_like(t) for n, t in want.items()}
    key = torch.arange(Sk, device="cuda")
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        for a in range(0, Sq, rows):
            i = slice(a, min(Sq, a + rows))
            last = Sk - 1
            if causal:
                last = torch.arange(i.start, i.stop, device="cuda")[:, None] + Sk - Sq
            seen = (key <= last).expand(i.stop - a, Sk)
            r = _grad.one_head(q[i, h], k[:, kv], v[:, kv], do[i, h], SCALE, seen)
            want["dq"][i, h] = r["dq"]
            want["dk"][:, kv] += r["dk"]
            want["dv"][:, kv] += r["dv"]
            if bounds:
                b = _grad.head_bounds(r, q[i, h], k[:, kv], do[i, h], SCALE, _grad.U)
                bound["dq"][i, h] = b["dq"]
                bound["dk"][:, kv] += b["dk"]
                bound["dv"][:, kv] += b["dv"]
            del r
    return {n: t.cpu() for n, t in want.items()}, {n: t.cpu() for n, t in bound.items()}


def test_long_sums_are_not_biased():
    """dK and dV of a key/value head of 8 query heads over 32768 queries each: 2048 tiles in one CTA
    (the call has a key tile for every SM). The signed error, relative to the sum of magnitudes, has
    to stay under a quarter of what one rounding to bf16 may take (2^-8 / 4): roundings to nearest
    average out over the 311296 elements, a truncated accumulation does not."""
    r = _rand(201)
    Sq, Sk, Hq, Hkv = 32768, 2432, 64, 8
    assert Hkv * ((Sk + 127) // 128) >= torch.cuda.get_device_properties(0).multi_processor_count
    q, k, v = r(1, Sq, Hq, 128), r(1, Sk, Hkv, 128), r(1, Sk, Hkv, 128)
    do = (r(1, Sq, Hq, 128).float() * 0.5 + 1).to(torch.bfloat16)
    out, lse = attn.attn_fwd_lse(q, k, v, layout="bshd")
    grads = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd")
    _ok()
    want, _ = _exact(q[0, :, :8], k[0, :, :1], v[0, :, :1], do[0, :, :8], False, 4096, bounds=False)
    for n, g in (("dk", grads[1][0, :, :1]), ("dv", grads[2][0, :, :1])):
        w = want[n]
        signed = ((g.cpu().double() - w) * w.sign()).sum() / w.abs().sum()
        assert abs(signed) < 2.0 ** -10, (n, float(signed))
        assert (g.cpu().double() - w).norm() <= 6e-3 * w.norm(), n


@pytest.mark.parametrize("Sq,Sk,causal", [
    (33100, 33100, True),    # up to 259 tiles in both kernels
    (300, 33000, False),     # the keys of few queries: shared between CTAs
    (20000, 33000, False),   # dQ: 258 key tiles, one CTA each
    (33000, 20000, False),   # dK and dV: 258 query tiles
    (32768, 32768, True),    # exactly 256
    (65700, 2000, True),     # rows without keys, then two accumulators
])
def test_long_ranges(Sq, Sk, causal):
    r = _rand(Sq + Sk)
    q, k, v, do = r(1, Sq, 1, 128), r(1, Sk, 1, 128), r(1, Sk, 1, 128), r(1, Sq, 1, 128)
    out, lse = attn.attn_fwd_lse(q, k, v, layout="bshd", causal=causal)
    grads = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd", causal=causal)
    again = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd", causal=causal)
    _ok()
    want, bound = _exact(q[0], k[0], v[0], do[0], causal)
    for n, g, a in zip(("dq", "dk", "dv"), grads, again):
        assert torch.equal(g.view(torch.int16), a.view(torch.int16)), n
        _grad.check(n, g[0], want[n], bound[n])


def test_grouped_and_packed():
    """A packed batch whose first sequence takes two accumulators of dK and dV (three heads of 100
    tiles) and whose others take one; rows behind the last sequence stay."""
    r = _rand(204)
    lq, lk, extra = [12700, 0, 900, 130], [1500, 40, 0, 131], 50
    nq, nk = sum(lq) + extra, sum(lk) + extra
    Hq, Hkv = 114, 38   # with these the plan leaves every key tile to one CTA
    q, do, k, v = r(nq, Hq, 128), r(nq, Hq, 128), r(nk, Hkv, 128), r(nk, Hkv, 128)
    B = len(lq)
    assert attn.bwd_varlen_workspace_bytes(B, Hq, Hkv, nq, nk, max(lq), max(lk)) == (
        Hq * (nq // 128 + B + 1) * 1024 + 2 * Hkv * (nk // 128 + B + 1) * 128 * 128 * 4)
    for t in (q, do, k, v):
        t[-extra:] = math.nan
    cu = [torch.tensor([0] + torch.tensor(x).cumsum(0).tolist(), dtype=torch.int32).cuda() for x in (lq, lk)]
    out, lse = torch.full_like(q, math.nan), torch.zeros(Hq, nq, device="cuda")
    attn.attn_fwd_varlen_lse(q, k, v, *cu, max(lq), out=out, lse=lse)
    grads = [torch.full_like(x, 9.0) for x in (q, k, v)]
    attn.attn_bwd_varlen(do, q, k, v, out, lse, *cu, max(lq), max(lk), dq=grads[0], dk=grads[1], dv=grads[2])
    _ok()
    assert all((x[-extra:] == 9.0).all() for x in grads)
    a = c = 0
    for b, (n, m) in enumerate(zip(lq, lk)):
        got = grads[0][a:a + n], grads[1][c:c + m], grads[2][c:c + m]
        if n == 0 or m == 0:
            assert all((x == 0).all() for x in got)
        else:
            for kv in (0, Hkv - 1):
                h = slice(3 * kv, 3 * kv + 3)
                want, bound = _exact(q[a:a + n, h], k[c:c + m, kv:kv + 1], v[c:c + m, kv:kv + 1], do[a:a + n, h],
                                     False, 8192)
                for name, x in zip(("dq", "dk", "dv"), (got[0][:, h], got[1][:, kv:kv + 1], got[2][:, kv:kv + 1])):
                    _grad.check(f"{name} of sequence {b}", x, want[name], bound[name])
        a, c = a + n, c + m


def test_shared_tiles_of_many_accumulators():
    """One query tile over 1.2 million keys: 32 CTAs share it, each over more than 256 tiles."""
    r = _rand(205)
    Sq, Sk = 100, 1_200_000
    q, k, v, do = r(1, Sq, 1, 128), r(1, Sk, 1, 128), r(1, Sk, 1, 128), r(1, Sq, 1, 128)
    out, lse = attn.attn_fwd_lse(q, k, v, layout="bshd")
    dq, dk, dv = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd")
    _ok()
    want, bound = _exact(q[0], k[0], v[0], do[0], False, 50)
    for n, g in zip(("dq", "dk", "dv"), (dq, dk, dv)):
        _grad.check(n, g[0], want[n], bound[n])


def test_non_finite_values_with_two_accumulators():
    """Causal, 259 tiles: a NaN in K near the end and one in dO near the start reach the pairs that
    see them and nothing else."""
    S, at_k, at_o, col = 33100, 33005, 70, 17
    r = _rand(206)
    q, k, v, do = (r(1, S, 1, 128) for _ in range(4))
    run = lambda: attn.attn_bwd(do, q, k, v, *attn.attn_fwd_lse(q, k, v, layout="bshd", causal=True), layout="bshd",
                                causal=True)
    clean = run()
    k[0, at_k, 0, col] = math.nan
    do[0, at_o, 0, col] = math.nan
    dq, dk, dv = run()
    _ok()
    bad_q = torch.zeros(S, dtype=torch.bool, device="cuda")
    bad_q[at_k:] = True
    bad_q[at_o] = True
    assert torch.isnan(dq[0, bad_q, 0]).all() and torch.isfinite(dq[0, ~bad_q, 0]).all()
    assert torch.equal(dq[0, ~bad_q].view(torch.int16), clean[0][0, ~bad_q].view(torch.int16))
    # The rows from at_k on have a NaN logit, so every key that they see gets NaN: all of them.
    assert torch.isnan(dk).all() and torch.isnan(dv).all()
    k[0, at_k, 0, col] = 0.5
    dq, dk, dv = run()
    _ok()
    seen = torch.arange(S, device="cuda") <= at_o
    assert torch.isnan(dk[0, seen]).all() and torch.isfinite(dk[0, ~seen]).all()
    assert torch.isnan(dv[0, seen, 0, col]).all() and torch.isfinite(dv[0, ~seen]).all()
    others = [c for c in range(128) if c != col]
    assert torch.isfinite(dv[0][:, 0, others]).all()
