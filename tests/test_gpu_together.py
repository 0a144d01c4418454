"""The sampling and training calls together, as a user runs them: completions of one prompt
sampled token by token against growing caches (attn_fwd_prefix), then one training step
on the sampled sequences, packed (attn_fwd_varlen_lse, attn_bwd_varlen)."""
import math

import pytest
import torch

import bf16_forward_attention_gb300 as attn
from bf16_forward_attention_gb300 import build

import _grad
from _parity import assert_parity, bits_of, compare

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    attn.load_library()


def test_sampling_then_training():
    B, Hq, Hkv, Sp, T = 3, 4, 2, 150, 40
    stop = [40, 23, 1]                       # completion lengths
    g = torch.Generator().manual_seed(77)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    kp, vp, qp = r(Sp, Hkv, 128), r(Sp, Hkv, 128), r(Sp, Hq, 128)
    q_new, k_new, v_new = r(T, B, Hq, 128), r(T, B, Hkv, 128), r(T, B, Hkv, 128)

    # ---- sampling: every step appends a token to the caches of the sequences still running.
    KP, VP = kp.cuda(), vp.cuda()
    cache_k = torch.full((B, T, Hkv, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    cache_v = cache_k.clone()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    steps = []
    ws = torch.empty(attn.prefix_workspace_bytes(B, Hq, Hkv, 1, Sp, T), dtype=torch.uint8, device="cuda")
    for t in range(T):
        for b in range(B):
            if t < stop[b]:
                cache_k[b, t], cache_v[b, t] = k_new[t, b].cuda(), v_new[t, b].cuda()
        lens.copy_(torch.tensor([min(t + 1, n) for n in stop], dtype=torch.int32))
        out, lse = attn.attn_fwd_prefix(q_new[t][:, None].cuda(), KP, VP, cache_k, cache_v, lens,
                                        layout="bshd", workspace=ws)
        steps.append((out[:, 0], lse[:, :, 0]))

    # ---- training on the whole sequences, prompt included, packed.
    seqs = [Sp + n for n in stop]
    cu = torch.tensor([0] + torch.tensor(seqs).cumsum(0).tolist(), dtype=torch.int32).cuda()
    cat = lambda p, new: torch.cat([torch.cat([p, new[:n, b]]) for b, n in enumerate(stop)])
    q, k, v = cat(qp, q_new), cat(kp, k_new), cat(vp, v_new)
    do = r(*q.shape)
    Q, K, V, DO = (x.cuda() for x in (q, k, v, do))
    out, lse = attn.attn_fwd_varlen_lse(Q, K, V, cu, cu, max(seqs), causal=True)
    grads = attn.attn_bwd_varlen(DO, Q, K, V, out, lse, cu, cu, max(seqs), max(seqs), causal=True)
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK

    at = 0
    sampled, exact = [], []
    for b, n in enumerate(stop):
        rows = slice(at, at + seqs[b])
        want, bound = _grad.sequence(q[rows], k[rows], v[rows], do[rows], SCALE, True)
        for name, x in zip(("dq", "dk", "dv"), grads):
            _grad.check(f"{name} of sequence {b}", x[rows], want[name], bound[name])
        assert_parity(compare(bits_of(out[rows]), want["out"].numpy(), "rtne"), excess=True)
        # Each sampled token attended to what its row attends to in training.
        for t in range(n):
            o, l = steps[t]
            sampled.append(o[b])
            exact.append(want["out"][Sp + t])
            assert (l[b].cpu().double() - want["lse"][:, Sp + t]).abs().max() <= 1e-4
            assert (l[b] - lse[:, at + Sp + t]).abs().max() <= 2e-5
        at += seqs[b]
    # All sampled tokens as one: the contract's share of outputs beyond one unit in the last
    # place (0.1%) is under one output of a token's 512, so a token by itself cannot be held
    # to it.
    assert_parity(compare(bits_of(torch.stack(sampled)), torch.stack(exact).numpy(), "rtne"), excess=True)


def test_large_offsets():
    """Tensors of more than 2^31 elements: the last batch entry of a cache, and the last rows
    of a backward pass, lie beyond 32-bit offsets."""
    g = torch.Generator(device="cuda").manual_seed(78)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    cap = 8_500_000                          # 2 * cap * 128 > 2^31
    k = torch.empty(2, cap, 1, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    n = [700, cap]
    for b, m in enumerate(n):                # the first 700 keys, and entry 1's last 700, are drawn
        k[b, :m], v[b, :m] = 0, 0
        k[b, m - 700:m], v[b, m - 700:m] = r(700, 1, 128), r(700, 1, 128)
    q, kp, vp = r(2, 1, 4, 128), r(130, 1, 128), r(130, 1, 128)
    out, lse = attn.attn_fwd_prefix(q, kp, vp, k, v, torch.tensor(n, dtype=torch.int32, device="cuda"),
                                    layout="bshd")
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    for b, m in enumerate(n):
        keys = torch.cat([kp[:, 0], k[b, m - 700:m, 0]]).double()
        vals = torch.cat([vp[:, 0], v[b, m - 700:m, 0]]).double()
        s = q[b, 0].double() @ keys.T * SCALE
        w = torch.exp(s)
        total = w.sum(1, keepdim=True) + (m - 700)     # zero keys: weight 1 each, value 0
        want = (w @ vals) / total
        assert (lse[b, :, 0].double() - torch.log(total[:, 0])).abs().max() <= 1e-4
        # out: one unit in the last place and, for 8.5 million terms, fp32 sums of them.
        assert ((out[b, 0].double() - want).abs() <= 2 ** -8 * want.abs() + 1e-4 * want.abs().max()).all()
    del k, v
    Sq, H, Sk = 2_150_000, 8, 60             # Sq * H * 128 > 2^31
    q, k, v = torch.zeros(1, Sq, H, 128, dtype=torch.bfloat16, device="cuda"), r(1, Sk, H, 128), r(1, Sk, H, 128)
    do = torch.zeros_like(q)
    q[0, -300:], do[0, -300:] = r(300, H, 128), r(300, H, 128)
    out, lse = attn.attn_fwd_lse(q, k, v, layout="bshd")
    dq, dk, dv = attn.attn_bwd(do, q, k, v, out, lse, layout="bshd")
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    # The other rows have dout = 0 and give nothing.
    want, bound = _grad.sequence(q[0, -300:].cpu(), k[0].cpu(), v[0].cpu(), do[0, -300:].cpu(), SCALE, False)
    assert (dq[0, :-300] == 0).all()
    _grad.check("dq", dq[0, -300:], want["dq"], bound["dq"])
    _grad.check("dk", dk[0], want["dk"], bound["dk"])
    _grad.check("dv", dv[0], want["dv"], bound["dv"])


def test_two_graphs_and_two_streams():
    """Two captured graphs that share the pool of a capture, replayed in turn, and eager calls on
    two streams at once: each call has a workspace of its own."""
    g = torch.Generator().manual_seed(79)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    sets = [(r(1, 500, 4, 128), r(1, 500, 2, 128), r(1, 500, 2, 128), r(1, 500, 4, 128)) for _ in range(2)]

    def step(q, k, v, do):
        out, lse = attn.attn_fwd_lse(q, k, v, layout="bshd", causal=True)
        return attn.attn_bwd(do, q, k, v, out, lse, layout="bshd", causal=True)

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    graphs, held = [], []
    pool = torch.cuda.graph_pool_handle()
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            held.append(step(*s))
        graphs.append(graph)
    for _ in range(3):
        for graph, h, w in zip(graphs, held, want):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(h, w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    assert attn.attn_fwd_last_error() == attn.ATTN_OK
    for i in range(2):
        for x in got[i]:
            assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(x, want[i]))
