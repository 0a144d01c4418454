"""The operators of a training step and of batched sampling, as measured cases.

  fwd_lse  attention that also leaves every row's log-sum-exp (dense or packed)
  bwd      attention's backward pass from q, k, v, the output, the log-sum-exp and the
           output's gradient (dense or packed)
  prefix   attention of a batch whose sequences share a prompt: every query sees the
           whole shared prefix and its own sequence's keys

With ``own`` false, run() computes them in plain torch operations in 32 bits; with
``own`` true it calls the library.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)


# ---------------------------------------------------------------- cases

def _dense(op, name, layout, B, Hq, Hkv, Sq, Sk, causal):
    return {"name": name, "op": op, "layout": layout, "B": B, "Hq": Hq, "Hkv": Hkv, "Sq": Sq, "Sk": Sk,
            "causal": causal, "packed": False}


def _packed(op, name, n_seq, Hq, Hkv, min_len, max_len, causal, len_seed):
    return {"name": name, "op": op, "packed": True, "n_seq": n_seq, "Hq": Hq, "Hkv": Hkv, "min_len": min_len,
            "max_len": max_len, "causal": causal, "len_seed": len_seed}


def _prefix(name, layout, B, Sq, Hq, Hkv, Sp, cap, min_len, causal, len_seed):
    return {"name": name, "op": "prefix", "layout": layout, "B": B, "Sq": Sq, "Hq": Hq, "Hkv": Hkv, "Sp": Sp,
            "cap": cap, "min_len": min_len, "causal": causal, "len_seed": len_seed}


def listed():
    return [
        # A training forward on the benchmark's 8K length, grouped heads, causal.
        _dense("fwd_lse", "fwd_lse_causal8k", "bshd", 2, 16, 4, 8192, 8192, True),
        # A ragged packed batch of short samples, forward.
        _packed("fwd_lse", "fwd_lse_packed", 13, 8, 8, 17, 1500, True, 5),
        # The smallest training step: two heads of 256 tokens, where latency counts.
        _dense("bwd", "bwd_tiny", "bhsd", 1, 2, 2, 256, 256, False),
        # The 8K self-attention workload, backward.
        _dense("bwd", "bwd_self8k", "bshd", 2, 16, 16, 8192, 8192, False),
        # A causal training step with grouped heads at an ordinary length.
        _dense("bwd", "bwd_causal4k_gqa", "bshd", 1, 32, 8, 4096, 4096, True),
        # Cross-attention to a short ragged key range (text conditioning): few key tiles, many rows.
        _dense("bwd", "bwd_cross77", "bshd", 2, 16, 16, 4096, 77, False),
        # Odd, unequal lengths.
        _dense("bwd", "bwd_ragged", "bhsd", 3, 6, 3, 1021, 1533, False),
        # A packed batch of samples of mixed length, causal, grouped heads.
        _packed("bwd", "bwd_packed", 16, 16, 4, 100, 3800, True, 7),
        # Sampling a handful of completions of a short prompt: latency.
        _prefix("prefix_small", "bshd", 4, 1, 8, 2, 1000, 64, 0, False, 3),
        # 64 completions of an 8K prompt, single tokens.
        _prefix("prefix_decode", "bshd", 64, 1, 32, 8, 8192, 512, 1, False, 11),
        # Drafted tokens: five at a time, odd group of seven heads, head-major caches.
        _prefix("prefix_draft", "bhsd", 48, 5, 28, 4, 5003, 700, 5, True, 13),
        # 256 completions of a 32K prompt, each already up to 2K long.
        _prefix("prefix_large", "bshd", 256, 1, 32, 8, 32768, 2048, 100, False, 17),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd_lse", "bwd", "bwd", "prefix"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 1, 2, 3, 4, 7])
    causal = rng.random() < 0.5
    layout = rng.choice(["bshd", "bhsd"])
    if op == "prefix":
        B = _log(rng, 1, 200)
        Sq = rng.choice([1, 1, 1, 2, 5])
        cap = _log(rng, 8, 1500)
        return {**_prefix("", layout, B, Sq, Hkv * group, Hkv, _log(rng, 64, 24000), cap, min(cap, Sq), causal,
                          rng.randrange(1 << 20))}
    if rng.random() < 0.3:
        return _packed(op, "", _log(rng, 1, 24), Hkv * group, Hkv, 8, _log(rng, 40, 2500), causal,
                       rng.randrange(1 << 20))
    # At most half of the largest dense case's pairs.
    Sq, Sk, B = _log(rng, 8, 6000), _log(rng, 16, 6000), rng.choice([1, 1, 2, 3])
    while B * Hkv * group * Sq * Sk > 16 * 8192 * 8192:
        Sq, Sk = max(8, Sq // 2), max(16, Sk // 2)
    if causal:
        Sk = max(Sq, Sk)
        while B * Hkv * group * Sq * Sk > 16 * 8192 * 8192:
            Sk = max(Sq, Sk // 2)
            Sq = max(8, Sq // 2)
    return _dense(op, "", layout, B, Hkv * group, Hkv, Sq, Sk, causal)


def _lengths(n, lo, hi, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, (n,), generator=g).tolist()


def _case_lengths(case):
    if case["op"] == "prefix":
        return _lengths(case["B"], case["min_len"], case["cap"], case["len_seed"])
    return _lengths(case["n_seq"], case["min_len"], case["max_len"], case["len_seed"])


def _pairs(Sq, Sk, causal):
    """Visible (query, key) pairs of one head; causal aligned at the bottom right."""
    if not causal:
        return Sq * Sk
    off = Sk - Sq
    first = max(0, -off)  # rows before it see no key
    n = Sq - first
    lo, hi = first + off + 1, Sk
    return n * (lo + hi) // 2


def work(case):
    Hq, Hkv, causal = case["Hq"], case["Hkv"], case["causal"]
    if case["op"] == "prefix":
        B, Sq, Sp, lens = case["B"], case["Sq"], case["Sp"], _case_lengths(case)
        own_pairs = sum(sum(max(0, min(n, i + n - Sq + 1)) if causal else n for i in range(Sq)) for n in lens)
        rows = B * Sq * Hq
        return {"bytes": 2 * D * (2 * rows + 2 * Hkv * (Sp + sum(lens))) + 4 * rows + 4 * B,
                "flops": 4 * D * (rows * Sp + Hq * own_pairs)}
    if case["packed"]:
        lens = _case_lengths(case)
        pairs, tq, tk, extra = Hq * sum(_pairs(n, n, causal) for n in lens), sum(lens), sum(lens), 8 * (len(lens) + 1)
    else:
        B = case["B"]
        pairs, tq, tk, extra = B * Hq * _pairs(case["Sq"], case["Sk"], causal), B * case["Sq"], B * case["Sk"], 0
    if case["op"] == "fwd_lse":
        return {"bytes": 2 * D * (2 * tq * Hq + 2 * tk * Hkv) + 4 * tq * Hq + extra, "flops": 4 * D * pairs}
    return {"bytes": 2 * D * (4 * tq * Hq + 4 * tk * Hkv) + 4 * tq * Hq + extra, "flops": 10 * D * pairs}


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Hq, Hkv = case["Hq"], case["Hkv"]
    st = dict(case)
    if case["op"] == "prefix":
        B, Sq, Sp, cap = case["B"], case["Sq"], case["Sp"], case["cap"]
        if case["layout"] == "bshd":
            st["q"] = _randn(g, B, Sq, Hq, D)
            st["kp"], st["vp"] = _randn(g, Sp, Hkv, D), _randn(g, Sp, Hkv, D)
            st["k"], st["v"] = _randn(g, B, cap, Hkv, D), _randn(g, B, cap, Hkv, D)
        else:
            st["q"] = _randn(g, B, Hq, Sq, D)
            st["kp"], st["vp"] = _randn(g, Hkv, Sp, D), _randn(g, Hkv, Sp, D)
            st["k"], st["v"] = _randn(g, B, Hkv, cap, D), _randn(g, B, Hkv, cap, D)
        st["lens"] = torch.tensor(_case_lengths(case), dtype=torch.int32, device="cuda")
        return st
    if case["packed"]:
        lens = _case_lengths(case)
        n = sum(lens)
        st["max_len_here"] = max(lens)
        st["cu"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        st["q"], st["k"], st["v"] = _randn(g, n, Hq, D), _randn(g, n, Hkv, D), _randn(g, n, Hkv, D)
    else:
        B, Sq, Sk = case["B"], case["Sq"], case["Sk"]
        qs, ks = ((B, Sq, Hq, D), (B, Sk, Hkv, D)) if case["layout"] == "bshd" else ((B, Hq, Sq, D), (B, Hkv, Sk, D))
        st["q"], st["k"], st["v"] = _randn(g, *qs), _randn(g, *ks), _randn(g, *ks)
    if case["op"] == "bwd":
        st["dout"] = _randn(g, *st["q"].shape)
        st["out"], st["lse"] = _plain_fwd(st)
    return st


# ---------------------------------------------------------------- plain forms

def _split(st):
    """q as (B, Hkv, g, Sq, D) and k, v as (B, Hkv, 1, Sk, D) in 32 bits, the mask of visible
    pairs (or None), and a function that takes a (B, Hkv, g, S, ...) result back to the
    caller's layout. Packed batches are padded to their longest sequence."""
    Hq, Hkv = st["Hq"], st["Hkv"]
    group = Hq // Hkv
    if st["packed"]:
        cu = st["cu"].long()
        lens = cu[1:] - cu[:-1]
        S = st["max_len_here"]
        pos = torch.arange(S, device="cuda")
        inside = pos < lens[:, None]                                     # (n_seq, S)
        at = torch.where(inside, cu[:-1, None] + pos, 0)
        pad = lambda t: torch.where(inside[..., None, None], t[at].float(), 0.0).transpose(1, 2)
        visible = inside[:, None, :] & inside[:, :, None]                # (n_seq, Sq, Sk)
        if st["causal"]:
            visible = visible & (pos[None, :] <= pos[:, None])
        visible = visible[:, None, None]

        def back(t):                                                     # (n_seq, H, S, ...) -> (tokens, H, ...)
            return t.transpose(1, 2)[inside]
    else:
        pad = lambda t: t.float() if st["layout"] == "bhsd" else t.float().transpose(1, 2)
        Sq, Sk = st["Sq"], st["Sk"]
        visible = None
        if st["causal"]:
            visible = torch.arange(Sk, device="cuda") <= torch.arange(Sq, device="cuda")[:, None] + (Sk - Sq)

        def back(t):
            return t if st["layout"] == "bhsd" else t.transpose(1, 2)
    heads = lambda t: t.unflatten(1, (Hkv, group))
    return pad, heads, visible, back


def _probabilities(q, k, visible):
    s = (q @ k.transpose(-1, -2)) * SCALE
    if visible is not None:
        s = torch.where(visible, s, -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    return e / total.clamp_min(1e-37), (m + torch.log(total)).squeeze(-1)


def _plain_fwd(st):
    pad, heads, visible, back = _split(st)
    q, k, v = heads(pad(st["q"])), pad(st["k"])[:, :, None], pad(st["v"])[:, :, None]
    p, lse = _probabilities(q, k, visible)
    out = back((p @ v).flatten(1, 2)).to(torch.bfloat16)
    lse = lse.flatten(1, 2)
    if st["packed"]:
        lse = back(lse).transpose(0, 1)
    return out.contiguous(), lse.contiguous()


def _plain_bwd(st):
    pad, heads, visible, back = _split(st)
    q, k, v = heads(pad(st["q"])), pad(st["k"])[:, :, None], pad(st["v"])[:, :, None]
    do = heads(pad(st["dout"]))
    p, _ = _probabilities(q, k, visible)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    del p, dp
    dq = ((ds @ k) * SCALE).flatten(1, 2)
    dk = ((ds.transpose(-1, -2) @ q) * SCALE).sum(2)
    return tuple(back(t).to(torch.bfloat16).contiguous() for t in (dq, dk, dv))


def _prefix_parts(st, to):
    """q (B, Hkv, g, Sq, D), prefix keys and values (Hkv, Sp, D), the sequences' own
    (B, Hkv, cap, D), and which of the latter each query sees (B, Sq, cap)."""
    group = st["Hq"] // st["Hkv"]
    major = (lambda t: t) if st["layout"] == "bhsd" else (lambda t: t.transpose(-2, -3))
    q = major(st["q"]).to(to).unflatten(1, (st["Hkv"], group))
    kp, vp, k, v = (major(st[n]).to(to) for n in ("kp", "vp", "k", "v"))
    j = torch.arange(st["cap"], device="cuda")
    n = st["lens"].long()[:, None, None]
    limit = n
    if st["causal"]:
        limit = torch.minimum(n, torch.arange(st["Sq"], device="cuda")[None, :, None] + n - st["Sq"] + 1)
    seen = (j[None, None, :] < limit).expand(-1, st["Sq"], -1)
    return q, kp, vp, k, v, seen


def _plain_prefix(st):
    q, kp, vp, k, v, seen = _prefix_parts(st, torch.float32)
    B, Hkv, g, Sq, _ = q.shape
    Sp = kp.shape[1]
    rows = q.permute(1, 0, 2, 3, 4).reshape(Hkv, B * g * Sq, D)
    s_shared = (rows @ kp.transpose(-1, -2)).view(Hkv, B, g, Sq, Sp) * SCALE
    s_own = (q.flatten(2, 3) @ k.transpose(-1, -2)).view(B, Hkv, g, Sq, -1).permute(1, 0, 2, 3, 4) * SCALE
    s_own = torch.where(seen[None, :, None], s_own, -math.inf)
    m = torch.maximum(s_shared.amax(-1, keepdim=True), s_own.amax(-1, keepdim=True))
    e_shared, e_own = torch.exp(s_shared - m), torch.exp(s_own - m)
    total = e_shared.sum(-1, keepdim=True) + e_own.sum(-1, keepdim=True)
    v_own = torch.where((torch.arange(st["cap"], device="cuda") < st["lens"].long()[:, None])[:, None, :, None], v, 0.0)
    o = (e_shared.reshape(Hkv, B * g * Sq, Sp) @ vp).view(Hkv, B, g, Sq, D)
    o = o + (e_own.permute(1, 0, 2, 3, 4).reshape(B, Hkv, g * Sq, -1) @ v_own).view(B, Hkv, g, Sq, D).transpose(0, 1)
    o = (o / total).transpose(0, 1).flatten(1, 2)                        # (B, Hq, Sq, D)
    lse = (m + torch.log(total)).squeeze(-1).transpose(0, 1).flatten(1, 2)
    if st["layout"] == "bshd":
        o = o.transpose(1, 2)
    return o.to(torch.bfloat16).contiguous(), lse.contiguous()


def run(st):
    if own:
        import bf16_forward_attention_gb300 as attn

        if st["op"] == "prefix":
            return attn.attn_fwd_prefix(st["q"], st["kp"], st["vp"], st["k"], st["v"], st["lens"],
                                        causal=st["causal"], layout=st["layout"])
        if st["op"] == "fwd_lse":
            if st["packed"]:
                return attn.attn_fwd_varlen_lse(st["q"], st["k"], st["v"], st["cu"], st["cu"], st["max_len_here"],
                                                causal=st["causal"])
            return attn.attn_fwd_lse(st["q"], st["k"], st["v"], causal=st["causal"], layout=st["layout"])
        if st["packed"]:
            return attn.attn_bwd_varlen(st["dout"], st["q"], st["k"], st["v"], st["out"], st["lse"], st["cu"],
                                        st["cu"], st["max_len_here"], st["max_len_here"], causal=st["causal"])
        return attn.attn_bwd(st["dout"], st["q"], st["k"], st["v"], st["out"], st["lse"], causal=st["causal"],
                             layout=st["layout"])
    if st["op"] == "prefix":
        return _plain_prefix(st)
    return _plain_fwd(st) if st["op"] == "fwd_lse" else _plain_bwd(st)


# ---------------------------------------------------------------- 64 bits, by the definition

def _attention64(q, k, v, seen):
    """Rows of one head by the definition: q (Sq, D), k and v (Sk, D) in 64 bits."""
    s = torch.einsum("id,jd->ij", q, k) / math.sqrt(D)
    if seen is not None:
        s = s.masked_fill(~seen, -math.inf)
    return torch.softmax(s, -1) @ v, torch.logsumexp(s, -1)


def _sequences(st):
    """For every sequence: the slices of q-like and k-like tensors as (S, H, D) views."""
    if st["packed"]:
        cu = st["cu"].tolist()
        return [(lambda t, a=a, b=b: t[a:b]) for a, b in zip(cu, cu[1:])]
    major = (lambda t: t) if st["layout"] == "bshd" else (lambda t: t.transpose(0, 1))
    return [(lambda t, b=b: major(t[b])) for b in range(st["B"])]


def exact(case, seed):
    w = work(case)
    if w["flops"] > 1.2e13:  # some 20 seconds in 64 bits
        return None
    st = prepare(case, seed)
    Hq, Hkv = case["Hq"], case["Hkv"]
    group = Hq // Hkv
    if case["op"] == "prefix":
        of = (lambda n: st[n].double()) if case["layout"] == "bhsd" else (lambda n: st[n].double().transpose(-2, -3))
        q, kp, vp, k, v = (of(n) for n in ("q", "kp", "vp", "k", "v"))   # head-major
        B, Sq, Sp, g = case["B"], case["Sq"], case["Sp"], group
        o = torch.empty(B, Hq, Sq, D, dtype=torch.float64, device="cuda")
        lse = torch.empty(B, Hq, Sq, dtype=torch.float64, device="cuda")
        lens = st["lens"].tolist()
        for b in range(B):
            n = lens[b]
            mask = torch.ones(Sq, Sp + n, dtype=torch.bool, device="cuda")
            if case["causal"]:
                mask[:, Sp:] = mask[:, Sp:].tril(n - Sq)
            for h in range(Hkv):
                rows = q[b, h * g:(h + 1) * g].reshape(g * Sq, D)
                ob, lb = _attention64(rows, torch.cat([kp[h], k[b, h, :n]]), torch.cat([vp[h], v[b, h, :n]]),
                                      mask.repeat(g, 1))
                o[b, h * g:(h + 1) * g], lse[b, h * g:(h + 1) * g] = ob.view(g, Sq, D), lb.view(g, Sq)
        return (o if case["layout"] == "bhsd" else o.transpose(1, 2).contiguous()), lse
    grads = case["op"] == "bwd"
    outs = {n: torch.empty(t.shape, dtype=torch.float64, device="cuda")
            for n, t in (("o", st["q"]), ("dq", st["q"]), ("dk", st["k"]), ("dv", st["v"]))}
    lse = torch.empty((Hq, st["q"].shape[0]) if case["packed"] else (st["B"], Hq, st["Sq"]), dtype=torch.float64,
                      device="cuda")
    at = 0
    for b, of in enumerate(_sequences(st)):
        Sq, Sk = of(st["q"]).shape[0], of(st["k"]).shape[0]
        seen = None
        if case["causal"]:
            seen = torch.ones(Sq, Sk, dtype=torch.bool, device="cuda").tril(Sk - Sq)
        for h in range(Hkv):
            k = of(st["k"])[:, h].double().requires_grad_(grads)
            v = of(st["v"])[:, h].double().requires_grad_(grads)
            dk, dv = torch.zeros_like(k), torch.zeros_like(v)
            for i in range(h * group, (h + 1) * group):
                q = of(st["q"])[:, i].double().requires_grad_(grads)
                o, l = _attention64(q, k, v, seen)
                if grads:
                    gq, gk, gv = torch.autograd.grad(o, (q, k, v), of(st["dout"])[:, i].double())
                    of(outs["dq"])[:, i] = gq
                    dk, dv = dk + gk, dv + gv
                else:
                    of(outs["o"])[:, i] = o
                    (lse[i, at:at + Sq] if case["packed"] else lse[b, i]).copy_(l)
            if grads:
                of(outs["dk"])[:, h], of(outs["dv"])[:, h] = dk.detach(), dv.detach()
        at += Sq
    return (outs["dq"], outs["dk"], outs["dv"]) if grads else (outs["o"], lse)
