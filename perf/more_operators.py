"""The steps around attention over a paged cache and around a training step's attention, as
measured cases.

  rope      per-head RMS norms of queries and keys with the position rotation
  rope_bwd  its gradients: queries, keys and both norm weights
  append    the same step in serving: rotated keys, and the values, go to a paged cache
  paged     attention of new tokens over a paged cache, with or without the accumulation of
            every key's attention weight
  evict     the cache kept to a budget: each key/value head keeps its keys of greatest
            accumulated weight and the latest ones, moved together in order

With ``own`` false, run() computes them in plain torch operations in 32 bits; with
``own`` true it calls the library.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
EPS = 1e-6
THETA = 10000.0


# ---------------------------------------------------------------- cases

def _rope(op, name, layout, B, S, Hq, Hkv, rot, interleaved, fused):
    return {"name": name, "op": op, "layout": layout, "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "rot": rot,
            "interleaved": interleaved, "fused": fused}


def _append(name, layout, B, S, Hq, Hkv, rot, interleaved, page, cap):
    return {"name": name, "op": "append", "layout": layout, "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "rot": rot,
            "interleaved": interleaved, "page": page, "cap": cap}


def _paged(name, layout, B, Sq, Hq, Hkv, page, cap, min_len, causal, mass, len_seed):
    return {"name": name, "op": "paged", "layout": layout, "B": B, "Sq": Sq, "Hq": Hq, "Hkv": Hkv, "page": page,
            "cap": cap, "min_len": min_len, "causal": causal, "mass": mass, "len_seed": len_seed}


def _evict(name, layout, B, Hkv, page, cap, min_len, budget, recent, len_seed):
    return {"name": name, "op": "evict", "layout": layout, "B": B, "Hkv": Hkv, "page": page, "cap": cap,
            "min_len": min_len, "budget": budget, "recent": recent, "len_seed": len_seed}


def listed():
    return [
        # The smallest training step: two heads of 256 tokens, where latency counts.
        _rope("rope", "rope_tiny", "bhsd", 1, 256, 2, 2, 128, False, False),
        # Training at the benchmark's 8K length, grouped heads, queries and keys still in one projection's output.
        _rope("rope", "rope_8k", "bshd", 2, 8192, 16, 4, 128, False, True),
        # Odd sizes, head-major, half of each head rotated, neighbouring columns paired.
        _rope("rope_bwd", "rope_bwd_ragged", "bhsd", 3, 1021, 6, 3, 64, True, False),
        # The 8K training step's gradients, all heads.
        _rope("rope_bwd", "rope_bwd_8k", "bshd", 2, 8192, 16, 16, 128, False, False),
        # One new token for each of 64 sequences.
        _append("append_decode", "bshd", 64, 1, 32, 8, 128, False, 64, 512),
        # A prompt's tokens, 4096 of each of 4 sequences, into small pages.
        _append("append_prompt", "bhsd", 4, 4096, 32, 8, 128, False, 16, 5003),
        # Sampling for a handful of users from short caches: latency.
        _paged("paged_small", "bshd", 4, 1, 8, 2, 16, 1000, 1, False, True, 3),
        # 64 users, caches of any length up to 8K.
        _paged("paged_decode", "bshd", 64, 1, 32, 8, 64, 8192, 1, False, False, 11),
        # Drafted tokens: five at a time, odd group of seven heads, head-major pages of an odd size.
        _paged("paged_draft", "bhsd", 48, 5, 28, 4, 20, 5003, 5, True, False, 13),
        # Two very long contexts, whose keys' weights are accumulated for a later eviction.
        _paged("paged_long", "bshd", 2, 1, 32, 8, 128, 131072, 100000, False, True, 17),
        # A handful of short caches halved.
        _evict("evict_small", "bshd", 4, 2, 16, 1000, 513, 512, 64, 19),
        # 32 caches of up to 16K keys cut to 4096, of which the last 512 stay.
        _evict("evict_large", "bhsd", 32, 8, 64, 16384, 1000, 4096, 512, 23),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "paged", "paged", "evict"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 1, 2, 3, 4, 7])
    layout = rng.choice(["bshd", "bhsd"])
    rot = rng.choice([128, 128, 64, 32, 96])
    inter = rng.random() < 0.3
    page = rng.choice([16, 16, 64, 128, 1, 20, 33, 256])
    seed = rng.randrange(1 << 20)
    if op in ("rope", "rope_bwd"):
        # Rows of one head: at most a quarter of the largest listed case's.
        B, S = rng.choice([1, 1, 2, 5]), _log(rng, 1, 16384)
        while B * S * Hkv * (group + 1) > 131072:
            S = max(1, S // 2)
        return _rope(op, "", layout, B, S, Hkv * group, Hkv, rot, inter, layout == "bshd" and rng.random() < 0.5)
    if op == "append":
        B, S = _log(rng, 1, 200), rng.choice([1, 1, 5, _log(rng, 2, 2000)])
        while B * S * Hkv * (group + 2) > 131072:
            B = max(1, B // 2)
        return _append("", layout, B, S, Hkv * group, Hkv, rot, inter, page, S + _log(rng, 1, 500))
    # Caches: at most the larger listed ones' size.
    B, cap = _log(rng, 1, 128), _log(rng, 8, 40000)
    while B * cap * Hkv > 64 * 8192 * 4:
        B, cap = max(1, B // 2), max(8, cap * 3 // 4)
    if op == "paged":
        Sq = rng.choice([1, 1, 1, 2, 5])
        return _paged("", layout, B, Sq, Hkv * group, Hkv, page, cap, min(cap, Sq), rng.random() < 0.5,
                      rng.random() < 0.4, seed)
    budget = _log(rng, 4, max(5, cap))
    return _evict("", layout, B, Hkv, page, cap, 1, budget, rng.choice([0, 1, budget // 8, budget // 2, budget]), seed)


def _lengths(case):
    g = torch.Generator().manual_seed(case["len_seed"])
    return torch.randint(case["min_len"], case["cap"] + 1, (case["B"],), generator=g).tolist()


def _slots(case):
    """Key slots of a sequence: its pages are whole."""
    return -(-case["cap"] // case["page"]) * case["page"]


def work(case):
    Hkv, B, op = case["Hkv"], case["B"], case["op"]
    if op in ("rope", "rope_bwd", "append"):
        Hq, T = case["Hq"], B * case["S"]
        rows = T * (Hq + Hkv)
        small = 4 * T + 4 * case["rot"] * case["S"] + 4 * D
        if op == "rope":
            return {"bytes": 2 * D * 2 * rows + small, "flops": 10 * D * rows}
        if op == "rope_bwd":
            return {"bytes": 2 * D * 3 * rows + small + 8 * D, "flops": 24 * D * rows}
        return {"bytes": 2 * D * 2 * (rows + T * Hkv) + small + 4 * T, "flops": 10 * D * rows}
    lens, slots = _lengths(case), _slots(case)
    if op == "paged":
        Hq, Sq = case["Hq"], case["Sq"]
        pairs = sum(sum(max(0, min(n, i + n - Sq + 1)) if case["causal"] else n for i in range(Sq)) for n in lens)
        rows = B * Sq * Hq
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": 2 * D * (2 * rows + 2 * Hkv * sum(lens)) + 4 * rows + 4 * B + 4 * pages
                + (8 * Hkv * sum(lens) if case["mass"] else 0), "flops": 4 * D * Hq * pairs}
    # Every kept key of a cache over its budget moves, but for the few before its first evicted one.
    moved = Hkv * sum(case["budget"] for n in lens if n > case["budget"])
    return {"bytes": 2 * 2 * 2 * D * moved + 4 * Hkv * (sum(lens) + B * slots) + 8 * B, "flops": Hkv * sum(lens)}


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _table(n, rot):
    """cos and sin of position times frequency, formed in 64 bits, kept in 32."""
    f = THETA ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def _pages(g, case):
    """Pages of all sequences in an order that mixes them, and the table that says which are whose."""
    B, page, per = case["B"], case["page"], _slots(case) // case["page"]
    n = B * per
    shape = (n, page, case["Hkv"], D) if case["layout"] == "bshd" else (n, case["Hkv"], page, D)
    table = torch.randperm(n, generator=g, device="cuda").view(B, per).to(torch.int32)
    return _randn(g, *shape), _randn(g, *shape), table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    op, B, Hkv = case["op"], case["B"], case["Hkv"]
    if op in ("rope", "rope_bwd", "append"):
        S, Hq = case["S"], case["Hq"]
        shape = (lambda H: (B, S, H, D)) if case["layout"] == "bshd" else (lambda H: (B, H, S, D))
        if case.get("fused"):
            st["q"], st["k"], _ = _randn(g, B, S, Hq + 2 * Hkv, D).split((Hq, Hkv, Hkv), 2)
        else:
            st["q"], st["k"] = _randn(g, *shape(Hq)), _randn(g, *shape(Hkv))
        st["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        st["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        if op == "append":
            st["v"] = _randn(g, *shape(Hkv))
            st["k_pages"], st["v_pages"], table = _pages(g, case)
            # The S new tokens come after each sequence's earlier ones.
            first = torch.randint(0, case["cap"] - S + 1, (B,), generator=g, device="cuda")
            pos = first[:, None] + torch.arange(S, device="cuda")
            st["slots"] = (torch.gather(table.long(), 1, pos // case["page"]) * case["page"] + pos % case["page"])
            st["slots"] = st["slots"].to(torch.int32)
            st["positions"] = pos.to(torch.int32)
            st["cos"], st["sin"] = _table(case["cap"], case["rot"])
            return st
        st["positions"] = torch.arange(S, device="cuda", dtype=torch.int32).repeat(B, 1)
        st["cos"], st["sin"] = _table(S, case["rot"])
        if op == "rope_bwd":
            st["dq_out"], st["dk_out"] = _randn(g, *shape(Hq)), _randn(g, *shape(Hkv))
        return st
    st["k_pages"], st["v_pages"], st["table"] = _pages(g, case)
    st["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if op == "paged":
        Sq, Hq = case["Sq"], case["Hq"]
        st["q"] = _randn(g, *((B, Sq, Hq, D) if case["layout"] == "bshd" else (B, Hq, Sq, D)))
        if case["mass"]:  # what earlier steps have accumulated
            st["weight"] = torch.rand(B, Hkv, _slots(case), generator=g, device="cuda")
        return st
    # Accumulated weights are skewed: few keys hold most of it, and some were never looked at.
    m = torch.exp(2 * torch.randn(B, Hkv, _slots(case), generator=g, device="cuda") - 4)
    st["weight"] = torch.where(torch.rand(m.shape, generator=g, device="cuda") < 0.1, 0.0, m)
    return st


# ---------------------------------------------------------------- plain forms

def _heads_last(st, t):
    """(B, S, H, ...) from either layout."""
    return t if st["layout"] == "bshd" else t.transpose(1, 2)


def _laid(st, t):
    """(B, S, H, ...) back to the case's layout."""
    return (t if st["layout"] == "bshd" else t.transpose(1, 2)).contiguous()


def _pairs(st, u):
    """The two columns of every rotated pair, each (..., rot / 2)."""
    r = st["rot"]
    return (u[..., 0:r:2], u[..., 1:r:2]) if st["interleaved"] else (u[..., :r // 2], u[..., r // 2:r])


def _unpaired(st, a, b, u):
    both = torch.stack((a, b), -1).flatten(-2) if st["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((both, u[..., st["rot"]:]), -1)


def _angles(st):
    pos = st["positions"].long()
    return st["cos"][pos][:, :, None], st["sin"][pos][:, :, None]


def _norm(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _norm_rotate(st, x, w):
    u = _norm(_heads_last(st, x).float()) * w.float()
    a, b = _pairs(st, u)
    c, s = _angles(st)
    return _laid(st, _unpaired(st, a * c - b * s, b * c + a * s, u).to(torch.bfloat16))


def _norm_rotate_bwd(st, dy, x, w):
    x, dy = _heads_last(st, x).float(), _heads_last(st, dy).float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    a, b = _pairs(st, dy)
    c, s = _angles(st)
    du = _unpaired(st, a * c + b * s, b * c - a * s, dy)
    dn = du * w.float()
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return _laid(st, dx.to(torch.bfloat16)), (du * n).flatten(0, 2).sum(0)


def _put(st, pages, t):
    """Rows t (B, S, Hkv, D) into their slots."""
    slot = st["slots"].long().flatten()
    page, at = slot // st["page"], slot % st["page"]
    rows = t.flatten(0, 1).to(torch.bfloat16)
    if st["layout"] == "bshd":
        pages[page, at] = rows
    else:
        pages[page, :, at] = rows


def _plain_append(st):
    _put(st, st["k_pages"], _heads_last(st, _norm_rotate(st, st["k"], st["wk"])))
    _put(st, st["v_pages"], _heads_last(st, st["v"]))
    return _norm_rotate(st, st["q"], st["wq"]), st["k_pages"], st["v_pages"]


def _gathered(st, pages):
    """(B, Hkv, slots, D) of all sequences, as they lie."""
    t = pages[st["table"].long()]                                        # (B, per, page, Hkv, D), or heads first
    if st["layout"] == "bhsd":
        t = t.transpose(2, 3)
    return t.flatten(1, 2).transpose(1, 2)


def _plain_paged(st):
    Sq, Hkv, group = st["Sq"], st["Hkv"], st["Hq"] // st["Hkv"]
    k, v = _gathered(st, st["k_pages"]).float(), _gathered(st, st["v_pages"]).float()
    B, slots = k.shape[0], k.shape[2]
    q = _heads_last(st, st["q"]).float().transpose(1, 2).unflatten(1, (Hkv, group))   # (B, Hkv, g, Sq, D)
    n = st["lens"].long()[:, None]
    limit = n.expand(B, Sq)
    if st["causal"]:
        limit = torch.minimum(limit, n - Sq + 1 + torch.arange(Sq, device="cuda"))
    seen = (torch.arange(slots, device="cuda") < limit[..., None])[:, None, None]     # (B, 1, 1, Sq, slots)
    s = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (group, Sq)) * SCALE
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    o = (e.flatten(2, 3) @ v).unflatten(2, (group, Sq)) / total
    lse = (m + torch.log(total)).squeeze(-1).flatten(1, 2)               # (B, Hq, Sq)
    out = _laid(st, o.flatten(1, 2).transpose(1, 2).to(torch.bfloat16))
    if not st["mass"]:
        return out, lse
    st["weight"] += torch.where(seen & (total > 0), e / total, 0.0).sum((2, 3))
    return out, lse, st["weight"]


def _plain_evict(st):
    budget, recent, page = st["budget"], st["recent"], st["page"]
    w, n = st["weight"], st["lens"].long()[:, None, None]
    B, Hkv, slots = w.shape
    j = torch.arange(slots, device="cuda")
    old, late = j < n - recent, (j >= n - recent) & (j < n)
    order = torch.sort(torch.where(old, w, -1.0), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, j.expand_as(order))
    keep = torch.where(n > budget, late | (old & (rank < budget - recent)), j < n)
    # Kept keys in order: slot d takes the d-th kept key; the slots after them keep what they hold.
    to = torch.where(keep, keep.long().cumsum(-1) - 1, slots)
    src = j.expand(B, Hkv, slots).contiguous()
    src = torch.cat((src, src[..., :1]), -1).scatter(2, to, j.expand_as(to))[..., :slots]
    left = torch.minimum(n, torch.full_like(n, budget))
    src = torch.where(j < left, src, j)
    weight = torch.where(j < left, torch.gather(w, 2, src), 0.0)
    for pages in (st["k_pages"], st["v_pages"]):
        rows = torch.gather(_gathered(st, pages), 2, src[..., None].expand(-1, -1, -1, D))   # (B, Hkv, slots, D)
        rows = rows.unflatten(2, (-1, page))
        rows = rows.permute(0, 2, 3, 1, 4) if st["layout"] == "bshd" else rows.transpose(1, 2)
        pages[st["table"].long()] = rows
    return left.flatten().to(torch.int32), weight, st["k_pages"], st["v_pages"]


def run(st):
    op = st["op"]
    if own:
        import bf16_forward_attention_gb300 as attn

        if op in ("rope", "rope_bwd", "append"):
            kw = {"eps": EPS, "interleaved": st["interleaved"], "layout": st["layout"]}
            if op == "rope":
                return attn.attn_qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], st["cos"], st["sin"],
                                              st["positions"], **kw)
            if op == "rope_bwd":
                return attn.attn_qk_norm_rope_bwd(st["dq_out"], st["dk_out"], st["q"], st["k"], st["wq"], st["wk"],
                                                  st["cos"], st["sin"], st["positions"], **kw)
            q = attn.attn_qk_norm_rope_paged(st["q"], st["k"], st["v"], st["wq"], st["wk"], st["cos"], st["sin"],
                                             st["positions"], st["slots"], st["k_pages"], st["v_pages"], **kw)
            return q, st["k_pages"], st["v_pages"]
        if op == "paged":
            got = attn.attn_fwd_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                      causal=st["causal"], layout=st["layout"], mass=st.get("weight"))
            return (*got, st["weight"]) if st["mass"] else got
        lens, weight = attn.attn_cache_evict(st["k_pages"], st["v_pages"], st["table"], st["lens"], st["weight"],
                                             st["budget"], recent=st["recent"], layout=st["layout"])
        return lens, weight, st["k_pages"], st["v_pages"]
    if op == "rope":
        return _norm_rotate(st, st["q"], st["wq"]), _norm_rotate(st, st["k"], st["wk"])
    if op == "rope_bwd":
        (dq, dwq), (dk, dwk) = (_norm_rotate_bwd(st, st["d" + n + "_out"], st[n], st["w" + n]) for n in "qk")
        return dq, dk, dwq, dwk
    return {"append": _plain_append, "paged": _plain_paged, "evict": _plain_evict}[op](st)


# ---------------------------------------------------------------- 64 bits, by the definition

def _rotation64(st):
    """(tokens, rot / 2) complex unit numbers of the table's angles, as they are kept."""
    pos = st["positions"].flatten().long()
    return torch.complex(st["cos"].double()[pos], st["sin"].double()[pos])


def _rows64(st, t):
    """(tokens, H, D) in 64 bits."""
    t = t.double() if st["layout"] == "bshd" else t.double().permute(0, 2, 1, 3)
    return t.reshape(-1, t.shape[2], D)


def _turned64(st, x, w, z):
    """Rows (tokens, H, D) normed, weighted and turned: pairs as complex numbers."""
    u = w * x / torch.sqrt(torch.einsum("thd,thd->th", x, x)[..., None] / D + EPS)
    h = st["rot"] // 2
    if st["interleaved"]:
        a, b = torch.arange(h, device="cuda") * 2, torch.arange(h, device="cuda") * 2 + 1
    else:
        a, b = torch.arange(h, device="cuda"), torch.arange(h, device="cuda") + h
    p = torch.complex(u[..., a], u[..., b]) * z[:, None]
    return u.index_copy(2, a, p.real).index_copy(2, b, p.imag)


def _back64(st, rows):
    t = rows.unflatten(0, (st["B"], -1))
    return t.contiguous() if st["layout"] == "bshd" else t.permute(0, 2, 1, 3).contiguous()


def _exact_rope(st):
    z = _rotation64(st)
    wq, wk = st["wq"].double(), st["wk"].double()
    q, k = _rows64(st, st["q"]), _rows64(st, st["k"])
    if st["op"] == "rope":
        return _back64(st, _turned64(st, q, wq, z)), _back64(st, _turned64(st, k, wk, z))
    if st["op"] == "rope_bwd":
        got = []
        for x, w, dy in ((q, wq, st["dq_out"]), (k, wk, st["dk_out"])):
            x.requires_grad_(True)
            w.requires_grad_(True)
            got.append(torch.autograd.grad(_turned64(st, x, w, z), (x, w), _rows64(st, dy)))
        return _back64(st, got[0][0]), _back64(st, got[1][0]), got[0][1], got[1][1]
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    slots = st["slots"].flatten().long()
    for pages, rows in ((kp, _turned64(st, k, wk, z)), (vp, _rows64(st, st["v"]))):
        flat = pages if st["layout"] == "bshd" else pages.transpose(1, 2).contiguous()
        flat.view(-1, st["Hkv"], D).index_copy_(0, slots, rows)
        if st["layout"] == "bhsd":
            pages.copy_(flat.transpose(1, 2))
    return _back64(st, _turned64(st, q, wq, z)), kp, vp


def _exact_paged(st):
    B, Sq, Hq, Hkv, page = (st[n] for n in ("B", "Sq", "Hq", "Hkv", "page"))
    group = Hq // Hkv
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Hq, Sq, dtype=torch.float64, device="cuda")
    weight = st["weight"].double() if st["mass"] else None
    lens, table = st["lens"].tolist(), st["table"].tolist()
    bshd = st["layout"] == "bshd"
    for b, n in enumerate(lens):
        mine = torch.tensor(table[b][:-(-n // page)], device="cuda")
        for h in range(Hkv):
            keys, vals = ((t[mine, :, h] if bshd else t[mine, h]).reshape(-1, D)[:n].double()
                          for t in (st["k_pages"], st["v_pages"]))
            for i in range(Sq):
                m = max(0, min(n, i + n - Sq + 1)) if st["causal"] else n
                heads = slice(h * group, (h + 1) * group)
                q = (st["q"][b, i, heads] if bshd else st["q"][b, heads, i]).double()
                s = torch.einsum("gd,jd->gj", q, keys[:m]) / math.sqrt(D)
                p = torch.softmax(s, -1)
                (out[b, i, heads] if bshd else out[b, heads, i]).copy_(p @ vals[:m])
                lse[b, heads, i] = torch.logsumexp(s, -1)
                if weight is not None:
                    weight[b, h, :m] += p.sum(0)
    return (out, lse, weight) if weight is not None else (out, lse)


def _exact_evict(st):
    budget, recent, page, bshd = st["budget"], st["recent"], st["page"], st["layout"] == "bshd"
    kp, vp, w = st["k_pages"].double(), st["v_pages"].double(), st["weight"].double()
    left, slots = st["lens"].clone(), w.shape[2]
    where = torch.arange(slots, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        w[b, :, n:] = 0
        if n <= budget:
            continue
        left[b] = budget
        at = st["table"][b].long()[where // page]
        for h in range(st["Hkv"]):
            # Ascending by (-weight, index): a stable sort of the negated weights.
            first = torch.argsort(-w[b, h, :n - recent], stable=True)[:budget - recent]
            kept = torch.cat((first.sort().values, where[n - recent:n]))
            for t in (kp, vp):
                if bshd:
                    t[at[:budget], where[:budget] % page, h] = t[at[kept], kept % page, h]
                else:
                    t[at[:budget], h, where[:budget] % page] = t[at[kept], h, kept % page]
            w[b, h, :budget] = w[b, h, kept]
        w[b, :, budget:] = 0
    return left, w, kp, vp


def exact(case, seed):
    st = prepare(case, seed)
    return {"paged": _exact_paged, "evict": _exact_evict}.get(case["op"], _exact_rope)(st)
