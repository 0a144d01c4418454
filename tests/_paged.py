"""Attention over a paged cache by its definition in 64 bits (test helper)."""
import math

import torch

SCALE = 1.0 / math.sqrt(128)


def pages_of(layout, n, page, Hkv, g=None, fill=None):
    shape = (n, page, Hkv, 128) if layout == "bshd" else (n, Hkv, page, 128)
    if fill is not None:
        return [torch.full(shape, fill, dtype=torch.bfloat16) for _ in range(2)]
    return [torch.randn(*shape, generator=g).to(torch.bfloat16) for _ in range(2)]


def inputs(layout, B, Sq, Hq, Hkv, page, max_pages, lens, seed, spare=3):
    """q, k_pages, v_pages, table, lens: every sequence's pages in a mixed order; slots past a
    sequence's last key and pages of nobody hold NaN, table entries past its last page are wrong."""
    g = torch.Generator().manual_seed(seed)
    n = B * max_pages + spare
    q = torch.randn(*((B, Sq, Hq, 128) if layout == "bshd" else (B, Hq, Sq, 128)), generator=g).to(torch.bfloat16)
    kp, vp = pages_of(layout, n, page, Hkv, g)
    table = torch.randperm(n, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32)
    used = torch.zeros(n, page, dtype=torch.bool)
    for b, m in enumerate(lens):
        j = torch.arange(m)
        used[table[b, j // page].long(), j % page] = True
        table[b, -(-m // page):] = -7 if b % 2 else n + 5
    for t in (kp, vp):
        (t if layout == "bshd" else t.transpose(1, 2))[~used] = math.nan
    return q, kp, vp, table, lens


def rows(pages, table, b, m, layout):
    """(m, Hkv, 128): sequence b's first m keys (or values)."""
    page = pages.shape[1 if layout == "bshd" else 2]
    j = torch.arange(m)
    p, i = table[b, j // page].long(), j % page
    return pages[p, i] if layout == "bshd" else pages[p, :, i]


def exact(q, kp, vp, table, lens, layout, causal, scale=SCALE):
    """(out, lse, mass, mass's error bound) in 64 bits, heads first; mass (B, Hkv, slots).

    A logit is a sum of 128 products whose partial sums are each off by 2^-23 at most, relative to
    the products' magnitudes: |ds| <= 128 * 2^-23 scale sum|q k|. A weight's exponent is off by
    that, by as much in lse, and by a few roundings of fp32 numbers up to 2^7 (2^-15 in all)."""
    if layout == "bhsd":
        q = q.transpose(1, 2)
    B, Sq, Hq, d = q.shape
    Hkv = kp.shape[2 if layout == "bshd" else 1]
    page = kp.shape[1 if layout == "bshd" else 2]
    g, slots = Hq // Hkv, table.shape[1] * page
    out = torch.full((B, Hq, Sq, d), math.nan, dtype=torch.float64)
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64)
    mass, bound = torch.zeros(B, Hkv, slots, dtype=torch.float64), torch.zeros(B, Hkv, slots, dtype=torch.float64)
    for b, n in enumerate(lens):
        k, v = rows(kp, table, b, n, layout).double(), rows(vp, table, b, n, layout).double()
        for i in range(Sq):
            m = max(0, n - (Sq - 1 - i)) if causal else n
            if m == 0:
                continue
            for h in range(Hq):
                x = q[b, i, h].double()
                s = k[:m, h // g] @ x * scale
                lse[b, h, i] = torch.logsumexp(s, 0)
                p = torch.exp(s - lse[b, h, i])
                out[b, h, i] = p @ v[:m, h // g]
                mass[b, h // g, :m] += p
                off = 128 * 2.0 ** -23 * abs(scale) * (k[:m, h // g].abs() @ x.abs())
                bound[b, h // g, :m] += p * (off + off.max() + 2.0 ** -15)
    return out, lse, mass, bound
