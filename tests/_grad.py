"""Attention's log-sum-exp and gradients by their definition in 64 bits, with the
error each gradient element may have (test helper).

What the kernels round, and by how much at most (u = 2^-8 for rounding to nearest in
bf16, 2^-7 toward zero):
  * P, as an operand of dV: u |P_ij| per pair -> u sum_i |P_ij| |dO_ic|
  * dS, as an operand of dK and dQ: u |dS_ij|
  * out, from which D = sum_c dO O is formed: |D error| <= u_out sum_c |dO_ic O_ic|,
    which enters dS as P_ij |D error|
  * the result: u_mode |result|
Everything else is fp32: a logit is a sum of 128 products, each partial sum off by
at most 2^-23 relative (the tensor pipe truncates), so exp is off by a factor of
about 1 + 2^-23 * 128 * scale * sum_c |q_c k_c|, some 2e-5 * |logit mass|; FP32
allows 1e-3 of the pair terms' magnitude for it, for dP's sum alike and for sums
over up to 2^12 rows.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8
FP32 = 1e-3


def visible(Sq, Sk, causal):
    if not causal:
        return torch.ones(Sq, Sk, dtype=torch.bool)
    return torch.ones(Sq, Sk, dtype=torch.bool).tril(Sk - Sq)


def one_head(q, k, v, do, scale, seen):
    """float64 (S, d) tensors of one query head. Returns a dict of out, lse, the three
    gradients' terms and, for each, the pair terms' magnitude that the bounds use. A
    hidden pair takes no part: it is left out of every sum."""
    s = (q @ k.T) * scale
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, 1) if k.shape[0] else torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    p = torch.where(seen & torch.isfinite(lse)[:, None], torch.exp(s - lse[:, None]), torch.zeros_like(s))
    o = p @ v
    dp = do @ v.T
    D = (p * dp).sum(1)
    ds = torch.where(seen, p * (dp - D[:, None]), torch.zeros_like(p))
    mag_D = (do.abs() * o.abs()).sum(1)
    mag_dp = do.abs() @ v.abs().T
    return dict(out=o, lse=lse, dq=scale * ds @ k, dk=scale * ds.T @ q, dv=p.T @ do,
                ds=ds.abs(), pD=p * mag_D[:, None], pdp=p * (mag_dp + mag_D[:, None]), p=p)


def head_bounds(r, q, k, do, scale, u_out):
    """Bounds of the gradients' errors before their own rounding."""
    e = U * r["ds"] + u_out * r["pD"] + FP32 * r["pdp"]
    a = abs(scale)
    return dict(dq=a * e @ k.abs(), dk=a * e.T @ q.abs(), dv=(U + FP32) * r["p"].T @ do.abs())


def sequence(q, k, v, do, scale, causal, u_out=U):
    """(S, H, d) tensors of one sequence (any float type, CPU): gradients, lse and bounds in
    float64, dk and dv summed over the query heads of each key/value head."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    Sq, Hq, d = q.shape
    Sk, Hkv, _ = k.shape
    g = Hq // Hkv
    seen = visible(Sq, Sk, causal)
    z = torch.zeros
    out = dict(dq=z(Sq, Hq, d, dtype=torch.float64), dk=z(Sk, Hkv, d, dtype=torch.float64),
               dv=z(Sk, Hkv, d, dtype=torch.float64), lse=z(Hq, Sq, dtype=torch.float64),
               out=z(Sq, Hq, d, dtype=torch.float64))
    bound = {n: torch.zeros_like(out[n]) for n in ("dq", "dk", "dv")}
    for h in range(Hq):
        kv = h // g
        r = one_head(q[:, h], k[:, kv], v[:, kv], do[:, h], scale, seen)
        b = head_bounds(r, q[:, h], k[:, kv], do[:, h], scale, u_out)
        out["dq"][:, h], out["lse"][h], out["out"][:, h] = r["dq"], r["lse"], r["out"]
        bound["dq"][:, h] = b["dq"]
        for n in ("dk", "dv"):
            out[n][:, kv] += r[n]
            bound[n][:, kv] += b[n]
    return out, bound


def check(name, got, want, bound, u_mode=U, norm=6e-3):
    """got (bf16) against want: element by element within the bound and its own rounding;
    and as a whole within `norm` relative: three independent roundings (operand, D or
    partner, result) of rms 2^-8 / sqrt(3) * 0.75 = 1.7e-3 each give 3e-3; twice that
    (4 times for rounding toward zero, whose errors do not average out)."""
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    over = err - (bound + u_mode * (want.abs() + bound))
    at = int(over.argmax()) if over.numel() else 0
    assert over.numel() == 0 or over.max() <= 1e-30, (
        name, float(over.max()), float(err.flatten()[at]), float(bound.flatten()[at]))
    n = want.norm()
    if n > 0:
        assert err.norm() <= norm * n, (name, float(err.norm() / n))
