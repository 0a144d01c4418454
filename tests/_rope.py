"""Per-head norms with the position rotation, by their definition in 64 bits (test helper).

Errors that the kernels may have, with u = 2^-8 for rounding to nearest in bf16 (half a step)
and 2^-7 toward zero:
  * forward: a sum of 128 squares (relative 2^-17 at worst, halved by the root), a handful of
    fp32 operations and two products per element, so |error| <= 2^-16 (|u_a cos| + |u_b sin|),
    then the rounding of the result;
  * backward: two such sums, |error| <= 2^-16 r (|dn| + |x r| mean|dn x r|) + rounding;
  * weights: fp32 sums whose longest chain has at most 128 additions in these tests (a lane's
    rows, a warp's four, four warps, every 32nd block, 32 terms) over terms off by some 2^-17
    themselves: |error| <= 2^-16 sum |terms|.
"""
import torch

FP32 = 2.0 ** -16
U = {"rtne": 2.0 ** -8, "rtna": 2.0 ** -8, "rtz": 2.0 ** -7}


def table(n, rot, theta=10000.0):
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def columns(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def forward(x, w, cos, sin, positions, interleaved, eps=1e-6):
    """x (tokens, H, 128), positions (tokens,): (y, magnitude) in float64."""
    x, w = x.double(), w.double()
    c, s = cos.double()[positions.long()][:, None], sin.double()[positions.long()][:, None]
    u = x * w / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    a, b = columns(2 * cos.shape[1], interleaved)
    y, mag = u.clone(), u.abs()
    y[..., a], y[..., b] = u[..., a] * c - u[..., b] * s, u[..., b] * c + u[..., a] * s
    mag[..., a] = (u[..., a] * c).abs() + (u[..., b] * s).abs()
    mag[..., b] = (u[..., b] * c).abs() + (u[..., a] * s).abs()
    return y, mag


def backward(dy, x, w, cos, sin, positions, interleaved, eps=1e-6):
    """(dx, magnitude, dw, magnitude) in float64, from the formulas."""
    dy, x, w = dy.double(), x.double(), w.double()
    c, s = cos.double()[positions.long()][:, None], sin.double()[positions.long()][:, None]
    a, b = columns(2 * cos.shape[1], interleaved)
    du, mdu = dy.clone(), dy.abs()
    du[..., a], du[..., b] = dy[..., a] * c + dy[..., b] * s, dy[..., b] * c - dy[..., a] * s
    mdu[..., a] = (dy[..., a] * c).abs() + (dy[..., b] * s).abs()
    mdu[..., b] = (dy[..., b] * c).abs() + (dy[..., a] * s).abs()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n, dn, mdn = x * r, du * w, mdu * w.abs()
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    mag = r * (mdn + n.abs() * (mdn * n.abs()).mean(-1, keepdim=True))
    return dx, mag, (du * n).sum((0, 1)), (mdu * n.abs()).sum((0, 1))


def check(name, got, want, mag, mode="rtne"):
    got = got.detach().cpu().double()
    e = FP32 * mag
    u = U[mode] if got.numel() and mode else 0.0
    over = (got - want).abs() - (e + u * (want.abs() + e))
    assert torch.isfinite(got).all(), name
    assert over.numel() == 0 or over.max() <= 1e-30, (name, float(over.max()))


def check_weight(name, got, want, mag):
    assert got.dtype == torch.float32, name
    over = (got.detach().cpu().double() - want).abs() - FP32 * mag
    assert over.max() <= 1e-30, (name, float(over.max()))
