"""Plain 64-bit forms of the norm and rotation of queries and keys, and of their
gradients, with bounds on the error of fp32 work and one rounding, for the tests."""
from __future__ import annotations

import math

import torch

# half a step of the type, relative to the value; the smallest step besides
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}
# fp32: sums of 12 terms in a row, a reciprocal root within 2^-22, cosines of angles within 2^-24 of a turn (2^-21), and
# half a dozen products, 2^-24 each
E = 2.0 ** -19


def partner(rot, d, interleaved):
    """Partner, pair and sign of each feature (pair -1: not rotated)."""
    at, pair, sign = list(range(d)), [-1] * d, [0.0] * d
    for i in range(rot // 2):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        at[lo], at[hi], pair[lo], pair[hi], sign[lo], sign[hi] = hi, lo, i, i, -1.0, 1.0
    return torch.tensor(at), torch.tensor(pair), torch.tensor(sign, dtype=torch.float64)


def turns(pos, freq, axis, d, interleaved, rot_scale, back):
    """cos and signed sin of each row and feature [.., 1, d]; pos [.., rows] or [axes, .., rows] with axis."""
    rot = 2 * len(freq)
    _, pair, sign = partner(rot, d, interleaved)
    p = pos.double()
    p = p[axis.long()].movedim(0, -1) if axis is not None else p[..., None].expand(*p.shape, rot // 2)
    # fractions of a turn, so that far positions keep their angle
    turn = p * (freq.double() / (2 * math.pi))
    a = 2 * math.pi * (turn - turn.round())
    c, s = torch.cos(a) * rot_scale, torch.sin(a) * rot_scale
    one = torch.ones(*p.shape[:-1], d, dtype=torch.float64)
    on = pair >= 0
    cs = torch.where(on, c[..., pair.clamp(min=0)] if rot else one, one)
    sn = torch.where(on, s[..., pair.clamp(min=0)] if rot else one, 0.0) * sign * (-1 if back else 1)
    return cs[..., None, :], sn[..., None, :]


def forward(x, w, pos, freq, *, axis=None, eps=1e-6, weight_offset=0.0, interleaved=False, rot_scale=1.0):
    """y and the bound on its error, x [.., rows, h, d] (w None: no norm)."""
    d, dt = x.shape[-1], x.dtype
    f = x.double()
    at, _, _ = partner(2 * len(freq), d, interleaved)
    if w is not None:
        f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + eps) * (w.double() + weight_offset)
    cs, sn = turns(pos, freq, axis, d, interleaved, rot_scale, False)
    y = f * cs + f[..., at] * sn
    size = f.abs() + (f[..., at].abs() if len(freq) else 0)
    return y, U[dt] * y.abs() + E * size * max(1.0, abs(rot_scale)) + TINY[dt]


def backward(g, x, w, pos, freq, *, axis=None, eps=1e-6, weight_offset=0.0, interleaved=False, rot_scale=1.0):
    """(dx, its bound, dw, its bound)."""
    d, dt = g.shape[-1], g.dtype
    at, _, _ = partner(2 * len(freq), d, interleaved)
    cs, sn = turns(pos, freq, axis, d, interleaved, rot_scale, True)
    f = g.double()
    u = f * cs + f[..., at] * sn
    eu = E * (f.abs() + f[..., at].abs()) * max(1.0, abs(rot_scale))
    if w is None:
        return u, U[dt] * u.abs() + eu + TINY[dt], None, None
    w = w.double() + weight_offset
    xx = x.double()
    r = torch.rsqrt((xx * xx).mean(-1, keepdim=True) + eps)
    n = xx * r
    dot = (w * u * n).mean(-1, keepdim=True)
    dx = r * (w * u - n * dot)
    edot = (w.abs() * n.abs() * (eu + E * u.abs())).mean(-1, keepdim=True)
    edx = r * (w.abs() * eu + n.abs() * (edot + E * dot.abs()) + E * (w * u).abs())
    rows = n.numel() // d
    dw = (u * n).reshape(-1, d).sum(0)
    edw = ((eu + E * u.abs()) * n.abs()).reshape(-1, d).sum(0) + (u * n).abs().reshape(-1, d).sum(0) * rows * 2.0 ** -24
    return dx, U[dt] * dx.abs() + edx * (1 + U[dt]) + TINY[dt], dw, edw
