"""The expert products in float64 torch operations, for shapes too large for
the numpy oracle in a test's time, and what a kernel may be off by."""
from __future__ import annotations

import torch

EPS32, EPS16 = 2.0 ** -24, 2.0 ** -11   # half a step of float32 and binary16, relative


def gathered(x, at):
    """Rows of x in float64 for each row of Y; zeros where the index is outside x."""
    ok = (at >= 0) & (at < len(x))
    rows = x[at.clamp(0, max(len(x) - 1, 0)).long()].double()
    return rows * (ok if x.dim() == 1 else ok[:, None])


def grouped(offsets, w, x, at, bias=None, ws=None, xs=None):
    """Y in float64 (NaN in rows of no expert), and what its errors are relative to: sum |x w| + |b|, or with scales
    (exact integer sums) |product| + |b|.  offsets is a list, w [experts][n][k]."""
    y = torch.full((len(at), w.shape[1]), float("nan"), dtype=torch.float64, device=w.device)
    size = y.clone()
    for e in range(len(w)):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        xe, we = gathered(x, at[a:b]), w[e].double().t().contiguous()
        p = torch.mm(xe, we)
        if ws is None:
            s = torch.mm(xe.abs(), we.abs())
        else:
            p = p * gathered(xs, at[a:b])[:, None] * ws[e].double()
            s = p.abs()
        y[a:b] = p if bias is None else p + bias[e].double()
        size[a:b] = s if bias is None else s + bias[e].double().abs()
    return y, size


def rounded(y, t, half):
    """Tolerance t and the last rounding to Y's type: half a step, or half binary16's smallest subnormal."""
    return t + (1 + EPS16) * (EPS16 * (y.abs() + t) + 2.0 ** -25) if half else t


def tolerance(y, size, k, scaled):
    """Before the rounding to Y's type.  8 bits: fma(float(sum) * xs, ws, b), two roundings on the product, the fma's
    on the result, one more for second-order terms.  binary16: products are exact in float32, and k + 1 additions
    round by at most a step each (the matrix cores may cut instead of rounding to nearest)."""
    if scaled:
        return 3 * EPS32 * size + EPS32 * y.abs() + 2.0 ** -126
    return (k + 2) * 2 * EPS32 * size + 2.0 ** -126


def joined(g, u, eg, eu):
    """silu(g) * u, and its tolerance from those of g and u: |silu'| <= 1.1; e^-g within 2 steps, the sum, the quotient
    and the product half a step each.  e^-g overflows past g = -88, where |silu| < 1e-36."""
    s = g * torch.sigmoid(g)
    h = s * u
    return h, 1.1 * eg * u.abs() + s.abs() * eu + 2 * eg * eu + 8 * EPS32 * h.abs() + 1e-35 * (1 + u.abs())
