"""64-bit references of the layer operators, and bounds on what fp32 arithmetic and one rounding may differ by.

Every bound is elementwise and worst-case.  U is the unit roundoff of a type (2^-p for p significand bits), TINY half
its smallest subnormal.  A sum of n fp32 terms in any order is within n EPS sum|terms| (EPS = 2^-23 also covers an
accumulator that truncates).  ACT bounds the absolute error of an activation's fp32 evaluation relative to |z|, and of
its slope: a few units of 2^-24 in erf, exp and the quotient, times an exponent's argument of up to about 20 where the
result still matters, below 2^-18.  No activation here has a slope above 1.2.
"""

import math

import torch

EPS = 2.0 ** -23
ACT = 2.0 ** -18
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
# Longest chain of additions in a row's sums: a thread's share (at most 128 values before it is joined), a warp, a block.
CHAIN = 160


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    c = math.sqrt(2 / math.pi)
    u = 2 * c * (z + 0.044715 * z ** 3)
    return torch.sigmoid(u) + z * torch.sigmoid(u) * torch.sigmoid(-u) * 2 * c * (1 + 3 * 0.044715 * z * z)


def linear64(x, w, b=None, r=None, act="none"):
    """(y, bound of y, z, bound of z) for the type of x."""
    u, tiny = U[x.dtype], TINY[x.dtype]
    xd, wd = x.double(), w.double()
    z = xd @ wd.t()
    mag = xd.abs() @ wd.abs().t()
    if b is not None:
        z = z + b.double()
        mag = mag + b.double().abs()
    ez = (x.shape[1] + 2) * EPS * mag
    y = act64(z, act)
    ey = 1.2 * ez + ACT * z.abs()
    if r is not None:
        y = y + r.double()
        ey = ey + EPS * y.abs()
    return y, u * y.abs() + (1 + u) * ey + tiny, z, u * z.abs() + (1 + u) * ez + tiny


def linear_backward64(dy, x, w, pre=None, act="none"):
    """((dx, dw, db), their bounds): dz is rounded to the type for the products, not for db."""
    u, tiny = U[x.dtype], TINY[x.dtype]
    xd, wd, dyd = x.double(), w.double(), dy.double()
    m, n = dy.shape
    if act == "none":
        dz, edz, erd = dyd, torch.zeros_like(dyd), torch.zeros_like(dyd)
    else:
        dz = dyd * slope64(pre.double(), act)
        edz = 2 * ACT * dyd.abs()              # before rounding
        erd = edz + u * (dz.abs() + edz) + tiny  # after rounding
    zmag = dz.abs() + erd
    dx, edx = dz @ wd, erd @ wd.abs() + (n + 2) * EPS * (zmag @ wd.abs())
    dw, edw = dz.t() @ xd, erd.t() @ xd.abs() + (m + 2) * EPS * (zmag.t() @ xd.abs())
    db, edb = dz.sum(0), edz.sum(0) + (m + 2) * EPS * zmag.sum(0)

    def done(v, e):
        return u * v.abs() + (1 + u) * e + tiny
    return (dx, dw, db), (done(dx, edx), done(dw, edw), done(db, edb))


def norm64(x, weight=None, bias=None, eps=1e-5):
    """((y, mean, rstd), their bounds)."""
    u, tiny = U[x.dtype], TINY[x.dtype]
    xd = x.double()
    h = max(x.shape[1], 1)
    mean = xd.sum(1, keepdim=True) / h
    d = xd - mean
    var = (d * d).sum(1, keepdim=True) / h
    rstd = (var + eps) ** -0.5
    w = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    emean = CHAIN * EPS * xd.abs().sum(1, keepdim=True) / h
    ed = emean + EPS * d.abs()
    evar = (2 * d.abs() * ed + ed * ed).sum(1, keepdim=True) / h + CHAIN * EPS * var
    rel = 0.5 * evar / (var + eps) + 4 * EPS
    # A relative error of the variance above 1/2 says nothing any more (a row of equal values, eps tiny).
    y = d * rstd * w + b
    ey = w.abs() * rstd * (ed + (d.abs() + ed) * rel) * (1 + rel) + 4 * EPS * ((d * rstd * w).abs() + b.abs())
    return (y, mean[:, 0], rstd[:, 0]), (u * y.abs() + (1 + u) * ey + tiny, emean[:, 0] + EPS * mean[:, 0].abs(),
                                         (rstd * rel * (1 + rel))[:, 0])


def norm_backward64(dy, x, mean, rstd, weight=None, dr=None):
    """((dx, dweight, dbias), their bounds) for the statistics as given."""
    u, tiny = U[x.dtype], TINY[x.dtype]
    rows, h = x.shape
    xd, g0 = x.double(), dy.double()
    mu, rs = mean.double().unsqueeze(1), rstd.double().unsqueeze(1)
    w = torch.ones(h, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    xh = (xd - mu) * rs
    exh = 2 * EPS * xh.abs()
    g = g0 * w
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    ec1 = (CHAIN + 2) * EPS * g.abs().mean(1, keepdim=True)
    ec2 = (CHAIN + 4) * EPS * (g * xh).abs().mean(1, keepdim=True)
    dx = rs * (g - c1 - xh * c2)
    edx = rs * (4 * EPS * (g.abs() + c1.abs() + (xh * c2).abs()) + ec1 + exh * c2.abs() + xh.abs() * ec2)
    if dr is not None:
        dx = dx + dr.double()
        edx = edx + EPS * dx.abs()
    dw, db = (g0 * xh).sum(0), g0.sum(0)
    edw = (rows + 4) * EPS * (g0 * xh).abs().sum(0)
    edb = (rows + 2) * EPS * g0.abs().sum(0)
    up, tp = (u, tiny) if weight is None else (U[weight.dtype], TINY[weight.dtype])

    def done(v, e, u, tiny):
        return u * v.abs() + (1 + u) * e + tiny
    return (dx, dw, db), (done(dx, edx, u, tiny), done(dw, edw, up, tp), done(db, edb, up, tp))


def worst(got, want, bound):
    """Largest error as a multiple of its bound (0 for an empty result); got must be finite where want is."""
    if got.numel() == 0:
        return 0.0
    assert got.shape == want.shape
    assert bool(torch.isfinite(got).all())
    return float(((got.double() - want).abs() / bound).max())
