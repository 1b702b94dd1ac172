"""Plain 64-bit forms of the norms around a block and of the gated activation,
with the bounds that the GPU tests hold the kernels to.

A rounding to BF16 is off by at most 2^-8 of the value, one to FP32 by 2^-24.
An FP32 chain of the kernels is at most about 20 operations plus a sum of
depth 45 (8 in a thread, 5 in a warp, up to 32 warps), and sums over tokens
add 16 in a thread, 8 or 16 over a cluster and rows / 1024 + 8 over clusters:
below 128 operations up to 65536 rows, so FP32 noise is below 2^-17 of the sum
of the magnitudes that enter.
"""
from __future__ import annotations

import torch

BF16 = 2.0 ** -8
NOISE = 2.0 ** -17


def norm_forward(x, h, w_post, gate, scale, eps):
    """(y before its rounding, bound of the rounded y, r1)."""
    x = x.double()
    r1 = None
    if h is None:
        return x, torch.zeros_like(x), r1
    hn = h.double()
    if w_post is not None:
        r1 = (hn.square().mean(1) + eps) ** -0.5
        hn = hn * r1[:, None] * w_post.double()
    if gate is not None:
        hn = hn * gate.double()
    y = x + scale * hn
    return y, BF16 * y.abs() + NOISE * (x.abs() + (scale * hn).abs()), r1


def norm_of(y, w_pre, eps):
    """(n before its rounding, its bound, r2) of the stored y."""
    y = y.double()
    r2 = (y.square().mean(1) + eps) ** -0.5
    n = y * r2[:, None] * w_pre.double()
    return n, (BF16 + NOISE) * n.abs(), r2


def norm_backward(dn, y, rstd, w_pre, h=None, dy=None, w_post=None, rstd_post=None, gate=None, scale=1.0):
    """{name: (value, bound)} for dx, dw_pre and, with h, dh, dw_post, dgate (bounds: results in BF16 or FP32)."""
    dn, y, r2, w = dn.double(), y.double(), rstd.double()[:, None], w_pre.double()
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    t, nh = dn * w, y * r2
    zero = torch.zeros_like(dn)
    g0 = dy.double() if dy is not None else zero
    g = g0 + r2 * (t - nh * mean(t * nh))
    size = g0.abs() + r2 * (t.abs() + nh.abs() * mean((t * nh).abs()))   # magnitudes that enter g
    out = {"dx": (g, BF16 * g.abs() + NOISE * size),
           "dw_pre": ((dn * nh).sum(0), NOISE * (dn * nh).abs().sum(0))}
    if h is None:
        return out
    r1 = rstd_post.double()[:, None] if w_post is not None else 1.0
    wp = w_post.double() if w_post is not None else 1.0
    gt = gate.double() if gate is not None else 1.0
    hh = h.double() * r1
    if gate is not None:
        dg, sg = scale * g * hh * wp, abs(scale) * size * (hh * wp).abs()
        if gate.shape[1] == 1:
            out["dgate"] = (dg.sum(1, keepdim=True), NOISE * sg.sum(1, keepdim=True))
        elif gate.shape[0] == 1:
            out["dgate"] = (dg.sum(0, keepdim=True), NOISE * sg.sum(0, keepdim=True))
        else:
            out["dgate"] = (dg, BF16 * dg.abs() + NOISE * sg)
    u, su = scale * gt * g, (scale * gt * size).abs() if gate is not None else abs(scale) * size
    if w_post is None:
        out["dh"] = (u, BF16 * u.abs() + NOISE * su)
        return out
    out["dw_post"] = ((u * hh).sum(0), NOISE * (su * hh.abs()).sum(0))
    v, sv = u * wp, su * wp.abs()
    dh = r1 * (v - hh * mean(v * hh))
    out["dh"] = (dh, BF16 * dh.abs() + NOISE * r1 * (sv + hh.abs() * mean(sv * hh.abs())))
    return out


# sigmoid(g) = 1 / (1 + exp(-g)) in FP32: from -g = 126 ln 2 on, 1 + exp(-g) passes 2^126, and the quotient, below
# FP32's normal range, comes out as zero.  s itself is then at most 2^-126, which bounds its error; each result is s
# times other factors, so the error is at most 2^-126 times those.
FLUSHED = 2.0 ** -126


def swiglu(gu):
    f = gu.shape[1] // 2
    g, u = gu[:, :f].double(), gu[:, f:].double()
    # exp(-g) carries |g| 2^-24 of relative noise from its argument
    a = g * torch.sigmoid(g) * u
    return a, (BF16 + NOISE + g.abs() * 2.0 ** -22) * a.abs() + FLUSHED * (g * u).abs() + 2.0 ** -133


def swiglu_backward(da, gu):
    f = gu.shape[1] // 2
    g, u, da = gu[:, :f].double(), gu[:, f:].double(), da.double()
    s = torch.sigmoid(g)
    ds = da * s
    dg, du = ds * u * (1 + g * (1 - s)), ds * g
    noise = NOISE + g.abs() * 2.0 ** -22
    size = (ds * u).abs() * (1 + g.abs() * (1 - s))
    return (torch.cat([dg, du], 1),
            torch.cat([BF16 * dg.abs() + noise * size + FLUSHED * (da * u).abs() * (1 + g.abs()),
                       (BF16 + noise) * du.abs() + FLUSHED * (da * g).abs()], 1) + 2.0 ** -133)
