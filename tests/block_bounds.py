"""First-order rounding-error bounds of the LayerNorm and dense-linear kernels (fp64 tensors).

u = 2^-8 is bf16's unit roundoff, v = 2^-24 fp32's.  A sum of n fp32 terms in any fixed tree is off by at
most n v sum|t|; the kernels' row sums add at most 64 terms in sequence and then reduce in a tree (about 75
additions deep at most), the column sums at most `depth` (given by the caller).  The tensor cores may
truncate when they add, so a product of depth K is bounded by K 2 v sum|p q|.  Elementary functions and the
few operations around them are held to 16 v of their result's scale.
"""
import torch

from oracle import block as K

U, V = 2.0 ** -8, 2.0 ** -24
ROW = 96 * V     # a row reduction and the handful of operations that use it


def layernorm_fwd(x, g, b, eps):
    """y, mean, rstd and their bounds."""
    d = x.shape[1]
    mean = x.mean(1)
    c = x - mean[:, None]
    var = (c * c).mean(1)
    rstd = (var + eps) ** -0.5
    y = K.layernorm(x, g, b, eps)
    amean = ROW * x.abs().mean(1)
    # the centred values are off by the mean's error plus a rounding; var by their squares' sums
    ec = amean[:, None] + V * c.abs()
    evar = ROW * var + 2 * (c.abs() * ec).mean(1) + (ec * ec).mean(1)
    erstd = 0.5 * rstd ** 3 * evar + 4 * V * rstd
    ey = (rstd[:, None] * ec + c.abs() * erstd[:, None]) * g.abs() + 8 * V * y.abs()
    if b is not None:
        ey = ey + 8 * V * b.abs()
    return {"y": (y, ey * (1 + U) + U * y.abs()), "mean": (mean, amean + V * mean.abs()), "rstd": (rstd, erstd)}


def layernorm_bwd(dy, x, g, mean, rstd, res, depth):
    """dx (+ res), dg, db from the statistics as given, and their bounds."""
    xh = (x - mean[:, None]) * rstd[:, None]
    exh = 4 * V * xh.abs()
    a = dy * g
    m1, m2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    em1, em2 = ROW * a.abs().mean(1, keepdim=True), ROW * (a * xh).abs().mean(1, keepdim=True)
    dx = rstd[:, None] * (a - m1 - xh * m2)
    mag = rstd[:, None] * (a.abs() + m1.abs() + (xh * m2).abs())
    edx = rstd[:, None] * (em1 + xh.abs() * em2 + exh * m2.abs()) + 16 * V * mag
    out = dx if res is None else dx + res
    if res is not None:
        edx = edx + 4 * V * res.abs()
    t = dy * xh
    return {"dx": (out, edx * (1 + U) + U * out.abs()),
            "dg": (t.sum(0), ((depth + 8) * V) * t.abs().sum(0)),
            "db": (dy.sum(0), ((depth + 8) * V) * dy.abs().sum(0))}


def linear_fwd(x, w, b, kind, res):
    z, y = K.linear(x, w, b, kind, res)
    ez = x.shape[1] * 2 * V * (x.abs() @ w.abs().T) + 4 * V * z.abs()
    if b is not None:
        ez = ez + 4 * V * b.abs()
    a = K.act(z, kind)
    ey = 1.2 * ez + 16 * V * (a.abs() + z.abs())       # every activation's slope is at most 1.13
    if res is not None:
        ey = ey + 4 * V * res.abs()
    return {"z": (z, ez * (1 + U) + U * z.abs()), "y": (y, ey * (1 + U) + U * y.abs())}


def linear_bwd(dy, x, w, z, kind, depth, dw_f32=False):
    """depth: additions behind one element of db (the contraction of dw is the rows of dy)."""
    if kind == "none":
        dz, e32, e16 = dy, torch.zeros_like(dy), torch.zeros_like(dy)
    else:
        zz = z.detach().clone().requires_grad_(True)
        (dz,) = torch.autograd.grad(K.act(zz, kind), zz, grad_outputs=dy)
        # act' is a sum of terms up to 1 + |z| phi in size: their rounding, not act' itself, sets the error
        e32 = 32 * V * dy.abs() * (1 + z.abs().clamp(max=8))
        e16 = e32 * (1 + U) + U * dz.abs()
    m, n = dy.shape
    dx, dw, db = dz @ w, dz.T @ x, dz.sum(0)
    a = dz.abs()
    edx = e16 @ w.abs() + n * 2 * V * (a @ w.abs())
    edw = e16.T @ x.abs() + m * 2 * V * (a.T @ x.abs())
    return {"dx": (dx, edx * (1 + U) + U * dx.abs()),
            "dw": (dw, edw + 4 * V * dw.abs() if dw_f32 else edw * (1 + U) + U * dw.abs()),
            "db": (db, e32.sum(0) + ((depth + 8) * V) * a.sum(0))}
