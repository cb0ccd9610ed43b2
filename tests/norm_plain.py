"""Group norm with an activation in 64 bits, written from its definition, and
the error bounds the float32 kernels are held to."""
import math

import torch

from deformable_convolution_gb300 import binding as B

U = 2.0 ** -24  # half a unit in the last place of float32; bf16's, with 8 significant bits, is 2^-8


def act(z, kind):
    if kind == B.DC_ACT_RELU:
        return z.clamp_min(0)
    if kind == B.DC_ACT_SILU:
        return z / (1 + torch.exp(-z))
    if kind == B.DC_ACT_GELU:
        return z * 0.5 * (1 + torch.erf(z / math.sqrt(2)))
    return z


def slope(z, kind):
    if kind == B.DC_ACT_RELU:
        return (z > 0).double()
    if kind == B.DC_ACT_SILU:
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    if kind == B.DC_ACT_GELU:
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def grouped(p, t):
    """float64 [n, groups, channels of a group, pixels]."""
    t = t.double()
    if p.layout == B.DC_NHWC:
        t = t.permute(0, 3, 1, 2)
    return t.reshape(p.n, p.groups, p.c // p.groups, p.h * p.w)


def layout(p, t):
    t = t.reshape(p.n, p.c, p.h, p.w)
    return t.permute(0, 2, 3, 1) if p.layout == B.DC_NHWC else t


def affine(p, gamma, beta):
    g = torch.ones(p.c) if gamma is None else gamma
    b = torch.zeros(p.c) if beta is None else beta
    return (v.double().reshape(1, p.groups, -1, 1) for v in (g, b))


def forward(p, x, gamma, beta):
    """dict of y, mean, rstd and of bounds on the kernels' error in them.

    The float32 sums add at most about 2 log2(m) + 8 terms in a row (a batch,
    a thread's batches of a bounded segment, shuffles, parts): each rounds by
    U of the running sum, at most of max|x|; 64 covers every size tested.
    z inherits the mean's error times rstd * gamma, and an error relative to
    the distance from the mean; the activations add a few units of z."""
    xg = grouped(p, x)
    g, b = affine(p, gamma, beta)
    mean = xg.mean((2, 3), keepdim=True)
    var = (xg - mean).square().mean((2, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + p.eps)
    xh = (xg - mean) * rstd
    z = xh * g + b
    y = act(z, p.act)
    top = xg.abs().amax((2, 3), keepdim=True)
    d_mean = 64 * U * top
    # var's error: relative from its own sums, and the mean's error squared
    d_rstd = rstd * (64 * U + 0.5 * rstd * rstd * d_mean ** 2 + rstd * d_mean * 2 * U)
    d_z = (d_mean * rstd + xh.abs() * 96 * U) * g.abs() + xh.abs() * g.abs() * d_rstd / rstd + 8 * U * (z.abs() + b.abs())
    d_y = 1.2 * d_z + 32 * U * (z.abs() + 1)
    if p.dtype == B.DC_BF16:
        d_y = d_y + (y.abs() + d_y) * 2.0 ** -8 * 1.01
    return dict(y=layout(p, y), d_y=layout(p, d_y), mean=mean[:, :, 0, 0], d_mean=d_mean[:, :, 0, 0] + 1e-40,
                rstd=rstd[:, :, 0, 0], d_rstd=d_rstd[:, :, 0, 0], z=layout(p, z), d_z=layout(p, d_z))


def backward(p, x, gamma, beta, mean, rstd, gy):
    """Gradients for the given (float32) mean and rstd, with bounds.

    dz carries the activation slope's error (a few units, and where z is
    within its own error of the ReLU's kink, all of gy); the sums of dz and
    dz * xh add at most 64 roundings of their absolute sums; grad_x is a
    difference of three terms, each with its own relative error."""
    xg, gyg = grouped(p, x), grouped(p, gy)
    g, b = affine(p, gamma, beta)
    mu, r = (t.double()[:, :, None, None] for t in (mean, rstd))
    xh = (xg - mu) * r
    z = xh * g + b
    d_xh = (2 * U) * (xh.abs() + 1e-30)
    d_z = d_xh * g.abs() + 4 * U * (z.abs() + b.abs())
    dz = gyg * slope(z, p.act)
    d_dz = gyg.abs() * (32 * U * (1 + z.abs()) + (1.2 * d_z if p.act in (B.DC_ACT_SILU, B.DC_ACT_GELU) else 0 * d_z))
    if p.act == B.DC_ACT_RELU:
        d_dz = d_dz + gyg.abs() * (z.abs() <= d_z)
    m = xg.shape[2] * xg.shape[3]
    A, Bs = dz.sum(3, keepdim=True), (dz * xh).sum(3, keepdim=True)
    d_A = d_dz.sum(3, keepdim=True) + 64 * U * dz.abs().sum(3, keepdim=True)
    d_B = (d_dz * xh.abs() + dz.abs() * d_xh).sum(3, keepdim=True) + 64 * U * (dz * xh).abs().sum(3, keepdim=True)
    s1, s2 = (g * A).sum(2, keepdim=True) / m, (g * Bs).sum(2, keepdim=True) / m
    d_s1 = (g.abs() * (d_A + 64 * U * A.abs())).sum(2, keepdim=True) / m
    d_s2 = (g.abs() * (d_B + 64 * U * Bs.abs())).sum(2, keepdim=True) / m
    gx = r * (g * dz - s1 - xh * s2)
    d_gx = r * (g.abs() * d_dz + d_s1 + xh.abs() * d_s2 + d_xh * s2.abs()
                + 4 * U * ((g * dz).abs() + s1.abs() + (xh * s2).abs()))
    if p.dtype == B.DC_BF16:
        d_gx = d_gx + (gx.abs() + d_gx) * 2.0 ** -8 * 1.01
    per = lambda t: t.sum(0).reshape(-1)  # noqa: E731
    return dict(grad_x=layout(p, gx), d_grad_x=layout(p, d_gx) + 1e-38,
                grad_gamma=per(Bs), d_grad_gamma=per(d_B + 64 * U * Bs.abs()) + 1e-38,
                grad_beta=per(A), d_grad_beta=per(d_A + 64 * U * A.abs()) + 1e-38)
