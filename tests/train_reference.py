"""Plain 64-bit forms of the layer norm (forward, backward) and the grouped
products, and the error bounds their fp32 kernels are held to.

Bounds.  u = 2^-24 is half a step of fp32, ut half a step of the output type.
A sum of n fp32 terms, in any order, is off by at most n*u*sum|terms|; the
kernels' sums are trees or at most `depth` additions long, so depth*u*sum|terms|
bounds them.  Each bound is the output's own rounding ut*|out| plus the fp32
errors carried to the output."""
import math

import torch

U = 2.0 ** -24
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
CODES = {"fp16": 0, "bf16": 1, "fp32": 2}
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp32": 2.0 ** -126}   # half a step below the normal range (fp32: flushed)


def half_step(name):
    return torch.finfo(TYPES[name]).eps / 2


def act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z


def act_slope(name, z):
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def norm_forward(x, res, gamma, beta, eps):
    s = x.double() if res is None else x.double() + res.double()
    mean = s.mean(1, keepdim=True)
    var = ((s - mean) ** 2).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    y = (s - mean) * rstd
    if gamma is not None:
        y = y * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return s, mean[:, 0], rstd[:, 0], y


def norm_forward_bounds(name, s, mean, rstd, y, gamma, beta):
    """(sum, mean, rstd, y).  The row sum has at most depth additions; d = s - mean is off by
    2u|s| + the mean's error; rstd by a relative error of at most twice d's largest over the
    standard deviation (plus the sum's own)."""
    depth = 32 + s.shape[1] // 64
    ut = half_step(name)
    g = torch.ones_like(s[0]) if gamma is None else gamma.double().abs()
    b = torch.zeros_like(s[0]) if beta is None else beta.double().abs()
    e_mean = depth * U * s.abs().mean(1) + U * mean.abs()
    e_d = 2 * U * s.abs() + e_mean[:, None]
    rel = 2 * e_d.amax(1) * rstd + (depth + 8) * U
    e_y = g * (e_d * rstd[:, None] + (s - mean[:, None]).abs() * (rstd * rel)[:, None]) + 4 * U * (y.abs() + b)
    tiny = TINY[name]
    return ut * s.abs() + U * s.abs() + tiny, e_mean + 1e-38, rstd * rel, ut * y.abs() + (1 + ut) * e_y + tiny


def norm_backward(dy, x, gamma, mean, rstd, dres):
    dy, x = dy.double(), x.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    w = dy if gamma is None else dy * gamma.double()
    dx = rstd * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * xh).sum(0), dy.sum(0)


def norm_backward_bounds(name, dy, x, gamma, mean, rstd, dres, dx):
    """(dx, dgamma, dbeta).  xh is off by 2u*rstd*(|x| + |mean|); the row sums have at most `depth`
    additions, the column sums at most one per row."""
    dy, x = dy.double(), x.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    w = dy if gamma is None else dy * gamma.double()
    depth = 32 + x.shape[1] // 64
    e_xh = 2 * U * rstd * (x.abs() + mean.abs()) + 2 * U * xh.abs()
    e_c1 = (depth + 2) * U * w.abs().mean(1, keepdim=True)
    c2 = (w * xh).mean(1, keepdim=True)
    e_c2 = (w.abs() * e_xh).mean(1, keepdim=True) + (depth + 3) * U * (w * xh).abs().mean(1, keepdim=True)
    inner = w.abs() + w.abs().mean(1, keepdim=True) + (xh * c2).abs()
    e = rstd * (e_c1 + xh.abs() * e_c2 + e_xh * c2.abs() + 6 * U * inner)
    if dres is not None:
        e = e + 2 * U * dres.double().abs()
    rows = x.shape[0] + 8
    e_dgamma = (dy.abs() * e_xh).sum(0) + rows * U * (dy * xh).abs().sum(0)
    return half_step(name) * dx.abs() + 2 * e + TINY[name], e_dgamma + 1e-37, rows * U * dy.abs().sum(0) + 1e-37


def grouped(offsets, rows, cols, product):
    """[rows][cols] of `product(e, slice)` over the groups, NaN outside them."""
    out = torch.full((rows, cols), float("nan"), dtype=torch.float64, device="cuda")
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            out[lo:hi] = product(e, slice(lo, hi))
    return out


def product_error(depth, magnitude):
    """fp32 error of a product's sum of `depth` terms whose magnitudes add up to `magnitude`: one
    rounding (or truncation, twice that) per addition."""
    return 2 * (depth + 32) * U * magnitude
