"""The linear layer and the group normalisation in float64, from their
definitions, with the error that each output of the float32 arithmetic may have.

u is float32's unit roundoff. A sum of n products in any order, with tensor-core
steps that truncate, is off by at most (n + 16) u times the sum of their
magnitudes; an activation multiplies an error by its steepest slope, at most
1.13 (gelu), and adds a few roundings of its own; an output is rounded once, by
at most half a step of its type.
"""
import math

import torch

U = 2.0 ** -24
SLOPE = 1.13


def act(z, a):
    if a == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if a == "silu":
        return z * torch.sigmoid(z)
    if a == "gelu":
        return z * torch.special.ndtr(z)
    return z


def slope(s, a):
    if a == "relu":
        return (s > 0).to(s.dtype)
    if a == "silu":
        g = torch.sigmoid(s)
        return g * (1 + s * (1 - g))
    if a == "gelu":
        return torch.special.ndtr(s) + s * torch.exp(-s * s / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(s)


def half_step(t):
    return torch.finfo(t).eps / 2


def check(name, got, ref, tol):
    """|got - ref| <= tol elementwise (tensors of one shape)."""
    assert tuple(got.shape) == tuple(ref.shape), (name, got.shape, ref.shape)
    off = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), "%s: not finite" % name
    over = off - tol
    if over.numel() and float(over.max()) > 0:
        i = int(over.argmax())
        raise AssertionError("%s: off by %.3g (allowed %.3g) at %d: %.9g for %.9g; %d of %d values" % (
            name, off.flatten()[i], tol.flatten()[i], i, got.flatten()[i], ref.flatten()[i], int((over > 0).sum()),
            over.numel()))


def linear_forward(x, w, b, r, a):
    """{y, z: (reference, tolerance)}"""
    t = x.dtype
    x, w = x.double(), w.double()
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    for v in (b, r):
        if v is not None:
            z, mag = z + v.double(), mag + v.double().abs()
    err = (x.shape[-1] + 16) * U * mag
    y = act(z, a)
    tiny = torch.finfo(torch.float32).tiny
    return {"y": (y, SLOPE * err + 8 * U * z.abs() + half_step(t) * (y.abs() + SLOPE * err) + tiny),
            "z": (z, err + half_step(t) * (z.abs() + err) + tiny)}


def linear_backward(x, w, saved, gy, a):
    """{grad_x, grad_weight, grad_bias, grad_residual: (reference, tolerance)}"""
    t = x.dtype
    x, w, gy = x.double(), w.double(), gy.double()
    dz = gy if a == "none" else gy * slope(saved.double(), a)
    # slopes of silu and gelu: a few roundings of terms of size up to 1 + |s|
    smooth = a in ("silu", "gelu")
    edz = 16 * U * gy.abs() * (1 + saved.double().abs()) if smooth else torch.zeros_like(dz)
    # grad_x of a bfloat16 layer reads dz rounded to bfloat16 (exact for none and relu)
    edx = edz + half_step(t) * (dz.abs() + edz) if smooth and t == torch.bfloat16 else edz
    N, M = dz.shape[-1], dz.shape[0]
    gx, egx = dz @ w, (N + 16) * U * (dz.abs() @ w.abs()) + edx @ w.abs()
    gw, egw = dz.t() @ x, (M + 16) * U * (dz.abs().t() @ x.abs()) + edz.t() @ x.abs()
    gb, egb = dz.sum(0), (M + 16) * U * dz.abs().sum(0) + edz.sum(0)
    h, f = half_step(t), U
    tiny = torch.finfo(torch.float32).tiny
    return {"grad_x": (gx, egx + h * (gx.abs() + egx) + tiny), "grad_weight": (gw, egw + f * gw.abs() + tiny),
            "grad_bias": (gb, egb + f * gb.abs() + tiny), "grad_residual": (dz, edz + h * (dz.abs() + edz) + tiny)}


def norm_stats(x, groups, eps):
    B, H, W, C = x.shape
    v = x.double().reshape(B, H * W, groups, C // groups)
    var, mean = torch.var_mean(v, dim=(1, 3), correction=0)
    return mean, (var + eps).rsqrt()


def _spread(v, C):
    """[B, groups] -> [B, 1, 1, C]"""
    return v.repeat_interleave(C // v.shape[1], dim=1)[:, None, None, :]


def norm_forward(x, ga, be, groups, eps, a):
    """{y, mean, rstd: (reference, tolerance)}. A sum goes through chains of at most a few hundred additions whose
    roundings are independent: 64 u of the values' size is over twice the square root of their number. The mean and
    the variance are off by that, rstd by half of the variance's; hat takes on both."""
    B, H, W, C = x.shape
    t = x.dtype
    mean, rstd = norm_stats(x, groups, eps)
    size = x.double().abs().reshape(B, H * W, groups, C // groups).mean(dim=(1, 3)) + 1 / rstd
    em = 64 * U * size
    er = rstd * (64 * U * (1 + mean.abs() * rstd))
    m, r = _spread(mean, C), _spread(rstd, C)
    xd = x.double()
    hat = (xd - m) * r
    g = torch.ones(C, dtype=torch.float64, device=x.device) if ga is None else ga.double()
    b = torch.zeros_like(g) if be is None else be.double()
    z = hat * g + b
    ehat = _spread(em, C) * r + hat.abs() * _spread(er, C) / r + 4 * U * (hat.abs() + 0 * r)
    err = ehat * g.abs() + 4 * U * (z.abs() + b.abs())
    y = act(z, a)
    return {"y": (y, SLOPE * err + 8 * U * z.abs() + half_step(t) * (y.abs() + SLOPE * err)),
            "mean": (mean, em + U * mean.abs()), "rstd": (rstd, er + U * rstd)}


def norm_backward(x, ga, be, stats, gy, groups, a):
    """{grad_x, grad_gamma, grad_beta: (reference, tolerance)}; stats as given, float32."""
    B, H, W, C = x.shape
    t = x.dtype
    n = H * W * (C // groups)
    m, r = (_spread(stats[..., k].double(), C) for k in (0, 1))
    hat = (x.double() - m) * r
    g = torch.ones(C, dtype=torch.float64, device=x.device) if ga is None else ga.double()
    b = torch.zeros_like(g) if be is None else be.double()
    z = hat * g + b
    gy = gy.double()
    dz = gy * slope(z, a)
    # the slope of silu and gelu changes by at most 0.8 for a step of 1 in z
    ez = 8 * U * (hat.abs() * g.abs() + b.abs())
    edz = gy.abs() * (16 * U * (1 + z.abs()) + 0.8 * ez) if a in ("silu", "gelu") else torch.zeros_like(dz)
    over = lambda v: v.reshape(B, H * W, groups, C // groups).sum(dim=(1, 3))  # noqa: E731
    dh = dz * g
    c1, c2 = over(dh) / n, over(dh * hat) / n
    e1 = over((64 * U * dz.abs() + edz) * g.abs()) / n
    e2 = over((64 * U * dz.abs() + edz) * g.abs() * hat.abs()) / n
    gx = r * (dh - _spread(c1, C) - hat * _spread(c2, C))
    egx = r * (edz * g.abs() + _spread(e1, C) + hat.abs() * _spread(e2, C)
               + 8 * U * (dh.abs() + _spread(c1.abs(), C) + hat.abs() * _spread(c2.abs(), C)))
    px = lambda v: v.sum(dim=(0, 1, 2))  # noqa: E731
    tiny = torch.finfo(torch.float32).tiny
    return {"grad_x": (gx, egx + half_step(t) * (gx.abs() + egx) + tiny),
            "grad_gamma": (px(dz * hat), px((64 * U * dz.abs() + edz) * hat.abs()) + tiny),
            "grad_beta": (px(dz), px(64 * U * dz.abs() + edz) + tiny)}
