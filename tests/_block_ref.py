"""The operators around the products in 64 bits, from their formulas, with
bounds on what 32-bit evaluation may be off (nothing here calls the library)."""
from __future__ import annotations

import torch

U = 2.0 ** -24          # half a step of fp32, relative
SUM = 64                # roundings that an fp32 sum over a row may collect: at most 32
#                         values one after another in a thread, 10 levels of the tree,
#                         the squares' and the factors' own


def half_step(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


def norm(v, w, b, kind, eps, err):
    """(n(v), bound on its error) of v with an error of at most err a value."""
    if kind is None:
        return v, err
    if kind == "layer":
        mean = v.mean(dim=1, keepdim=True)
        # the mean's own error, and the rounding of v - mean
        err = err + err.mean(dim=1, keepdim=True) + SUM * U * v.abs().mean(dim=1, keepdim=True) + U * (v.abs() + mean.abs())
        v = v - mean
    q = (v * v).mean(dim=1, keepdim=True) + eps
    f = torch.rsqrt(q)
    rel = SUM * U + (err * v.abs()).mean(dim=1, keepdim=True) / q + 0.5 * err.square().mean(dim=1, keepdim=True) / q
    out, bound = v * f, f * (err + v.abs() * (rel + 4 * U))
    if w is not None:
        out, bound = out * w.double(), bound * w.double().abs()
    if b is not None:
        out = out + b.double()
        bound = bound + U * out.abs()
    return out, bound


def residual(x, y, gate, scale, post, pre, sigmoid=False):
    """((x', bound), (h, bound)) in 64 bits on the CPU; post, pre: (w, b, kind, eps)."""
    x = x.cpu().double()
    err = torch.zeros_like(x)
    if y is not None:
        d, derr = norm(y.cpu().double(), *post, torch.zeros_like(x))
        if gate is not None:
            g = gate.cpu().double()
            if sigmoid:
                g = torch.sigmoid(g)
                derr = derr + d.abs() * 8 * U
            d, derr = d * g, derr * g.abs()
        x = x + scale * d
        err = abs(scale) * (derr + 4 * U * d.abs()) + U * x.abs()
    h = norm(x, *pre, err) if pre[2] is not None else None
    return (x, err), h


def lies_between(got, want, err):
    """Whether got is the rounding of something within err of want: all of it."""
    t = got.dtype
    g = got.cpu().double()
    tiny = torch.finfo(t).smallest_normal * half_step(t) * 2  # half a step of a subnormal, and more
    return bool(((g - want).abs() <= err + half_step(t) * (want.abs() + err) + tiny).all())
