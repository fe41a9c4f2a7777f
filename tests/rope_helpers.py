"""64-bit references of the norms per head and the position rotation, from their definitions, with the bounds that the
kernel's fp32 arithmetic gives.

Bound of an element z = a c - b s (or b c + a s) of a row of D dims, with e = the relative error of a and b:
  * with a norm: the mean's D squares summed in fp32, each partial sum off by 2^-24 of it, half of that through the square
    root; the reciprocal root, its product and the weight's: 8 * 2^-24 at most. e = (D / 2 + 8) 2^-24; without one e = 0
  * two products and their difference: 3 * 2^-24 of |a c| + |b s|
  * the result's rounding to bf16: 2^-8 |z|
"""
from __future__ import annotations

import torch

F64 = torch.float64


def pair_dims(R, interleaved):
    i = torch.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def angles(cos_sin, positions, axes):
    """(cos, sin) [T, R / 2] in 64 bits; positions [T] or [A, T] and the pairs' axes; outside the table: an angle of 0."""
    P, R = cos_sin.shape
    pos = positions if positions.dim() == 2 else positions[None]
    ax = torch.zeros(R // 2, dtype=torch.long) if axes is None else axes.long()
    known = (ax >= 0) & (ax < pos.shape[0])
    at = pos[ax.clamp(0, pos.shape[0] - 1)].T.long()  # [T, R / 2]
    known = known[None] & (at >= 0) & (at < P)
    at, i = at.clamp(0, P - 1), torch.arange(R // 2)
    c, s = cos_sin[at, i].to(F64), cos_sin[at, R // 2 + i].to(F64)
    return torch.where(known, c, torch.ones_like(c)), torch.where(known, s, torch.zeros_like(s)), bool((~known).any())


def rope_ref(x, weight, eps, cos, sin, interleaved, rounded=True):
    """(reference, bound) of the rows of x [T, H, D] (CPU); cos and sin [T, R / 2]. Bound: of the fp32 value before its
    rounding to bf16, and with `rounded` of the result."""
    D = x.shape[-1]
    y = x.to(F64)
    e = 0.0
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * weight.to(F64)
        e = (D / 2 + 8) * 2.0 ** -24
    ref, size = y.clone(), y.abs()
    a, b = pair_dims(2 * cos.shape[1], interleaved)
    c, s = cos[:, None], sin[:, None]
    ref[..., a] = y[..., a] * c - y[..., b] * s
    ref[..., b] = y[..., b] * c + y[..., a] * s
    size[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
    size[..., b] = (y[..., b] * c).abs() + (y[..., a] * s).abs()
    tol = size * (e + 3 * 2.0 ** -24) * 1.01 + 2.0 ** -133
    return ref, tol + (2.0 ** -8 * (ref.abs() + tol) if rounded else 0.0)


def rope_f32(x, cos, sin, interleaved):
    """The rotation without a norm as fp32 arithmetic gives it, product by product (cos and sin: fp32 values)."""
    y = x.float()
    z = y.clone()
    a, b = pair_dims(2 * cos.shape[1], interleaved)
    c, s = cos[:, None].float(), sin[:, None].float()
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    return z


def table(P, R, theta=10000.0):
    i = torch.arange(R // 2, dtype=F64)
    t = torch.arange(P, dtype=F64)[:, None] * theta ** (-2 * i / R)
    return torch.cat([t.cos(), t.sin()], 1).float()
