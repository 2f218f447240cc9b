"""Normed rotary rows and their gradient in 64 bits, from their definitions; nothing here is shared with the library."""
import torch

import block_reference as ref


def turn(x, positions, sections, theta, pairing, sign=1, **kw):
    return ref.rope(x, positions, sections, theta, pairing, sign=sign, **kw)


def scale(x, eps):
    return 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + eps)


def forward(x, w, positions, sections, eps, theta=1e4, pairing="half", **kw):
    """(y, tol): the fp32 kernel's bound before the output's rounding.  r: sums of at most 25 roundings a path
    (half of them under the root) and 2 ulp of the root, 2^-19.9; weights, products and the turn four roundings; the angle
    2^-21 of |a| + |b|: 2^-19 of twice the head's largest |x r w| in all."""
    n = x.double() * scale(x, eps) * w.double()
    size = 2 * n.abs().amax(-1, keepdim=True)
    return turn(n, positions, sections, theta, pairing, **kw), size * 2.0 ** -19


def gradient(x, dy, w, positions, sections, eps, theta=1e4, pairing="half", **kw):
    """(dx, dx's tol, dw, dw's tol).  g is off by 2^-21 of twice the head's largest |dy| and a product's roundings,
    r as above; sum u x by 25 roundings of its terms; 2^-18 of each term's largest covers them.  dw: the terms'
    2^-18, and at most 256 additions in a row, 2^-16 of the sum of the terms' largest."""
    x, w = x.double(), w.double()
    r = scale(x, eps)
    g = turn(dy, positions, sections, theta, pairing, sign=-1, **kw)
    u, h = g * w, x * r
    d = x.shape[-1]
    m = (u * x).sum(-1, keepdim=True) * r * r / d
    dx = r * (u - x * m)
    big = 2 * dy.double().abs().amax(-1, keepdim=True)
    em = (big * (w * x).abs()).sum(-1, keepdim=True) * r * r / d
    tol = r * (big * w.abs() + x.abs() * (em + m.abs())) * 2.0 ** -18
    return dx, tol, (g * h).sum((0, 1)), (big * h.abs()).sum((0, 1)) * 2.0 ** -16 + 1e-30
