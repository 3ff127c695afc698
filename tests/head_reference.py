"""Plain definitions of the rotary positions and of the norm of each head, for the tests: torch on the
tensors' own device, in float64."""
from __future__ import annotations

import torch


def pairs(n, layout, device):
    """elements a and b of the n pairs"""
    i = torch.arange(n, device=device)
    return (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)


def angles(positions, freqs):
    """[tokens, 1, n]"""
    return positions.double()[:, None, None] * freqs.double()


def rotate(x, positions, freqs, layout, scale=1.0, inverse=False):
    """(rotated x, and for every element the sum of the magnitudes that made it)"""
    x = x.double()
    y, terms = x.clone(), x.abs()
    if freqs is None or freqs.numel() == 0:
        return y, terms
    a, b = pairs(freqs.numel(), layout, x.device)
    t = angles(positions, freqs)
    c, s = t.cos() * scale, t.sin() * scale * (-1 if inverse else 1)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    both = (x[..., a].abs() + x[..., b].abs()) * abs(scale)
    terms[..., a], terms[..., b] = both, both
    return y, terms


def rstd(x, eps):
    return 1.0 / (x.double().square().mean(-1, keepdim=True) + eps).sqrt()


def norm_rope(x, weight, positions, freqs, eps, layout, scale=1.0):
    """(y, magnitudes)"""
    v = x.double() * rstd(x, eps)
    if weight is not None:
        v = v * weight.double()
    return rotate(v, positions, freqs, layout, scale)


def norm_rope_backward(dy, x, weight, positions, freqs, eps, layout, scale=1.0):
    """(dx, dweight, magnitudes of dx's terms, of dweight's)"""
    r = rstd(x, eps)
    xh = x.double() * r
    w = torch.ones_like(xh[0, 0]) if weight is None else weight.double()
    u, ua = rotate(dy, positions, freqs, layout, scale, inverse=True)
    g, ga = u * w, ua * w.abs()
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    mag = r * (ga + xh.abs() * (ga * xh.abs()).mean(-1, keepdim=True))
    return dx, (u * xh).sum((0, 1)), mag, (ua * xh.abs()).sum((0, 1))
