"""Plain definitions of the block-128 FP8 operators and of the norm, for the tests: torch on the
tensors' own device, sums in float64.  The quantizer's fp32 operations are written out one by one
(each rounds once), so its codes and scales have one right value each."""
from __future__ import annotations

import torch

BLK = 128
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOOR = 2.0 ** -100
# half a step: relative for normal values, absolute (in units of the scale) for subnormal ones
HALF_REL = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
HALF_SUB = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}


def cdiv(a, b):
    return -(-a // b)


def block_amax(v, tile):
    """largest |v| (or NaN / inf) of every block along the last dim: [rows or tiles, blocks]"""
    rows, k = v.shape
    out = torch.stack([v[:, k0:k0 + BLK].abs().amax(1) for k0 in range(0, k, BLK)], 1)
    if tile:
        out = torch.stack([out[r:r + BLK].amax(0) for r in range(0, rows, BLK)])
    return out


def quantize(x, fmt, mode="row"):
    """(codes uint8 [n x k], scales fp32 [blocks x n or tiles]) of a bf16 or fp32 matrix"""
    v = x.float()
    if mode.endswith("transpose"):
        v = v.t().contiguous()
    tile = mode.startswith("tile")
    amax = block_amax(v, tile)
    bad = ~torch.isfinite(amax)
    amax = torch.where(bad, torch.zeros_like(amax), amax).clamp(min=FLOOR)
    fmax = torch.full_like(amax, FMAX[fmt])
    scales, inv = amax / fmax, fmax / amax
    scales = torch.where(bad, torch.full_like(scales, float("nan")), scales)
    per = lambda t: spread(t, v.shape, tile)
    q = torch.where(per(bad), torch.zeros_like(v), v) * per(inv)
    codes = q.clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)
    codes = torch.where(per(bad), torch.zeros_like(codes), codes)
    return codes, scales.t().contiguous()


def spread(t, shape, tile):
    """[rows or tiles, blocks] -> one value for every element of shape"""
    if tile:
        t = t.repeat_interleave(BLK, 0)[:shape[0]]
    return t.repeat_interleave(BLK, 1)[:, :shape[1]]


def values(codes, scales, fmt, tile=False):
    """float64 values of an operand"""
    return codes.contiguous().view(F8[fmt]).double() * spread(scales.double().t(), codes.shape, tile)


def gemm(a, fa, b, fb, tile):
    """(C, sum of |terms|) in float64"""
    va, vb = values(*a, fa), values(*b, fb, tile)
    return va @ vb.t().contiguous(), va.abs() @ vb.abs().t().contiguous()


def norm(x, weight, bias, eps, rms):
    """(y, mean, rstd) in float64"""
    v = x.double()
    mean = torch.zeros_like(v[:, 0]) if rms else v.mean(1)
    d = v - mean[:, None]
    rstd = 1.0 / (d.square().mean(1) + eps).sqrt()
    y = d * rstd[:, None]
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y, mean, rstd


def norm_backward(dy, x, weight, mean, rstd, rms):
    """(dx, dweight, dbias) in float64"""
    v, d = x.double(), dy.double()
    xh = (v if rms else v - mean.double()[:, None]) * rstd.double()[:, None]
    g = d if weight is None else d * weight.double()
    inner = g - xh * (g * xh).mean(1, keepdim=True)
    if not rms:
        inner = inner - g.mean(1, keepdim=True)
    return inner * rstd.double()[:, None], (d * xh).sum(0), d.sum(0)
