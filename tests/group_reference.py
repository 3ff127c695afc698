"""Plain definitions of the block-128 operators by group, for the tests, on block_reference's: one group at a time."""
from __future__ import annotations

import torch

import block_reference as ref
from block_reference import BLK, cdiv


def ranges(ends, rows):
    """(first row, end) of every group: an end is at most `rows` and at least the ends before it"""
    out, at = [], 0
    for e in ends:
        e = max(at, min(e, rows))
        out.append((at, e))
        at = e
    return out


def blocks(ends, rows):
    """(first block, end) of every group in the transposed form"""
    out, b = [], 0
    for lo, hi in ranges(ends, rows):
        out.append((b, b + cdiv(hi - lo, BLK)))
        b = out[-1][1]
    return out


def bound(rows, groups):
    """the most columns of the transposed form"""
    return (rows + (BLK - 1) * min(rows, groups)) // BLK * BLK


def quantize(x, ends, fmt, fill_codes=0, fill_scales=0.0):
    """(codes [cols x bound], scales [bound / 128 x cols]), what is not written filled"""
    rows, cols = x.shape
    k = bound(rows, len(ends))
    codes = torch.full((cols, k), fill_codes, dtype=torch.uint8, device=x.device)
    scales = torch.full((k // BLK, cols), fill_scales, device=x.device)
    for (lo, hi), (b0, b1) in zip(ranges(ends, rows), blocks(ends, rows)):
        if hi > lo:
            codes[:, b0 * BLK:b1 * BLK] = 0
            c, s = ref.quantize(x[lo:hi], fmt, "transpose")
            codes[:, b0 * BLK:b0 * BLK + hi - lo] = c
            scales[b0:b1] = s
    return codes, scales


def gemm(a, fa, b, fb, ends, tile):
    """(C, sum of |terms|) in float64, zeros in rows of no group; b: codes [G x N x K], scales [G x blocks x tiles or N]"""
    rows, n = a[0].shape[0], b[0].shape[1]
    C = torch.zeros(rows, n, dtype=torch.float64, device=a[0].device)
    S = torch.zeros_like(C)
    for i, (lo, hi) in enumerate(ranges(ends, rows)):
        if hi > lo:
            C[lo:hi], S[lo:hi] = ref.gemm((a[0][lo:hi], a[1][:, lo:hi]), fa, (b[0][i], b[1][i]), fb, tile)
    return C, S


def gemm_k(a, fa, b, fb, ends):
    """(C [G x M x N], sum of |terms|) in float64"""
    cols = a[0].shape[1]
    out = []
    for b0, b1 in blocks(ends, cols):
        b0, b1 = min(b0, cols // BLK), min(b1, cols // BLK)
        cut = lambda t: (t[0][:, b0 * BLK:b1 * BLK], t[1][b0:b1])
        if b1 > b0:
            out.append(ref.gemm(cut(a), fa, cut(b), fb, False))
        else:
            z = torch.zeros(a[0].shape[0], b[0].shape[0], dtype=torch.float64, device=a[0].device)
            out.append((z, z))
    return torch.stack([c for c, _ in out]), torch.stack([s for _, s in out])
