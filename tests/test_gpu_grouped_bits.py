"""The products by group, bit for bit the single product of each group where both take the kernel for any alignment, or
share K among eight waves: a group's place among the others changes nothing in the order of its sums."""
import pytest

import block_reference as ref
import group_reference as grp
from test_gpu_grouped import data, ends_of, mx, weights  # noqa: F401 (mx is a fixture)

pytestmark = pytest.mark.gpu
TYPES = [("float32", True), ("bfloat16", True), ("bfloat16", False)]


def unaligned(codes):
    """the same codes in rows of an odd number of bytes"""
    import torch
    n, k = codes.shape
    buf = torch.zeros(n, (k + 17) | 1, dtype=torch.uint8, device="cuda")
    buf[:, 3:3 + k] = codes
    return buf[:, 3:3 + k]


@pytest.mark.parametrize("K", [640, 200])
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("dtype,full", TYPES)
def test_rows(mx, K, tile, dtype, full):
    import torch
    sizes = [300, 0, 512, 2, 200]
    ends, dtype = ends_of(sizes), getattr(torch, dtype)
    c, s = mx.block_quantize(data(1020, K, seed=81), "e4m3")
    a, b = (unaligned(c), s), weights(mx, 5, 384, K, "e5m2", tile, 82)
    assert a[0].stride(0) % 16 != 0
    got = torch.full((1020, 384), 7.0, dtype=dtype, device="cuda")
    mx.block_gemm_grouped(*a, "e4m3", *b, "e5m2", ends, out_dtype=dtype, full_sums=full, out=got)
    for i, (lo, hi) in enumerate(grp.ranges(ends.tolist(), 1020)):
        if hi > lo:
            one = mx.block_gemm(a[0][lo:hi], a[1][:, lo:hi], "e4m3", b[0][i], b[1][i], "e5m2", out_dtype=dtype, full_sums=full)
            assert torch.equal(got[lo:hi], one)
    assert (got[ends[-1]:] == 7).all()


# whole blocks in rows of odd length; 64 x 32 tiles of which either call makes less than two rounds
@pytest.mark.parametrize("odd", [True, False])
@pytest.mark.parametrize("dtype,full", TYPES)
def test_columns(mx, odd, dtype, full):
    import torch
    sizes = [700, 0, 513, 128, 1300]
    ends, dtype = ends_of(sizes), getattr(torch, dtype)
    a = mx.block_quantize_grouped(data(2641, 200, seed=83), ends, "e4m3")
    b = mx.block_quantize_grouped(data(2641, 136, seed=84), ends, "e5m2")
    if odd:
        a, b = (unaligned(a[0]), a[1]), (unaligned(b[0]), b[1])
    got = mx.block_gemm_grouped_k(*a, "e4m3", *b, "e5m2", ends, out_dtype=dtype, full_sums=full)
    for i, (lo, hi) in enumerate(grp.blocks(ends.tolist(), 2641)):
        if hi > lo:
            cut = lambda t: (t[0][:, 128 * lo:128 * hi], t[1][lo:hi])
            ca, cb = cut(a), cut(b)
            one = mx.block_gemm(*ca, "e4m3", *cb, "e5m2", out_dtype=dtype, full_sums=full)
            assert torch.equal(got[i], one)
        else:
            assert (got[i] == 0).all()
