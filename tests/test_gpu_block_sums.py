"""Block-128 products to bf16 with sums in fp32: the fp32 product rounded once, bit for bit, from every kernel; and the
term that the FP8 instruction's window loses is there."""
import pytest

import block_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_block_amax_amd as m
    m.lib()
    return m


def data(rows, cols, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, cols, device="cuda", generator=g).bfloat16()


# few rows (8 to 64, one and two rounds), 64 x 32, 128 x 128 and 256 x 128 tiles, K in whole chunks and not, K = 0
SIZES = [(1, 1, 1), (1, 300, 4001), (8, 4096, 256), (16, 130, 1024), (31, 515, 640), (48, 512, 2048), (64, 640, 1152), (64, 9000, 272),
         (100, 1000, 144), (300, 300, 15), (1100, 1100, 15), (1111, 1301, 401), (1100, 1102, 384), (2300, 4100, 272), (4100, 4251, 401),
         (5, 7, 0)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("aligned", [True, False])
def test_full_sums_are_the_fp32_product_rounded(mx, M, N, K, tile, aligned):
    """C dense and inside a buffer whose other elements stay"""
    import torch
    print("case", M, N, K, tile, aligned, flush=True)
    for fa, fb in (("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")):
        a, b = mx.block_quantize(data(M, K, 1), fa), mx.block_quantize(data(N, K, 2), fb, "tile" if tile else "row")
        if not aligned:
            buf = torch.full((M, K + 3), 0x7F, dtype=torch.uint8, device="cuda")
            buf[:, 1:1 + K] = a[0]
            a = (buf[:, 1:1 + K], a[1])
        want = mx.block_gemm(*a, fa, *b, fb, out_dtype=torch.float32)
        if K:
            C, S = ref.gemm(a, fa, b, fb, tile)
            assert ((want.double() - C).abs() <= (130 + ref.cdiv(K, 128)) * 2.0 ** -24 * S).all()
        want = want.bfloat16()
        assert torch.equal(mx.block_gemm(*a, fa, *b, fb, full_sums=True), want)
        for off, pad in ((1, 2), (4, 4)):
            buf = torch.full((M + 2, off + N + pad), 3.0, dtype=torch.bfloat16, device="cuda")
            c = buf[1:1 + M, off:off + N]
            mx.block_gemm(*a, fa, *b, fb, out=c, full_sums=True)
            assert torch.equal(c, want)
            c.fill_(3.0)
            assert (buf == 3.0).all(), "elements outside C were written"


@pytest.mark.parametrize("M,N", [(1, 64), (40, 64), (300, 256), (1200, 1200), (4200, 4100)])
def test_full_sums_keep_what_a_cancelled_pair_leaves(mx, M, N):
    """448 * 448 and its negative in one step of 32 products, and 1: fp32 holds the 1 to half a step of the running
    sum, 2^-7 at each of the two additions that meet the pair; half a step of bf16 at 1 is 2^-8"""
    import torch
    a = torch.zeros(M, 256, dtype=torch.uint8, device="cuda")
    b = torch.zeros(N, 256, dtype=torch.uint8, device="cuda")
    a[:, 3], b[:, 3] = 0x38, 0x38
    a[:, 5], b[:, 5] = 0x7E, 0x7E
    a[:, 6], b[:, 6] = 0x7E, 0xFE
    s = torch.ones(2, M, device="cuda"), torch.ones(2, N, device="cuda")
    c = mx.block_gemm(a, s[0], "e4m3", b, s[1], "e4m3", full_sums=True)
    assert ((c.double() - 1).abs() <= 2 * 2.0 ** -7 + 2.0 ** -8).all()


def test_full_sums_nan_and_inf(mx):
    """a NaN scale and an Inf code come through the rounding"""
    import torch
    for M, N in ((40, 300), (300, 300), (1200, 1200)):
        a, b = mx.block_quantize(data(M, 400, 1), "e5m2"), mx.block_quantize(data(N, 400, 2), "e4m3")
        a[0][0, 7], a[1][1, 3] = 0x7C, float("nan")
        b[0][:, 7] = 0x38
        c = mx.block_gemm(*a, "e5m2", *b, "e4m3", full_sums=True)
        assert (c[0] == float("inf")).all() and c[3].isnan().all() and c[1:3].isfinite().all() and c[4:].isfinite().all()
    x = mx.block_gemm(*a, "e5m2", *b, "e4m3", out_dtype=torch.float32)
    assert x.dtype == torch.float32 and torch.equal(mx.block_gemm(*a, "e5m2", *b, "e4m3", out_dtype=torch.float32, full_sums=True)[4:], x[4:])
