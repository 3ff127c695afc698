"""Block-128 products of operands that are not aligned to 16 bytes, in every form of scales and pair of formats, and
the bound of the fp32 sums, on sums made to lose the most.

Tolerance of fp32 sums: products are exact; a block's 128 of them are at most 127 additions, its scales' product one
rounding, and each of the ceil(K / 128) blocks one more of the running sum: (130 + ceil(K / 128)) 2^-24 of the sum of
|terms|, second-order terms included.  bf16 output adds half a step of the result (2^-8), and on the FP8
instruction the window of test_gpu_block.py (2^-8 of the sum of |terms|)."""
import pytest

import block_reference as ref

pytestmark = pytest.mark.gpu
FORMATS = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")]


@pytest.fixture(scope="module")
def mx():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_block_amax_amd as m
    m.lib()
    return m


def sums_bound(K):
    return (130 + ref.cdiv(K, 128)) * 2.0 ** -24


def operand(mx, n, k, fmt, tile, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, k, device="cuda", generator=g)
    x = x * torch.exp2(torch.randint(-3, 4, (n, 1), device="cuda", generator=g).float())
    x = x * torch.exp2(torch.randint(-3, 4, (1, k), device="cuda", generator=g).float())
    return mx.block_quantize(x.bfloat16(), fmt, "tile" if tile else "row")


def inside(t, off, pad, fill):
    """t within a larger buffer of `fill`, rows `off` elements in and the pitch t's width + off + pad"""
    import torch
    buf = torch.full((t.shape[0] + 2, off + t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    v = buf[1:1 + t.shape[0], off:off + t.shape[1]]
    v.copy_(t)
    return v


def check(c, a, fa, b, fb, tile, K):
    import torch
    C, S = ref.gemm(a, fa, b, fb, tile)
    tol = sums_bound(K) * S if c.dtype == torch.float32 else 2.0 ** -8 * (C.abs() + S) + 2.0 ** -134
    bad = ~((c.double() - C).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


# one tile and part of one, more than one tile either way with odd edges; K of several blocks and a remainder, whole
# blocks, and less than one
SIZES = [(1, 1, 3), (1, 300, 645), (129, 131, 257), (257, 385, 1000), (300, 129, 640), (140, 520, 100), (513, 260, 901)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
def test_unaligned_operands(mx, M, N, K, tile, bf16):
    """both operands, one of them, or only their pitch unaligned; NaN codes and NaN scales around them, and C inside a
    buffer whose other elements stay"""
    import torch
    print("case", M, N, K, tile, bf16, flush=True)
    dt = torch.bfloat16 if bf16 else torch.float32
    for fa, fb in FORMATS:
        a, b = operand(mx, M, K, fa, False, M + K), operand(mx, N, K, fb, tile, N + K + 1)
        for (oa, pa), (ob, pb) in (((1, 6), (3, 4)), ((5, 11), (16, 16 - K % 16)), ((16, 16 - K % 16), (7, 0)), ((0, 1), (8, 8))):
            nan = float("nan")
            buf = torch.full((M + 2, N + 9), 3.0, dtype=dt, device="cuda")
            c = buf[1:1 + M, oa % 5:oa % 5 + N]
            mx.block_gemm(inside(a[0], oa, pa, 0x7F), inside(a[1], oa, pa, nan), fa, inside(b[0], ob, pb, 0x7F),
                          inside(b[1], ob, pb, nan), fb, out_dtype=dt, out=c)
            check(c, a, fa, b, fb, tile, K)
            c.fill_(3.0)
            assert (buf == 3.0).all(), "elements outside C were written"


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("tile", [True, False])
def test_unaligned_special_codes_and_scales(mx, bf16, tile):
    """NaN and Inf codes and a NaN scale, of an unaligned operand: the elements that they enter, and no others"""
    import torch
    dt = torch.bfloat16 if bf16 else torch.float32
    M, N, K = 300, 290, 400
    a, b = operand(mx, M, K, "e4m3", False, 1), operand(mx, N, K, "e5m2", tile, 2)
    a[0][:, 7] = 0x38                                    # 1
    b[0][289, 399], b[0][0, 7] = 0x7F, 0x7C             # NaN, Inf
    a[0][5, 130] = 0xFF                                  # NaN
    a[1][2, 140] = float("nan")
    c = mx.block_gemm(inside(a[0], 1, 2, 0x7F), a[1], "e4m3", inside(b[0], 3, 0, 0x7F), b[1], "e5m2", out_dtype=dt)
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[:, 289], want[5], want[140] = True, True, True
    assert torch.equal(c.isnan(), want)
    inf = torch.zeros_like(want)
    inf[:, 0] = True
    assert torch.equal(c == float("inf"), inf & ~want)


def test_one_block_scales_of_any_stride(mx):
    """with one block of K the stride between blocks of scales is never used, whatever it is"""
    import ctypes
    import torch
    M, N, K = 70, 300, 96
    a, b = operand(mx, M, K, "e4m3", False, 1), operand(mx, N, K, "e4m3", False, 2)
    c = torch.zeros(M, N, device="cuda")
    P = lambda t: ctypes.c_void_p(t.data_ptr())
    for ld in (1 << 40, 1 << 61, (1 << 63) - 1):
        c.zero_()
        assert mx.lib().mx_block_gemm(P(a[0]), K, P(a[1]), ld, 0, P(b[0]), K, P(b[1]), ld, 0, 0, M, N, K, P(c), 0, N,
                                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        check(c, a, "e4m3", b, "e4m3", False, K)


# every kernel: few rows (8 to 64), 64 x 32, 128 x 128 and 256 x 128 tiles, and any alignment
@pytest.mark.parametrize("M,N", [(1, 64), (40, 64), (64, 300), (300, 256), (1200, 1200), (4200, 4100)])
@pytest.mark.parametrize("aligned", [True, False])
def test_fp32_sums_that_lose_the_most(mx, M, N, aligned):
    """one term of 448 * 448 = 200704, whose fp32 step is 2^-6, among terms just under half a step and just under a
    step of it (15/16 2^-7 and 15/16 2^-6), in its block and in 300 others, before and after it: every addition loses
    nearly as much as it can"""
    import torch
    print("case", M, N, aligned, flush=True)
    K = 128 * 301
    one = lambda n: torch.ones(301, n, device="cuda")
    code = lambda v: int(torch.tensor([v]).to(torch.float8_e4m3fn).view(torch.uint8).item())
    place = (lambda t: t) if aligned else (lambda t: inside(t, 1, 2, 0x7F))
    for where in (0, 64, 127, 128 * 150 + 3, K - 1):
        for small in (1.875 * 2.0 ** -4, 1.875 * 2.0 ** -3):   # times 2^-4
            for every in (1, 128):                             # every term, or one of each block
                for sign in (0, 0x80):
                    a = torch.zeros(1, K, dtype=torch.uint8, device="cuda")
                    b = torch.zeros(1, K, dtype=torch.uint8, device="cuda")
                    a[0, ::every], b[0, ::every] = code(small) | sign, code(2.0 ** -4)
                    a[0, where], b[0, where] = code(448.0), code(448.0)
                    va, vb = a.view(ref.F8["e4m3"]).double(), b.view(ref.F8["e4m3"]).double()
                    C, S = (va * vb).sum().item(), (va * vb).abs().sum().item()
                    c = mx.block_gemm(place(a.repeat(M, 1)), one(M), "e4m3", place(b.repeat(N, 1)), one(N), "e4m3",
                                      out_dtype=torch.float32)
                    off = (c.double() - C).abs().max().item()
                    assert off <= sums_bound(K) * S, (where, small, every, sign, off / S * 2 ** 24)
