"""Block-128 FP8 quantizers and product on the GPU, against plain definitions (block_reference).

Codes and scales have one right value each.  Products: float32 output within 1e-5 of the sum of
|terms| (the products are exact and an fp32 sum of n terms in any order is off by at most
n 2^-24 of it; block sums of 128 and up to a few hundred blocks stay far below).  bfloat16 output:
half a step of the result (2^-8 relative) and the matrix instruction's window, at most 31 products
of a step losing less than 2^-13 of the largest each: 31 / 2^13 < 2^-8 of the sum of |terms|."""
import pytest

import block_reference as ref

pytestmark = pytest.mark.gpu
MODES = ("row", "transpose", "tile", "tile_transpose")


@pytest.fixture(scope="module")
def mx():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_block_amax_amd as m
    m.lib()
    return m


def data(rows, cols, seed, spread=0):
    """bf16 normal values, columns and rows scaled by powers of two up to 2^+-spread"""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    if spread:
        x = x * torch.exp2(torch.randint(-spread, spread + 1, (rows, 1), device="cuda", generator=g).float())
        x = x * torch.exp2(torch.randint(-spread, spread + 1, (1, cols), device="cuda", generator=g).float())
    return x.bfloat16()


def same_operand(got, want, what=""):
    import torch
    c, s = got
    assert c.shape == want[0].shape and s.shape == want[1].shape, what
    bad = (s != want[1]) & ~(s.isnan() & want[1].isnan())
    assert not bad.any(), "%s: %d scales differ, first at %s" % (what, int(bad.sum()), bad.nonzero()[0].tolist())
    bad = c != want[0]
    assert not bad.any(), "%s: %d codes differ, first at %s" % (what, int(bad.sum()), bad.nonzero()[0].tolist())


SIZES = [(1, 1), (1, 128), (3, 130), (127, 129), (128, 128), (129, 8), (256, 384), (1000, 520), (7, 4097), (385, 1023)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize(mx, rows, cols, fmt):
    x = data(rows, cols, rows * 7 + cols, 6)
    for mode in MODES:
        same_operand(mx.block_quantize(x, fmt, mode), ref.quantize(x, fmt, mode), mode)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("fr,ft", [("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_quantize_dual(mx, rows, cols, fr, ft):
    x = data(rows, cols, rows * 5 + cols, 6)
    for tile, (a, b) in ((False, MODES[:2]), (True, MODES[2:])):
        got = mx.block_quantize_dual(x, fr, ft, tile=tile)
        same_operand(got[:2], ref.quantize(x, fr, a), a)
        same_operand(got[2:], ref.quantize(x, ft, b), b)


def test_quantize_edges(mx):
    """zeros, the smallest and largest values, ties, infinities and NaN, each with neighbours unharmed"""
    import torch
    x = data(260, 520, 1)
    x[0:128, 0:128] = 0
    x[0, 5] = -0.0
    x[130, 140] = float("inf")
    x[131, 300] = float("nan")
    x[5, 300] = -float("inf")
    x[200] = x[200] * 2.0 ** -126          # subnormal and nearly so: below the smallest amax
    x[201] = 2.0 ** -133
    x[202] = 3.38e38
    x[203, 0::2], x[203, 1::2] = 1.0, 448.0
    x[204] = torch.arange(520, device="cuda").bfloat16()   # ties of the 8-bit grid
    for fmt in ("e4m3", "e5m2"):
        for mode in MODES:
            same_operand(mx.block_quantize(x, fmt, mode), ref.quantize(x, fmt, mode), (fmt, mode))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_every_bf16(mx, fmt):
    """every finite bf16 beside block maxima across the whole range"""
    import torch
    v = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    v = v[: v.numel() // 127 * 127].view(-1, 127)
    for top in (2.0 ** -120, 3.0e-20, 1.0, 447.0, 6.1e4, 3.3e38):
        x = torch.cat([v, torch.full_like(v[:, :1], top)], 1)
        same_operand(mx.block_quantize(x, fmt), ref.quantize(x, fmt), top)


def test_quantize_strides_and_guards(mx):
    """strided and unaligned inputs; outputs in strided buffers whose other bytes stay as they were"""
    import torch
    big = data(301, 700, 3)
    for r0, c0, rows, cols, step in ((1, 1, 200, 333, 1), (0, 3, 129, 257, 2), (2, 8, 64, 640, 1)):
        x = big[r0:r0 + rows * step:step, c0:c0 + cols]
        rows = x.shape[0]
        for mode in MODES:
            want = ref.quantize(x, "e4m3", mode)
            same_operand(mx.block_quantize(x, "e4m3", mode), want, mode)
            n, k = want[0].shape
            for off in (0, 3):
                buf = torch.full((n + 2, k + 37), 0xA5, dtype=torch.uint8, device="cuda")
                sbuf = torch.full((want[1].shape[0] + 2, want[1].shape[1] + 5), 7.0, device="cuda")
                c, s = buf[1:1 + n, off:off + k], sbuf[1:1 + want[1].shape[0], off:off + want[1].shape[1]]
                same_operand(mx.block_quantize(x, "e4m3", mode, out=(c, s)), want, mode)
                buf2, sbuf2 = buf.clone(), sbuf.clone()
                buf2[1:1 + n, off:off + k] = 0xA5
                sbuf2[1:1 + want[1].shape[0], off:off + want[1].shape[1]] = 7.0
                assert (buf2 == 0xA5).all() and (sbuf2 == 7.0).all(), "bytes outside the outputs were written"


def test_quantize_empty(mx):
    import torch
    for rows, cols in ((0, 5), (5, 0), (0, 0)):
        x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        for mode in MODES:
            c, s = mx.block_quantize(x, "e4m3", mode)
            assert c.numel() == 0 and s.numel() == 0
        assert len(mx.block_quantize_dual(x, "e4m3", "e5m2")) == 4


def test_quantize_large_equals_its_parts(mx):
    """input above the size from which it is read past the cache: every form equals that of its parts"""
    import torch
    rows, cols = 8320, 8200
    x = data(rows, cols, 11, 3)
    parts = [x[:4096], x[4096:]]
    for fmt in ("e4m3", "e5m2"):
        for mode in MODES:
            c, s = mx.block_quantize(x, fmt, mode)
            got = [mx.block_quantize(p, fmt, mode) for p in parts]
            t = mode.endswith("transpose")
            assert torch.equal(c, torch.cat([g[0] for g in got], 1 if t else 0)), (fmt, mode)
            assert torch.equal(s, torch.cat([g[1] for g in got], 0 if t else 1)), (fmt, mode)
    same_operand((c[:256, :4096], s[:32, :2]), ref.quantize(x[:4096, :256], "e5m2", "tile_transpose"))


def test_quantize_beyond_31_bits(mx):
    """more than 2^31 elements: offsets of x and of both forms' codes need 64 bits"""
    import torch
    rows, cols = 70016, 32768
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 8752):
        x[r:r + 8752] = data(8752, cols, r)
    c, s, ct, st = mx.block_quantize_dual(x, "e4m3", "e5m2")
    for r0, r1 in ((0, 256), (65536, 65536 + 130), (rows - 100, rows)):
        same_operand((c[r0:r1], s[:, r0:r1]), ref.quantize(x[r0:r1], "e4m3"), r0)
    b0 = rows // 128 - 2    # whole row blocks near the end, and the last, short one
    for q0, q1 in ((0, 128), (cols - 130, cols)):
        want = ref.quantize(x[b0 * 128:, q0:q1].contiguous(), "e5m2", "transpose")
        same_operand((ct[q0:q1, b0 * 128:], st[b0:, q0:q1]), want, q0)


# ---------------------------------------------------------------------------

def operand(mx, n, k, fmt, tile, seed, spread=0):
    c, s = mx.block_quantize(data(n, k, seed, spread), fmt, "tile" if tile else "row")
    return c, s


def check_product(c, a, fa, b, fb, tile, bf16):
    import torch
    C, S = ref.gemm(a, fa, b, fb, tile)
    err = (c.double() - C).abs()
    tol = 1e-5 * S
    if bf16:
        tol = 2.0 ** -8 * C.abs() + 2.0 ** -8 * S + 2.0 ** -134
    bad = ~(err <= tol)
    assert not bad.any(), "%d of %d off, first at %s: %r, %r, S %r" % (
        int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), c[bad][0].item(), C[bad][0].item(), S[bad][0].item())
    if C.numel() > 1000 and bf16:
        # over many elements: rounding to bf16 is uniform within half a step, at most 2^-8 / sqrt(3) in the
        # 2-norm; the window's errors are a few 2^-13 of terms that do not all point the same way: 2^-11
        assert err.norm() <= (2.0 ** -8 / 3 ** 0.5 + 2.0 ** -11) * C.norm(), (err.norm() / C.norm()).item()


GEMM_SIZES = [(1, 1, 1), (1, 128, 128), (1, 300, 4001), (70, 1, 1001), (300, 1, 250), (1, 6144, 512), (2, 300, 64), (5, 77, 333), (16, 256, 1024), (17, 130, 4097), (31, 515, 640),
              (33, 96, 128), (48, 512, 2048), (64, 640, 1152), (65, 128, 260), (100, 1000, 144), (128, 128, 128), (129, 257, 384),
              (256, 512, 512), (300, 301, 302), (333, 640, 1000), (512, 768, 1280), (513, 1025, 272), (1024, 512, 896)]


@pytest.mark.parametrize("M,N,K", GEMM_SIZES)
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
def test_gemm(mx, M, N, K, tile, bf16):
    import torch
    print("case", M, N, K, tile, bf16, flush=True)
    for fa, fb in (("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")):
        a, b = operand(mx, M, K, fa, False, M + K, 3), operand(mx, N, K, fb, tile, N + K + 1, 3)
        c = mx.block_gemm(*a, fa, *b, fb, out_dtype=torch.bfloat16 if bf16 else torch.float32)
        check_product(c, a, fa, b, fb, tile, bf16)


# sizes beyond the small tiles: 128 x 128 (whole and ragged K, long rows), 256 x 256 and 256 x 128 tiles, odd edges
LARGE = [(1100, 1100, 384), (1111, 1301, 4001), (1100, 1100, 130), (2048, 2048, 12352), (2051, 2177, 12304), (4096, 4096, 272),
         (4100, 4250, 400), (4096, 2048, 144), (2300, 4100, 1000), (8200, 4099, 16)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
def test_gemm_large(mx, M, N, K, tile, bf16):
    import torch
    print("case", M, N, K, tile, bf16, flush=True)
    for fa, fb in (("e4m3", "e4m3"), ("e5m2", "e4m3")):
        a, b = operand(mx, M, K, fa, False, M + K, 3), operand(mx, N, K, fb, tile, N + K + 1, 3)
        c = mx.block_gemm(*a, fa, *b, fb, out_dtype=torch.bfloat16 if bf16 else torch.float32)
        check_product(c, a, fa, b, fb, tile, bf16)


# K ends inside 16 bytes: every tile size, a reduction of less than 16, whole blocks and one element, long rows
RAGGED_K = [(40, 300, 257), (100, 300, 15), (1100, 1100, 1), (1100, 1100, 15), (1100, 1100, 17), (1111, 1301, 129), (1100, 1100, 255),
            (2048, 2048, 12353), (4096, 2048, 135), (4100, 4250, 401), (4096, 4096, 1037), (8200, 4099, 31)]


@pytest.mark.parametrize("M,N,K", RAGGED_K)
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
def test_gemm_ragged_k(mx, M, N, K, tile, bf16):
    """rows of whole 16 bytes whose bytes past K are NaN codes, as those around the operands are"""
    import torch
    print("case", M, N, K, tile, bf16, flush=True)

    def inside(t):
        buf = torch.full((t.shape[0] + 2, (K + 15) // 16 * 16 + 32), 0x7F, dtype=torch.uint8, device="cuda")
        v = buf[1:1 + t.shape[0], 16:16 + K]
        v.copy_(t)
        return v

    for fa, fb in (("e4m3", "e4m3"), ("e5m2", "e4m3")):
        a, b = operand(mx, M, K, fa, False, M + K, 3), operand(mx, N, K, fb, tile, N + K + 1, 3)
        c = mx.block_gemm(inside(a[0]), a[1], fa, inside(b[0]), b[1], fb, out_dtype=torch.bfloat16 if bf16 else torch.float32)
        check_product(c, a, fa, b, fb, tile, bf16)


@pytest.mark.parametrize("M,N,K", [(1, 200, 256), (40, 200, 300), (300, 520, 640), (520, 300, 272), (1200, 1160, 272), (1201, 1160, 301),
                                   (4200, 4100, 272)])
@pytest.mark.parametrize("bf16", [True, False])
def test_gemm_strides_and_guards(mx, M, N, K, bf16):
    """operands inside larger buffers whose other bytes are NaN codes and NaN scales, unaligned too; C inside a larger
    buffer whose other elements stay as they were"""
    import torch
    dt = torch.bfloat16 if bf16 else torch.float32
    a, b = operand(mx, M, K, "e4m3", False, 1), operand(mx, N, K, "e4m3", False, 2)
    for off, pad in ((0, 16), (16, 32), (5, 11), (1, 0)):
        def inside(t, fill, dtype):
            buf = torch.full((t.shape[0] + 2, off + t.shape[1] + pad + 16), fill, dtype=dtype, device="cuda")
            v = buf[1:1 + t.shape[0], off:off + t.shape[1]]
            v.copy_(t)
            return v
        ap, bp = inside(a[0], 0x7F, torch.uint8), inside(b[0], 0x7F, torch.uint8)
        asp, bsp = inside(a[1], float("nan"), torch.float32), inside(b[1], float("nan"), torch.float32)
        buf = torch.full((M + 2, N + 40), 3.0, dtype=dt, device="cuda")
        c = buf[1:1 + M, off:off + N]
        mx.block_gemm(ap, asp, "e4m3", bp, bsp, "e4m3", out_dtype=dt, out=c)
        check_product(c, a, "e4m3", b, "e4m3", False, bf16)
        buf[1:1 + M, off:off + N] = 3.0
        assert (buf == 3.0).all(), "elements outside C were written"


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_empty_k_and_sizes(mx, M):
    import torch
    for dt in (torch.float32, torch.bfloat16):
        z = lambda n: (torch.empty(n, 0, dtype=torch.uint8, device="cuda"), torch.empty(0, n, device="cuda"))
        out = torch.full((M, 70), 5.0, dtype=dt, device="cuda")
        assert (mx.block_gemm(*z(M), "e4m3", *z(70), "e4m3", out_dtype=dt, out=out) == 0).all()
    a, b = operand(mx, M, 64, "e4m3", False, 1), operand(mx, 0, 64, "e4m3", False, 2)
    assert mx.block_gemm(*a, "e4m3", *b, "e4m3").shape == (M, 0)
    assert mx.block_gemm(*b, "e4m3", *a, "e4m3").shape == (0, M)


@pytest.mark.parametrize("M,N", [(1, 300), (24, 300), (60, 300), (200, 300), (600, 300), (1200, 1200), (4200, 4100)])
@pytest.mark.parametrize("bf16", [True, False])
def test_gemm_nan_scales(mx, M, N, bf16):
    """a NaN scale of A's row m makes row m NaN, one of B's row n column n, and nothing else"""
    import torch
    dt = torch.bfloat16 if bf16 else torch.float32
    K = 640
    x, w = data(M, K, 5), data(N, K, 6)
    x[M - 1, 200] = float("inf")
    w[37, 5] = float("nan")
    a, b = mx.block_quantize(x, "e4m3"), mx.block_quantize(w, "e4m3")
    c = mx.block_gemm(*a, "e4m3", *b, "e4m3", out_dtype=dt)
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[M - 1] = True
    want[:, 37] = True
    assert torch.equal(c.isnan(), want)
    bt = mx.block_quantize(w, "e4m3", "tile")
    c = mx.block_gemm(*a, "e4m3", *bt, "e4m3", out_dtype=dt)
    want[:, 0:128] = True
    assert torch.equal(c.isnan(), want)
    # every row and column in turn at the edges of the kernels' tiles, in the first and in the last block
    for m in {0, 4, 31, 63, 130, 140} & set(range(M)):
        for blk in (0, 4):
            a, b = mx.block_quantize(data(M, K, 5), "e4m3"), mx.block_quantize(data(N, K, 6), "e4m3")
            a[1][blk, m], b[1][blk, 299 - m] = float("nan"), float("inf")
            c = mx.block_gemm(*a, "e4m3", *b, "e4m3", out_dtype=dt)
            assert c[m].isnan().all() and not c[:, 299 - m].isfinite().any()
            rest = torch.ones(M, N, dtype=torch.bool, device="cuda")
            rest[m], rest[:, 299 - m] = False, False
            assert c[rest].isfinite().all()


@pytest.mark.parametrize("M,N", [(1, 300), (40, 300), (300, 300), (1200, 1200), (4200, 4100)])
@pytest.mark.parametrize("bf16", [True, False])
def test_gemm_special_codes(mx, M, N, bf16):
    """NaN codes, and E5M2's infinities, make the elements that they enter NaN and Inf, and no others"""
    import torch
    dt = torch.bfloat16 if bf16 else torch.float32
    K = 400
    a, b = operand(mx, M, K, "e5m2", False, 1), operand(mx, N, K, "e4m3", True, 2)
    b[0][:, 7] = 0x38                                    # 1
    a[0][M - 1, 399], a[0][0, 7] = 0x7F, 0x7C           # NaN, Inf
    b[0][5, 130] = 0xFF                                  # NaN
    c = mx.block_gemm(*a, "e5m2", *b, "e4m3", out_dtype=dt)
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[M - 1], want[:, 5] = True, True
    assert torch.equal(c.isnan(), want)
    inf = torch.zeros_like(want)
    inf[0] = True
    assert torch.equal(c == float("inf"), inf & ~want)


@pytest.mark.parametrize("M,N", [(1, 64), (40, 64), (300, 256), (1200, 1200), (4200, 4100)])
def test_gemm_small_terms_kept_in_fp32(mx, M, N):
    """float32 output: 1 + 2^-18 in one block, the small term 2^-9 * 2^-9, is exact.  Beside a large pair that cancels,
    fp32 holds the small terms to a step of the running sum only: the terms 448 * 448 = 200704 and their negative add
    up to 2^18.6, half a step of fp32 there is 2^-7, and each of the two additions that meet it may lose as much"""
    import torch
    a = torch.zeros(M, 256, dtype=torch.uint8, device="cuda")
    b = torch.zeros(N, 256, dtype=torch.uint8, device="cuda")
    one, tiny, big = 0x38, 0x01, 0x7E                    # 1, 2^-9, 448
    a[:, 3], b[:, 3] = one, one
    a[:, 17], b[:, 17] = tiny, tiny
    s = torch.ones(2, M, device="cuda"), torch.ones(2, N, device="cuda")
    c = mx.block_gemm(a, s[0], "e4m3", b, s[1], "e4m3", out_dtype=torch.float32)
    assert (c == 1 + 2.0 ** -18).all()
    a[:, 40], b[:, 40] = big, big
    a[:, 41], b[:, 41] = big, big | 0x80
    c = mx.block_gemm(a, s[0], "e4m3", b, s[1], "e4m3", out_dtype=torch.float32)
    assert ((c - (1 + 2.0 ** -18)).abs() <= 2 * 2.0 ** -7).all()


@pytest.mark.parametrize("M", [1, 40, 300, 1200, 4200])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_gemm_smallest_and_largest_codes(mx, M, fa, fb):
    """subnormal codes are numbers: their products, all multiples of one power of two and their sums below 2^24 of it,
    are exact in float32; so are the largest codes' (128 of one product per block, an integer of 24 bits times a power of two)"""
    import torch
    N, K = 300 if M < 1000 else 1160 if M < 4000 else 4096, 256
    g = torch.Generator(device="cuda").manual_seed(7)
    top = {"e4m3": 8, "e5m2": 4}
    rnd = lambda n, f: (torch.randint(0, top[f], (n, K), device="cuda", generator=g) +
                        128 * torch.randint(0, 2, (n, K), device="cuda", generator=g)).to(torch.uint8)
    one = lambda n: torch.ones(2, n, device="cuda")
    a, b = rnd(M, fa), rnd(N, fb)
    c = mx.block_gemm(a, one(M), fa, b, one(N), fb, out_dtype=torch.float32)
    want = a.view(ref.F8[fa]).double() @ b.view(ref.F8[fb]).double().t().contiguous()
    assert torch.equal(c.double(), want) and bool((want != 0).any())
    big = {"e4m3": 0x7E, "e5m2": 0x7B}
    a, b = torch.full_like(a, big[fa]), torch.full_like(b, big[fb])
    c = mx.block_gemm(a, one(M), fa, b, one(N), fb, out_dtype=torch.float32)
    assert (c.double() == 256 * ref.FMAX[fa] * ref.FMAX[fb]).all()


@pytest.mark.parametrize("bf16", [True, False])
def test_gemm_beyond_31_bits(mx, bf16):
    """C and B of more than 2^31 elements"""
    import torch
    dt = torch.bfloat16 if bf16 else torch.float32
    M, N, K = 66048, 36864, 64
    a, b = operand(mx, M, K, "e4m3", False, 1), operand(mx, N, K, "e4m3", True, 2)
    c = mx.block_gemm(*a, "e4m3", *b, "e4m3", out_dtype=dt)
    for r0, r1 in ((0, 64), (58300, 58364), (M - 64, M)):
        check_product(c[r0:r1], (a[0][r0:r1], a[1][:, r0:r1]), "e4m3", b, "e4m3", True, bf16)
    del c
    N, K = 70000, 32768
    b = (torch.randint(0, 0x78, (N, K), dtype=torch.uint8, device="cuda"), torch.rand(K // 128, N, device="cuda"))
    for M in (2, 160):
        a = operand(mx, M, K, "e4m3", False, 3)
        c = mx.block_gemm(*a, "e4m3", *b, "e4m3", out_dtype=dt)
        for n0, n1 in ((0, 32), (65530, 65562), (N - 32, N)):
            check_product(c[:, n0:n1], a, "e4m3", (b[0][n0:n1], b[1][:, n0:n1]), "e4m3", False, bf16)


def test_gemm_repeats_bits_on_streams_and_in_graphs(mx):
    """the same inputs give the same bits: on another stream, beside another call, and replayed from a graph between
    eager calls"""
    import torch
    for M, N, K, dt, tile in ((1, 1024, 2048, torch.bfloat16, True), (40, 512, 4096, torch.float32, False),
                              (300, 512, 1024, torch.bfloat16, True), (1300, 1200, 1024, torch.float32, False),
                              (1300, 1200, 1001, torch.bfloat16, True), (4200, 4200, 640, torch.bfloat16, True),
                              (4200, 4200, 640, torch.float32, False)):
        a, b = operand(mx, M, K, "e4m3", False, 1), operand(mx, N, K, "e4m3", tile, 2)
        a2 = operand(mx, M, K, "e4m3", False, 9)
        want, want2 = (mx.block_gemm(*t, "e4m3", *b, "e4m3", out_dtype=dt) for t in (a, a2))
        check_product(want, a, "e4m3", b, "e4m3", tile, dt == torch.bfloat16)
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        c1 = mx.block_gemm(*a, "e4m3", *b, "e4m3", out_dtype=dt, stream=s1)
        c2 = mx.block_gemm(*a2, "e4m3", *b, "e4m3", out_dtype=dt, stream=s2.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(c1, want) and torch.equal(c2, want2)
        x = data(M, K, 1)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q = mx.block_quantize(x, "e4m3")
            c = mx.block_gemm(*q, "e4m3", *b, "e4m3", out_dtype=dt)
        for i in range(3):
            c.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(c, want)
            assert torch.equal(mx.block_gemm(*a2, "e4m3", *b, "e4m3", out_dtype=dt), want2)


def test_gemm_refuses(mx):
    import torch
    a, b = operand(mx, 8, 256, "e4m3", False, 1), operand(mx, 300, 256, "e4m3", False, 2)
    ok = lambda **k: mx.block_gemm(k.get("a", a[0]), k.get("as_", a[1]), k.get("fa", "e4m3"), k.get("b", b[0]),
                                   k.get("bs", b[1]), "e4m3", out_dtype=k.get("dt", torch.bfloat16), out=k.get("out"))
    ok()
    for bad in (dict(fa="e2m1"), dict(as_=a[1].t()), dict(as_=a[1][:1]), dict(bs=b[1][:, :299]), dict(bs=b[1].double()),
                dict(b=b[0][:, :128]), dict(a=a[0].to(torch.int8)), dict(dt=torch.float16), dict(a=a[0][0]),
                dict(out=torch.empty(8, 300, device="cuda")), dict(a=a[0].cpu()), dict(as_=a[1].cpu()),
                dict(out=torch.empty(300, 8, dtype=torch.bfloat16, device="cuda").t()), dict(a=a[0].t().contiguous().t())):
        with pytest.raises(ValueError):
            ok(**bad)
    shared = torch.zeros(8, 300, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mx.MXError):   # C over A's codes
        ok(a=shared.view(torch.uint8)[:, :256], out=shared)
    with pytest.raises(mx.MXError):   # rows of C on top of each other
        ok(out=shared[:1].expand(8, 300))
    with pytest.raises(ValueError):
        mx.block_quantize(data(4, 4, 1), "e2m1")
    with pytest.raises(ValueError):
        mx.block_quantize(data(4, 4, 1), "e4m3", "column")
    with pytest.raises(ValueError):
        mx.block_quantize(data(4, 4, 1).t(), "e4m3")
