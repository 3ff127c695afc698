"""Block-128 operators by group on the GPU, against plain definitions (group_reference), one group at a time.

Codes and scales have one right value each.  Products as those of block_gemm: fp32 sums within (130 + blocks of K) 2^-24
of the sum of |terms|, FP8 sums (bf16 output) within 31 2^-13 < 2^-8 of it, a bf16 output off by half a step more."""
import pytest

import block_reference as ref
import group_reference as grp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_block_amax_amd as m
    m.lib()
    return m


def data(*shape, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).bfloat16()


def ends_of(sizes):
    import torch
    return torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32)


def check(c, C, S, nk, full):
    tol = S * ((130 + nk) * 2.0 ** -24 if full else 2.0 ** -8 + nk * 2.0 ** -24)
    if c.element_size() == 2:
        tol = tol + 2.0 ** -8 * (C.abs() + tol)
    err = (c.double() - C).abs()
    assert (err <= tol).all(), "off by %g of the tolerance" % (err / tol).max().item()


def weights(mx, groups, n, k, fmt, tile, seed):
    import torch
    w = data(groups, n, k, seed=seed)
    q = [mx.block_quantize(x, fmt, "tile" if tile else "row") for x in w.unbind()]
    codes = torch.zeros(groups, n, ref.cdiv(k, 16) * 16, dtype=torch.uint8, device="cuda")[:, :, :k]
    for i, (c, _) in enumerate(q):
        codes[i] = c
    return codes, torch.stack([s for _, s in q])


# sizes of the groups, rows behind the last one
GROUPS = [([1], 0), ([0], 3), ([300], 0), ([0, 5, 0, 130, 1, 0, 300], 7), ([128, 128, 256], 0), ([1] * 200, 0),
          ([0] * 70 + [9, 20] + [0] * 60 + [31, 2], 5), ([40] * 30, 1), ([17, 0, 63, 64, 65, 127, 129], 0), ([700, 3, 600, 900], 0),
          ([0, 0, 0], 4)]


@pytest.mark.parametrize("sizes,behind", GROUPS, ids=str)
@pytest.mark.parametrize("cols", [1, 128, 200, 520])
def test_quantize(mx, sizes, behind, cols):
    import torch
    rows, ends = sum(sizes) + behind, ends_of(sizes)
    x = data(rows, cols, seed=rows + cols)
    if rows > 4:
        x[rows // 2, cols // 2] = float("inf")
        x[3] = 0
    k = grp.bound(rows, len(sizes))
    assert mx.block_grouped_cols(rows, len(sizes)) == k
    for fr, ft in (("e4m3", "e5m2"), ("e5m2", "e5m2"), ("e4m3", "e4m3")):
        buf = torch.full((cols + 1, k + 7), 0xA5, dtype=torch.uint8, device="cuda")
        sbuf = torch.full((k // 128 + 1, cols + 3), 7.0, device="cuda")
        out = (buf[:cols, 3:3 + k], sbuf[:k // 128, 1:1 + cols])
        want = grp.quantize(x, ends.tolist(), ft, 0xA5, 7.0)
        same = lambda got: torch.equal(got[0], want[0]) and torch.equal(got[1].nan_to_num(-1), want[1].nan_to_num(-1))
        mx.block_quantize_grouped(x, ends, ft, out=out)
        assert same(out)
        out[0].fill_(0xA5)
        out[1].fill_(7.0)
        assert (buf == 0xA5).all() and (sbuf == 7).all(), "bytes outside the output were written"
        rc = torch.full((rows, cols), 0x11, dtype=torch.uint8, device="cuda")
        rs = torch.full((ref.cdiv(cols, 128), rows), 3.0, device="cuda")
        mx.block_quantize_grouped_dual(x, ends, fr, ft, out=(rc, rs) + out)
        assert same(out)
        live = rows - behind
        if live:
            wc, ws = ref.quantize(x[:live], fr)
            assert torch.equal(rc[:live], wc) and torch.equal(rs[:, :live].nan_to_num(-1), ws.nan_to_num(-1))
        assert (rc[live:] == 0x11).all() and (rs[:, live:] == 3).all()


@pytest.mark.parametrize("rows,cols", [(16500, 4096), (500, 200), (500, 208), (500, 203)])
def test_quantize_formats(mx, rows, cols):
    """every pair of formats, and more than 2^26 elements, against each group quantized by itself"""
    import torch
    ends = ends_of([rows // 3, 0, 129, rows // 2])                        # of 500 rows the last end is cut
    live = min(int(ends[-1]), rows)
    x = data(rows, cols, seed=45)
    pieces = list(zip(grp.ranges(ends.tolist(), rows), grp.blocks(ends.tolist(), rows)))
    for fr in ("e4m3", "e5m2"):
        for ft in ("e4m3", "e5m2"):
            rc, rs, tc, ts = mx.block_quantize_grouped_dual(x, ends, fr, ft)
            wc, ws = mx.block_quantize(x[:live], fr)
            assert torch.equal(rc[:live], wc) and torch.equal(rs[:, :live], ws)
            oc, os = mx.block_quantize_grouped(x, ends, ft)
            for (lo, hi), (b0, b1) in pieces:
                if hi == lo:
                    continue
                wc, ws = mx.block_quantize(x[lo:hi], ft, "transpose")
                for codes, scales in ((tc, ts), (oc, os)):
                    assert torch.equal(codes[:, 128 * b0:128 * b0 + hi - lo], wc) and torch.equal(scales[b0:b1], ws)
                    assert (codes[:, 128 * b0 + hi - lo:128 * b1] == 0).all()


# N, K: whole tiles and not, K in whole blocks, chunks of 16 bytes and neither
SIZES = [(256, 256), (130, 400), (300, 129), (16, 1), (515, 640), (128, 15), (1, 48)]


@pytest.mark.parametrize("sizes,behind", GROUPS, ids=str)
@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("tile", [True, False])
def test_rows(mx, sizes, behind, N, K, tile):
    import torch
    print("case", sizes, behind, N, K, tile, flush=True)
    rows, groups, ends = sum(sizes) + behind, len(sizes), ends_of(sizes)
    fa, fb = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")][(N + groups) % 4]
    a = mx.block_quantize(data(rows, K, seed=1), fa)
    b = weights(mx, groups, N, K, fb, tile, 2)
    live = rows - behind
    C, S = grp.gemm(a, fa, b, fb, ends.tolist(), tile and ref.cdiv(N, 128) != N)
    nk = ref.cdiv(K, 128)
    for dtype, full in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
        buf = torch.full((rows + 1, N + 5), 9.0, dtype=dtype, device="cuda")
        c = buf[:rows, 2:2 + N]
        mx.block_gemm_grouped(*a, fa, *b, fb, ends, out_dtype=dtype, out=c, full_sums=full)
        check(c[:live], C[:live], S[:live], nk, full)
        assert (c[live:] == 9).all(), "rows behind the last group were written"
        c.fill_(9.0)
        assert (buf == 9).all(), "elements outside C were written"


# mean rows of a group on either side of every rule, tiles of 8 to 256 rows, N beyond one tile of any kernel
@pytest.mark.parametrize("mean", [3, 8, 9, 16, 17, 32, 33, 60, 120, 250, 511, 520, 1100])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_rows_of_every_kernel(mx, mean, fa, fb):
    import torch
    sizes = [mean, 2 * mean + 1, 0, mean // 2, mean + mean // 2 - 1]   # 5 groups, 5 * mean rows
    ends = ends_of(sizes)
    rows = sum(sizes)
    for N, K, tile in ((640, 1152, True), (300, 1040, True), (272, 777, False), (272, 512, False), (520, 1000, True)):
        print("case", mean, fa, fb, N, K, tile, flush=True)
        a = mx.block_quantize(data(rows, K, seed=3), fa)
        b = weights(mx, 5, N, K, fb, tile, 4)
        C, S = grp.gemm(a, fa, b, fb, ends.tolist(), tile)
        for dtype, full in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
            check(mx.block_gemm_grouped(*a, fa, *b, fb, ends, out_dtype=dtype, full_sums=full), C, S, ref.cdiv(K, 128), full)


# groups, rows, N, K where 128 x 128 tiles in two groups of waves are taken (with fp32 sums, with FP8 sums), 128 x 128,
# and 256 x 256 (FP8 sums, B in tiles)
@pytest.mark.parametrize("groups,rows,N,K", [(16, 80, 2048, 512), (16, 79, 2040, 505), (16, 80, 2048, 1536), (16, 79, 2040, 1531),
                                             (5, 300, 4096, 1152), (5, 299, 4090, 1147),
                                             (16, 2600, 2048, 512), (16, 2599, 2044, 505)])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_rows_of_large_tiles(mx, groups, rows, N, K, fa, fb):
    import torch
    print("case", groups, rows, N, K, fa, fb, flush=True)
    share = [i % 5 for i in range(groups)]                                # none, or one to four parts
    sizes = [rows * w // sum(share) for w in share]
    sizes[-1] += rows - sum(sizes)
    ends = ends_of(sizes)
    a = mx.block_quantize(data(rows, K, seed=41), fa)
    for tile in (True, False):
        b = weights(mx, groups, N, K, fb, tile, 42)
        C, S = grp.gemm(a, fa, b, fb, ends.tolist(), tile)
        for dtype, full in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
            check(mx.block_gemm_grouped(*a, fa, *b, fb, ends, out_dtype=dtype, full_sums=full), C, S, ref.cdiv(K, 128), full)


def test_rows_are_the_single_products(mx):
    """every group's rows, bit for bit, where the single product takes a kernel of the same order of sums"""
    import torch
    sizes = [300, 0, 512, 200]
    ends = ends_of(sizes)
    a, b = mx.block_quantize(data(1012, 640, seed=5), "e4m3"), weights(mx, 4, 384, 640, "e4m3", True, 6)
    for full, dtype in ((True, torch.float32),):
        c = mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends, out_dtype=dtype, full_sums=full)
        C, S = grp.gemm(a, "e4m3", b, "e4m3", ends.tolist(), True)
        at = 0
        for i, n in enumerate(sizes):
            if n:
                one = mx.block_gemm(a[0][at:at + n], a[1][:, at:at + n], "e4m3", b[0][i], b[1][i], "e4m3", out_dtype=dtype)
                assert ((one - c[at:at + n]).abs().double() <= 2 * 135 * 2.0 ** -24 * S[at:at + n]).all()
            at += n


def test_weights_quantized_as_one_matrix(mx):
    """both forms of the stacked weights, viewed as B for the product and for its gradient"""
    import torch
    E, N, K = 6, 256, 384
    sizes = [10, 0, 200, 1, 128, 61]
    ends, w = ends_of(sizes), data(6, 256, 384, seed=7)
    cr, sr, ct, st = mx.block_quantize_dual(w.view(E * N, K), "e4m3", "e4m3", tile=True)
    b = (cr.view(E, N, K), sr.view(K // 128, E, N // 128).transpose(0, 1))
    bt = (ct.view(K, E, N).transpose(0, 1), st.view(E, N // 128, K // 128))
    a, d = mx.block_quantize(data(400, K, seed=8), "e4m3"), mx.block_quantize(data(400, N, seed=9), "e5m2")
    for x, fx, y, n, k in ((a, "e4m3", b, N, K), (d, "e5m2", bt, K, N)):
        C, S = grp.gemm(x, fx, y, "e4m3", ends.tolist(), True)
        check(mx.block_gemm_grouped(*x, fx, *y, "e4m3", ends), C, S, k // 128, False)


@pytest.mark.parametrize("K", [256, 200])
def test_unaligned_rows(mx, K):
    """the general kernel: rows that do not start at multiples of 16 bytes, either operand"""
    import torch
    sizes = [0, 5, 130, 1, 300]
    ends = ends_of(sizes)
    a, b = mx.block_quantize(data(436, K, seed=10), "e4m3"), weights(mx, 5, 200, K, "e4m3", True, 11)
    au = torch.full((436, K + 3), 0x7F, dtype=torch.uint8, device="cuda")
    au[:, 1:1 + K] = a[0]
    bu = torch.full((5, 200, K + 16), 0x7F, dtype=torch.uint8, device="cuda")[:, :, 5:5 + K]
    bu.copy_(b[0])
    C, S = grp.gemm(a, "e4m3", b, "e4m3", ends.tolist(), True)
    for x, y in (((au[:, 1:1 + K], a[1]), b), (a, (bu, b[1])), ((au[:, 1:1 + K], a[1]), (bu, b[1]))):
        for dtype, full in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
            c = torch.full((436, 200), 9.0, dtype=dtype, device="cuda")
            mx.block_gemm_grouped(*x, "e4m3", *y, "e4m3", ends, out_dtype=dtype, out=c, full_sums=full)
            check(c, C, S, ref.cdiv(K, 128), full)


def test_no_columns(mx):
    """K = 0 clears the groups' rows and no other"""
    import torch
    a = (torch.empty(20, 0, dtype=torch.uint8, device="cuda"), torch.empty(0, 20, device="cuda"))
    b = (torch.empty(3, 50, 0, dtype=torch.uint8, device="cuda"), torch.empty(3, 0, 1, device="cuda"))
    for dtype in (torch.bfloat16, torch.float32):
        c = torch.full((20, 50), 9.0, dtype=dtype, device="cuda")
        mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends_of([4, 0, 9]), out_dtype=dtype, out=c)
        assert (c[:13] == 0).all() and (c[13:] == 9).all()


@pytest.mark.parametrize("sizes,behind", GROUPS, ids=str)
@pytest.mark.parametrize("M,N", [(256, 256), (130, 300), (64, 515), (1, 7), (300, 128)])
def test_cols(mx, sizes, behind, M, N):
    import torch
    print("case", sizes, behind, M, N, flush=True)
    rows, groups, ends = sum(sizes) + behind, len(sizes), ends_of(sizes)
    fa, fb = [("e5m2", "e4m3"), ("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")][(N + groups) % 4]
    a = mx.block_quantize_grouped(data(rows, M, seed=12), ends, fa)
    b = mx.block_quantize_grouped(data(rows, N, seed=13), ends, fb)
    C, S = grp.gemm_k(a, fa, b, fb, ends.tolist())
    nk = max(ref.cdiv(s, 128) for s in sizes)
    for dtype, full in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
        buf = torch.full((groups, M + 1, N + 5), 9.0, dtype=dtype, device="cuda")
        c = buf[:, :M, 2:2 + N]
        mx.block_gemm_grouped_k(*a, fa, *b, fb, ends, out_dtype=dtype, out=c, full_sums=full)
        check(c, C, S, nk, full)
        c.fill_(9.0)
        assert (buf == 9).all(), "elements outside C were written"


@pytest.mark.parametrize("M,N", [(4100, 2304), (1300, 1030), (520, 4100)])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_cols_of_every_kernel(mx, M, N, fa, fb):
    import torch
    for sizes in ([1000, 3, 0, 600], [70, 0, 130, 1, 128, 40]):
        rows, ends = sum(sizes), ends_of(sizes)
        a = mx.block_quantize_grouped(data(rows, M, seed=14), ends, fa)
        b = mx.block_quantize_grouped(data(rows, N, seed=15), ends, fb)
        C, S = grp.gemm_k(a, fa, b, fb, ends.tolist())
        for dtype, full in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
            check(mx.block_gemm_grouped_k(*a, fa, *b, fb, ends, out_dtype=dtype, full_sums=full), C, S, 8, full)


@pytest.mark.parametrize("groups", [1, 3])
@pytest.mark.parametrize("M,N", [(384, 80), (65, 33), (1, 500), (700, 900), (1100, 600)])
def test_long_columns_of_few_tiles(mx, groups, M, N):
    """waves that share the blocks of K: whole eighths and not, a group without rows among them"""
    import torch
    for rows in (700, 3000, 5000):
        sizes = [rows] if groups == 1 else [rows * 2, 0, rows]
        ends = ends_of(sizes)
        a = mx.block_quantize_grouped(data(sum(sizes), M, seed=31), ends, "e5m2")
        b = mx.block_quantize_grouped(data(sum(sizes), N, seed=32), ends, "e4m3")
        C, S = grp.gemm_k(a, "e5m2", b, "e4m3", ends.tolist())
        for dtype, full in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
            check(mx.block_gemm_grouped_k(*a, "e5m2", *b, "e4m3", ends, out_dtype=dtype, full_sums=full), C, S,
                  ref.cdiv(max(sizes), 128), full)


# few tiles: the blocks of K shared by eight waves, by two groups of waves; one row of tiles
@pytest.mark.parametrize("sizes", [[1500], [700, 0, 1300], [0, 900, 129, 600]], ids=str)
@pytest.mark.parametrize("M,N", [(130, 70), (1050, 1100), (64, 33)])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_columns_shared(mx, sizes, M, N, fa, fb):
    import torch
    rows, ends = sum(sizes), ends_of(sizes)
    a = mx.block_quantize_grouped(data(rows, M, seed=43), ends, fa)
    b = mx.block_quantize_grouped(data(rows, N, seed=44), ends, fb)
    C, S = grp.gemm_k(a, fa, b, fb, ends.tolist())
    buf = torch.full((M, a[0].shape[1] + 3), 0x7F, dtype=torch.uint8, device="cuda")
    odd = buf[:, 1:1 + a[0].shape[1]]                                     # rows of no alignment: the general kernel
    odd.copy_(a[0])
    for dtype, full in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
        for codes in (a[0], odd):
            check(mx.block_gemm_grouped_k(codes, a[1], fa, *b, fb, ends, out_dtype=dtype, full_sums=full), C, S, 12, full)


def test_unaligned_columns(mx):
    import torch
    sizes = [5, 0, 300, 130]
    ends = ends_of(sizes)
    a, b = (mx.block_quantize_grouped(data(435, n, seed=n), ends, "e4m3") for n in (200, 136))
    C, S = grp.gemm_k(a, "e4m3", b, "e4m3", ends.tolist())
    buf = torch.full((200, a[0].shape[1] + 3), 0x7F, dtype=torch.uint8, device="cuda")
    u = buf[:, 1:1 + a[0].shape[1]]
    u.copy_(a[0])
    for dtype, full in ((torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, True)):
        check(mx.block_gemm_grouped_k(u, a[1], "e4m3", *b, "e4m3", ends, out_dtype=dtype, full_sums=full), C, S, 3, full)


def test_ends_that_are_no_ranges(mx):
    """decreasing ends and ends past the rows are taken as the nearest ones that are ranges; nothing else is touched"""
    import torch
    ends = torch.tensor([5, 3, 900, -1, 60], dtype=torch.int32, device="cuda")
    x = data(100, 256, seed=16)
    want = grp.quantize(x, ends.tolist(), "e4m3", 1, 2.0)
    k = grp.bound(100, 5)
    out = (torch.full((256, k), 1, dtype=torch.uint8, device="cuda"), torch.full((k // 128, 256), 2.0, device="cuda"))
    mx.block_quantize_grouped(x, ends, "e4m3", out=out)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    a, b = mx.block_quantize(x, "e4m3"), weights(mx, 5, 130, 256, "e4m3", True, 17)
    C, S = grp.gemm(a, "e4m3", b, "e4m3", ends.tolist(), True)
    check(mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends), C, S, 2, False)
    ones = (torch.full((150, 384), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(3, 150, device="cuda"))
    for e in ([200, 100, 2000], [500, 600, 700], [-5, -1, 130]):
        t = torch.tensor(e, dtype=torch.int32, device="cuda")
        C, S = grp.gemm_k(ones, "e4m3", ones, "e4m3", e)
        check(mx.block_gemm_grouped_k(*ones, "e4m3", *ones, "e4m3", t), C, S, 3, True)


@pytest.mark.parametrize("groups", [64, 65, 255, 256, 257, 511, 700, 1025])
def test_many_groups(mx, groups):
    """as many groups as one read of the ends holds, and more: rows at either side of its border and behind it"""
    import torch
    g = torch.Generator().manual_seed(groups)
    sizes = torch.randint(0, 3, (groups,), generator=g)
    sizes[torch.randint(0, groups, (3,), generator=g)] = 140
    sizes[-1] = 5
    sizes = sizes.tolist()
    rows, ends = sum(sizes) + 4, ends_of(sizes)
    e = ends.tolist()
    x, y = data(rows, 64, seed=34), data(rows, 48, seed=35)
    k = grp.bound(rows, groups)
    out = lambda n: (torch.zeros(n, k, dtype=torch.uint8, device="cuda"), torch.zeros(k // 128, n, device="cuda"))
    qx, qy = mx.block_quantize_grouped(x, ends, "e4m3", out=out(64)), mx.block_quantize_grouped(y, ends, "e5m2", out=out(48))
    for got, want in ((qx, grp.quantize(x, e, "e4m3")), (qy, grp.quantize(y, e, "e5m2"))):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    C, S = grp.gemm_k(qy, "e5m2", qx, "e4m3", e)
    check(mx.block_gemm_grouped_k(*qy, "e5m2", *qx, "e4m3", ends), C, S, 2, True)
    a, w = mx.block_quantize(x, "e4m3"), data(groups, 40, 64, seed=36)
    cw, sw = mx.block_quantize(w.view(groups * 40, 64), "e4m3")
    b = (cw.view(groups, 40, 64), sw.view(1, groups, 40).transpose(0, 1))
    C, S = grp.gemm(a, "e4m3", b, "e4m3", e, False)
    c = torch.full((rows, 40), 9.0, device="cuda")
    mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends, out_dtype=torch.float32, out=c)
    check(c[:rows - 4], C[:rows - 4], S[:rows - 4], 1, True)
    assert (c[rows - 4:] == 9).all()


def test_offsets_beyond_31_bits(mx):
    """C of more than 2^31 elements, by rows and by groups; a stack of weights of more than 2^31 bytes"""
    import torch
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB of GPU memory")
    g = torch.Generator(device="cuda").manual_seed(33)
    codes = lambda *s: torch.randint(0x20, 0x48, s, device="cuda", generator=g, dtype=torch.uint8)
    rows, N = 70100, 32768
    a, b = (codes(rows, 16), torch.ones(1, rows, device="cuda")), (codes(2, N, 16), torch.ones(2, 1, N // 128, device="cuda"))
    ends = torch.tensor([60000, rows], dtype=torch.int32, device="cuda")
    c = mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends)
    v = lambda t: t.view(torch.float8_e4m3fn).double()
    for lo, i in ((0, 0), (59990, 0), (60000, 1), (rows - 200, 1)):
        want = v(a[0][lo:lo + 10]) @ v(b[0][i]).t().contiguous()
        assert ((c[lo:lo + 10].double() - want).abs() <= 2.0 ** -7 * want).all()  # (all terms positive)
    del c
    a, b = (codes(16384, 1152), torch.ones(9, 16384, device="cuda")), (codes(16384, 1152), torch.ones(9, 16384, device="cuda"))
    ends = torch.arange(128, 1153, 128, dtype=torch.int32, device="cuda")
    c = mx.block_gemm_grouped_k(*a, "e4m3", *b, "e4m3", ends, out_dtype=torch.bfloat16, full_sums=True)
    for i in (0, 7, 8):
        cut = slice(128 * i, 128 * i + 128)
        want = v(a[0][-40:, cut].contiguous()) @ v(b[0][:, cut].contiguous()).t().contiguous()
        assert ((c[i, -40:].double() - want).abs() <= (2.0 ** -8 + 130 * 2.0 ** -24) * want).all()
    del c, a, b
    w = (codes(3, 32768, 32768), torch.ones(3, 256, 256, device="cuda"))
    a = (codes(40, 32768), torch.ones(256, 40, device="cuda"))
    ends = torch.tensor([7, 7, 40], dtype=torch.int32, device="cuda")
    c = mx.block_gemm_grouped(*a, "e4m3", *w, "e4m3", ends, out_dtype=torch.float32)
    for lo, hi, i in ((0, 7, 0), (7, 40, 2)):
        want = v(a[0][lo:hi]) @ v(w[0][i, -300:]).t().contiguous()
        assert ((c[lo:hi, -300:].double() - want).abs() <= (130 + 256) * 2.0 ** -24 * want).all()


def test_special_values(mx):
    """a NaN scale or code reaches its own row, or its own group, only"""
    import torch
    sizes = [50, 100, 0, 30]
    ends = ends_of(sizes)
    x = data(180, 256, seed=18)
    x[60, 7] = float("nan")
    a, b = mx.block_quantize(x, "e4m3"), weights(mx, 4, 140, 256, "e4m3", True, 19)
    b[1][3, 0, 0] = float("nan")
    for dtype in (torch.bfloat16, torch.float32):
        c = mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends, out_dtype=dtype)
        bad = torch.isnan(c)
        assert bad[60].all() and bad[150:, :128].all() and not bad[150:, 128:].any()
        bad[60] = False
        assert not bad[:150].any()
        at = mx.block_quantize_grouped(x, ends, "e4m3")
        g = mx.block_gemm_grouped_k(*at, "e4m3", *at, "e4m3", ends, out_dtype=dtype)
        assert torch.isnan(g[1, 7]).all() and torch.isnan(g[1, :, 7]).all() and not torch.isnan(g[[0, 2, 3]]).any()


def test_refusals(mx):
    import torch
    sizes = [50, 100]
    ends = ends_of(sizes)
    x = data(150, 256, seed=20)
    a, b = mx.block_quantize(x, "e4m3"), weights(mx, 2, 140, 256, "e4m3", True, 21)
    at = mx.block_quantize_grouped(x, ends, "e4m3")
    g = lambda **k: mx.block_gemm_grouped(k.get("a", a[0]), k.get("s", a[1]), k.get("f", "e4m3"), k.get("b", b[0]), k.get("t", b[1]),
                                          "e4m3", k.get("ends", ends), k.get("dtype", torch.bfloat16), k.get("out"))
    h = lambda **k: mx.block_gemm_grouped_k(k.get("a", at[0]), k.get("s", at[1]), "e4m3", *at, "e4m3", k.get("ends", ends),
                                            k.get("dtype", torch.float32), k.get("out"))
    bad = [lambda: g(ends=ends.long()), lambda: g(ends=ends.cpu()), lambda: g(ends=ends[:1]), lambda: g(ends=ends[None]),
           lambda: g(f="e2m1"), lambda: g(a=a[0][:, :128]), lambda: g(s=a[1][:1]), lambda: g(t=b[1][:, :, :1]), lambda: g(b=b[0][0]),
           lambda: g(dtype=torch.float16), lambda: g(out=torch.empty(150, 139, dtype=torch.bfloat16, device="cuda")),
           lambda: g(out=a[0].view(torch.bfloat16)[:, :140]), lambda: h(ends=ends.float()), lambda: h(a=at[0][:, :128]),
           lambda: h(s=at[1][1:]), lambda: h(dtype=torch.float64), lambda: h(out=torch.empty(1, 256, 256, device="cuda")),
           lambda: mx.block_quantize_grouped(x.float(), ends, "e4m3"), lambda: mx.block_quantize_grouped(x, ends, "e2m1"),
           lambda: mx.block_quantize_grouped(x, ends, "e4m3", out=(at[0][:, :128], at[1])),
           lambda: mx.block_quantize_grouped_dual(x, ends, "e4m3", "e4m3", out=(a[0], a[1], at[0], a[1]))]
    for call in bad:
        with pytest.raises((ValueError, mx.MXError)):
            call()


def test_empty(mx):
    import torch
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = data(0, 64, seed=1)
    q = mx.block_quantize_grouped(x, ends_of([0, 0]), "e4m3")
    assert q[0].shape == (64, 0)
    assert (mx.block_gemm_grouped_k(*q, "e4m3", *q, "e4m3", ends_of([0, 0])) == 0).all()
    assert mx.block_gemm_grouped_k(*q, "e4m3", *q, "e4m3", none).shape == (0, 64, 64)
    c = mx.block_gemm_grouped(*mx.block_quantize(x, "e4m3"), "e4m3", *weights(mx, 2, 30, 64, "e4m3", True, 2), "e4m3", ends_of([0, 0]))
    assert c.shape == (0, 30)


def test_layer(mx):
    """an expert layer forward and backward behind a norm and the normalised, rotated queries and keys of the QKV product, as
    a training step calls them; captured, and replayed with other rows per expert"""
    import torch
    T, D, H, E, heads, kv, hd = 200, 256, 384, 6, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(22)
    x = data(T, D, seed=23)
    nw, wqkv = (1 + 0.1 * data(D, seed=24).float()).bfloat16(), 0.06 * data((heads + 2 * kv) * hd, D, seed=25)
    qw = (1 + 0.1 * data(hd, seed=26).float()).bfloat16()
    w1 = (0.06 * data(E * H, D, seed=27).float()).bfloat16()
    pos, freqs = torch.arange(T, device="cuda"), mx.rope_frequencies(hd)
    index = torch.randint(0, T, (2 * T,), device="cuda", generator=g)
    dy = (1e-2 * data(2 * T, H, seed=28).float()).bfloat16()
    wq = mx.block_quantize(wqkv.bfloat16(), "e4m3", "tile")
    cr, sr, ct, st = mx.block_quantize_dual(w1, "e4m3", "e4m3", tile=True)
    b = (cr.view(E, H, D), sr.view(D // 128, E, H // 128).transpose(0, 1))
    bt = (ct.view(D, E, H).transpose(0, 1), st.view(E, H // 128, D // 128))
    ends = ends_of([100, 0, 57, 128, 100, 15])

    def step():
        hc, hs, _, rstd = mx.layer_norm_quantize(x, nw, rms=True)
        qkv = mx.block_gemm(hc, hs, "e4m3", *wq, "e4m3").view(T, heads + 2 * kv, hd)
        q, k = mx.qk_norm_rope(qkv[:, :heads], qkv[:, heads:heads + kv], qw, qw, pos, freqs)
        rows = x[index]                                      # tokens in their experts' order
        rc, rs, tc, ts = mx.block_quantize_grouped_dual(rows, ends, "e4m3", "e4m3")
        y = mx.block_gemm_grouped(rc, rs, "e4m3", *b, "e4m3", ends)
        dc, ds, dtc, dts = mx.block_quantize_grouped_dual(dy, ends, "e5m2", "e5m2")
        dx = mx.block_gemm_grouped(dc, ds, "e5m2", *bt, "e4m3", ends)
        dw = mx.block_gemm_grouped_k(dtc, dts, "e5m2", tc, ts, "e4m3", ends)
        return qkv, q, k, rows, (rc, rs), (tc, ts), y, (dc, ds), (dtc, dts), dx, dw

    def verify(out):
        import head_reference as head
        qkv, q, k, rows, r, t, y, d, dt, dx, dw = out
        for got, raw in ((q, qkv[:, :heads]), (k, qkv[:, heads:heads + kv])):
            want, mag = head.norm_rope(raw, qw, pos, freqs, 1e-5, "half")
            assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * mag).all()
        e = ends.tolist()
        check(y, *grp.gemm(r, "e4m3", b, "e4m3", e, True), 2, False)
        check(dx, *grp.gemm(d, "e5m2", bt, "e4m3", e, True), 3, False)
        check(dw, *grp.gemm_k(dt, "e5m2", t, "e4m3", e), 1, True)
        # the layer itself: quantized values are off by half a step of 8 bits, each operand's amax being its rows'
        lo = 0
        for i, hi in enumerate(e):
            if hi > lo:
                W, X = w1.view(E, H, D)[i].double(), rows[lo:hi].double()
                rel = 2.0 ** -4 + 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -8
                tiny = (X.abs().amax() * 2.0 ** -17 * W.abs().amax()) * D
                assert ((y[lo:hi].double() - X @ W.t()).abs() <= 1.1 * rel * (X.abs() @ W.abs().t()) + tiny).all()
            lo = hi

    verify(step())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for sizes in ([100, 0, 57, 128, 100, 15], [0, 0, 400, 0, 0, 0], [66, 67, 67, 66, 67, 67], [1, 2, 3, 4, 5, 385]):
        ends.copy_(ends_of(sizes))
        x.copy_(data(T, D, seed=sum(i * n for i, n in enumerate(sizes))))
        graph.replay()
        torch.cuda.synchronize()
        verify(out)
        again = step()
        for i in (1, 2, 6, 9, 10):
            assert torch.equal(out[i], again[i])


def test_other_stream(mx):
    import torch
    sizes = [300, 5, 0, 100]
    ends = ends_of(sizes)
    x = data(405, 256, seed=29)
    a, b = mx.block_quantize(x, "e4m3"), weights(mx, 4, 512, 256, "e4m3", True, 30)
    want = mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends)
    wq = mx.block_quantize_grouped(x, ends, "e4m3")
    wk = mx.block_gemm_grouped_k(*wq, "e4m3", *wq, "e4m3", ends)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends, stream=s)
    q = mx.block_quantize_grouped(x, ends, "e4m3", stream=s)
    k = mx.block_gemm_grouped_k(*q, "e4m3", *q, "e4m3", ends, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want) and torch.equal(k, wk)
