"""Ends that lie above the rows, through the quantizer and the product along the rows, whose buffers hold NaN scales
and codes wherever the quantizer does not write.  The want is made of each group's own rows, cut to those that exist.

Tolerances as in test_gpu_grouped: nk blocks of a group."""
import pytest

import block_reference as ref
import group_reference as grp
from test_gpu_grouped import check, data, mx  # noqa: F401 (mx is a fixture)

pytestmark = pytest.mark.gpu


def operand(mx, x, fmt, ends, extra=0, shift=0):
    """x quantized into buffers of NaN, `extra` blocks wider than needed, rows `shift` bytes off"""
    import torch
    rows, cols = x.shape
    k = grp.bound(rows, len(ends))
    codes = torch.full((cols, k + 128 * extra + 16), 0x7F, dtype=torch.uint8, device="cuda")[:, shift:shift + k + 128 * extra]
    scales = torch.full((k // 128 + extra, cols), float("nan"), device="cuda")
    mx.block_quantize_grouped(x, ends, fmt, out=(codes[:, :k], scales[:k // 128]))
    return codes, scales


def want(x, fx, y, fy, ends):
    """(C, sum of |terms|), and the most blocks of a group"""
    import torch
    C, S, nk = [], [], 1
    for lo, hi in grp.ranges(ends, x.shape[0]):
        if hi > lo:
            c, s = ref.gemm(ref.quantize(x[lo:hi], fx, "transpose"), fx, ref.quantize(y[lo:hi], fy, "transpose"), fy, False)
        else:
            c = s = torch.zeros(x.shape[1], y.shape[1], dtype=torch.float64, device="cuda")
        C.append(c), S.append(s)
        nk = max(nk, ref.cdiv(hi - lo, 128))
    return torch.stack(C), torch.stack(S), nk


# rows and ends: one block more, several, a later end above the rows too, decreasing, all above, within the last block,
# more groups than one read of the ends holds, as far as a number goes
CASES = [(200, [100, 400]), (200, [100, 250, 300]), (100, [5, 3, 900, -1, 60]), (300, [500]), (130, [140, 150, 7, 2 ** 31 - 1]),
         (384, [100, 385]), (250, [251]), (1, [5, 9]), (700, [2 * i for i in range(349)] + [2000, 900]), (900, [300, 5000, 6000, 7000])]


@pytest.mark.parametrize("rows,ends", CASES, ids=lambda v: str(v)[:30])
@pytest.mark.parametrize("M,N", [(40, 72), (130, 260)])
@pytest.mark.parametrize("extra,shift", [(0, 0), (2, 0), (1, 5)])
def test_ends_above_the_rows(mx, rows, ends, M, N, extra, shift):
    import torch
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    x, y = data(rows, M, seed=51), data(rows, N, seed=52)
    a, b = operand(mx, x, "e5m2", e, extra, shift), operand(mx, y, "e4m3", e, extra, shift)
    C, S, nk = want(x, "e5m2", y, "e4m3", ends)
    for dtype, full in ((torch.float32, True), (torch.bfloat16, True), (torch.bfloat16, False)):
        c = torch.full((len(ends), M, N), float("nan"), dtype=dtype, device="cuda")
        mx.block_gemm_grouped_k(*a, "e5m2", *b, "e4m3", e, out_dtype=dtype, full_sums=full, out=c, rows=rows)
        check(c, C, S, nk, full)


# sizes where K is shared by eight waves, by two groups of waves, and not
@pytest.mark.parametrize("rows,ends,M,N", [(1700, [500, 1600, 9999], 200, 136), (2000, [800, 1500, 4000], 1024, 1024),
                                           (900, [100, 250, 250, 251, 700, 650, 901, 3000], 1030, 520)])
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
def test_every_kernel(mx, rows, ends, M, N, fa):
    import torch
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    x, y = data(rows, M, seed=53), data(rows, N, seed=54)
    a, b = operand(mx, x, fa, e), operand(mx, y, "e4m3", e)
    C, S, nk = want(x, fa, y, "e4m3", ends)
    for dtype in (torch.float32, torch.bfloat16):
        check(mx.block_gemm_grouped_k(*a, fa, *b, "e4m3", e, out_dtype=dtype, rows=rows), C, S, nk, dtype is torch.float32)


def test_ends_within_the_rows(mx):
    """with and without the number of rows: the same bits"""
    import torch
    e = torch.tensor([10, 10, 300, 431], dtype=torch.int32, device="cuda")
    x = data(440, 96, seed=55)
    q = operand(mx, x, "e4m3", e)
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(mx.block_gemm_grouped_k(*q, "e4m3", *q, "e4m3", e, out_dtype=dtype),
                           mx.block_gemm_grouped_k(*q, "e4m3", *q, "e4m3", e, out_dtype=dtype, rows=440))


def test_more_routed_than_held(mx):
    """one graph over a buffer of fixed size, replayed with routings that it holds and that it does not"""
    import torch
    x, y = data(256, 64, seed=56), data(256, 128, seed=57)
    e = torch.tensor([64, 128, 192, 256], dtype=torch.int32, device="cuda")
    k = grp.bound(256, 4)
    qx, qy = [(torch.full((n, k), 0x7F, dtype=torch.uint8, device="cuda"), torch.full((k // 128, n), float("nan"), device="cuda"))
              for n in (64, 128)]

    def step():
        mx.block_quantize_grouped(x, e, "e4m3", out=qx)
        mx.block_quantize_grouped(y, e, "e4m3", out=qy)
        return mx.block_gemm_grouped_k(*qy, "e4m3", *qx, "e4m3", e, rows=256)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for ends in ([64, 128, 192, 256], [200, 260, 500, 600], [0, 0, 0, 900], [100, 200, 250, 300]):
        e.copy_(torch.tensor(ends, dtype=torch.int32))
        for t in (qx[1], qy[1]):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(out, *want(y, "e4m3", x, "e4m3", ends), True)
        assert torch.equal(out, step())


@pytest.mark.parametrize("rows", [384, 385, 1 << 20, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 1])
@pytest.mark.parametrize("ends", [[2 ** 31 - 1], [100, 2 ** 31 - 1, 2 ** 31 - 1], [0, 2 ** 31 - 100, 5], [200, 384, 1 << 30]], ids=str)
def test_more_rows_than_columns(mx, rows, ends):
    """a number of rows beyond the columns: groups have the blocks that there are"""
    import torch
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    for M, N in ((70, 40), (150, 300)):
        a, b = ((torch.full((n, 384), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(3, n, device="cuda")) for n in (M, N))
        C, S = grp.gemm_k(a, "e4m3", b, "e4m3", ends)
        for dtype in (torch.float32, torch.bfloat16):
            c = mx.block_gemm_grouped_k(*a, "e4m3", *b, "e4m3", e, out_dtype=dtype, rows=rows)
            check(c, C, S, 3, dtype is torch.float32)


def test_refusals(mx):
    import torch
    e = torch.tensor([100, 200], dtype=torch.int32, device="cuda")
    q = operand(mx, data(200, 64, seed=58), "e4m3", e)
    for rows in (-1, 1 << 31):
        with pytest.raises(mx.MXError):
            mx.block_gemm_grouped_k(*q, "e4m3", *q, "e4m3", e, rows=rows)
