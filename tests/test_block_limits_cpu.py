"""Sizes at the edges of the block-128 and norm calls' index ranges and overlap rules, refused or
accepted on the host (pointers are only compared)."""
import ctypes
import os

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
E4M3, F32, BF16 = 0, 0, 1
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from precision_block_amax_amd import build as libbuild
    if not os.path.exists(libbuild.LIB_PATH):
        libbuild.build()
    import precision_block_amax_amd as mx
    return mx.lib()


@pytest.mark.parametrize("out", [F32, BF16])
def test_block_gemm_longest_k(L, out):
    """The kernels count K, rounded up to whole blocks, in 31 bits: a K above 2^31 - 128 would round to 2^31
    and past it, so it is refused, not answered with zeros."""
    for K in ((1 << 31) - 127, (1 << 31) - 1, 1 << 31, 1 << 40):
        args = [P(1 << 44), K, P(1 << 45), 1, E4M3, P(1 << 46), K, P(1 << 47), 1, E4M3, 0, 1, 1, K, P(1 << 32), out, 1, None]
        assert L.mx_block_gemm(*args) == UNSUPPORTED, K


def test_interleaved_rows_that_touch(L):
    """Rows in the gaps of another buffer's rows are refused where one byte is shared, where the strides differ, and
    where a run of other memory lies between them (pointers are compared on the host only)."""
    x = 0x100000000
    y = lambda **k: [P(x), 10, 64, k.get("ldx", 200), None, None, BF16, 0, 1e-5, P(x + k.get("at", 128)), k.get("ldy", 200),
                     P(k.get("mean", 0x200000000)), P(0x300000000), None]
    for bad in (dict(at=126), dict(at=274), dict(at=0), dict(ldy=201), dict(at=128 + 2 * 200 * 3 + 146), dict(at=-2 * 200 * 3 + 126),
                dict(mean=x + 300), dict(mean=x + 260)):
        assert L.mx_layer_norm(*y(**bad)) == INVALID, bad
    q = lambda s, ld: [P(x), 256, 64, 64, E4M3, 1, P(0x400000000), 512, P(0x400000000 + s), ld, None]  # 64 rows of 256 codes, 2 of scales
    for s, ld in ((252, 128), (257, 128), (256, 129), (256, 64)):
        assert L.mx_block_quantize(*q(s, ld)) == INVALID, (s, ld)


def test_interleaved_rows_of_different_counts_are_counted_whole(L):
    """(rows - 1) strides and a width that leave 64 bits are refused, a single row with any stride is not"""
    args = lambda ld, rows: [P(0x100000000), rows, 64, ld, None, None, BF16, 0, 1e-5, None, 64, None, None, None]
    assert L.mx_layer_norm(*args(1 << 62, 3)) == INVALID
    assert L.mx_layer_norm(*args(1 << 62, 0)) == OK


def test_block_gemm_sums_rejects(L):
    args = lambda **k: [P(0x100000000), 208, P(0x200000000), 70, k.get("fa", E4M3), P(0x300000000), 208, P(0x400000000), 300, E4M3,
                        k.get("tile", 0), k.get("M", 70), 300, k.get("K", 200), P(k.get("c", 0x500000000)), k.get("out", BF16), 300,
                        k.get("sums", 1), None]
    f = L.mx_block_gemm_sums
    for bad in (dict(sums=2), dict(sums=-1), dict(sums=0, out=F32), dict(sums=1, out=2), dict(sums=0, out=3), dict(fa=2), dict(tile=2),
                dict(M=-1), dict(c=0x100000000)):
        assert f(*args(**bad)) == INVALID, bad
    for sums, out in ((0, BF16), (1, BF16), (1, F32)):
        assert f(*args(sums=sums, out=out, M=0)) == OK
        assert f(*args(sums=sums, out=out, K=(1 << 31) - 1)) != OK


def test_single_rows_of_any_width(L):
    """one row whose bytes leave 64 bits is refused, whatever the stride"""
    for cols in ((1 << 62), (1 << 62) + 5, (1 << 63) - 1):
        args = [P(1 << 20), 1, cols, (1 << 63) - 1, E4M3, 0, P(1 << 30), (1 << 63) - 1, P(1 << 40), 1, None]
        assert L.mx_block_quantize(*args) == INVALID, cols
    assert L.mx_layer_norm(P(1 << 20), 1, 1 << 62, 1 << 62, None, None, BF16, 0, 1e-5, P(1 << 30), 1 << 62, None, None, None) == UNSUPPORTED
