"""Block-128 operators by group on the host: arguments that are refused before any HIP call (pointers are only
compared), empty calls, sizes, and the reference definitions the GPU tests rely on."""
import ctypes
import os
import random

import pytest
import torch

import block_reference as ref
import group_reference as grp

OK, INVALID, UNSUPPORTED = 0, 1, 2
E4M3, E5M2, E2M1 = 0, 1, 2
F32, BF16 = 0, 1
FP8SUMS, FULL = 0, 1
P = ctypes.c_void_p
X, E, C, S, C2, S2, A, AS, B, BS, Y = (P(0x100000000 * (i + 1)) for i in range(11))


@pytest.fixture(scope="module")
def L():
    from precision_block_amax_amd import build as libbuild
    if not os.path.exists(libbuild.LIB_PATH):
        libbuild.build()
    import precision_block_amax_amd as mx
    return mx.lib()


def test_columns_are_enough(L):
    """the bound holds for any groups and is met by some"""
    f = L.mx_block_grouped_cols
    rng = random.Random(1)
    for _ in range(300):
        rows, groups = rng.randint(1, 2000), rng.randint(1, 40)
        ends = sorted(rng.randint(0, rows) for _ in range(groups))
        assert grp.blocks(ends, rows)[-1][1] * 128 <= f(rows, groups) == grp.bound(rows, groups)
    for rows, groups in ((1, 1), (128, 1), (129, 1), (5, 9), (300, 2), (1000, 8)):
        n = min(rows, groups)   # one row in all groups but the first, the rest there, cut to leave whole blocks and a row
        most = max(sum(ref.cdiv(s, 128) for s in [rows - (n - 1) - 128 * j] + [1 + 128 * j] + [1] * (n - 2)) if n > 1
                   else ref.cdiv(rows, 128) for j in range(max(1, (rows - n) // 128 + 1)) if rows - (n - 1) - 128 * j > 0)
        assert most * 128 == f(rows, groups)
    assert f(0, 5) == 0 and f(5, 0) == 0 and f(-1, 3) == 0 and f(1 << 31, 1) == 0 and f(5, (1 << 16) + 1) == 0


def quant(**k):   # 300 rows in 5 groups: at most 7 blocks
    return [k.get("x", X), k.get("rows", 300), k.get("cols", 200), k.get("ldx", 200), k.get("ends", E), k.get("groups", 5),
            k.get("fmt", E4M3), k.get("c", C), k.get("ldc", 896), k.get("s", S), k.get("lds", 200), None]


def dual(**k):
    return [k.get("x", X), k.get("rows", 300), k.get("cols", 200), k.get("ldx", 200), k.get("ends", E), k.get("groups", 5),
            k.get("fr", E4M3), k.get("cr", C2), k.get("ldcr", 200), k.get("sr", S2), k.get("ldsr", 300),
            k.get("fmt", E5M2), k.get("c", C), k.get("ldc", 896), k.get("s", S), k.get("lds", 200), None]


def test_quantize_rejects(L):
    assert L.mx_block_grouped_cols(300, 5) == 896
    for f, args in ((L.mx_block_quantize_grouped, quant), (L.mx_block_quantize_grouped_dual, dual)):
        for bad in (dict(rows=-1), dict(cols=-1), dict(groups=-1), dict(ldx=199), dict(fmt=E2M1), dict(fmt=7), dict(ldc=895),
                    dict(lds=199), dict(x=None), dict(ends=None), dict(c=None), dict(s=None), dict(c=X), dict(s=X), dict(c=E),
                    dict(s=P(E.value + 16)), dict(s=P(C.value + 199 * 896)), dict(ldx=1 << 62), dict(ldc=1 << 62),
                    dict(x=P(C.value + 896 * 200 - 2))):
            assert f(*args(**bad)) == INVALID, bad
        assert f(*args(groups=(1 << 16) + 1)) == UNSUPPORTED
        assert f(*args(rows=1 << 31)) == UNSUPPORTED
        none = dict(x=None, ends=None, c=None, s=None, cr=None, sr=None)
        assert f(*args(rows=0, **none)) == OK
        assert f(*args(groups=0, **none)) == OK
        assert f(*args(cols=0, ldx=0, **none)) == OK
    f = L.mx_block_quantize_grouped_dual
    for bad in (dict(fr=E2M1), dict(ldcr=199), dict(ldsr=299), dict(cr=None), dict(sr=None), dict(cr=C), dict(sr=S), dict(cr=E)):
        assert f(*dual(**bad)) == INVALID, bad


def rows_args(**k):  # 5 groups, 300 rows, N = 260, K = 200
    return [k.get("a", A), k.get("lda", 208), k.get("as_", AS), k.get("ldsa", 300), k.get("fa", E4M3), k.get("b", B),
            k.get("ldbg", 260 * 208), k.get("ldb", 208), k.get("bs", BS), k.get("ldsbg", 520), k.get("ldsb", 260), k.get("fb", E5M2),
            k.get("tile", 0), k.get("ends", E), k.get("groups", 5), k.get("rows", 300), k.get("N", 260), k.get("K", 200),
            k.get("c", Y), k.get("out", BF16), k.get("ldc", 260), k.get("sums", FP8SUMS), None]


def test_rows_rejects(L):
    f = L.mx_block_gemm_grouped
    for bad in (dict(rows=-1), dict(N=-1), dict(K=-1), dict(groups=-1), dict(fa=E2M1), dict(fb=E2M1), dict(fa=9), dict(out=2),
                dict(tile=2), dict(sums=2), dict(sums=-1), dict(out=F32), dict(lda=199), dict(ldb=199), dict(ldsa=299), dict(ldsb=259),
                dict(ldbg=-1), dict(ldsbg=-1), dict(ldc=259), dict(a=None), dict(as_=None), dict(b=None), dict(bs=None),
                dict(ends=None), dict(c=None), dict(c=A), dict(c=AS), dict(c=P(B.value + 4 * 260 * 208 + 259 * 208)),
                dict(c=P(BS.value + 4 * (4 * 520 + 260 + 259))), dict(c=P(E.value + 16)), dict(lda=1 << 62), dict(ldbg=1 << 62),
                dict(ldsbg=1 << 62), dict(ldc=1 << 62), dict(ldb=1 << 62)):
        assert f(*rows_args(**bad)) == INVALID, bad
    big = dict(lda=1 << 40, ldb=1 << 40)
    for bad in (dict(rows=1 << 31, ldsa=1 << 31, a=P(1 << 50), c=P(1 << 54)), dict(groups=(1 << 16) + 1),
                dict(K=(1 << 31) - 127, a=P(1 << 50), b=P(1 << 55), as_=P(1 << 57), bs=P(1 << 58), c=P(1 << 60), **big),
                dict(rows=1 << 26, N=1 << 10, ldc=1 << 10, ldsa=1 << 26, ldsb=1 << 10, a=P(1 << 50), as_=P(1 << 52), c=P(1 << 54))):
        assert f(*rows_args(**bad)) == UNSUPPORTED, bad
    none = dict(a=None, as_=None, b=None, bs=None, ends=None, c=None)
    assert f(*rows_args(rows=0, **none)) == OK
    assert f(*rows_args(N=0, **none)) == OK
    assert f(*rows_args(groups=0, **none)) == OK


def cols_args(**k):  # 5 groups, M = 70, N = 260, 896 columns
    return [k.get("a", A), k.get("lda", 896), k.get("as_", AS), k.get("ldsa", 70), k.get("fa", E4M3), k.get("b", B),
            k.get("ldb", 896), k.get("bs", BS), k.get("ldsb", 260), k.get("fb", E5M2), k.get("ends", E), k.get("groups", 5),
            k.get("M", 70), k.get("N", 260), k.get("cols", 896), k.get("c", Y), k.get("out", F32), k.get("ldcg", 70 * 260),
            k.get("ldc", 260), k.get("sums", FULL), None]


def test_cols_rejects(L):
    f = L.mx_block_gemm_grouped_k
    for bad in (dict(M=-1), dict(N=-1), dict(cols=-1), dict(cols=895), dict(groups=-1), dict(fa=E2M1), dict(fb=E2M1), dict(out=2),
                dict(sums=2), dict(sums=FP8SUMS), dict(lda=895), dict(ldb=895), dict(ldsa=69), dict(ldsb=259), dict(ldc=259),
                dict(ldcg=70 * 260 - 1), dict(ldcg=-1), dict(a=None), dict(as_=None), dict(b=None), dict(bs=None), dict(ends=None),
                dict(c=None), dict(c=A), dict(c=B), dict(c=AS), dict(c=BS), dict(c=E), dict(a=P(Y.value + 4 * 5 * 70 * 260 - 1)),
                dict(lda=1 << 62), dict(ldc=1 << 61), dict(ldcg=1 << 62)):
        assert f(*cols_args(**bad)) == INVALID, bad
    for bad in (dict(groups=(1 << 16) + 1), dict(M=1 << 20, N=1 << 20, ldsa=1 << 20, ldsb=1 << 20, ldc=1 << 20, ldcg=1 << 40,
                                                 a=P(1 << 50), b=P(1 << 51), as_=P(1 << 52), bs=P(1 << 53), c=P(1 << 55))):
        assert f(*cols_args(**bad)) == UNSUPPORTED, bad
    none = dict(a=None, as_=None, b=None, bs=None, ends=None, c=None)
    assert f(*cols_args(M=0, **none)) == OK
    assert f(*cols_args(N=0, **none)) == OK
    assert f(*cols_args(groups=0, **none)) == OK


def test_reference():
    """the parts by group add up to the whole where a group's products may be written as one matrix product"""
    g = torch.Generator().manual_seed(1)
    x, dy = torch.randn(400, 30, generator=g).bfloat16(), torch.randn(400, 20, generator=g).bfloat16()
    ends = [0, 130, 130, 131, 390]
    assert grp.ranges([5, 3, 900, -1], 100) == [(0, 5), (5, 5), (5, 100), (100, 100)]
    qx, qy = grp.quantize(x, ends, "e4m3"), grp.quantize(dy, ends, "e5m2")
    assert qx[0].shape == (30, grp.bound(400, 5))
    C, S = grp.gemm_k(qy, "e5m2", qx, "e4m3", ends)
    assert C.shape == (5, 20, 30) and (C[0] == 0).all() and (C[2] == 0).all() and (S.sum(0) > 0).all()
    whole = ref.values(*qy, "e5m2") @ ref.values(*qx, "e4m3").t()
    assert torch.allclose(C.sum(0), whole, rtol=0, atol=1e-10)
    a = ref.quantize(x, "e4m3")
    w = [ref.quantize(torch.randn(7, 30, generator=g).bfloat16(), "e4m3", "tile") for _ in ends]
    b = (torch.stack([c for c, _ in w]), torch.stack([s for _, s in w]))
    C, _ = grp.gemm(a, "e4m3", b, "e4m3", ends, True)
    assert (C[390:] == 0).all()
    assert torch.allclose(C[130], ref.values(a[0][130:131], a[1][:, 130:131], "e4m3")[0] @ ref.values(*w[3], "e4m3", True).t())
