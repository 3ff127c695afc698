"""Block-128 FP8 and norm entry points on the host: arguments that are refused before any HIP call
(pointers are only compared), empty calls, and the reference definitions the GPU tests rely on."""
import ctypes
import os

import pytest
import torch

import block_reference as ref

OK, INVALID, UNSUPPORTED = 0, 1, 2
E4M3, E5M2, E2M1 = 0, 1, 2
F32, BF16 = 0, 1
P = ctypes.c_void_p
X, C, S, C2, S2, W, B, Y, M_, R_ = (P(0x100000000 * (i + 1)) for i in range(10))


@pytest.fixture(scope="module")
def L():
    from precision_block_amax_amd import build as libbuild
    if not os.path.exists(libbuild.LIB_PATH):
        libbuild.build()
    import precision_block_amax_amd as mx
    return mx.lib()


def test_block_quantize_rejects(L):
    args = lambda **k: [k.get("x", X), k.get("rows", 300), k.get("cols", 200), k.get("ldx", 200), k.get("fmt", E4M3),
                        k.get("mode", 0), k.get("c", C), k.get("ldc", 208), k.get("s", S), k.get("lds", 300), None]
    f = L.mx_block_quantize
    assert f(*args(rows=-1)) == INVALID
    assert f(*args(cols=-1)) == INVALID
    assert f(*args(ldx=199)) == INVALID
    assert f(*args(fmt=E2M1)) == INVALID                    # FP8 formats only
    assert f(*args(fmt=9)) == INVALID
    assert f(*args(mode=4)) == INVALID
    assert f(*args(mode=-1)) == INVALID
    assert f(*args(ldc=199)) == INVALID                     # rows of codes overlap
    assert f(*args(lds=299)) == INVALID                     # blocks of scales overlap
    assert f(*args(mode=1, ldc=299)) == INVALID             # transposed: 200 rows of 300 codes
    assert f(*args(mode=1, ldc=300, lds=199)) == INVALID
    assert f(*args(mode=2, lds=2)) == INVALID               # 3 tiles of rows
    assert f(*args(mode=3, ldc=300, lds=1)) == INVALID      # 2 tiles of columns
    assert f(*args(x=None)) == INVALID
    assert f(*args(c=None)) == INVALID
    assert f(*args(s=None)) == INVALID
    assert f(*args(c=X)) == INVALID                         # overlaps
    assert f(*args(s=P(X.value + 2 * 300 * 200 - 2))) == INVALID
    assert f(*args(s=P(C.value + 299 * 208))) == INVALID
    assert f(*args(ldx=1 << 62)) == INVALID                 # extent beyond 64 bits
    assert f(*args(rows=1 << 30, cols=1 << 30, ldx=1 << 30, ldc=1 << 30, lds=1 << 30, x=P(1 << 12), c=P(1 << 61),
                   s=P(1 << 62))) in (INVALID, UNSUPPORTED)
    assert f(*args(rows=0, x=None, c=None, s=None)) == OK
    assert f(*args(cols=0, ldx=0, x=None, c=None, s=None)) == OK


def test_block_quantize_dual_rejects(L):
    args = lambda **k: [k.get("x", X), k.get("rows", 300), k.get("cols", 200), k.get("ldx", 200), k.get("tile", 0),
                        k.get("fr", E4M3), k.get("c", C), 200, k.get("s", S), k.get("lds", 300), k.get("ft", E5M2),
                        k.get("ct", C2), k.get("ldct", 300), k.get("st", S2), k.get("ldst", 200), None]
    f = L.mx_block_quantize_dual
    assert f(*args(tile=2)) == INVALID
    assert f(*args(fr=E2M1)) == INVALID
    assert f(*args(ft=E2M1)) == INVALID
    assert f(*args(ldct=299)) == INVALID
    assert f(*args(ldst=199)) == INVALID
    assert f(*args(ct=C)) == INVALID
    assert f(*args(st=S)) == INVALID
    assert f(*args(st=P(C2.value + 199 * 300))) == INVALID
    assert f(*args(ct=None)) == INVALID
    assert f(*args(rows=0, x=None, c=None, s=None, ct=None, st=None)) == OK


def test_block_gemm_rejects(L):
    args = lambda **k: [k.get("a", X), k.get("lda", 208), k.get("as_", S), k.get("ldsa", 70), k.get("fa", E4M3),
                        k.get("b", C), k.get("ldb", 208), k.get("bs", S2), k.get("ldsb", 300), k.get("fb", E5M2),
                        k.get("tile", 0), k.get("M", 70), k.get("N", 300), k.get("K", 200), k.get("c", Y),
                        k.get("out", BF16), k.get("ldc", 300), None]
    f = L.mx_block_gemm
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(fa=E2M1), dict(fb=E2M1), dict(out=2), dict(tile=2),
                dict(lda=199), dict(ldb=199), dict(ldsa=69), dict(ldsb=299), dict(tile=1, ldsb=2), dict(ldc=299),
                dict(a=None), dict(as_=None), dict(b=None), dict(bs=None), dict(c=None), dict(c=X),
                dict(c=P(S.value + 4 * (70 + 69))), dict(c=P(C.value + 299 * 208)), dict(lda=1 << 62),
                dict(ldc=1 << 62)):
        assert f(*args(**bad)) == INVALID, bad
    assert f(*args(M=1 << 31, ldsa=1 << 31, c=P(1 << 60), a=P(1 << 58), as_=P(1 << 59))) == UNSUPPORTED
    assert f(*args(M=0, a=None, as_=None, c=None)) == OK
    assert f(*args(N=0, b=None, bs=None, c=None)) == OK


def test_layer_norm_rejects(L):
    args = lambda **k: [k.get("x", X), k.get("rows", 4), k.get("cols", 100), k.get("ldx", 100), k.get("w", W),
                        k.get("b", B), k.get("param", BF16), k.get("kind", 0), k.get("eps", 1e-5), k.get("y", Y),
                        k.get("ldy", 100), k.get("mean", M_), k.get("rstd", R_), None]
    f = L.mx_layer_norm
    for bad in (dict(rows=-1), dict(cols=-1), dict(ldx=99), dict(param=2), dict(kind=2), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(ldy=99), dict(x=None), dict(y=None), dict(y=X),
                dict(y=W), dict(mean=Y), dict(rstd=M_), dict(rstd=B)):
        assert f(*args(**bad)) == INVALID, bad
    assert f(*args(cols=40000, ldx=40000, ldy=40000)) == UNSUPPORTED
    assert f(*args(rows=0, x=None, y=None)) == OK
    assert f(*args(cols=0, x=None, y=None)) == OK


def test_layer_norm_quantize_rejects(L):
    args = lambda **k: [k.get("x", X), k.get("rows", 4), k.get("cols", 96), 96, W, B, BF16, 0, 1e-5, k.get("fmt", E2M1),
                        k.get("c", C), k.get("s", S), M_, R_, None]
    f = L.mx_layer_norm_quantize
    for bad in (dict(cols=80), dict(fmt=7), dict(c=None), dict(s=None), dict(s=C), dict(c=X), dict(s=M_)):
        assert f(*args(**bad)) == INVALID, bad
    assert f(*args(rows=0, x=None, c=None, s=None)) == OK
    blk = lambda **k: [k.get("x", X), k.get("rows", 4), k.get("cols", 100), 100, W, B, BF16, 1, 1e-5, k.get("fmt", E4M3),
                       k.get("c", C), k.get("ldc", 112), k.get("s", S), k.get("lds", 4), None, R_, None]
    g = L.mx_layer_norm_block_quantize
    for bad in (dict(fmt=E2M1), dict(ldc=99), dict(lds=3), dict(s=None), dict(s=P(C.value + 3 * 112)), dict(rows=-4)):
        assert g(*blk(**bad)) == INVALID, bad
    assert g(*blk(rows=0, x=None, c=None, s=None)) == OK


def test_layer_norm_backward_rejects(L):
    need = L.mx_layer_norm_backward_workspace(100, 64)
    assert need > 0 and L.mx_layer_norm_backward_workspace(0, 64) == 0 and L.mx_layer_norm_backward_workspace(5, -1) == 0
    args = lambda **k: [k.get("dy", Y), k.get("lddy", 64), k.get("x", X), 64, k.get("rows", 100), k.get("cols", 64), W,
                        k.get("param", BF16), k.get("kind", 0), k.get("mean", M_), k.get("rstd", R_), k.get("dx", C),
                        k.get("lddx", 64), k.get("dw", S), k.get("db", S2), k.get("ws", C2), k.get("n", need), None]
    f = L.mx_layer_norm_backward
    for bad in (dict(rows=-1), dict(lddy=63), dict(lddx=63), dict(param=3), dict(kind=-1), dict(dy=None), dict(x=None),
                dict(mean=None), dict(rstd=None), dict(dx=None), dict(ws=None), dict(n=need - 1),
                dict(ws=P(C2.value + 4)), dict(dx=X), dict(dx=Y), dict(dw=S2), dict(ws=C), dict(db=R_)):
        assert f(*args(**bad)) == INVALID, bad
    assert f(*args(cols=0, dy=None, x=None)) == OK
    assert f(*args(rows=0, dy=None, x=None, dw=None, db=None)) == OK


def test_binding_refuses():
    import precision_block_amax_amd as mx
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(2, 4)
    for call in (lambda: mx.block_quantize(x, "e4m3"), lambda: mx.block_quantize_dual(x, "e4m3", "e4m3"),
                 lambda: mx.layer_norm(x), lambda: mx.layer_norm_quantize(x),
                 lambda: mx.layer_norm_backward(x, x, None, None, s, rms=True),
                 lambda: mx.block_gemm(c, s, "e4m3", c, s, "e4m3")):
        with pytest.raises(ValueError):  # tensors that are not on a GPU
            call()
    with pytest.raises(ValueError):
        mx._fp8("e2m1")


@pytest.mark.parametrize("cols", [8, 1024, 2048, 4096, 8192, 16384, 16392, 32768])
def test_norm_backward_workgroups_all_have_rows(cols):
    """Workgroup b of the backward pass takes rows b * per .. with per = ceil(rows / workgroups), and reads its
    first row before it looks at its count: the last one must have a row.  The workspace (two fp32 sums of
    cols for each workgroup) tells how many there are."""
    import precision_block_amax_amd as mx
    size = mx.lib().mx_layer_norm_backward_workspace
    assert size(0, cols) == 0
    for rows in [*range(1, 1200), 2049, 4095, 5000, 65537, (1 << 20) + 1, (1 << 31) - 1]:
        chunks, rest = divmod(size(rows, cols), 2 * 4 * cols)
        assert rest == 0 and 1 <= chunks <= 256
        assert (chunks - 1) * -(-rows // chunks) < rows


def test_reference_norm_gradient_against_differences():
    """The formula the kernels are held to, against central differences of the definition in float64:
    with step h the difference is off by h^2 times third derivatives of order 1 and by 2^-53 / h."""
    torch.manual_seed(0)
    rows, cols, eps, h = 3, 10, 1e-3, 1e-5
    x, dy = torch.randn(rows, cols, dtype=torch.float64), torch.randn(rows, cols, dtype=torch.float64)
    w, b = torch.randn(cols, dtype=torch.float64), torch.randn(cols, dtype=torch.float64)
    for rms in (False, True):
        _, mean, rstd = ref.norm(x, w, b, eps, rms)
        dx, dw, db = ref.norm_backward(dy, x, w, mean, rstd, rms)
        loss = lambda x_, w_, b_: (ref.norm(x_, w_, b_, eps, rms)[0] * dy).sum()
        for t, g, at in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
            for i in range(t.numel()):
                e = torch.zeros_like(t).view(-1)
                e[i] = h
                e = e.view_as(t)
                a, c = [x, w, b], [x, w, b]
                a[at], c[at] = t + e, t - e
                d = (loss(*a) - loss(*c)) / (2 * h)
                assert abs(d - g.reshape(-1)[i]) < 1e-7, (rms, at, i)


def test_reference_quantizer_by_hand():
    x = torch.zeros(2, 130)
    x[0, 0], x[0, 1], x[0, 129], x[1, 3] = 448.0, -1.0, 2.0, float("inf")
    codes, scales = ref.quantize(x, "e4m3")
    assert scales.shape == (2, 2) and scales[0, 0] == 1.0 and scales[1, 0] == torch.tensor(2.0) / 448.0
    assert codes[0, 0] == 0x7E and codes[0, 1] == 0xB8 and codes[0, 129] == 0x7E and codes[0, 2] == 0
    assert torch.isnan(scales[0, 1]) and (codes[1] == 0).all()
    assert scales[1, 1] == torch.tensor(2.0 ** -100) / 448.0
    t, st = ref.quantize(x.t().contiguous(), "e4m3", "transpose")
    assert torch.equal(t, codes) and torch.equal(st.nan_to_num(-1.0), scales.nan_to_num(-1.0))
