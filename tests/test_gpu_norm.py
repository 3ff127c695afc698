"""The norm in front of a linear layer on the GPU against its definition in float64
(block_reference), forward, to quantized operands, and backward; and a layer's run of the
block-128 operators together.

Tolerances.  fp32 sums of n terms taken as T threads of 8 U terms, a wave and its workgroup are
trees of depth d <= 8 U + 6 + T / 64 <= 54, off by at most d 2^-24 of the sum of |terms|; with
the few roundings per element that follow, 64 2^-24 = 2^-18 of the terms involved covers mean,
variance (and so rstd, relative) and y before its own rounding, which adds half a step."""
import pytest

import block_reference as ref

pytestmark = pytest.mark.gpu
E = 2.0 ** -18


@pytest.fixture(scope="module")
def mx():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_block_amax_amd as m
    m.lib()
    return m


def make(rows, cols, seed, dtype=None, shift=0.5):
    import torch
    dtype = dtype or torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    x = (r(rows, cols) * (1 + r(rows, 1).abs()) + shift).bfloat16()
    return x, (1 + 0.3 * r(cols)).to(dtype), (0.3 * r(cols)).to(dtype), (1e-2 * r(rows, cols)).bfloat16()


def y_error(x, w, rms, y, mean, rstd):
    """what fp32 may be off by in y, before its rounding: E of the terms that make it"""
    import torch
    v = x.double()
    a = v.abs() + v.abs().mean(1, keepdim=True) + (v - mean[:, None]).abs()
    a = a * rstd[:, None]
    if w is not None:
        a = a * w.double().abs()
    return E * (a + y.abs())


def check_stats(x, mean, rstd, want_mean, want_rstd, rms):
    v = x.double()
    if rms:
        assert mean is None
    else:
        assert ((mean.double() - want_mean).abs() <= E * v.abs().mean(1)).all()
    # d rstd / rstd = - d var / (2 (var + eps)); the mean's error enters var in second order
    assert ((rstd.double() / want_rstd - 1).abs() <= E).all()


SHAPES = [(1, 1), (1, 4096), (3, 5), (2, 8), (5, 100), (4, 512), (7, 513), (6, 1000), (3, 1024), (2, 1025), (9, 2048), (5, 2056),
          (3, 4096), (2, 4097), (300, 640), (3, 8192), (2, 8200), (2, 14336), (2, 16384), (2, 16392), (2, 28672), (1, 32768)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm(mx, rows, cols, rms):
    import torch
    print("case", rows, cols, rms, flush=True)
    for dtype in (torch.bfloat16, torch.float32):
        x, w, b, _ = make(rows, cols, rows + cols, dtype)
        for wt, bs in ((w, b), (w, None), (None, b), (None, None)):
            y, mean, rstd = mx.layer_norm(x, wt, bs, eps=1e-3, rms=rms)
            want, wm, wr = ref.norm(x, wt, bs, 1e-3, rms)
            check_stats(x, mean, rstd, wm, wr, rms)
            tol = 2.0 ** -8 * want.abs() + y_error(x, wt, rms, want, wm, wr) + 2.0 ** -134
            bad = ~((y.double() - want).abs() <= tol)
            assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


def deq_block(codes, scales, fmt):
    return ref.values(codes, scales, fmt)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_layer_norm_block_quantize(mx, rows, cols, rms, fmt):
    import torch
    x, w, b, _ = make(rows, cols, rows + 2 * cols)
    codes, scales, mean, rstd = mx.layer_norm_quantize(x, w, b, fmt, eps=1e-3, rms=rms)
    want, wm, wr = ref.norm(x, w, b, 1e-3, rms)
    check_stats(x, mean, rstd, wm, wr, rms)
    dy = y_error(x, w, rms, want, wm, wr)
    amax = ref.block_amax(want, False).clamp(min=ref.FLOOR)
    slack = ref.block_amax(dy, False) + 2.0 ** -22 * amax
    assert codes.shape == x.shape and scales.shape == (ref.cdiv(cols, 128), rows)
    assert ((scales.double().t() * ref.FMAX[fmt] - amax).abs() <= slack).all()
    # a code is within half a step of its value over its scale; the scale's own slack moves both alike
    sc = ref.spread(scales.double().t(), x.shape, False)
    tol = ref.HALF_REL[fmt] * want.abs() * (1 + 2.0 ** -10) + ref.HALF_SUB[fmt] * sc + 2 * dy + 2.0 ** -20 * want.abs()
    bad = ~((deq_block(codes, scales, fmt) - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("cols", [32, 96, 512, 544, 2048, 4096, 5120, 14336, 32768])
def test_layer_norm_quantize_exact(mx, cols):
    """rows of +-1: their RMS is 1 exactly and y = +-weight exactly, so the quantized forms equal the quantizers'
    own codes and scales of y, in both scalings and every format"""
    import torch
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.randint(0, 2, (70, cols), device="cuda", generator=g) * 2 - 1).bfloat16()
    w = torch.randn(cols, device="cuda", generator=g).bfloat16()
    y, _, rstd = mx.layer_norm(x, w, eps=0.0, rms=True)
    assert torch.equal(y, x * w) and (rstd == 1).all()
    for fmt in ("e4m3", "e5m2", "e2m1"):
        got = mx.layer_norm_quantize(x, w, None, fmt, eps=0.0, rms=True, scaling="mx")
        want = mx.quantize(y, fmt)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), fmt
        if fmt != "e2m1":
            got = mx.layer_norm_quantize(x, w, None, fmt, eps=0.0, rms=True)
            want = ref.quantize(y, fmt)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), fmt


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 4096), (130, 1056), (3, 16416)])
def test_layer_norm_mx_quantize(mx, fmt, rows, cols):
    """MX operand of a layer norm: the scale is the power of two under amax, and every code is within half a step of
    y, or at the largest value where y lies beyond it"""
    import torch
    x, w, b, _ = make(rows, cols, 5, torch.float32)
    codes, scales, mean, rstd = mx.layer_norm_quantize(x, w, b, fmt, eps=1e-5, scaling="mx")
    want, wm, wr = ref.norm(x, w, b, 1e-5, False)
    dy = y_error(x, w, False, want, wm, wr)
    emax, top, rel, sub = {"e4m3": (8, 448.0, 2.0 ** -4, 2.0 ** -10), "e5m2": (15, 57344.0, 2.0 ** -3, 2.0 ** -17),
                           "e2m1": (2, 6.0, 2.0 ** -2, 2.0 ** -2)}[fmt]
    amax = want.abs().view(rows, -1, 32).amax(2)
    slack = dy.view(rows, -1, 32).amax(2)
    e = scales.double() - 127
    assert (torch.exp2(e + emax) <= amax + slack).all() and (torch.exp2(e + emax + 1) > amax - slack).all()
    if fmt == "e2m1":
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device="cuda", dtype=torch.float64)
        nib = torch.stack([codes & 15, codes >> 4], 2).view(rows, cols)
        v = grid[nib.long()]
    else:
        v = codes.view(ref.F8[fmt]).double()
    sc = torch.exp2(e).repeat_interleave(32, 1)
    q = (want / sc).clamp(-top, top)
    tol = rel * q.abs() * (1 + 2.0 ** -10) + sub + 2 * dy / sc
    bad = ~((v - q).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


def test_layer_norm_edges(mx):
    """constant rows, a zero row, infinities and NaN (their own rows only), a huge offset, the largest values"""
    import torch
    x, w, b, _ = make(12, 700, 3)
    x[1] = 3.0
    x[2] = 0.0
    x[3, 50] = float("inf")
    x[4, 60] = float("nan")
    x[5] = x[5] * 1e-20
    x[6] = (x[6].float() + 3.0e4).bfloat16()
    for rms in (False, True):
        y, mean, rstd = mx.layer_norm(x, w, b, eps=1e-5, rms=rms)
        want, wm, wr = ref.norm(x, w, b, 1e-5, rms)
        bad_rows = torch.zeros(12, dtype=torch.bool, device="cuda")
        bad_rows[3] = bad_rows[4] = True
        good = ~bad_rows
        tol = 2.0 ** -8 * want.abs() + y_error(x, w, rms, want, wm, wr) + 2.0 ** -134
        assert ((y.double() - want).abs() <= tol)[good].all()
        assert y[4].isnan().all() and y[3, 50].isnan()
        codes, scales, _, _ = mx.layer_norm_quantize(x, w, b, "e4m3", eps=1e-5, rms=rms)
        assert scales[:, good].isfinite().all()
        assert scales[:, 4].isnan().all() and (codes[4] == 0).all() and scales[0, 3].isnan()
    assert mx.layer_norm(x, w, b, eps=1e-5)[1][1] == 3.0


def test_layer_norm_strides_empty_and_many_rows(mx):
    import torch
    big, w, b, dyb = make(64, 900, 4)
    for off, cols, step in ((0, 640, 1), (3, 700, 2), (1, 257, 1)):
        x, dy, wt, bs = big[::step, off:off + cols], dyb[::step, off:off + cols], w[:cols].clone(), b[:cols].clone()
        n = x.shape[0]
        want, mean, rstd = mx.layer_norm(x.contiguous(), wt, bs)
        buf = torch.full((n + 2, cols + 9), 3.0, dtype=torch.bfloat16, device="cuda")
        y, m2, r2 = mx.layer_norm(x, wt, bs, out=buf[1:1 + n, 5:5 + cols])
        assert torch.equal(y, want) and torch.equal(m2, mean) and torch.equal(r2, rstd)
        buf[1:1 + n, 5:5 + cols] = 3.0
        assert (buf == 3.0).all()
        c, s, _, _ = mx.layer_norm_quantize(x.contiguous(), wt, bs)
        cb = torch.full((n + 2, cols + 9), 9, dtype=torch.uint8, device="cuda")
        sb = torch.full((s.shape[0] + 2, n + 3), 9.0, device="cuda")
        out = cb[1:1 + n, 3:3 + cols], sb[1:1 + s.shape[0], 1:1 + n]
        mx.layer_norm_quantize(x, wt, bs, out=out)
        assert torch.equal(out[0], c) and torch.equal(out[1], s)
        out[0].fill_(9), out[1].fill_(9.0)
        assert (cb == 9).all() and (sb == 9.0).all()
        dx, dw, db = mx.layer_norm_backward(dy.contiguous(), x.contiguous(), wt, mean, rstd)
        d2 = mx.layer_norm_backward(dy, x, wt, mean, rstd, out=buf[1:1 + n, 5:5 + cols])
        assert torch.equal(d2[0], dx) and torch.equal(d2[1], dw) and torch.equal(d2[2], db)
        buf[1:1 + n, 5:5 + cols] = 3.0
        assert (buf == 3.0).all()
    e = torch.empty(0, 640, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = mx.layer_norm(e, w[:640].clone())
    assert y.shape == (0, 640) and rstd.shape == (0,)
    assert mx.layer_norm_quantize(e)[1].shape == (5, 0)
    dx, dw, db = mx.layer_norm_backward(e, e, None, mean, rstd)
    assert dx.shape == (0, 640) and (dw == 0).all() and (db == 0).all()
    # more rows than a launch takes, and than it has workgroups, two kinds of kernels
    for rows, cols in ((2 ** 25 + 4000, 8), (4500001, 8), (1048600, 1032)):
        g = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
        for rms in (False, True):
            y, mean, rstd = mx.layer_norm(x, rms=rms)
            at = torch.tensor([0, 1, rows // 2, 1048575, 1048576, 1048577, rows - 1], device="cuda")
            want, wm, wr = ref.norm(x[at], None, None, 1e-5, rms)
            tol = 2.0 ** -8 * want.abs() + y_error(x[at], None, rms, want, wm, wr)
            assert ((y[at].double() - want).abs() <= tol).all()
            assert bool(y.isfinite().all())
            if cols == 8:
                c, sc, _, _ = mx.layer_norm_quantize(x, fmt="e5m2", rms=rms)
                d = (ref.values(c[at], sc[:, at], "e5m2") - want).abs()
                assert (d <= 2.0 ** -3 * want.abs() * (1 + 2.0 ** -9) + 2.0 ** -17 * sc[:, at].double().t()).all()
            dx = mx.layer_norm_backward(y, x, None, mean, rstd, rms=rms, weight_grad=False, bias_grad=False)[0]
            want = ref.norm_backward(y[at], x[at], None, None if rms else mean[at], rstd[at], rms)[0]
            err = (dx[at].double() - want).abs()
            assert (err <= 2.0 ** -8 * want.abs() + 8 * E * rstd[at].double()[:, None] * (1 + x[at].double().abs()) ** 2).all()


BWD_SHAPES = [(1, 1), (1, 4096), (2, 8), (5, 100), (17, 512), (16, 513), (33, 1000), (300, 1024), (257, 1025), (1001, 2048),
              (65, 2056), (2049, 4096), (70, 4097), (129, 8192), (20, 8200), (19, 14336), (18, 16392), (5, 32768)]


@pytest.mark.parametrize("rows,cols", BWD_SHAPES)
@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_backward(mx, rows, cols, rms):
    """dx: each of its terms and the two means over the row carry E, then half a step of bf16; the sums over
    rows are trees of chunks, at most rows / 128 + 16 + 128 terms one after another: 2^-24 of that many of the
    sum of |terms|, and the few roundings of a term"""
    import torch
    print("case", rows, cols, rms, flush=True)
    for dtype in (torch.bfloat16, torch.float32):
        x, w, b, dy = make(rows, cols, rows + cols, dtype)
        for wt in (w, None):
            _, mean, rstd = mx.layer_norm(x, wt, b, eps=1e-3, rms=rms)
            dx, dw, db = mx.layer_norm_backward(dy, x, wt, mean, rstd, rms=rms)
            wx, ww, wb = ref.norm_backward(dy, x, wt, mean, rstd, rms)
            v, d, r = x.double(), dy.double(), rstd.double()[:, None]
            off = v.abs() + (0 if rms else mean.double().abs()[:, None])
            xh = off * r
            g = d.abs() if wt is None else d.abs() * wt.double().abs()
            tol = 2.0 ** -8 * wx.abs() + 2.0 ** -134
            tol = tol + 2 * E * r * (g + g.mean(1, keepdim=True) + xh * (g * xh).mean(1, keepdim=True))
            bad = ~((dx.double() - wx).abs() <= tol)
            assert not bad.any(), ("dx", int(bad.sum()), bad.nonzero()[0].tolist())
            n = (rows / 128 + 16 + 128 + 8) * 2.0 ** -24
            assert ((dw.double() - ww).abs() <= n * (d.abs() * xh).sum(0)).all(), "dweight"
            assert ((db.double() - wb).abs() <= n * d.abs().sum(0)).all(), "dbias"
    one = mx.layer_norm_backward(dy, x, wt, mean, rstd, rms=rms, bias_grad=False)
    assert torch.equal(one[0], dx) and torch.equal(one[1], dw) and one[2] is None
    one = mx.layer_norm_backward(dy, x, wt, mean, rstd, rms=rms, weight_grad=False)
    assert torch.equal(one[0], dx) and one[1] is None and torch.equal(one[2], db)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("cols", [640, 1000, 2048, 4096, 8192, 16384])
def test_norm_large_equals_its_parts(mx, cols, rms):
    """input above the size from which it is read past the cache: rows equal those of smaller calls, the gradients of
    the parameters are within the rounding of their sums"""
    import torch
    rows = 2 ** 26 // cols + 600
    x, w, b, dy = make(rows, cols, 2)
    cut = rows // 2
    for call in (lambda t: mx.layer_norm(t, w, b, rms=rms), lambda t: mx.layer_norm_quantize(t, w, b, rms=rms),
                 lambda t: mx.layer_norm_quantize(t[:, :cols // 32 * 32], fmt="e2m1", scaling="mx", rms=rms)):
        all_, p, q = call(x), call(x[:cut]), call(x[cut:])
        for a, u, v in zip(all_, p, q):
            if a is not None:
                d = 1 if a.dim() == 2 and a.shape[0] != rows else 0
                assert torch.equal(a, torch.cat([u, v], d))
    _, mean, rstd = mx.layer_norm(x, w, b, rms=rms)
    dx, dw, db = mx.layer_norm_backward(dy, x, w, mean, rstd, rms=rms)
    m = lambda a, c: None if rms else mean[a:c]
    dx1 = mx.layer_norm_backward(dy[:cut], x[:cut], w, m(0, cut), rstd[:cut], rms=rms)[0]
    dx2 = mx.layer_norm_backward(dy[cut:], x[cut:], w, m(cut, rows), rstd[cut:], rms=rms, weight_grad=False, bias_grad=False)[0]
    assert torch.equal(dx, torch.cat([dx1, dx2]))
    wx, ww, wb = ref.norm_backward(dy, x, w, mean, rstd, rms)
    d = dy.double().abs()
    xh = (x.double().abs() + (0 if rms else mean.double().abs()[:, None])) * rstd.double()[:, None]
    n = (rows / 256 + 16 + 256 + 8) * 2.0 ** -24   # rows of a chunk, then at most 256 chunks, one after another
    assert ((dw.double() - ww).abs() <= n * (d * xh).sum(0)).all() and ((db.double() - wb).abs() <= n * d.sum(0)).all()


def test_norm_repeats_bits_on_streams_and_in_graphs(mx):
    """the same bits from other streams at once (each call has its own workspace), and replayed from two graphs
    between eager calls"""
    import torch
    for rows, cols in ((1, 4096), (777, 4096), (300, 600)):
        x, w, b, dy = make(rows, cols, 1)
        x2, _, _, dy2 = make(rows, cols, 2)
        def step(x_, dy_, s=None):
            c, sc, mean, rstd = mx.layer_norm_quantize(x_, w, b, stream=s)
            return (c, sc, mean, rstd) + mx.layer_norm_backward(dy_, x_, w, mean, rstd, stream=s)
        want, want2 = step(x, dy), step(x2, dy2)
        same = lambda a, c: all(torch.equal(p, q) for p, q in zip(a, c))
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = [step(x, dy, s1), step(x2, dy2, s2.cuda_stream), step(x, dy, s1)]
        torch.cuda.synchronize()
        assert same(got[0], want) and same(got[1], want2) and same(got[2], want)
        graphs = []
        for xx, dd in ((x, dy), (x2, dy2)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = step(xx, dd)
            graphs.append((g, out))
        for i in range(3):
            for (g, out), wnt in zip(graphs, (want, want2)):
                for t in out:
                    t.zero_()
                g.replay()
                torch.cuda.synchronize()
                assert same(out, wnt)
                assert same(step(x2, dy2), want2)


def test_norm_refuses(mx):
    import torch
    x, w, b, dy = make(4, 256, 1)
    _, mean, rstd = mx.layer_norm(x, w, b)
    for call in (lambda: mx.layer_norm(x, w.float(), b), lambda: mx.layer_norm(x, w[:255], b),
                 lambda: mx.layer_norm(x, w.half(), None), lambda: mx.layer_norm(x.float(), w, b),
                 lambda: mx.layer_norm(x, w, b.cpu()), lambda: mx.layer_norm(x.t(), None, None),
                 lambda: mx.layer_norm(x, w.repeat(2)[::2], b),
                 lambda: mx.layer_norm(x, w, b, out=torch.empty(4, 256, device="cuda")),
                 lambda: mx.layer_norm_quantize(x, w, b, "e2m1"), lambda: mx.layer_norm_quantize(x, w, b, scaling="tensor"),
                 lambda: mx.layer_norm_backward(dy[:3], x, w, mean, rstd), lambda: mx.layer_norm_backward(dy, x, w, None, rstd),
                 lambda: mx.layer_norm_backward(dy, x, w, mean[:3], rstd), lambda: mx.layer_norm_backward(dy, x, w, mean, rstd.double())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mx.layer_norm(x, w, b, eps=-1.0), lambda: mx.layer_norm(x, w, b, eps=float("nan")),
                 lambda: mx.layer_norm(x, w, b, out=x), lambda: mx.layer_norm_quantize(x[:, :40], scaling="mx"),
                 lambda: mx.layer_norm(torch.zeros(1, 40000, dtype=torch.bfloat16, device="cuda")),
                 lambda: mx.layer_norm_backward(dy, x, w, mean, rstd, out=dy)):
        with pytest.raises(mx.MXError):
            call()


@pytest.mark.parametrize("tokens", [1, 77, 1000])
def test_layer_forward_and_backward(mx, tokens):
    """one linear layer behind its norm as a training step runs it: norm to operand, Fprop, both forms of dY from one
    read, Dgrad, Wgrad, norm backward; every product against the float64 product of its own operands, and the whole
    against the layer in float64 with the 8-bit roundings' error: an operand's elements are off by up to 2^-4 (E4M3)
    or 2^-3 (E5M2) of themselves, independently, so a product's 2-norm is off by less than the sum of the two
    operands' relative 2-norm errors"""
    import torch
    hidden, width = 640, 384
    x, gamma, beta, _ = make(tokens, hidden, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    w = (0.05 * torch.randn(width, hidden, device="cuda", generator=g)).bfloat16()
    dy = (1e-3 * torch.randn(tokens, width, device="cuda", generator=g)).bfloat16()
    cw, sw, cwt, swt = mx.block_quantize_dual(w, "e4m3", "e4m3", tile=True)
    cn, sn, mean, rstd = mx.layer_norm_quantize(x, gamma, beta)
    y = mx.block_gemm(cn, sn, "e4m3", cw, sw, "e4m3")
    cd, sd, cdt, sdt = mx.block_quantize_dual(dy, "e5m2", "e5m2")
    dn = mx.block_gemm(cd, sd, "e5m2", cwt, swt, "e4m3")
    n = mx.layer_norm(x, gamma, beta)[0]
    cnt, snt = mx.block_quantize(n, "e4m3", "transpose")
    dw = mx.block_gemm(cdt, sdt, "e5m2", cnt, snt, "e4m3", out_dtype=torch.float32)
    dx, dgamma, dbeta = mx.layer_norm_backward(dn, x, gamma, mean, rstd)
    def near(got, a, fa, b, fb, tile):
        C, S = ref.gemm(a, fa, b, fb, tile)
        tol = 1e-5 * S if got.dtype == torch.float32 else 2.0 ** -8 * (C.abs() + S)
        assert ((got.double() - C).abs() <= tol).all()
    near(y, (cn, sn), "e4m3", (cw, sw), "e4m3", True)
    near(dn, (cd, sd), "e5m2", (cwt, swt), "e4m3", True)
    near(dw, (cdt, sdt), "e5m2", (cnt, snt), "e4m3", False)
    n64 = ref.norm(x, gamma, beta, 1e-5, False)[0]
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    dn64 = dy.double() @ w.double()
    dx64, dg64, db64 = ref.norm_backward(dn64, x, gamma, mean, rstd, False)
    assert rel(y, n64 @ w.double().t()) <= 2 * 2.0 ** -4
    assert rel(dn, dn64) <= 2.0 ** -3 + 2.0 ** -4
    assert rel(dw, dy.double().t() @ n64) <= 2.0 ** -3 + 2.0 ** -4
    assert rel(dx, dx64) <= 0.25 and rel(dgamma, dg64) <= 0.25 and rel(dbeta, db64) <= 0.25
