"""The norm on rows that a rounding of the mean shows up in, and its backward pass beside large means."""
import pytest

import block_reference as ref

pytestmark = pytest.mark.gpu
E = 2.0 ** -18   # test_gpu_norm.py: fp32 sums of a row and the few roundings after them


@pytest.fixture(scope="module")
def mx():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_block_amax_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("cols", [1, 100, 513, 896, 1000, 1792, 3584, 4096, 7168, 14336, 16392, 28672, 32768])
def test_constant_rows(mx, cols):
    """every bf16 significand, repeated: the fp32 sum of up to 2^15 equal numbers of 8 bits is exact in any order, so
    the mean is the number itself, every x - mean is 0 and y is the bias, in every output form; with eps = 0 rstd is
    Inf and y NaN"""
    import torch
    print("case", cols, flush=True)
    sig = torch.arange(128, 256, device="cuda").double()
    x = torch.cat([sig * 2.0 ** -7, -sig * 2.0 ** 6, sig * 2.0 ** -40]).bfloat16()[:, None].repeat(1, cols)
    g = torch.Generator(device="cuda").manual_seed(cols)
    w, b = ((torch.randn(cols, device="cuda", generator=g)).bfloat16() for _ in range(2))
    y, mean, rstd = mx.layer_norm(x, w, b, eps=1e-5)
    assert torch.equal(mean, x[:, 0].float())
    assert ((rstd.double() * 1e-5 ** 0.5 - 1).abs() <= 2.0 ** -22).all()
    assert torch.equal(y, b.expand_as(y))
    want = ref.quantize(b[None], "e4m3")
    codes, scales, mean, _ = mx.layer_norm_quantize(x, w, b, "e4m3", eps=1e-5)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(codes, want[0].expand_as(codes)) and torch.equal(scales, want[1].expand_as(scales))
    if cols % 32 == 0:
        want = mx.quantize(b[None].contiguous(), "e2m1")
        codes, scales, _, _ = mx.layer_norm_quantize(x, w, b, "e2m1", eps=1e-5, scaling="mx")
        assert torch.equal(codes, want[0].expand_as(codes)) and torch.equal(scales, want[1].expand_as(scales))
    y, mean, rstd = mx.layer_norm(x, w, b, eps=0.0)
    assert torch.equal(mean, x[:, 0].float()) and (rstd == float("inf")).all() and y.isnan().all()


@pytest.mark.parametrize("cols", [1, 7, 100, 513, 1000, 4096, 7168, 16392])
def test_mean_is_the_rounded_quotient(mx, cols):
    """rows of small whole numbers: the sum is exact in any order, and the mean is its quotient rounded to fp32 once;
    a row with an Inf has that mean, and one whose sum leaves fp32 an infinite one"""
    import torch
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randint(-255, 256, (300, cols), device="cuda", generator=g).bfloat16()
    want = (x.double().sum(1) / cols).float()   # a quotient of 24 bits by 15 rounded to 53 first: no double rounding
    x[7, cols // 2] = float("inf")
    x[8, 0] = -float("inf")
    x[9] = 3e38
    want[7], want[8], want[9] = float("inf"), -float("inf"), float("inf") if cols > 1 else x[9, 0].float()
    mean = mx.layer_norm(x)[1]
    assert torch.equal(mean, want)


@pytest.mark.parametrize("rows,cols", [(9, 100), (300, 513), (33, 1000), (300, 1024), (11, 2056), (65, 4096), (3, 8200), (5, 16392)])
@pytest.mark.parametrize("params", [True, False])
def test_backward_beside_a_large_mean(mx, rows, cols, params):
    """constant rows of 1e33 between ordinary ones, eps = 1e-12: mean * rstd is beyond fp32, but x - mean is 0 in every
    column, and nothing of it reaches dx, the parameters' sums or other rows.  Each term carries the roundings of
    E's derivation, relative to itself; the sums over rows those of test_gpu_norm.py"""
    import torch
    print("case", rows, cols, params, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    x, w, dy = r(rows, cols).bfloat16(), (1 + 0.3 * r(cols)).bfloat16(), (1e-2 * r(rows, cols)).bfloat16()
    x[0::4], x[2::4] = 1e33, -1e33
    _, mean, rstd = mx.layer_norm(x, w, eps=1e-12)
    assert torch.equal(mean[0::2], x[0::2, 0].float()) and bool((rstd * mean)[0::2].isinf().all())
    dx, dw, db = mx.layer_norm_backward(dy, x, w, mean, rstd, weight_grad=params, bias_grad=params)
    wx, ww, wb = ref.norm_backward(dy, x, w, mean, rstd, False)
    d, k = dy.double().abs(), rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]).abs() * k
    t = d * w.double().abs()
    tol = 2.0 ** -8 * wx.abs() + 2.0 ** -134 + 2 * E * k * (t + t.mean(1, keepdim=True) + xh * (t * xh).mean(1, keepdim=True))
    assert ((dx.double() - wx).abs() <= tol).all()
    if params:
        n = (rows / 128 + 16 + 128 + 8) * 2.0 ** -24
        assert ((dw.double() - ww).abs() <= n * (d * xh).sum(0)).all() and ((db.double() - wb).abs() <= n * d.sum(0)).all()


def test_single_column_of_any_stride(mx):
    """rows of one element are contiguous whatever the stride of that dimension says"""
    import torch
    x = torch.randn(1, 300, device="cuda").bfloat16()
    col = x.t()
    assert col.shape == (300, 1) and col.stride(1) == 300
    for mode in ("row", "transpose", "tile", "tile_transpose"):
        got, want = mx.block_quantize(col, "e4m3", mode), ref.quantize(col, "e4m3", mode)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    y, mean, rstd = mx.layer_norm(col, eps=1.0)
    assert (y == 0).all() and torch.equal(mean, x[0].float()) and (rstd == 1).all()
    dx, dw, db = mx.layer_norm_backward(col, col, None, mean, rstd)
    assert (dx == 0).all() and (dw == 0).all()
