"""Outputs of the block-128 and norm calls in the gaps between the rows of their inputs or of each other: the same
values as in buffers of their own, and every other byte as it was."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_block_amax_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("rows,cols", [(2, 5), (70, 257), (300, 640), (1100, 4096)])
@pytest.mark.parametrize("y_first", [False, True])
def test_norm_within_one_buffer(mx, rows, cols, y_first):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows)
    buf = torch.randn(rows, 2 * cols + 6, device="cuda", generator=g).bfloat16()
    dy = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
    x0, y0 = (cols + 3, 1) if y_first else (1, cols + 3)
    x, y = buf[:, x0:x0 + cols], buf[:, y0:y0 + cols]
    keep = buf.clone()
    want, mean, rstd = mx.layer_norm(x.contiguous())
    got, m2, r2 = mx.layer_norm(x, out=y)
    assert got.data_ptr() == y.data_ptr() and torch.equal(y, want) and torch.equal(m2, mean) and torch.equal(r2, rstd)
    wx, ww, wb = mx.layer_norm_backward(dy, x.contiguous(), None, mean, rstd)
    dx, dw, db = mx.layer_norm_backward(dy, x, None, mean, rstd, out=y)
    assert torch.equal(y, wx) and torch.equal(dw, ww) and torch.equal(db, wb)
    want = mx.layer_norm_quantize(x.contiguous())
    codes = buf.view(torch.uint8)[:, 2 * y0:2 * y0 + cols]
    scales = torch.empty_like(want[1])
    mx.layer_norm_quantize(x, out=(codes, scales))
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    y.copy_(keep[:, y0:y0 + cols])
    assert torch.equal(buf, keep)


@pytest.mark.parametrize("rows,cols", [(256, 384), (300, 300), (1000, 520)])
def test_both_forms_within_one_buffer(mx, rows, cols):
    """a square's two forms side by side, and a form's codes beside the rows that they were made from"""
    import torch
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
    want = mx.block_quantize_dual(x, "e4m3", "e5m2")
    buf = torch.full((max(rows, cols), rows + cols + 5), 0xA5, dtype=torch.uint8, device="cuda")
    c, ct = buf[:rows, 2:2 + cols], buf[:cols, cols + 4:cols + 4 + rows]
    s, st = torch.empty_like(want[1]), torch.empty_like(want[3])
    mx.block_quantize_dual(x, "e4m3", "e5m2", out=(c, s, ct, st))
    for got, w in zip((c, s, ct, st), want):
        assert torch.equal(got, w)
    c.fill_(0xA5), ct.fill_(0xA5)
    assert (buf == 0xA5).all()
    buf = torch.zeros(rows, 2 * cols, dtype=torch.bfloat16, device="cuda")
    buf[:, :cols] = x
    c = buf.view(torch.uint8)[:, 2 * cols:3 * cols]
    mx.block_quantize(buf[:, :cols], "e4m3", out=(c, s))
    assert torch.equal(c, want[0]) and torch.equal(s, want[1]) and torch.equal(buf[:, :cols], x)


@pytest.mark.parametrize("M,N,K", [(40, 64, 300), (300, 256, 640), (1200, 1160, 301), (4200, 4100, 272)])
@pytest.mark.parametrize("bf16", [True, False])
def test_product_beside_its_operand(mx, M, N, K, bf16):
    """C in the gaps between the rows of A's codes, straight after each row's last byte or 16"""
    import torch
    g = torch.Generator(device="cuda").manual_seed(K)
    r = lambda n: torch.randn(n, K, device="cuda", generator=g).bfloat16()
    a, b = mx.block_quantize(r(M), "e4m3"), mx.block_quantize(r(N), "e4m3", "tile")
    dt, size = (torch.bfloat16, 2) if bf16 else (torch.float32, 4)
    want = mx.block_gemm(*a, "e4m3", *b, "e4m3", out_dtype=dt)
    for k0 in (-(-K // size) * size, -(-K // 16) * 16):
        buf = torch.full((M, -(-(k0 + N * size) // 16) * 16), 0x7F, dtype=torch.uint8, device="cuda")
        codes, c = buf[:, :K], buf.view(dt)[:, k0 // size:k0 // size + N]
        codes.copy_(a[0])
        mx.block_gemm(codes, a[1], "e4m3", *b, "e4m3", out_dtype=dt, out=c)
        assert torch.equal(c, want) and torch.equal(codes, a[0])
