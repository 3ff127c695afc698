"""Calls by group and on heads whose operands are views: weights that all groups share, ends, positions and weights that
start anywhere, outputs within wider buffers, one stream beside another.  Tolerances as in test_gpu_grouped and
test_gpu_rope."""
import pytest

import block_reference as ref
import group_reference as grp
import head_reference as head
from test_gpu_grouped import check, data, ends_of, mx, weights  # noqa: F401 (mx is a fixture)
from test_gpu_rope import close
from test_gpu_rope import data as heads

pytestmark = pytest.mark.gpu
SIZES = [3, 0, 140, 1, 64, 200]


def part(t, ahead):
    """the same values `ahead` elements into a buffer"""
    import torch
    buf = torch.zeros(t.numel() + ahead, dtype=t.dtype, device=t.device)
    buf[ahead:] = t.flatten()
    return buf[ahead:].view(t.shape)


@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("N,K", [(260, 384), (40, 200), (1, 17), (520, 16), (130, 31)])
def test_shared_weights(mx, tile, N, K):
    """one weight for all groups: a step of 0 from one to the next"""
    import torch
    ends = part(ends_of(SIZES), 1)
    a = mx.block_quantize(data(408, K, seed=91), "e4m3")
    w = weights(mx, 1, N, K, "e4m3", tile, 92)
    b = (w[0].expand(6, -1, -1), w[1].expand(6, -1, -1))
    C, S = grp.gemm(a, "e4m3", b, "e4m3", ends.tolist(), tile)
    one = (w[0][0], w[1][0])
    for dtype, full in ((torch.bfloat16, False), (torch.float32, True)):
        c = mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends, out_dtype=dtype, full_sums=full)
        check(c, C, S, ref.cdiv(K, 128), full)
        check(mx.block_gemm(*a, "e4m3", *one, "e4m3", out_dtype=dtype), *ref.gemm(a, "e4m3", one, "e4m3", tile), ref.cdiv(K, 128), full)


@pytest.mark.parametrize("N", [64, 129, 300])
@pytest.mark.parametrize("ahead,wider", [(0, 0), (1, 1), (8, 8), (3, 4)])
@pytest.mark.parametrize("dtype,full", [("float32", True), ("bfloat16", True), ("bfloat16", False)])
def test_outputs_in_wider_buffers(mx, N, ahead, wider, dtype, full):
    """what lies beside C, and its rows of no group, is left as it was; any alignment of rows"""
    import torch
    ends, dtype = ends_of(SIZES), getattr(torch, dtype)
    a, b = mx.block_quantize(data(413, 256, seed=93), "e4m3"), weights(mx, 6, N, 256, "e4m3", True, 94)
    C, S = grp.gemm(a, "e4m3", b, "e4m3", ends.tolist(), True)
    buf = torch.full((413, ahead + N + wider), 7.0, dtype=dtype, device="cuda")
    c = buf[:, ahead:ahead + N]
    mx.block_gemm_grouped(*a, "e4m3", *b, "e4m3", ends, out_dtype=dtype, full_sums=full, out=c)
    check(c[:408], C[:408], S[:408], 2, full)
    assert (c[408:] == 7).all() and (buf[:, :ahead] == 7).all() and (buf[:, ahead + N:] == 7).all()
    q = mx.block_quantize_grouped(data(413, 70, seed=95), ends, "e5m2"), mx.block_quantize_grouped(data(413, N, seed=96), ends, "e4m3")
    C, S = grp.gemm_k(q[0], "e5m2", q[1], "e4m3", ends.tolist())
    buf = torch.full((6, 73, ahead + N + wider), 7.0, dtype=dtype, device="cuda")
    c = buf[:, 1:71, ahead:ahead + N]
    mx.block_gemm_grouped_k(*q[0], "e5m2", *q[1], "e4m3", ends, out_dtype=dtype, full_sums=full, out=c)
    check(c, C, S, 2, full)
    assert (buf[:, 0] == 7).all() and (buf[:, 71:] == 7).all() and (buf[:, :, :ahead] == 7).all() and (buf[:, :, ahead + N:] == 7).all()


@pytest.mark.parametrize("dim,rot,layout", [(128, 128, "half"), (120, 40, "interleaved"), (100, 20, "half"), (100, 50, "interleaved"), (65, 64, "half")])
@pytest.mark.parametrize("ptype", ["int32", "int64"])
def test_views_of_positions_and_weights(mx, dim, rot, layout, ptype):
    import torch
    q, k, w, pos, f, (dq, dk) = heads(37, 5, 2, dim, 97, rot, first=-60)
    pos, f = part(pos.to(getattr(torch, ptype)), 1), part(f, 1)
    for wq, wk in ((part(w[0], 1), part(w[1], 3)), (part(w[0].float(), 1), None)):
        y = mx.qk_norm_rope(q, k, wq, wk, pos, f, eps=1e-6, layout=layout, scale=-0.5)
        g = mx.qk_norm_rope_backward(part(dq, 1), dk, q, k, wq, wk, pos, f, eps=1e-6, layout=layout, scale=-0.5)
        for x, d, wt, out, dx, dw in zip((q, k), (dq, dk), (wq, wk), y, g[:2], g[2:]):
            close(out, *head.norm_rope(x, wt, pos, f, 1e-6, layout, -0.5))
            want, wantw, mag, magw = head.norm_rope_backward(d, x, wt, pos, f, 1e-6, layout, -0.5)
            close(dx, want, mag)
            assert ((dw.double() - wantw).abs() <= 2.0 ** -15 * magw).all()
    y, _ = mx.rope(q, None, pos, f, layout=layout, scale=0.0)
    assert (y[..., :rot] == 0).all() and torch.equal(y[..., rot:], q[..., rot:])


def test_streams_side_by_side(mx):
    """the same calls on two streams at once, other inputs on each: none meets the other's memory"""
    import torch
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for i in range(2):
        q, k, w, pos, f, g = heads(3000, 6, 2, 128, 98 + i, 128)
        sizes = [1000 * (i + 1), 0, 700, 1300 - 900 * i]
        x = data(3000, 512, seed=100 + i)
        sets.append((q, k, w, pos, f, g, ends_of(sizes), x, weights(mx, 4, 384, 512, "e4m3", True, 102 + i)))

    def step(s, stream):
        q, k, w, pos, f, (dq, dk), ends, x, b = s
        out = mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f, stream=stream)
        r = mx.block_quantize_grouped_dual(x, ends, "e4m3", "e5m2", stream=stream)
        c = mx.block_gemm_grouped(r[0], r[1], "e4m3", *b, "e4m3", ends, stream=stream)
        d = mx.block_gemm_grouped_k(r[2], r[3], "e5m2", r[2], r[3], "e5m2", ends, stream=stream, rows=3000)
        n = int(ends[-1])
        return [*out, c[:n], d]

    want = [step(s, None) for s in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [step(s, t) for s, t in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
