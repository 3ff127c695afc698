"""Rotary positions and the norm of each head on the GPU against their definitions in float64 (head_reference).

Tolerances.  An angle is off by 2^-21 at most (and by p f 2^-51 for position p, in both sides' fp64), its cosine and
sine by two roundings more, the rotation by three: 2^-19 of the magnitudes that meet in an element, scale * (|a| + |b|).
Sums over a head are 16 terms in a row and a tree of six steps at most: 2^-18 of their terms with what surrounds them.
So 2^-17 of the magnitudes covers y and dx before their rounding, which adds half a step, 2^-8 of the value (2^-134
below bf16's normal range).  A weight's sum takes one term for each pass of a wave's tokens in a row (below 300 in these
tests) and about 70 in trees: 2^-15 of its terms."""
import pytest

import head_reference as ref

pytestmark = pytest.mark.gpu
E = 2.0 ** -17


@pytest.fixture(scope="module")
def mx():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import precision_block_amax_amd as m
    m.lib()
    return m


def close(got, want, mag, angle=0.0):
    tol = 2.0 ** -8 * want.abs() * (1 + E) + (E + angle) * mag + 2.0 ** -134
    err = (got.double() - want).abs()
    assert (err <= tol).all(), "off by %g of the tolerance" % (err / tol).max().item()


def data(tokens, hq, hk, dim, seed, rot, first=0, pos64=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    qkv = (r(tokens, hq + 2 * hk, dim) * (1 + r(tokens, 1, 1).abs())).bfloat16()
    w = [(1 + 0.3 * r(dim)).bfloat16() for _ in range(2)]
    pos = (first + torch.randint(0, 4 * tokens, (tokens,), device="cuda", generator=g)).to(torch.int64 if pos64 else torch.int32)
    f = 500000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / max(rot, 1))
    grads = [(1e-2 * r(tokens, h, dim)).bfloat16() for h in (hq, hk)]
    return qkv[:, :hq], qkv[:, hq:hq + hk], w, pos, f, grads


# tokens, query heads, key heads, dim, rot
SHAPES = [(1, 1, 1, 2, 2), (1, 32, 8, 128, 128), (3, 6, 1, 64, 64), (5, 3, 2, 40, 40), (4, 5, 5, 40, 20), (7, 2, 0, 80, 80),
          (2, 9, 2, 80, 20), (6, 4, 1, 96, 48), (3, 7, 3, 96, 24), (2, 4, 4, 128, 64), (5, 3, 2, 128, 0), (3, 5, 1, 256, 64),
          (2, 3, 2, 512, 512), (2, 3, 1, 320, 64), (3, 2, 1, 100, 50), (2, 2, 2, 65, 64), (1, 1, 1, 1, 0), (4, 3, 1, 16, 16),
          (2, 1, 1, 511, 510), (3, 2, 2, 250, 0), (300, 16, 4, 128, 128), (1000, 3, 1, 64, 32), (17, 33, 9, 192, 192),
          (5, 2, 1, 24, 8), (3, 300, 2, 48, 16)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", SHAPES)
def test_rope(mx, tokens, hq, hk, dim, rot, layout):
    import torch
    q, k, _, pos, f, _ = data(tokens, hq, hk, dim, 1, rot)
    for inverse, scale in ((False, 1.0), (True, 1.25)):
        out = mx.rope(q, k, pos, f, layout=layout, scale=scale, inverse=inverse)
        for x, y in zip((q, k), out):
            want, mag = ref.rotate(x, pos, f, layout, scale, inverse)
            assert torch.equal(y[..., rot:], x[..., rot:])
            close(y, want, mag)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", SHAPES)
def test_norm(mx, tokens, hq, hk, dim, rot, layout):
    import torch
    q, k, w, pos, f, _ = data(tokens, hq, hk, dim, 2, rot, pos64=False)
    for ws in (w, [None, None], [w[0].float(), None]):
        out = mx.qk_norm_rope(q, k, *ws, pos, f, eps=1e-6, layout=layout, scale=0.75)
        for x, wt, y in zip((q, k), ws, out):
            close(y, *ref.norm_rope(x, wt, pos, f, 1e-6, layout, 0.75))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", SHAPES)
def test_backward(mx, tokens, hq, hk, dim, rot, layout):
    import torch
    q, k, w, pos, f, (dq, dk) = data(tokens, hq, hk, dim, 3, rot)
    for ws in (w, [None, w[1].float()]):
        out = mx.qk_norm_rope_backward(dq, dk, q, k, *ws, pos, f, eps=1e-6, layout=layout, scale=1.5)
        for x, d, wt, dx, dw in zip((q, k), (dq, dk), ws, out[:2], out[2:]):
            want, wantw, mag, magw = ref.norm_rope_backward(d, x, wt, pos, f, 1e-6, layout, 1.5)
            close(dx, want, mag)
            assert ((dw.double() - wantw).abs() <= 2.0 ** -15 * magw).all()
        again = mx.qk_norm_rope_backward(dq, dk, q, k, *ws, pos, f, eps=1e-6, layout=layout, scale=1.5)
        assert all(torch.equal(a, b) for a, b in zip(out, again))
    assert mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f, weight_grad=False)[2:] == (None, None)


# more than 2^25 elements, which go past the caches: a size of head for every width of load, and below it the one that
# the other tests have no head for
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hk,dim,rot,n", [(8, 2, 64, 64, 1 << 25), (7, 2, 128, 96, 1 << 25), (3, 2, 256, 64, 1 << 25),
                                             (3, 1, 512, 512, 1 << 25), (9, 3, 72, 24, 1 << 25), (5, 4, 36, 12, 1 << 25),
                                             (6, 1, 100, 20, 1 << 25), (3, 2, 148, 20, 1 << 25), (4, 3, 50, 26, 1 << 25),
                                             (3, 2, 148, 20, 4000)])
def test_large(mx, hq, hk, dim, rot, n, layout):
    import torch
    tokens = n // ((hq + hk) * dim) + 3
    q, k, w, pos, f, (dq, dk) = data(tokens, hq, hk, dim, 14, rot)
    out = mx.rope(q, k, pos, f, layout=layout)
    for x, y in zip((q, k), out):
        assert torch.equal(y[..., rot:], x[..., rot:])
        close(y, *ref.rotate(x, pos, f, layout))
    out = mx.qk_norm_rope(q, k, *w, pos, f, eps=1e-6, layout=layout)
    for x, wt, y in zip((q, k), w, out):
        close(y, *ref.norm_rope(x, wt, pos, f, 1e-6, layout))
    out = mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f, eps=1e-6, layout=layout)
    for x, d, wt, dx, dw in zip((q, k), (dq, dk), w, out[:2], out[2:]):
        want, wantw, mag, magw = ref.norm_rope_backward(d, x, wt, pos, f, 1e-6, layout)
        close(dx, want, mag)
        assert ((dw.double() - wantw).abs() <= 2.0 ** -15 * magw).all()


def test_gradient_is_the_difference(mx):
    """dx and dweight along a direction against differences of the definition's forward pass"""
    import torch
    q, k, w, pos, f, (dq, dk) = data(40, 4, 2, 64, 4, 64)
    dxq, _, dwq, _ = mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f, eps=1e-6)
    g = torch.Generator(device="cuda").manual_seed(5)
    v = torch.randn(q.shape, device="cuda", generator=g).double()
    vw = torch.randn(64, device="cuda", generator=g).double()
    value = lambda x, wt: (ref.norm_rope(x, wt, pos, f, 1e-6, "half")[0] * dq.double()).sum()
    h = 2.0 ** -12
    _, _, mag, magw = ref.norm_rope_backward(dq, q, w[0], pos, f, 1e-6, "half")
    # central differences are off by h^2 / 6 of the third derivative, which is below 100 times the magnitudes here
    slope = (value(q.double() + h * v, w[0]) - value(q.double() - h * v, w[0])) / (2 * h)
    tol = ((2.0 ** -8 + E + 100 * h * h) * mag * v.abs() * (1 + v.abs()) ** 2).sum()
    assert (slope - (dxq.double() * v).sum()).abs() <= tol
    slope = (value(q, w[0].double() + h * vw) - value(q, w[0].double() - h * vw)) / (2 * h)
    assert (slope - (dwq.double() * vw).sum()).abs() <= ((2.0 ** -15 + h * h) * magw * vw.abs()).sum()


@pytest.mark.parametrize("first,pos64", [(-100000, True), (131072, False), (2 ** 31 - 5000, False), (2 ** 40, True)])
def test_far_positions(mx, first, pos64):
    q, k, w, pos, f, _ = data(9, 4, 2, 128, 6, 128, first, pos64)
    # both sides' angles are fp64 products, off by p f 2^-51
    slack = float(max(abs(first), 1)) * 2.0 ** -50
    for x, y in zip((q, k), mx.rope(q, k, pos, f)):
        close(y, *ref.rotate(x, pos, f, "half"), angle=slack)
    for x, wt, y in zip((q, k), w, mx.qk_norm_rope(q, k, *w, pos, f)):
        close(y, *ref.norm_rope(x, wt, pos, f, 1e-5, "half"), angle=slack)


def test_position_zero_is_exact(mx):
    import torch
    q, k, _, _, f, _ = data(5, 3, 2, 128, 7, 128)
    zero = torch.zeros(5, dtype=torch.int64, device="cuda")
    oq, ok = mx.rope(q, k, zero, f)
    assert torch.equal(oq, q) and torch.equal(ok, k)


@pytest.mark.parametrize("dim,rot", [(128, 64), (40, 20), (96, 24)])
def test_special_values(mx, dim, rot):
    """Inf and NaN stay within their head, and out of the rotated part where they lie behind it; heads of zeros"""
    import torch
    q, k, w, pos, f, (dq, dk) = data(6, 4, 2, dim, 8, rot)
    x = q.clone()
    x[1, 2, rot + 1] = float("inf")
    x[3, 0, rot + 2] = float("nan")
    x[4, 1] = 0
    y, _ = mx.rope(x, None, pos, f)
    want, mag = ref.rotate(x, pos, f, "half")
    fine = torch.isfinite(mag)
    assert torch.equal(y[..., rot:].view(torch.int16), x[..., rot:].view(torch.int16))
    close(y[fine], want[fine], mag[fine])
    y, _ = mx.qk_norm_rope(x, None, w[0], None, pos, f)
    good = torch.isfinite(x).all(-1)
    want, mag = ref.norm_rope(x, w[0], pos, f, 1e-5, "half")
    close(y[good], want[good], mag[good])
    assert not torch.isfinite(y[3, 0]).any() and (y[4, 1] == 0).all()
    assert torch.isnan(mx.qk_norm_rope(x, None, w[0], None, pos, f, eps=0.0)[0][4, 1]).all()
    dx, _, dw, _ = mx.qk_norm_rope_backward(dq, None, x, None, w[0], None, pos, f)
    want, _, mag, _ = ref.norm_rope_backward(dq, x, w[0], pos, f, 1e-5, "half")
    close(dx[good], want[good], mag[good])
    assert torch.isnan(dw).all()


def test_strides(mx):
    """heads outermost, unaligned starts, outputs within wider rows: what lies between is left alone"""
    import torch
    q, k, w, pos, f, (dq, dk) = data(11, 4, 2, 64, 9, 64)
    want = mx.qk_norm_rope(q, k, *w, pos, f)
    outer = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    flat = torch.empty(11 * 4 * 64 + 3, dtype=torch.bfloat16, device="cuda")
    odd = flat[3:].view(11, 4, 64)
    odd.copy_(q)
    for a, b in ((outer(q), outer(k)), (odd, k)):
        out = mx.qk_norm_rope(a, b, *w, pos, f)
        assert all(torch.equal(s, t) for s, t in zip(out, want))
    buf = torch.full((11, 7, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    out = (buf[:, :4, 1:65], buf[:, 4:6, 3:67])
    mx.qk_norm_rope(q, k, *w, pos, f, out=out)
    assert all(torch.equal(s, t) for s, t in zip(out, want))
    left = torch.ones_like(buf, dtype=torch.bool)
    left[:, :4, 1:65] = left[:, 4:6, 3:67] = False
    assert (buf[left] == 5).all()
    want = mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f)
    out = mx.qk_norm_rope_backward(outer(dq), dk, odd, outer(k), *w, pos, f,
                                   out=(outer(torch.empty_like(dq)), torch.empty_like(dk)))
    assert all(torch.equal(s, t) for s, t in zip(out, want))
    with pytest.raises(mx.MXError):
        mx.rope(q, None, pos, f, out=(q, None))                      # in place
    with pytest.raises(mx.MXError):
        mx.rope(q[:, :1].expand(11, 4, 64), None, pos, f, out=(q[:, :1].expand(11, 4, 64), None))


def test_refusals(mx):
    import torch
    q, k, w, pos, f, (dq, dk) = data(4, 3, 2, 64, 10, 64)
    bad = [lambda: mx.rope(q.float(), k, pos, f), lambda: mx.rope(q, k[:3], pos, f), lambda: mx.rope(q, k, pos[:3], f),
           lambda: mx.rope(q, k, pos.float(), f), lambda: mx.rope(q, k, pos, f.float()), lambda: mx.rope(q, k, pos.cpu(), f),
           lambda: mx.rope(q, k, None, f), lambda: mx.rope(q, k, pos, torch.cat([f, f])), lambda: mx.rope(q, k, pos, f, "both"),
           lambda: mx.rope(q[:, :, ::2], None, pos, f[:16]), lambda: mx.rope(q, None, pos, f, out=(None, k)),
           lambda: mx.qk_norm_rope(q, k, w[0][:32], w[1], pos, f), lambda: mx.qk_norm_rope(q, k, w[0], w[1].float(), pos, f),
           lambda: mx.qk_norm_rope_backward(dq, None, q, k, *w, pos, f),
           lambda: mx.qk_norm_rope_backward(dq[:3], dk, q, k, *w, pos, f)]
    for call in bad:
        with pytest.raises((ValueError, mx.MXError)):
            call()


def test_offsets_beyond_31_bits(mx):
    """more than 2^31 elements, tokens outermost and heads outermost"""
    import torch
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of GPU memory")
    T, H, D = 270000, 64, 128
    g = torch.Generator(device="cuda").manual_seed(13)
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    q.normal_(generator=g)
    f, w = mx.rope_frequencies(D, 500000.0), (1 + 0.3 * torch.randn(D, device="cuda", generator=g)).bfloat16()
    pos = torch.arange(T, device="cuda")
    at = torch.tensor([0, 1, 131072, T // 2 + 7, T - 1], device="cuda")
    y, _ = mx.rope(q, None, pos, f)
    close(y[at], *ref.rotate(q[at], pos[at], f, "half"))
    dx, _, dw, _ = mx.qk_norm_rope_backward(y, None, q, None, w, None, pos, f, weight_grad=False)
    want, _, mag, _ = ref.norm_rope_backward(y[at], q[at], w, pos[at], f, 1e-5, "half")
    close(dx[at], want, mag)
    del dx
    outer = q.view(H, T, D).transpose(0, 1)
    y, _ = mx.qk_norm_rope(outer, None, w, None, pos, f)
    close(y[at], *ref.norm_rope(outer[at], w, pos[at], f, 1e-5, "half"))


def test_empty(mx):
    import torch
    q, k, w, pos, f, (dq, dk) = data(4, 3, 2, 64, 11, 64)
    y, _ = mx.rope(q[:0], None, pos[:0], f)
    assert y.shape == (0, 3, 64)
    _, _, dwq, dwk = mx.qk_norm_rope_backward(dq[:0], dk[:0], q[:0], k[:0], *w, pos[:0], f)
    assert (dwq == 0).all() and (dwk == 0).all()
    _, _, dwq, dwk = mx.qk_norm_rope_backward(dq, dk[:, :0], q, k[:, :0], *w, pos, f)
    assert (dwk == 0).all() and (dwq != 0).any()


def test_other_stream_and_capture(mx):
    """on a stream of its own; captured, and replayed with other contents and eager work in between"""
    import torch
    q, k, w, pos, f, (dq, dk) = data(50, 8, 2, 128, 12, 128)
    q, k = q.clone(), k.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = mx.qk_norm_rope(q, k, *w, pos, f, stream=s)
    b = mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(a, mx.qk_norm_rope(q, k, *w, pos, f)))
    assert all(torch.equal(x, y) for x, y in zip(b, mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f)))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = mx.qk_norm_rope(q, k, *w, pos, f)
        g = mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f)
        r = mx.rope(y[0], y[1], pos, f, inverse=True)
    for i in range(3):
        q.copy_((q.float() * (1.5 + i)).bfloat16() + i)
        pos.add_(1000 * i)
        graph.replay()
        torch.cuda.synchronize()
        want = mx.qk_norm_rope(q, k, *w, pos, f)
        assert all(torch.equal(s, t) for s, t in zip(y, want))
        assert all(torch.equal(s, t) for s, t in zip(g, mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f)))
        assert all(torch.equal(s, t) for s, t in zip(r, mx.rope(*want, pos, f, inverse=True)))
