"""Rotary positions and the norm of each head on the host: arguments that are refused before any HIP call
(pointers are only compared), empty calls, the frequencies, and the reference definitions the GPU tests rely on."""
import ctypes
import math
import os

import pytest
import torch

import head_reference as ref

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
P = ctypes.c_void_p
Q, K, PO, FR, QO, KO, QW, KW, DQ, DK, GQ, GK, WS = (P(0x100000000 * (i + 1)) for i in range(13))


@pytest.fixture(scope="module")
def L():
    from precision_block_amax_amd import build as libbuild
    if not os.path.exists(libbuild.LIB_PATH):
        libbuild.build()
    import precision_block_amax_amd as mx
    return mx.lib()


# 10 tokens, 6 query and 2 key heads of 64 within rows of 10 heads
def heads(k):
    return [k.get("q", Q), k.get("ldq", 640), k.get("ldqh", 64), k.get("hq", 6), k.get("k", K), k.get("ldk", 640),
            k.get("ldkh", 64), k.get("hk", 2), k.get("tokens", 10), k.get("dim", 64)]


def rotation(k):
    return [k.get("pos", PO), k.get("pt", 1), k.get("fr", FR), k.get("rot", 64), k.get("layout", 0), k.get("scale", 1.0)]


def outs(k):
    return [k.get("qo", QO), k.get("ldqo", 384), k.get("ldqoh", 64), k.get("ko", KO), k.get("ldko", 128), k.get("ldkoh", 64)]


def rope(**k):
    return heads(k) + rotation(k) + [k.get("inverse", 0)] + outs(k) + [None]


def norm(**k):
    return heads(k) + [k.get("qw", QW), k.get("kw", KW), k.get("param", BF16), k.get("eps", 1e-5)] + rotation(k) + outs(k) + [None]


def back(**k):
    return ([k.get("dq", DQ), 384, 64, k.get("dk", DK), 128, 64] + heads(k) +
            [k.get("qw", QW), k.get("kw", KW), k.get("param", BF16), k.get("eps", 1e-5)] + rotation(k) + outs(k) +
            [k.get("gq", GQ), k.get("gk", GK), k.get("ws", WS), k.get("wsb", 1 << 30), None])


COMMON = [dict(hq=-1), dict(hk=-1), dict(tokens=-1), dict(dim=-1), dict(rot=-2), dict(rot=63), dict(rot=66), dict(pt=2),
          dict(layout=2), dict(layout=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(k=None),
          dict(qo=None), dict(ko=None), dict(pos=None), dict(fr=None),
          dict(ldqh=63),                                  # heads overlap
          dict(ldq=383),                                  # tokens overlap, and heads lie in each other's tokens
          dict(ldq=64, ldqh=639),                         # heads outermost: 10 tokens of 64 do not fit 639
          dict(ldqo=0), dict(ldqoh=0),                    # broadcast
          dict(qo=Q), dict(ko=Q), dict(ko=QO),            # overlaps
          dict(qo=P(Q.value + 2 * 639)), dict(ko=P(QO.value + 2 * 384 * 10 - 2)), dict(ko=PO), dict(qo=P(FR.value + 8 * 31)),
          dict(ldq=1 << 62), dict(ldqo=1 << 62)]


@pytest.mark.parametrize("bad", COMMON, ids=str)
def test_rejects(L, bad):
    assert L.mx_rope(*rope(**bad)) == INVALID
    assert L.mx_qk_norm_rope(*norm(**bad)) == INVALID
    assert L.mx_qk_norm_rope_backward(*back(**bad)) == INVALID


def test_rejects_of_each(L):
    assert L.mx_rope(*rope(inverse=2)) == INVALID
    for f, args in ((L.mx_qk_norm_rope, norm), (L.mx_qk_norm_rope_backward, back)):
        for bad in (dict(param=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(qo=QW),
                    dict(ko=P(KW.value + 2 * 63))):
            assert f(*args(**bad)) == INVALID, bad
    need = L.mx_qk_norm_rope_backward_workspace(10, 6, 2, 64)
    assert need > 0
    for bad in (dict(dq=None), dict(dk=None), dict(ws=None), dict(wsb=need - 1), dict(ws=P(WS.value + 8)), dict(gq=GK),
                dict(gq=Q), dict(ws=GQ), dict(qo=DQ), dict(gk=QO), dict(ws=P(QO.value + 16))):
        assert L.mx_qk_norm_rope_backward(*back(**bad)) == INVALID, bad


def test_limits(L):
    for f, args in ((L.mx_rope, rope), (L.mx_qk_norm_rope, norm), (L.mx_qk_norm_rope_backward, back)):
        assert f(*args(dim=514, ldq=6000, ldqh=514, ldk=6000, ldkh=514)) == UNSUPPORTED
        assert f(*args(hq=(1 << 16) + 1)) == UNSUPPORTED
        assert f(*args(tokens=(1 << 31) + 1)) == UNSUPPORTED
    assert L.mx_qk_norm_rope_backward_workspace(0, 6, 2, 64) == 0
    assert L.mx_qk_norm_rope_backward_workspace(10, 0, 0, 64) == 0
    assert L.mx_qk_norm_rope_backward_workspace(1 << 31, 64, 64, 512) < 1 << 26


def test_empty_calls(L):
    none = dict(q=None, k=None, qo=None, ko=None, pos=None, fr=None)
    for f, args in ((L.mx_rope, rope), (L.mx_qk_norm_rope, norm)):
        assert f(*args(tokens=0, **none)) == OK
        assert f(*args(hq=0, hk=0, **none)) == OK
        assert f(*args(dim=0, rot=0, **none)) == OK
    assert L.mx_qk_norm_rope_backward(*back(tokens=0, gq=None, gk=None, ws=None, dq=None, dk=None, **none)) == OK
    assert L.mx_qk_norm_rope_backward(*back(dim=0, rot=0, ws=None, dq=None, dk=None, **none)) == OK


def test_python_refusals():
    import precision_block_amax_amd as mx
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mx.rope(x, None, None, None)               # not on a GPU
    with pytest.raises(ValueError):
        mx.rope(x[0], None, None, None)
    with pytest.raises(ValueError):
        mx.rope_frequencies(64, scaling="other", device="cpu")
    with pytest.raises(mx.MXError):
        mx.rope_frequencies(63, device="cpu")
    with pytest.raises(mx.MXError):
        mx.rope_frequencies(64, scaling="bands", factor=8.0, low=4.0, high=4.0, device="cpu")
    with pytest.raises(mx.MXError):
        mx.rope_frequencies(64, scaling="linear", factor=0.0, device="cpu")


def test_frequencies():
    import precision_block_amax_amd as mx
    f = mx.rope_frequencies(128, 500000.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (64,)
    for i in (0, 1, 31, 63):
        assert math.isclose(f[i].item(), math.exp(-2 * i / 128 * math.log(500000.0)), rel_tol=1e-14)
    assert torch.equal(mx.rope_frequencies(128, 500000.0, "linear", 4.0, device="cpu"), f / 4)
    g = mx.rope_frequencies(128, 500000.0, "bands", 8.0, 1.0, 4.0, 8192.0, device="cpu")
    wavelength = 2 * math.pi / f
    short, long = wavelength < 8192 / 4, wavelength > 8192 / 1
    assert short.any() and long.any() and (~short & ~long).any()
    assert torch.equal(g[short], f[short]) and torch.equal(g[long], f[long] / 8)
    mid = ~short & ~long
    keep = (8192 / wavelength - 1) / 3
    assert torch.allclose(g[mid], ((1 - keep) * f / 8 + keep * f)[mid], rtol=1e-14, atol=0)
    assert mx.rope_frequencies(0, device="cpu").numel() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_reference(layout):
    """the definitions: the inverse is the transpose, turns add, and the gradient is the derivative"""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    pos, f = torch.tensor([0, 3, -2, 70]), torch.tensor([1.0, 0.1, 0.01], dtype=torch.float64)
    x, dy, w = r(4, 3, 10), r(4, 3, 10), r(10)
    y, mag = ref.rotate(x, pos, f, layout, 0.7)
    assert torch.equal(y[..., 6:], x[..., 6:])
    assert (mag >= y.abs() - 1e-12).all()
    back, _ = ref.rotate(dy, pos, f, layout, 0.7, inverse=True)
    assert math.isclose((y * dy).sum().item(), (x * back).sum().item(), rel_tol=1e-12)
    two, _ = ref.rotate(ref.rotate(x, pos, f, layout)[0], pos, f, layout)
    assert torch.allclose(two, ref.rotate(x, 2 * pos, f, layout)[0], atol=1e-12)
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    a, b = ref.pairs(3, layout, x.device)
    v = xg * (xg.square().mean(-1, keepdim=True) + 1e-3).rsqrt() * wg
    t = ref.angles(pos, f)
    out = v.index_copy(-1, a, v[..., a] * t.cos() * 0.7 - v[..., b] * t.sin() * 0.7)
    out = out.index_copy(-1, b, v[..., b] * t.cos() * 0.7 + v[..., a] * t.sin() * 0.7)
    assert torch.allclose(out, ref.norm_rope(x, w, pos, f, 1e-3, layout, 0.7)[0], atol=1e-12)
    (out * dy).sum().backward()
    dx, dw, _, _ = ref.norm_rope_backward(dy, x, w, pos, f, 1e-3, layout, 0.7)
    assert torch.allclose(xg.grad, dx, atol=1e-11) and torch.allclose(wg.grad, dw, atol=1e-11)
