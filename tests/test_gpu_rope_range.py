"""The norm of heads whose squares leave fp32's range, above and below, beside ordinary heads of the same wave.

Tolerances as in test_gpu_rope: a head scaled by a power of two has the roundings of any other."""
import pytest

import head_reference as ref
from test_gpu_rope import close, data, mx  # noqa: F401 (mx is a fixture)

pytestmark = pytest.mark.gpu

# magnitude of the odd heads, eps, magnitude of their gradients (dx stays within bf16's normal range and g * x within fp32's)
MAGS = [(1e17, 1e-6, 1e10), (1e18, 1e-6, 1e10), (3e18, 0.0, 1e10), (1e19, 1e-6, 1e10), (1e20, 1e-6, 1e10), (1e20, 3e38, 1e10),
        (1e30, 1e-6, 1e20), (1e38, 1e-6, 1e20), (1e-14, 0.0, 1e-10), (1e-15, 1e-32, 1e-10), (1e-16, 0.0, 1e-10),
        (1e-20, 0.0, 1e-10), (1e-20, 1e-36, 1e-10), (1e-20, 1e-40, 1e-10), (1e-25, 0.0, 1e-15), (1e-38, 0.0, 1e-20),
        (1e-38, 1e-45, 1e-20), (1e-20, 1e-6, 1.0)]


@pytest.mark.parametrize("dim,rot,layout", [(128, 128, "half"), (64, 32, "interleaved"), (40, 20, "half"), (100, 50, "interleaved"),
                                            (72, 24, "half"), (512, 512, "half"), (511, 510, "interleaved"), (33, 0, "half")])
@pytest.mark.parametrize("mag,eps,grad", MAGS)
def test_norm_of_any_magnitude(mx, dim, rot, layout, mag, eps, grad):
    import torch
    eps = torch.tensor(eps, dtype=torch.float32).item()                     # as the call takes it (1e-45 is 2^-149)
    q, k, w, pos, f, (dq, dk) = data(6, 5, 2, dim, 31, rot)
    q = q.float() / q.float().abs().amax(-1, keepdim=True).clamp(min=1.0)   # at most 1
    q[::2, 1::2] *= mag
    dq = dq.float()
    dq[::2, 1::2] *= grad
    q, dq = q.bfloat16(), dq.bfloat16()
    y, _ = mx.qk_norm_rope(q, k, *w, pos, f, eps=eps, layout=layout)
    close(y, *ref.norm_rope(q, w[0], pos, f, eps, layout))
    dx, _, dw, _ = mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f, eps=eps, layout=layout)
    want, wantw, mags, magw = ref.norm_rope_backward(dq, q, w[0], pos, f, eps, layout)
    close(dx, want, mags)
    assert ((dw.double() - wantw).abs() <= 2.0 ** -15 * magw).all()


def test_ordinary_heads_beside(mx):
    """a head's bits do not depend on the other heads of its wave"""
    import torch
    q, k, w, pos, f, (dq, dk) = data(6, 8, 2, 128, 32, 128)
    other = q.clone()
    other[:, 3] = (other[:, 3].float() * 1e30).bfloat16()
    other[2, 5] = (other[2, 5].float() * 1e-30).bfloat16()
    same = torch.ones(6, 8, dtype=torch.bool, device="cuda")
    same[:, 3] = same[2, 5] = False
    a, b = mx.qk_norm_rope(q, k, *w, pos, f, eps=0.0), mx.qk_norm_rope(other, k, *w, pos, f, eps=0.0)
    assert torch.equal(a[0][same], b[0][same]) and torch.equal(a[1], b[1])
    a = mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f, eps=0.0)
    b = mx.qk_norm_rope_backward(dq, dk, other, k, *w, pos, f, eps=0.0)
    assert torch.equal(a[0][same], b[0][same]) and torch.equal(a[1], b[1])


def test_heads_of_zeros_and_infinities(mx):
    """zeros: 0 with any eps above 0, NaN with none; an infinite element: NaN there, its head's others 0"""
    import torch
    q, _, w, pos, f, _ = data(4, 3, 2, 64, 33, 64)
    q = q.clone()
    q[1, 1] = 0
    q[2, 0, 5] = float("inf")
    for eps in (1e-6, 1e-35, 1e-44):
        assert (mx.qk_norm_rope(q, None, None, None, eps=eps)[0][1, 1] == 0).all()
    y = mx.qk_norm_rope(q, None, None, None, eps=0.0)[0]
    assert torch.isnan(y[1, 1]).all() and torch.isnan(y[2, 0, 5]) and (y[2, 0, :5] == 0).all() and (y[2, 0, 6:] == 0).all()
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
