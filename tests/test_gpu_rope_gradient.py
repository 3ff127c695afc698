"""The gradients of the norm and rotation of heads against differences of the definition, along directions on which a
gradient that is zero, negated or half as large is seen.

Along v = the gradient itself, the slope is the sum of its squares, to which every element adds: bf16's rounding, half a
step of each element, is then at most 2^-8 of the slope, and 2^-17 of the magnitudes |v| (test_gpu_rope: E) come from
fp32.  A weight's gradient is within 2^-15 of its magnitudes.  The difference itself, of steps h and h / 2 in float64,
is off by a third of what these two differ by (its error goes with h^2); all of that is allowed, and 2^-40 of the
value's terms over the step for float64."""
import pytest

import head_reference as ref
from test_gpu_rope import E, data, mx  # noqa: F401 (mx is a fixture)

pytestmark = pytest.mark.gpu


def slope(value, terms, h):
    """(difference quotient, its error): value(t) at t = 0, terms: the sum of |terms| in it"""
    d = [(value(s) - value(-s)) / (2 * s) for s in (h, h / 2)]
    return d[1], (d[0] - d[1]).abs() + 2.0 ** -40 * terms / h


@pytest.mark.parametrize("dim,rot,layout,scale", [(64, 64, "half", 1.0), (128, 64, "interleaved", 0.75), (40, 20, "half", 1.25),
                                                  (100, 50, "interleaved", 1.0), (65, 64, "half", 1.0), (256, 0, "half", 1.0)])
@pytest.mark.parametrize("of", ["queries", "keys"])
def test_gradients(mx, dim, rot, layout, scale, of):
    import torch
    q, k, w, pos, f, (dq, dk) = data(40, 4, 2, dim, 61, rot)
    out = mx.qk_norm_rope_backward(dq, dk, q, k, *w, pos, f, eps=1e-6, layout=layout, scale=scale)
    i = of == "keys"
    x, dy, wt, dx, dw = (k, dk, w[1], out[1], out[3]) if i else (q, dq, w[0], out[0], out[2])
    x, dy, wt = x.double(), dy.double(), wt.double()
    want, wantw, mag, magw = ref.norm_rope_backward(dy, x, wt, pos, f, 1e-6, layout, scale)
    value = lambda a, b: (ref.norm_rope(a, b, pos, f, 1e-6, layout, scale)[0] * dy).sum()
    terms = (ref.norm_rope(x, wt, pos, f, 1e-6, layout, scale)[1] * dy.abs()).sum()

    v = want / want.abs().max()
    s, err = slope(lambda t: value(x + t * v, wt), terms, 2.0 ** -10)
    tol = err + (2.0 ** -8 * (1 + E) * want.abs() * v.abs() + E * mag * v.abs()).sum()
    assert tol < s / 64                        # zero, half or negated gradients are far outside
    assert (s - (dx.double() * v).sum()).abs() <= tol
    v = wantw / wantw.abs().max()
    s, err = slope(lambda t: value(x, wt + t * v), terms, 2.0 ** -10)
    tol = err + (2.0 ** -15 * magw * v.abs()).sum()
    assert tol < s / 64
    assert (s - (dw.double() * v).sum()).abs() <= tol


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_of_the_rotation(mx, layout):
    """the inverse rotation of dy, along itself"""
    import torch
    q, k, _, pos, f, (dq, _) = data(40, 4, 2, 64, 62, 48)
    x, dy = q.double(), dq.double()
    want, mag = ref.rotate(dy, pos, f, layout, 1.25, True)
    v = want / want.abs().max()
    value = lambda t: (ref.rotate(x + t * v, pos, f, layout, 1.25)[0] * dy).sum()
    s, err = slope(value, (ref.rotate(x, pos, f, layout, 1.25)[1] * dy.abs()).sum(), 2.0 ** -10)
    tol = err + (2.0 ** -8 * (1 + E) * want.abs() * v.abs() + E * mag * v.abs()).sum()
    assert tol < s / 64
    dx, _ = mx.rope(dq, None, pos, f, layout=layout, scale=1.25, inverse=True)
    assert (s - (dx.double() * v).sum()).abs() <= tol
