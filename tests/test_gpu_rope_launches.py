"""The forward calls on more tokens than one launch takes (2^25 waves): every launch has its own tokens, positions and
strides.  Tolerances as in test_gpu_rope; both sides' angles are fp64 products, off by p f 2^-51."""
import pytest

import head_reference as ref
from test_gpu_rope import close, mx  # noqa: F401 (mx is a fixture)

pytestmark = pytest.mark.gpu


# one head: a wave for each token, 2^25 of them per launch; nine heads of two elements: two waves, half as many tokens
@pytest.mark.parametrize("hq,hk,most", [(1, 0, 1 << 25), (8, 1, 1 << 24)])
@pytest.mark.parametrize("norm,wide", [(False, False), (True, True)])
def test_more_than_one_launch(mx, hq, hk, most, norm, wide):
    import torch
    T, H = most + 5, hq + hk
    g = torch.Generator(device="cuda").manual_seed(71)
    x = torch.empty(T, H, 4, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    buf = torch.full((T, H, 4), 5.0, dtype=torch.bfloat16, device="cuda")
    q, k = x[:, :hq, 1:3], x[:, hq:, 1:3] if hk else None
    out = (buf[:, :hq, 2:], buf[:, hq:, 2:] if hk else None)
    pos = torch.arange(T, device="cuda", dtype=torch.int64 if wide else torch.int32)
    f = torch.tensor([0.37], dtype=torch.float64, device="cuda")
    w = torch.tensor([1.5, -0.75], dtype=torch.float32, device="cuda")
    if norm:
        mx.qk_norm_rope(q, k, w, None, pos, f, out=out)
    else:
        mx.rope(q, k, pos, f, out=out)
    for lo, hi in ((0, 1000), (most // 2, most // 2 + 1000), (most - 1000, T)):
        for a, b, wt in ((q, out[0], w), (k, out[1], None)):
            if a is None:
                continue
            a, b, p = a[lo:hi], b[lo:hi], pos[lo:hi]
            want = ref.norm_rope(a, wt, p, f, 1e-5, "half") if norm else ref.rotate(a, p, f, "half")
            close(b, *want, angle=T * 2.0 ** -50)
    assert (buf[..., :2] == 5).all()
    # nothing is left out in between: of an element of 5.0 as many as its bf16 values' chance, none of whole tokens
    assert not (buf[..., 2:] == 5).all(-1).any()
