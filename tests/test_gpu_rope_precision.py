"""rope_rotate of float32 rows: what float32 products of correctly rounded cosines and sines may be off by, and no more, so
that cosines near 0 have their bits."""
import pytest
import torch

from nvfp4_block_scaled_moe_amd import ops
from tests.attention_util import frequencies

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot,start", [(1021, 6, 128, 64, 64), (300, 9, 96, 96, 0), (65, 3, 50, 22, 3)])
def test_float32_rows(T, H, D, rot, start, interleaved, grad):
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H, D), generator=g)
    pos = torch.randint(0, 1_000_000, (T,), generator=g)
    f, m = frequencies(rot), 1.25
    got = ops.rope_rotate(x.cuda(), pos.cuda(), ops.Rope(f.cuda(), start, interleaved, m), grad=grad).cpu()
    axis = -1 if interleaved else -2
    pairs = lambda t: t[..., start:start + rot].unflatten(-1, (rot // 2, 2) if interleaved else (2, rot // 2)).double()  # noqa: E731
    u, w = pairs(x).select(axis, 0), pairs(x).select(axis, 1)
    a = pos.double()[:, None, None] * f
    c, s = torch.cos(a) * m, torch.sin(a) * (-m if grad else m)
    step = 2.0 ** -24                                            # half of a float32's, relative
    for k, (p, q, sign) in enumerate(((u, w, -1.0), (w, u, 1.0))):
        want = p * c + sign * q * s
        # the cosine's and sine's rounding, that of q s, that of the sum; and the angle's in float64 on either side
        tol = step * ((p * c).abs() + 2.0 * (q * s).abs() + want.abs()) * (1.0 + 2.0 ** -20) + 2.0 ** -50 * (1.0 + a) * m * (p.abs() + q.abs())
        over = (pairs(got).select(axis, k) - want).abs() - tol
        assert (over <= 0).all(), (k, float(over.max()), int((over > 0).sum()))
    other = [d for d in range(D) if not start <= d < start + rot]
    assert torch.equal(got[..., other], x[..., other])
