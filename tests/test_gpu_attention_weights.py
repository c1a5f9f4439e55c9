"""The precision of the second product's weights over an E4M3 cache where rows are many: f16, 11 bits, not bf16's 8. Rows with a
few keys, or a few that count, whose outputs show a weight's rounding beside their own."""
import math

import pytest
import torch

from nvfp4_block_scaled_moe_amd import ops
from tests.attention_util import BF, HALF, Case, check

# (new tokens, tokens before them, query heads, key heads, D, page, scale)
CASES = [
    ([33], [0], 4, 2, 64, 16, None),
    ([20, 50], [0, 3], 6, 2, 96, 32, None),
    ([129], [0], 2, 1, 32, 64, None),
    ([40], [500], 8, 2, 64, 64, 0.5),       # (blocks that every row sees)
    ([70], [300], 4, 1, 128, 16, 0.3),
    ([30], [200], 4, 2, 160, 32, 0.3),
    ([24], [0], 3, 1, 256, 64, None),
    ([256], [0], 8, 2, 128, 64, None),      # (tiles of 256 rows, by a wide page table)
    ([300], [700], 4, 1, 128, 32, 0.3),
]
WIDE = [7, 8]


def _reference(c, scale, step, rounded=None):
    """float64 outputs and how far they may be off with weights of a half step ``step`` that end at 2^-25 (f16: half of its least
    number), taken 2^7 times as large as the largest key's is. ``rounded``: the outputs with weights of that type."""
    scale = c.D ** -0.5 if scale is None else scale
    G = c.Hq // c.Hkv
    out, tol = torch.zeros((c.T, c.Hq, c.D), dtype=torch.float64), torch.zeros((c.T, c.Hq, c.D), dtype=torch.float64)
    for b, (n, ctx) in enumerate(zip(c.new, c.ctx)):
        rows = slice(c.starts[b], c.starts[b] + n)
        sees = (ctx + torch.arange(n))[:, None] >= torch.arange(n + ctx)
        for h in range(c.Hq):
            q, k, v = c.q[rows, h].double(), c.keys[b][:, h // G], c.values[b][:, h // G]
            s = torch.where(sees, (q @ k.t()) * scale, -math.inf)
            e = torch.exp(s - s.amax(-1, keepdim=True))
            total = e.sum(-1, keepdim=True)
            if rounded is not None:
                e = (e * 128.0).to(rounded).double() / 128.0
            o, a = e @ v / total, e @ v.abs() / total
            d = torch.where(sees, (q.abs() @ k.abs().t()) * scale, 0.0).amax(-1, keepdim=True)
            # scores, exponentials and sums in float32 as in Case.attention; the largest key's weight is part of the total, so that
            # a weight's least step is at most 2^-25 / 2^7 of it
            rel = 2.0 * d * (c.D + 8) * 2.0 ** -24 + (n + ctx + 64) * 2.0 ** -23 + step
            off = rel * a + 2.0 ** -32 * torch.where(sees, 1.0, 0.0).double() @ v.abs()
            out[rows, h], tol[rows, h] = o, HALF[BF] * (o.abs() + off) + off
    return out, tol


def _case(case, **kw):
    return Case(*CASES[case][:-1], fp8=True, seed=400 + case, v_spread=3.0, **kw), CASES[case][-1]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_the_tolerance_tells_weights_of_two_types_apart(case):
    c, scale = _case(case, dev="cpu")
    want, tol = _reference(c, scale, 2.0 ** -11)
    check(_reference(c, scale, 0.0, torch.float16)[0].to(BF), want, tol, "f16")
    with pytest.raises(AssertionError):
        check(_reference(c, scale, 0.0, BF)[0].to(BF), want, tol, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights_of_many_rows(case):
    c, scale = _case(case)
    assert c.rows() > 16
    check(ops.kv_cache_attention(c.q.cuda(), c.cache, c.batch, scale=scale), *_reference(c, scale, 2.0 ** -11))


@pytest.mark.gpu
@pytest.mark.parametrize("case", WIDE)
def test_weights_of_tiles_of_256_rows(case):
    c, scale = _case(case)
    assert c.rows() >= 1024
    table = torch.full((1, 4096 // c.page), -1, dtype=torch.int32)
    table[0, :c.table.shape[1] - 1] = c.table[0, :-1]
    batch = ops.CacheBatch(table.cuda(), c.batch.lengths, c.batch.starts)
    check(ops.kv_cache_attention(c.q.cuda(), c.cache, batch, scale=scale), *_reference(c, scale, 2.0 ** -11))
