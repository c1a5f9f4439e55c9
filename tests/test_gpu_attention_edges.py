"""The attention half at the ends of what its calls take: starts outside the rows, rows whose scores are all -Inf."""
import pytest
import torch

from nvfp4_block_scaled_moe_amd import ops
from tests.attention_util import BF, Case, frequencies

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,ctx", [([4, 6], [14, 20]), ([30, 0, 50], [100, 7, 3]), ([1] * 1100, [i % 30 for i in range(1100)])])
def test_starts_outside_the_rows(new, ctx, fp8):
    """They count as the first and last row, in the append as in the attention over what it stored."""
    c = Case(new, ctx, 4, 2, 64, 16, fp8=fp8, seed=len(new))
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((c.T, 2, 64), generator=g).to(BF).cuda() for _ in range(2))
    rope = ops.Rope(frequencies(64).cuda())
    got = []
    for first, last in ((0, c.T), (-3, c.T + 5), (-2 ** 31, 2 ** 31 - 1)):
        starts = c.batch.starts.clone()
        starts[0], starts[-1] = first, last
        batch = ops.CacheBatch(c.batch.page_table, c.batch.lengths, starts)
        cache = ops.KVCache(c.cache.k.clone(), c.cache.v.clone(), c.cache.k_scale, c.cache.v_scale)
        q = ops.kv_cache_append(cache, batch, k, v, q=c.q.cuda(), rope=rope)
        bits = torch.uint8 if fp8 else torch.int16
        got.append((q, cache.k.view(bits), cache.v.view(bits), ops.kv_cache_attention(q, cache, batch)))
    assert torch.isfinite(got[0][3]).all()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,ctx", [([3], 70), ([2], 4200), ([40], 70), ([40], 4200), ([150], 4200)])
def test_rows_whose_scores_are_all_minus_infinity(new, ctx, fp8):
    """The softmax of such a row is NaN, in one part and across a join, and its neighbours' is theirs; the same row before its
    sequence, where it sees no key, gives zeros."""
    c = Case(new, [ctx], 8, 1, 128, 64, fp8=fp8, seed=20)
    n, head = new[0], 3
    k = c.cache.k.clone()
    k[:, :, :, 0] = torch.tensor(1.0).to(k.dtype)
    cache = ops.KVCache(k, c.cache.v, c.cache.k_scale, c.cache.v_scale)
    q = c.q.cuda()
    want = ops.kv_cache_attention(q, cache, c.batch)
    low = q.clone()
    low[n // 2, head, 0] = float("-inf")
    got = ops.kv_cache_attention(low, cache, c.batch)
    assert torch.isnan(got[n // 2, head]).all()
    got[n // 2, head] = want[n // 2, head]
    assert torch.equal(got, want)
    short = ops.CacheBatch(c.batch.page_table, torch.full_like(c.batch.lengths, n - n // 2 - 1), c.batch.starts)
    got = ops.kv_cache_attention(low, cache, short)
    assert (got[:n // 2 + 1] == 0).all() and torch.isfinite(got).all() and (got[n // 2 + 1:] != 0).any(-1).all()
