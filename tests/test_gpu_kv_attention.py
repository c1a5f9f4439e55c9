"""kv_cache_attention against float64: head layouts, sizes, lengths from nothing to many segments, pages, windows,
both caches, and what must not reach a row."""
import math

import pytest
import torch

from nvfp4_block_scaled_moe_amd import ops
from tests.attention_util import BF, Case, check

pytestmark = pytest.mark.gpu


def _run(c, **kw):
    out, tol = c.attention(kw.get("scale"), kw.get("window", 0))
    got = ops.kv_cache_attention(c.q.cuda(), c.cache, c.batch, **kw)
    check(got[:c.T], out, tol, str(kw))
    return got


# (new tokens, tokens before them, query heads, key heads, D, page)
DECODE = [
    ([1], [0], 1, 1, 32, 16),
    ([1], [15], 2, 1, 64, 16),
    ([1], [16], 16, 2, 64, 16),
    ([1, 1, 1], [0, 31, 32], 8, 8, 128, 32),
    ([1, 1], [63, 200], 12, 2, 96, 64),
    ([1] * 5, [5, 700, 64, 0, 129], 8, 1, 128, 64),
    ([1, 0, 1], [40, 70, 3000], 16, 1, 128, 16),
    ([1], [9000], 16, 2, 128, 128),
    ([1, 1], [513, 100], 6, 3, 160, 256),
    ([1, 1], [300, 2500], 5, 1, 192, 32),
    ([1], [777], 3, 1, 224, 16),
    ([1, 1], [1500, 20], 10, 2, 256, 64),
    ([2, 1, 3], [100, 50, 333], 8, 2, 64, 32),
    ([1] * 70, [3 * i for i in range(70)], 4, 2, 64, 16),
    ([40, 1, 1, 1, 1, 1, 1, 1], [10, 900, 30, 2, 77, 64, 128, 5], 4, 2, 128, 64),
    ([40] + [1] * 66, [7 * i for i in range(67)], 16, 2, 32, 16),
]
CHUNK = [   # up to 32 rows a sequence, up to 64, and more
    ([17], [0], 1, 1, 32, 16),
    ([128], [0], 1, 1, 64, 64),
    ([129], [63], 4, 2, 64, 32),
    ([33, 0, 70], [0, 5, 190], 6, 2, 96, 16),
    ([200], [1000], 8, 1, 128, 64),
    ([65, 1, 1], [128, 700, 0], 8, 2, 128, 128),
    ([50], [300], 7, 1, 160, 16),
    ([40], [333], 8, 4, 192, 32),
    ([30, 90], [64, 1], 4, 1, 224, 256),
    ([77], [500], 3, 1, 256, 64),
    ([5, 300], [2000, 100], 16, 1, 64, 16),
    ([2, 1], [900, 33], 16, 1, 128, 64),
    ([3, 1], [100, 700], 14, 1, 192, 16),
    ([4, 5], [3000, 64], 32, 2, 64, 32),
    ([7], [555], 8, 1, 128, 16),
    ([3, 4, 1], [1, 300, 2000], 32, 1, 256, 64),
    ([8, 8, 8], [0, 77, 1000], 24, 3, 96, 16),
    ([90] + [1] * 66, [7 * i for i in range(67)], 16, 2, 32, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_few_rows(case, fp8):
    c = Case(*DECODE[case], fp8=fp8, seed=case)
    assert c.rows() <= 16
    _run(c)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(CHUNK)))
def test_many_rows(case, fp8):
    c = Case(*CHUNK[case], fp8=fp8, seed=100 + case)
    _run(c)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 64, 100, 1000])
@pytest.mark.parametrize("many", [False, True])
def test_window(many, window):
    c = Case([150, 1], [333, 70], 4, 2, 64, 16, seed=window) if many else Case([1, 3, 1], [333, 70, 0], 4, 2, 128, 32, seed=window)
    assert (c.rows() > 64) == many
    _run(c, window=window)


def test_long_contexts_in_segments():
    """More blocks than a segment: sums of several workgroups are joined."""
    _run(Case([1, 1], [20000, 300], 8, 1, 64, 64, seed=1))
    _run(Case([1], [33000], 4, 1, 64, 16, fp8=True, seed=2))
    _run(Case([40], [9000], 8, 1, 64, 64, seed=3))
    _run(Case([19, 2], [5000, 6000], 16, 1, 128, 32, fp8=True, seed=4))


def test_large_scores():
    """Rows whose largest score comes late, and far above the others."""
    for new in ([1], [60]):
        c = Case(new, [400], 4, 1, 64, 16, seed=5)
        _run(c, scale=3.0)
        _run(c, scale=1e-3)


@pytest.mark.parametrize("new", [[1, 2], [70, 33]])
def test_rows_behind_the_last_sequence_stay(new):
    c = Case(new, [50, 90], 8, 2, 64, 32, seed=6, spare_rows=5)
    out = torch.full(c.q.shape, 7.0, dtype=BF, device="cuda")
    want, tol = c.attention()
    got = ops.kv_cache_attention(c.q.cuda(), c.cache, c.batch, out=out)
    assert got is out
    check(got[:c.T], want, tol)
    assert (got[c.T:] == 7.0).all()


@pytest.mark.parametrize("new", [[1, 2], [70, 33]])
def test_rows_apart(new):
    """Queries and outputs as views of wider rows, heads apart."""
    c = Case(new, [50, 90], 6, 2, 64, 32, seed=7)
    wide = torch.randn((c.T, 9, 72), device="cuda").to(BF)
    q = wide[:, 2:8, :64]
    q.copy_(c.q)
    room = torch.full((c.T, 7, 80), 3.0, dtype=BF, device="cuda")
    want, tol = c.attention()
    check(ops.kv_cache_attention(q, c.cache, c.batch, out=room[:, :6, :64]), want, tol)
    assert (room[:, 6:] == 3.0).all() and (room[:, :, 64:] == 3.0).all()
    odd = torch.empty(c.q.numel() + 1, dtype=BF, device="cuda")[1:].view(c.q.shape)   # 2 bytes off
    odd.copy_(c.q)
    check(ops.kv_cache_attention(odd, c.cache, c.batch), want, tol)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[6], [90]])
def test_nothing_leaks_from_unseen_tokens(new, fp8):
    """A NaN or Inf in a new token's key or value reaches the rows that see it, and no row before."""
    c = Case(new, [70], 2, 1, 64, 16, fp8=fp8, seed=8)
    clean = ops.kv_cache_attention(c.q.cuda(), c.cache, c.batch).cpu()
    p = 70 + new[0] // 2
    page, slot = int(c.table[0, p // 16]), p % 16
    for which in ("v nan", "v inf", "k nan"):
        k, v = c.cache.k.clone(), c.cache.v.clone()
        bits = 0x7F if fp8 else (0x7F80 if which == "v inf" else 0x7FC0)   # (E4M3 has no Inf: NaN)
        as_int = torch.uint8 if fp8 else torch.int16
        if which[0] == "v":
            v.view(as_int)[page, 0, 5, slot] = bits
        else:
            k.view(as_int)[page, 0, slot, 5] = bits
        got = ops.kv_cache_attention(c.q.cuda(), ops.KVCache(k, v, c.cache.k_scale, c.cache.v_scale), c.batch).cpu()
        before, after = got[:new[0] // 2], got[new[0] // 2:]
        assert torch.equal(before, clean[:new[0] // 2]), which
        if which[0] == "v":
            assert not torch.isfinite(after[:, :, 5]).any(), which
            keep = [d for d in range(64) if d != 5]
            assert torch.equal(after[:, :, keep], clean[new[0] // 2:][:, :, keep]), which
        else:
            assert torch.isnan(after).all(), which


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[4], [80]])
def test_missing_pages_give_nan_where_they_are_seen(new, fp8):
    c = Case(new, [100], 2, 1, 64, 16, fp8=fp8, seed=9)
    clean = ops.kv_cache_attention(c.q.cuda(), c.cache, c.batch, window=40).cpu()
    for bad in (-1, c.pages, -2 ** 31, 2 ** 31 - 1):
        table = c.table.clone()
        table[0, 4] = bad    # tokens 64 to 79
        batch = ops.CacheBatch(table.cuda(), c.batch.lengths, c.batch.starts)
        assert torch.isnan(ops.kv_cache_attention(c.q.cuda(), c.cache, batch)).all()
        got = ops.kv_cache_attention(c.q.cuda(), c.cache, batch, window=40).cpu()
        sees = torch.tensor([i for i in range(new[0]) if 100 + i - 40 < 79])
        other = torch.tensor([i for i in range(new[0]) if 100 + i - 40 >= 79], dtype=torch.long)
        assert torch.isnan(got[sees]).all() and torch.equal(got[other], clean[other])


@pytest.mark.parametrize("new", [[3], [50]])
def test_lengths_outside_the_table(new):
    """Longer than the page table, shorter than the new tokens, negative, and starts that say nothing."""
    c = Case(new, [60], 4, 2, 64, 16, seed=10)
    n = new[0]
    q = c.q.cuda()
    call = lambda lengths, starts: ops.kv_cache_attention(  # noqa: E731
        q, c.cache, ops.CacheBatch(c.batch.page_table[:, :-(-(60 + n) // 16)].contiguous(),
                                   torch.tensor([lengths], dtype=torch.int32, device="cuda"),
                                   torch.tensor(starts, dtype=torch.int32, device="cuda")),
        out=torch.full_like(q, 5.0))
    assert torch.isnan(call(2 ** 31 - 1, [0, n])).all()
    short = call(1, [0, n])       # the last row has position 0, the others lie before the sequence
    assert (short[:-1] == 0).all() and torch.isfinite(short[-1]).all() and (short[-1] != 0).any()
    assert (call(0, [0, n]) == 0).all()
    assert (call(-5, [0, n]) == 0).all()
    assert (call(60 + n, [n, n]) == 5.0).all()
    assert (call(60 + n, [n, 0]) == 5.0).all()
    assert (call(60 + n, [2 ** 31 - 1, 2 ** 31 - 1]) == 5.0).all()
    whole = call(60 + n, [-7, 2 ** 31 - 1])    # clipped to the rows that there are
    assert torch.equal(whole, call(60 + n, [0, n]))


def test_no_tokens():
    c = Case([1], [5], 2, 1, 64, 16)
    out = ops.kv_cache_attention(c.q.cuda()[:0], c.cache, c.batch)
    assert out.shape == (0, 2, 64)


@pytest.mark.parametrize("new", [[1, 1, 1], [64, 300, 2]])
def test_same_bits_every_time_and_in_graphs(new):
    """Eager calls, on another stream, and replays of a captured one between them; lengths change under the graph."""
    c = Case(new, [2000, 500, 4000], 8, 2, 128, 64, seed=11)
    q = c.q.cuda()
    first = ops.kv_cache_attention(q, c.cache, c.batch)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert torch.equal(ops.kv_cache_attention(q, c.cache, c.batch), first)
    torch.cuda.current_stream().wait_stream(s)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.kv_cache_attention(q, c.cache, c.batch, out=out)
    full = c.batch.lengths.clone()
    for less in (0, 100, 1, 0):
        c.batch.lengths.copy_(full - less)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ops.kv_cache_attention(q, c.cache, c.batch)), less
    assert torch.equal(out, first)


def test_pages_past_32_bits():
    """A cache of over 2^32 elements: the last page's offsets pass 32 bits."""
    pages, page, D = (1 << 32) // (64 * 128) + 2, 64, 128
    cache = ops.KVCache(torch.empty((pages, 1, page, D), dtype=BF, device="cuda"), torch.empty((pages, 1, D, page), dtype=BF, device="cuda"))
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32)
    for new in (1, 40):
        c = Case([new], [100 - new], 2, 1, D, page, seed=new)
        for i in range(2):
            cache.k[int(table[0, i])] = c.cache.k[int(c.table[0, i])]
            cache.v[int(table[0, i])] = c.cache.v[int(c.table[0, i])]
        want, tol = c.attention()
        got = ops.kv_cache_attention(c.q.cuda(), cache, ops.CacheBatch(table.cuda(), c.batch.lengths, c.batch.starts))
        check(got, want, tol)


# Tiles of 256 rows: heads of 128 dims, 1024 rows or more of a sequence on average, page tables of 4096 tokens or more.
WIDE = [
    ([150], [4200], 8, 1, 128, 64),
    ([128], [4000], 8, 1, 128, 16),          # the last tile whole
    ([300, 10, 0], [4100, 33, 0], 16, 1, 128, 32),
    ([257], [5000], 12, 3, 128, 128),
    ([1030], [3500], 1, 1, 128, 1024),
    ([40], [9000], 32, 1, 128, 64),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_tiles_of_256_rows(case, fp8):
    c = Case(*WIDE[case], fp8=fp8, seed=200 + case)
    assert c.rows() >= 1024 and c.table.shape[1] * c.page >= 4096
    _run(c)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [1, 63, 130, 1000])
def test_windows_of_tiles_of_256_rows(window, fp8):
    c = Case([150, 140], [4000, 30], 8, 1, 128, 16, fp8=fp8, seed=window)
    _run(c, window=window)


@pytest.mark.parametrize("fp8", [False, True])
def test_what_tiles_of_256_rows_do_not_see(fp8):
    c = Case([160], [4000], 8, 1, 128, 64, fp8=fp8, seed=12)
    clean = ops.kv_cache_attention(c.q.cuda(), c.cache, c.batch).cpu()
    p = 4000 + 100
    v = c.cache.v.clone()
    v.view(torch.uint8 if fp8 else torch.int16)[int(c.table[0, p // 64]), 0, 77, p % 64] = 0x7F if fp8 else 0x7FC0
    got = ops.kv_cache_attention(c.q.cuda(), ops.KVCache(c.cache.k, v, c.cache.k_scale, c.cache.v_scale), c.batch).cpu()
    keep = [d for d in range(128) if d != 77]
    assert torch.equal(got[:100], clean[:100]) and torch.equal(got[100:, :, keep], clean[100:, :, keep])
    assert torch.isnan(got[100:, :, 77]).all()
    for page, window in ((3, 0), (60, 150)):
        table = c.table.clone()
        table[0, page] = -1
        batch = ops.CacheBatch(table.cuda(), c.batch.lengths, c.batch.starts)
        want = ops.kv_cache_attention(c.q.cuda(), c.cache, c.batch, window=window).cpu()
        got = ops.kv_cache_attention(c.q.cuda(), c.cache, batch, window=window).cpu()
        sees = torch.tensor([not window or 4000 + i - window + 1 < 64 * page + 64 for i in range(160)])
        assert torch.isnan(got[sees]).all() and torch.equal(got[~sees], want[~sees])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1], [40], [150]])
def test_scores_that_grow(new, fp8):
    """Scores that rise along the keys by far more than exponentials hold, and fall again."""
    c = Case(new, [4200], 8, 1, 128, 64, fp8=fp8, seed=13)
    n = c.total[0]
    ramp = torch.cat((torch.linspace(0.0, 1.0, n // 2), torch.linspace(1.0, -1.0, n - n // 2)))
    if fp8:
        ramp = ramp / 0.02
    k = torch.zeros_like(c.cache.k).float()
    at = torch.arange(n)
    k[c.table[0].long()[at // 64].cuda(), 0, (at % 64).cuda(), 0] = ramp.cuda()
    k = k.to(c.cache.k.dtype)
    c.q[..., 0] = 8.0
    c.keys = [torch.zeros((n, 1, 128), dtype=torch.float64)]
    scale = c.k_scale.double() if fp8 else torch.ones(1).double()
    c.keys[0][:, 0, 0] = k.float().cpu()[c.table[0].long()[at // 64], 0, at % 64, 0].double() * scale
    c.cache = ops.KVCache(k, c.cache.v, c.cache.k_scale, c.cache.v_scale)
    _run(c, scale=12.0)      # up to about 100 above the first
    _run(c, scale=0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[1], [40], [150]])
def test_many_small_weights_beside_a_large_one(new, fp8):
    """The first key takes nearly all of each row, with a value of zero; the others, 2^-23 of it each, are the output."""
    c = Case(new, [4200], 8, 1, 128, 64, fp8=fp8, seed=14)
    n = c.total[0]
    k, v = torch.zeros_like(c.cache.k).float(), c.cache.v.float()
    first = int(c.table[0, 0])
    k[first, 0, 0, 0] = 16.0
    v[first, 0, :, 0] = 0.0
    c.q[..., 0] = 1.0
    scale = c.k_scale.double() if fp8 else torch.ones(1).double()
    c.keys = [torch.zeros((n, 1, 128), dtype=torch.float64)]
    c.keys[0][0, 0, 0] = 16.0 * scale[0]
    c.values[0][0] = 0.0
    c.cache = ops.KVCache(k.to(c.cache.k.dtype), v.to(c.cache.v.dtype), c.cache.k_scale, c.cache.v_scale)
    _run(c, scale=float(1.0 / scale[0]))


@pytest.mark.parametrize("new", [[1], [40], [150]])
def test_large_values(new):
    """Values near the end of bf16 (3.4e38), as far from it as 2^16 weights of up to 2^8 need."""
    c = Case(new, [4200], 8, 1, 128, 64, seed=15, v_spread=1e30)
    _run(c, scale=1.0)


# Groups of more query heads than a tile has rows.
GROUPS = [
    ([1, 0, 0], [200, 5, 0], 40, 1, 64, 16),
    ([1, 0], [900, 3], 32, 1, 128, 64),
    ([1, 2], [500, 30], 300, 1, 32, 16),
    ([1], [70], 514, 2, 96, 32),
    ([5], [4200], 320, 1, 128, 64),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_groups_larger_than_a_tile(case, fp8):
    _run(Case(*GROUPS[case], fp8=fp8, seed=300 + case))


@pytest.mark.parametrize("new", [[1, 1, 1], [90, 40]])
def test_windows_as_long_as_numbers(new):
    """A window past every sequence's length is none, and a length below the new tokens leaves rows before it empty."""
    c = Case(new, [100, 60, 5][:len(new)], 8, 2, 64, 16, seed=16)
    q = c.q.cuda()
    n = new[0]
    whole = ops.kv_cache_attention(q, c.cache, c.batch)
    short = ops.CacheBatch(c.batch.page_table, c.batch.lengths.clone(), c.batch.starts)
    short.lengths[0] = max(n // 2, 1)
    part = ops.kv_cache_attention(q, c.cache, short)
    assert (part[:n - max(n // 2, 1)] == 0).all() and torch.equal(part[n:], whole[n:])
    for window in (c.table.shape[1] * 16, 1 << 30, (1 << 31) - 1):
        assert torch.equal(ops.kv_cache_attention(q, c.cache, c.batch, window=window), whole)
        assert torch.equal(ops.kv_cache_attention(q, c.cache, short, window=window), part)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new", [[3], [90], [600]])
def test_a_row_that_is_not_finite_stays_alone(new, fp8):
    c = Case(new, [1000], 8, 2, 128, 64, fp8=fp8, seed=17)
    q = c.q.cuda()
    want = ops.kv_cache_attention(q, c.cache, c.batch)
    for bad in (float("nan"), float("inf")):
        spoiled = q.clone()
        spoiled[1, 3, 7] = bad
        got = ops.kv_cache_attention(spoiled, c.cache, c.batch)
        assert not torch.isfinite(got[1, 3]).any()
        got[1, 3] = want[1, 3]
        assert torch.equal(got, want)


def test_many_sequences():
    """More sequences than a wave's lanes, some of them split, in both kernels."""
    for first in (1, 2200):
        c = Case([first] + [i % 3 for i in range(299)], [4000] + [(37 * i) % 300 for i in range(299)], 4, 2, 64, 16, seed=first)
        _run(c)


def test_two_calls_at_once():
    """Two streams at work on the same cache and batch, each with its workspace."""
    c = Case([300, 1, 5], [3000, 4000, 90], 8, 1, 128, 64, seed=18)
    q = c.q.cuda()
    want = ops.kv_cache_attention(q, c.cache, c.batch)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for s, g in zip(streams, got):
            with torch.cuda.stream(s):
                g.append(ops.kv_cache_attention(q, c.cache, c.batch))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for g in got for x in g)


@pytest.mark.parametrize("new", [[1], [40], [150]])
def test_keys_of_minus_infinity_count_for_nothing(new):
    """The first keys' scores are -Inf, those of all others far below what exponentials hold."""
    c = Case(new, [4200], 8, 1, 128, 64, seed=19)
    q = c.q.cuda()
    q[..., 0], q[..., 1] = 1.0, 8.0
    got = []
    for low in (float("-inf"), -1e4):    # (weights of exactly 0 either way)
        k = c.cache.k.clone()
        at = torch.arange(c.total[0])
        page, slot = c.table[0].long()[at // 64].cuda(), (at % 64).cuda()
        k[page, 0, slot, 1] = -8.0
        k[page[:100], 0, slot[:100], 0] = low
        got.append(ops.kv_cache_attention(q, ops.KVCache(k, c.cache.v), c.batch, scale=4.0))
    assert torch.isfinite(got[0]).all() and (got[0] != 0).any(-1).all()
    assert torch.equal(*got)
