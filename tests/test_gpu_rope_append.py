"""rope_rotate and kv_cache_append against float64: layouts, parts of the head, far positions, gradients, types,
distances, pages, FP8 rounding, and what is left alone."""
import math

import pytest
import torch

from nvfp4_block_scaled_moe_amd import ops
from tests.attention_util import BF, F8, HALF, Case, check, frequencies, rotated

pytestmark = pytest.mark.gpu

# An angle becomes float32 as half turns in [-1, 1], off by 2^-25 of a half turn, its cosine and sine by a few
# 2^-24; products and sum in float32 add as much again.
TURN = 2.0 ** -21


def _tolerance(y, size, dtype):
    return HALF[dtype] * (y.abs() + TURN * size) + TURN * size


# (T, H, D, rot, start, interleaved)
ROPE = [
    (1, 1, 2, 2, 0, False),
    (1, 8, 64, 64, 0, False),
    (3, 5, 64, 32, 0, True),
    (7, 2, 96, 24, 72, False),
    (65, 3, 128, 64, 64, True),
    (33, 64, 128, 128, 0, False),
    (5, 1, 80, 10, 3, True),
    (4, 3, 20, 12, 4, False),
    (300, 1, 32, 16, 8, True),
    (1000, 4, 192, 64, 128, False),
    (2, 2, 4096, 4096, 0, False),
]


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("case", ROPE)
def test_rope(case, grad, dtype):
    T, H, D, rot, start, inter = case
    g = torch.Generator().manual_seed(T + D)
    x = torch.randn((T, H, D), generator=g).to(dtype)
    pos = torch.randint(0, 1_000_000, (T,), generator=g)
    pos[0] = 0
    f = frequencies(rot)
    want, size = rotated(x, pos, f, start, inter, 1.25, -1.0 if grad else 1.0)
    rope = ops.Rope(f.cuda(), start, inter, 1.25)
    tol = _tolerance(want, size, dtype)
    for p in (pos.to(torch.int32), pos):
        check(ops.rope_rotate(x.cuda(), p.cuda(), rope, grad=grad), want, tol)
    # in place; and views whose rows and heads lie apart, at odd addresses
    y = x.cuda()
    assert ops.rope_rotate(y, pos.cuda(), rope, grad=grad, out=y) is y
    check(y, want, tol)
    wide = torch.full((T, H + 1, D + 3), 5.0, dtype=dtype, device="cuda")
    view = wide[:, 1:, 1:D + 1]
    view.copy_(x)
    room = torch.full((T, H + 2, D + 1), 5.0, dtype=dtype, device="cuda")
    ops.rope_rotate(view, pos.cuda(), rope, grad=grad, out=room[:, 2:, :D])
    check(room[:, 2:, :D], want, tol)
    assert (room[:, :2] == 5.0).all() and (room[:, :, D:] == 5.0).all()


def test_rope_positions():
    """Negative ones, the largest int32 and ones past it."""
    pos = torch.tensor([-1, -12345, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 1, 0, 5])
    f = frequencies(64)
    x = torch.randn((7, 2, 64), generator=torch.Generator().manual_seed(0))
    want, size = rotated(x, pos, f)
    # (float64 angles of 2^40 radians: off by 2^-13 turns at most, on either side)
    tol = _tolerance(want, size, torch.float32) + size * (pos.double().abs() * 2.0 ** -50)[:, None, None]
    check(ops.rope_rotate(x.cuda(), pos.cuda(), ops.Rope(f.cuda())), want, tol)


def test_rope_gradient_by_differences():
    """The formula's gradient of sum(g * out) against central differences of the call in float32, which is linear:
    a step of 1 gives the derivative up to roundings of the sums."""
    gen = torch.Generator().manual_seed(3)
    T, H, D = 5, 2, 64
    x, g = torch.randn((T, H, D), generator=gen).cuda(), torch.randn((T, H, D), generator=gen).cuda()
    pos = torch.tensor([0, 3, 77, 4000, 100_000]).cuda()
    for inter in (False, True):
        rope = ops.Rope(frequencies(32).cuda(), 16, inter, 0.75)
        dx = ops.rope_rotate(g, pos, rope, grad=True)
        for _ in range(20):
            step = torch.randn((T, H, D), generator=gen).cuda()
            up, down = ops.rope_rotate(x + step, pos, rope), ops.rope_rotate(x - step, pos, rope)
            got = float((dx.double() * step.double()).sum())
            want = float((g.double() * (up.double() - down.double())).sum()) / 2.0
            # each element: roundings of x +- step, of two products and a sum, of the two outputs
            tol = 8.0 * 2.0 ** -21 * float((g.abs().double() * (x.abs() + step.abs() + 1.0).double()).sum() + (dx.abs() * step.abs()).sum())
            assert abs(got - want) <= tol, (got, want, tol)


def test_rope_nothing():
    rope = ops.Rope(frequencies(8).cuda())
    assert ops.rope_rotate(torch.empty((0, 3, 8), device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), rope).shape == (0, 3, 8)


def test_rope_nan_and_inf_stay_in_their_pair():
    f = frequencies(16)
    x = torch.randn((3, 1, 16), generator=torch.Generator().manual_seed(1))
    clean = ops.rope_rotate(x.cuda(), torch.arange(3).cuda(), ops.Rope(f.cuda())).cpu()
    x[1, 0, 2], x[2, 0, 9] = math.nan, math.inf
    got = ops.rope_rotate(x.cuda(), torch.arange(3).cuda(), ops.Rope(f.cuda())).cpu()
    hit = torch.zeros((3, 1, 16), dtype=torch.bool)
    hit[1, 0, [2, 10]] = True
    hit[2, 0, [1, 9]] = True
    assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], clean[~hit])


# (new, before, Hq, Hkv, D, page, rot, start, interleaved)
APPEND = [
    ([1], [0], 1, 1, 32, 16, 32, 0, False),
    ([1], [700], 64, 8, 128, 64, 128, 0, False),
    ([3, 0, 1, 9], [0, 5, 15, 31], 20, 4, 96, 16, 32, 0, True),
    ([100, 33], [60, 1], 4, 2, 64, 32, 64, 0, True),
    ([70, 1, 200], [0, 999, 77], 6, 3, 160, 128, 80, 80, False),
    ([17], [1000], 2, 1, 256, 256, 10, 3, False),
    ([64] * 3, [64, 0, 128], 8, 8, 64, 64, 64, 0, False),
    ([1] * 40, [7 * i for i in range(40)], 8, 2, 128, 16, 64, 64, False),
]


def _appended(c, k, v, f, start, inter, mag, positions=None):
    """float64 of the turned keys and queries, and where each new token goes: (sequence, position)."""
    where = [(b, ctx + i) for b, (n, ctx) in enumerate(zip(c.new, c.ctx)) for i in range(n)]
    pos = torch.tensor([p for _, p in where]) if positions is None else positions
    return where, rotated(c.q[:c.T], pos, f, start, inter, mag), rotated(k, pos, f, start, inter, mag)


def _check_cache(c, before, where, want_k, size_k, v):
    """The new tokens' places hold what they should, every other place its old bits."""
    kc, vc = c.cache.k.cpu(), c.cache.v.cpu()
    old_k, old_v = before
    bits = torch.uint8 if c.fp8 else torch.int16
    mask = torch.zeros((c.pages, c.page), dtype=torch.bool)
    for t, (b, p) in enumerate(where):
        pg, sl = int(c.table[b, p // c.page]), p % c.page
        mask[pg, sl] = True
        gk, gv = kc[pg, :, sl].double(), vc[pg, :, :, sl].double()
        if c.fp8:
            for got, want, size, s in ((gk, want_k[t], size_k[t], c.k_scale), (gv, v[t].double(), torch.zeros(v[t].shape), c.v_scale)):
                s = s.double().view(-1, 1)
                x = (want / s).clamp(-448, 448)
                # half a step of E4M3 (2^-10 below its normal numbers); the float32 quotient before it
                slack = TURN * size / s + 2.0 ** -22 * x.abs()
                check(got, x, torch.maximum(2.0 ** -4 * (x.abs() + slack), torch.tensor(2.0 ** -10).double()) + slack, "fp8")
        else:
            check(gk, want_k[t], _tolerance(want_k[t], size_k[t], BF), "k")
            assert torch.equal(gv, v[t].double())
    keep = ~mask
    assert torch.equal(kc.view(bits).transpose(1, 2)[keep], old_k.view(bits).transpose(1, 2)[keep])
    assert torch.equal(vc.view(bits).permute(0, 3, 1, 2)[keep], old_v.view(bits).permute(0, 3, 1, 2)[keep])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case, fp8):
    new, ctx, Hq, Hkv, D, page, rot, start, inter = APPEND[case]
    c = Case(new, ctx, Hq, Hkv, D, page, fp8=fp8, seed=case, spare_rows=2)
    g = torch.Generator().manual_seed(50 + case)
    rows = c.q.shape[0]
    qkv = torch.randn((rows, Hq + 2 * Hkv, D), generator=g).to(BF)
    c.q = qkv[:, :Hq]
    k, v = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    f = frequencies(rot)
    before = c.cache.k.cpu(), c.cache.v.cpu()
    where, (want_q, size_q), (want_k, size_k) = _appended(c, k[:c.T], v, f, start, inter, 1.5)
    x = qkv.cuda()
    rope = ops.Rope(f.cuda(), start, inter, 1.5)
    out = torch.full((rows, Hq, D), 3.0, dtype=BF, device="cuda")
    got = ops.kv_cache_append(c.cache, c.batch, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q=x[:, :Hq], rope=rope, q_out=out)
    assert got is out and (got[c.T:] == 3.0).all()
    check(got[:c.T], want_q, _tolerance(want_q, size_q, BF), "q")
    assert torch.equal(x.cpu(), qkv)
    _check_cache(c, before, where, want_k, size_k, v)
    # the queries in place, in the projection's rows; and at an address that allows no wide access
    kept = c.cache.k.clone(), c.cache.v.clone()
    bits = torch.uint8 if fp8 else torch.int16
    q = x[:, :Hq]
    assert ops.kv_cache_append(c.cache, c.batch, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q=q, rope=rope, q_out=q) is q
    assert torch.equal(x[:c.T, :Hq], got[:c.T]) and torch.equal(x[:, Hq:].cpu(), qkv[:, Hq:])
    assert torch.equal(x[c.T:].cpu(), qkv[c.T:])
    room = torch.empty(qkv.numel() + 1, dtype=BF, device="cuda")[1:].view(qkv.shape)
    room.copy_(qkv)
    c.cache.k.view(bits).zero_(), c.cache.v.view(bits).zero_()
    odd = ops.kv_cache_append(c.cache, c.batch, room[:, Hq:Hq + Hkv], room[:, Hq + Hkv:], q=room[:, :Hq], rope=rope)
    assert torch.equal(odd[:c.T], got[:c.T])
    zeros = [torch.zeros_like(t.cpu().view(bits)).view(t.dtype) for t in kept]
    _check_cache(c, zeros, where, want_k, size_k, v)


def test_append_without_queries_or_rotation():
    c = Case([5, 40], [30, 0], 2, 2, 64, 16, seed=20)
    g = torch.Generator().manual_seed(21)
    k, v = torch.randn((45, 2, 64), generator=g).to(BF), torch.randn((45, 2, 64), generator=g).to(BF)
    before = c.cache.k.cpu(), c.cache.v.cpu()
    assert ops.kv_cache_append(c.cache, c.batch, k.cuda(), v.cuda()) is None
    where = [(b, ctx + i) for b, (n, ctx) in enumerate(zip(c.new, c.ctx)) for i in range(n)]
    _check_cache(c, before, where, k.double(), torch.zeros(k.shape), v)


def test_append_positions():
    """Angles at positions of the caller's own; the places stay the sequences'."""
    for dt in (torch.int32, torch.int64):
        c = Case([5, 9], [30, 2], 2, 2, 64, 16, seed=22)
        g = torch.Generator().manual_seed(23)
        k, v = torch.randn((14, 2, 64), generator=g).to(BF), torch.randn((14, 2, 64), generator=g).to(BF)
        pos = torch.randint(-5, 100_000, (14,), generator=g)
        f = frequencies(64)
        before = c.cache.k.cpu(), c.cache.v.cpu()
        where, (want_q, size_q), (want_k, size_k) = _appended(c, k, v, f, 0, False, 1.0, pos)
        q = ops.kv_cache_append(c.cache, c.batch, k.cuda(), v.cuda(), q=c.q.cuda(), rope=ops.Rope(f.cuda()), positions=pos.to(dt).cuda())
        check(q, want_q, _tolerance(want_q, size_q, BF))
        _check_cache(c, before, where, want_k, size_k, v)


def test_append_extreme_values_to_fp8():
    """Saturation, NaN, infinities, zeros of both signs and numbers below the smallest code."""
    c = Case([1], [0], 1, 1, 32, 16, fp8=True, seed=24)
    c.cache.k_scale.fill_(0.5), c.cache.v_scale.fill_(0.5)
    x = torch.zeros((1, 1, 32))
    x[0, 0, :12] = torch.tensor([224.0, 225.0, -1e30, math.inf, -math.inf, math.nan, -0.0, 2.0 ** -11, 2.0 ** -10, 3 * 2.0 ** -11, 216.0, 232.0])
    ops.kv_cache_append(c.cache, c.batch, x.to(BF).cuda(), x.to(BF).cuda())
    want = (x.to(BF).float() / 0.5).clamp(-448, 448).to(F8)[0, 0].float()
    pg = int(c.table[0, 0])
    for got in (c.cache.k[pg, 0, 0].float().cpu(), c.cache.v[pg, 0, :, 0].float().cpu()):
        assert torch.equal(torch.nan_to_num(got, nan=9e9), torch.nan_to_num(want, nan=9e9)), (got, want)


def test_append_leaves_out_tokens_without_a_page():
    c = Case([4, 40], [14, 20], 2, 2, 64, 16, seed=25)
    g = torch.Generator().manual_seed(26)
    k, v = torch.randn((44, 2, 64), generator=g).to(BF), torch.randn((44, 2, 64), generator=g).to(BF)
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[0, 1] = bad       # tokens 16, 17 of the first sequence
        before = c.cache.k.cpu(), c.cache.v.cpu()
        ops.kv_cache_append(c.cache, ops.CacheBatch(table.cuda(), c.batch.lengths, c.batch.starts), k.cuda(), v.cuda(), q=c.q.cuda())
        where = [(0, 14), (0, 15)] + [(1, 20 + i) for i in range(40)]
        pick = [0, 1] + list(range(4, 44))
        _check_cache(c, before, where, k[pick].double(), torch.zeros((42, 2, 64)), v[pick])
    # lengths past the table's columns and below the new tokens; starts outside the rows
    i32 = dict(dtype=torch.int32, device="cuda")
    for lengths, starts in (([10 ** 6, 2 ** 31 - 1], [0, 4, 44]), ([0, -7], [0, 4, 44]), ([18, 60], [44, 44, 44]),
                            ([18, 60], [2 ** 31 - 1] * 3), ([18, 60], [5, 5, -3])):
        before = c.cache.k.cpu(), c.cache.v.cpu()
        b = ops.CacheBatch(c.batch.page_table, torch.tensor(lengths, **i32), torch.tensor(starts, **i32))
        ops.kv_cache_append(c.cache, b, k.cuda(), v.cuda(), q=c.q.cuda())
        _check_cache(c, before, [], None, None, None)


def test_append_many_sequences():
    """More sequences than have their starts in LDS."""
    B = 1500
    c = Case([1 if b % 3 else 0 for b in range(B)], [b % 40 for b in range(B)], 2, 1, 32, 16, seed=27)
    g = torch.Generator().manual_seed(28)
    k, v = torch.randn((c.T, 1, 32), generator=g).to(BF), torch.randn((c.T, 1, 32), generator=g).to(BF)
    f = frequencies(32)
    before = c.cache.k.cpu(), c.cache.v.cpu()
    where, (want_q, size_q), (want_k, size_k) = _appended(c, k, v, f, 0, True, 1.0)
    q = ops.kv_cache_append(c.cache, c.batch, k.cuda(), v.cuda(), q=c.q.cuda(), rope=ops.Rope(f.cuda(), interleaved=True))
    check(q, want_q, _tolerance(want_q, size_q, BF))
    _check_cache(c, before, where, want_k, size_k, v)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_then_attend_as_a_sequence_grows(fp8):
    """A prompt, a chunk and single tokens through append and attention, captured and replayed for the last ones, against
    float64 attention over what the cache holds."""
    Hq, Hkv, D, page, n = 8, 2, 64, 16, 130
    g = torch.Generator().manual_seed(31)
    qkv = torch.randn((n, Hq + 2 * Hkv, D), generator=g).to(BF).cuda()
    scale = torch.full((Hkv,), 0.01, device="cuda") if fp8 else None
    cache = ops.kv_cache(12, Hkv, page, D, F8 if fp8 else BF, k_scale=scale, v_scale=scale)
    rope = ops.Rope(frequencies(D).cuda())
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[7, 3, 0, 11, 2, 9, 5, 1, 10]], **i32)
    lengths, starts = torch.zeros(1, **i32), torch.zeros(2, **i32)
    batch = ops.CacheBatch(table, lengths, starts)
    rows, out = torch.empty((1, Hq + 2 * Hkv, D), dtype=BF, device="cuda"), torch.empty((1, Hq, D), dtype=BF, device="cuda")

    def step(x, o=None):
        q = ops.kv_cache_append(cache, batch, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q=x[:, :Hq], rope=rope)
        return q, ops.kv_cache_attention(q, cache, batch, out=o)

    got, queries = [], []
    for a, b in ((0, 77), (77, 110)):
        lengths.fill_(b)
        starts[1] = b - a
        q, o = step(qkv[a:b])
        queries.append(q), got.append(o)
    starts[1] = 1
    lengths.fill_(110)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lengths.add_(1)
        q1, _ = step(rows, out)
    for t in range(110, n):
        rows.copy_(qkv[t:t + 1])
        graph.replay()
        queries.append(q1.clone()), got.append(out.clone())
    q, o = torch.cat(queries), torch.cat(got)
    want_q, size_q = rotated(qkv[:, :Hq].cpu(), torch.arange(n), frequencies(D))
    check(q, want_q, _tolerance(want_q, size_q, BF))
    c = Case([n], [0], Hq, Hkv, D, page)
    order = torch.arange(n)
    kc, vc = (t.float().cpu().double() * (0.01 if fp8 else 1.0) for t in (cache.k, cache.v))
    if fp8:   # (the scale is a float32)
        kc, vc = (t.float().cpu().double() * float(scale[0]) for t in (cache.k, cache.v))
    pg = table.cpu()[0].long()[order // page]
    c.keys, c.values, c.q = [kc[pg, :, order % page]], [vc[pg, :, :, order % page]], q.cpu()
    want, tol = c.attention()
    check(o, want, tol + 2.0 ** -8 * want.abs())
    # the cache holds the turned keys and the values, within its type's rounding
    want_k, size_k = rotated(qkv[:, Hq:Hq + Hkv].cpu(), torch.arange(n), frequencies(D))
    tol_k = _tolerance(want_k, size_k, BF) if not fp8 else 2.0 ** -4 * want_k.abs() + 2.0 ** -10 * 0.01 + 2.0 ** -20 * size_k
    check(c.keys[0], want_k, tol_k)
