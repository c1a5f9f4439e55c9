"""layer.attention_block_forward: its parts called one by one, the block against float64, and whole decoder layers (this block
and the MoE block), eager and captured."""
import math

import pytest
import torch

from nvfp4_block_scaled_moe_amd import inputs, layer, ops
from tests.attention_util import BF, F8, frequencies, rotated

pytestmark = pytest.mark.gpu

H, HQ, HKV, D, PAGE = 256, 8, 2, 64, 16


def _weights(mx=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for R, C in (((HQ + 2 * HKV) * D, H), (H, HQ * D)):
        w = torch.randn((1, R, C), generator=g, device="cuda") * C ** -0.5
        out.append(ops.mxfp4_weights_tile(*ops.mxfp4_quantize(w)) if mx else ops.nvfp4_weights_tile(*ops.nvfp4_quantize(w)))
    return layer.AttentionWeights(out[0], out[1], HQ)


def _dequantized(w):
    """float64 rows of a matrix, as its products with unit rows."""
    eye = torch.eye(w.C, device="cuda").to(BF)
    mv = ops.nvfp4_matvec if isinstance(w, ops.TiledWeights) else ops.mxfp4_matvec
    return torch.cat([mv(eye[i:i + 16], w, out_dtype=torch.float32) for i in range(0, w.C, 16)]).t().double().cpu()


def _setting(new, ctx, dtype=BF, seed=1):
    g = torch.Generator().manual_seed(seed)
    total = [n + c for n, c in zip(new, ctx)]
    used = [-(-t // PAGE) for t in total]
    order = torch.randperm(sum(used) + 2, generator=g).to(torch.int32)
    table = torch.full((len(new), max(used) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    scale = torch.full((HKV,), 0.02, device="cuda") if dtype == F8 else None
    cache = ops.kv_cache(sum(used) + 2, HKV, PAGE, D, dtype, k_scale=scale, v_scale=scale)
    cache.k.copy_(torch.randn(cache.k.shape, generator=g).to(dtype).cuda())
    cache.v.copy_(torch.randn(cache.v.shape, generator=g).to(dtype).cuda())
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = ops.CacheBatch(table.cuda(), torch.tensor(total, **i32), torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], **i32))
    T = sum(new)
    resid = torch.randn((T, H), generator=g).cuda()
    pre = (1.0 + 0.1 * torch.randn(H, generator=g)).cuda()
    return cache, batch, resid, pre


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("new,few", [([1, 2, 1], None), ([1, 2, 1], False), ([40, 7], None)])
def test_block_is_its_parts(new, few, mx):
    w = _weights(mx)
    cache, batch, resid, pre = _setting(new, [30, 0, 100][:len(new)])
    other = ops.KVCache(cache.k.clone(), cache.v.clone())
    x = ops.moe_block_norm(resid, pre_w=pre)[1]
    rope = ops.Rope(frequencies(D).cuda())
    r, nxt = layer.attention_block_forward(resid, x, w, cache, batch, rope=rope, post_w=pre, scale=0.5, pre_w=pre, few=few)
    T = x.shape[0]
    use_few = T <= 16 if few is None else few
    qkv = layer._projection(x, w.qkv, BF, use_few).view(T, HQ + 2 * HKV, D)
    q = ops.kv_cache_append(other, batch, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], q=qkv[:, :HQ], rope=rope)
    a = ops.kv_cache_attention(q, other, batch)
    y = layer._projection(a.view(T, HQ * D), w.o, torch.float32, use_few)
    want = ops.moe_block_norm(resid, y, post_w=pre, scale=0.5, pre_w=pre)
    assert torch.equal(r, want[0]) and torch.equal(nxt, want[1])
    assert torch.equal(cache.k, other.k) and torch.equal(cache.v, other.v)


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("new", [[1, 3], [50, 33]])
def test_block_against_float64(new, window):
    """NVFP4 weights, bf16 cache. Roundings, of half a bf16 step (2^-8) at most each: q, k and v twice (the projection, the
    rotation), weights, the attention's output; a score of size s moves its weight by s times q's and k's. Scores stay
    below 4 here, so that the output is off by (2 + 1 + 1 + 2 * 2 * 4) * 2^-8 of its norm at most."""
    w = _weights()
    ctx = [30, 100]
    cache, batch, resid, pre = _setting(new, ctx)
    keys, values = cache.k.double().cpu(), cache.v.double().cpu()
    x = ops.moe_block_norm(resid, pre_w=pre)[1]
    f = frequencies(D)
    r, _ = layer.attention_block_forward(resid, x, w, cache, batch, rope=ops.Rope(f.cuda()), window=window, attention_scale=D ** -0.5 / 4)
    qkv = (x.double().cpu() @ _dequantized(w.qkv).t()).view(-1, HQ + 2 * HKV, D)
    y, at = [], 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        p = torch.arange(n + c)
        pg = batch.page_table.cpu()[b].long()[p // PAGE]
        k, v = keys[pg, :, p % PAGE], values[pg, :, :, p % PAGE]
        mine = qkv[at:at + n]
        at += n
        pos = torch.arange(c, c + n)
        q = rotated(mine[:, :HQ], pos, f)[0]
        k[c:], v[c:] = rotated(mine[:, HQ:HQ + HKV], pos, f)[0], mine[:, HQ + HKV:]
        far = pos[:, None] - p
        hidden = (far < 0) | ((far >= window) if window else torch.zeros_like(far, dtype=torch.bool))
        for_heads = []
        for h in range(HQ):
            s = (q[:, h] @ k[:, h // (HQ // HKV)].t()) * (D ** -0.5 / 4)
            assert s.abs().max() < 4.0
            for_heads.append(torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v[:, h // (HQ // HKV)])
        y.append(torch.stack(for_heads, 1).reshape(n, HQ * D))
    want = torch.cat(y) @ _dequantized(w.o).t()
    got = (r - resid).double().cpu()
    # (the residual's float32 sum: 2^-24 of it)
    off = float((got - want).norm() / want.norm())
    assert off <= 20 * 2.0 ** -8 + 2.0 ** -20, off


@pytest.mark.parametrize("new", [[1, 2], [30, 5]])
def test_layer_with_queries_alone(new):
    """A layer that reads the keys of the one before: nothing is written, queries are turned at the positions given. Its
    queries' weights are the first rows of a whole projection, whose own block, with keys in place, gives the same."""
    g = torch.Generator(device="cuda").manual_seed(9)
    full = torch.randn((1, (HQ + 2 * HKV) * D, H), generator=g, device="cuda") * H ** -0.5
    tile = lambda t: ops.mxfp4_weights_tile(*ops.mxfp4_quantize(t))  # noqa: E731  (scales by 32 columns: rows stand alone)
    o = _weights(mx=True).o
    cache, batch, resid, pre = _setting(new, [30, 100])
    x = ops.moe_block_norm(resid, pre_w=pre)[1]
    rope = ops.Rope(frequencies(D).cuda())
    r0, n0 = layer.attention_block_forward(resid, x, layer.AttentionWeights(tile(full), o, HQ), cache, batch, rope=rope, pre_w=pre)
    kept = cache.k.clone(), cache.v.clone()
    alone = layer.AttentionWeights(tile(full[:, :HQ * D].contiguous()), o, HQ)
    pos = torch.cat([torch.arange(c, c + n) for n, c in zip(new, [30, 100])]).cuda()
    r1, n1 = layer.attention_block_forward(resid, x, alone, cache, batch, rope=rope, positions=pos, pre_w=pre)
    assert torch.equal(cache.k, kept[0]) and torch.equal(cache.v, kept[1])
    assert torch.equal(r0, r1) and torch.equal(n0, n1)
    with pytest.raises(ValueError, match="positions"):
        layer.attention_block_forward(resid, x, alone, cache, batch, rope=rope)


@pytest.mark.parametrize("dtype", [BF, F8])
@pytest.mark.parametrize("new", [[1, 1, 1], [20, 1, 9]])
def test_decoder_layers(new, dtype):
    """Two layers of attention and MoE blocks, eager and as a graph replayed with other inputs between."""
    wl = inputs.WORKLOADS["tiny"]
    experts = layer.quantize_experts(wl, "cuda")
    router_w = torch.randn((wl.E, H), generator=torch.Generator().manual_seed(4)).cuda() / 16
    router = lambda rows: rows.float() @ router_w.t()  # noqa: E731
    layers = [_weights(seed=s) for s in (5, 6)]
    cache0, batch, resid, pre = _setting(new, [10, 40, 3], dtype)
    caches = [ops.KVCache(cache0.k.view(torch.uint8).clone().view(dtype) if dtype == F8 else cache0.k.clone(),
                          cache0.v.view(torch.uint8).clone().view(dtype) if dtype == F8 else cache0.v.clone(), cache0.k_scale, cache0.v_scale)
              for _ in layers]
    rope = ops.Rope(frequencies(D).cuda(), interleaved=True)

    def run(h):
        x = ops.moe_block_norm(h, pre_w=pre)[1]
        for w, c in zip(layers, caches):
            h, x = layer.attention_block_forward(h, x, w, c, batch, rope=rope, pre_w=pre)
            h, x = layer.moe_block_forward(h, x, wl.k, experts, router, pre_w=pre)
        return h, x

    first = run(resid)
    assert all(torch.isfinite(t).all() for t in first)
    graph = torch.cuda.CUDAGraph()
    here = resid.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = run(here)
    for scale in (1.0, 0.5, 1.0):
        here.copy_(resid * scale)
        graph.replay()
        torch.cuda.synchronize()
        want = run(resid * scale)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert torch.equal(out[0], first[0])
