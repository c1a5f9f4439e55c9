"""What the attention half's calls refuse before they reach the device, and the frequencies of rotary positions, on the CPU."""
import math

import pytest
import torch

from nvfp4_block_scaled_moe_amd import _lib, layer, ops

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
P = 1 << 20   # (addresses that are never read)


def _call(name, **args):
    fn = getattr(_lib.load(), name)
    st = fn(*args.values())
    return st, _lib.load().nvfp4moe_last_error().decode()


ROPE = dict(x=P, dtype=_lib.BF16, x_row=512, x_head=64, T=4, H=8, D=64, positions=P, pos_bytes=4, freqs=P, rot=64, start=0,
            interleaved=0, grad=0, magnitude=1.0, out=2 * P, o_row=512, o_head=64, stream=None)
APPEND = dict(q=P, q_row=1024, q_head=64, k=P + 1024, k_row=1024, k_head=64, v=P + 1280, v_row=1024, v_head=64, T=4, Hq=8, Hkv=2,
              D=64, positions=None, pos_bytes=4, freqs=P, rot=64, start=0, interleaved=0, magnitude=1.0, page_table=P, ld_table=5,
              cols=5, lengths=P, starts=P, B=2, k_cache=4 * P, v_cache=8 * P, fp8=0, pages=6, page=16, k_scale=None, v_scale=None,
              q_out=2 * P, qo_row=512, qo_head=64, stream=None)
ATTEND = dict(q=P, q_row=512, q_head=64, T=4, Hq=8, Hkv=2, D=64, page_table=P, ld_table=5, cols=5, lengths=P, starts=P, B=2,
              k_cache=4 * P, v_cache=8 * P, fp8=0, pages=6, page=16, k_scale=None, v_scale=None, scale=0.125, window=0, out=2 * P,
              o_row=512, o_head=64, ws=16 * P, ws_bytes=1 << 40, stream=None)


def _refused(name, base, change, word=""):
    st, why = _call(name, **{**base, **change})
    assert st in (_lib.ERR_INVALID_ARG, _lib.ERR_WORKSPACE) and why.startswith(name) and word in why, (change, st, why)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(out=None), dict(positions=None), dict(freqs=None), dict(dtype=7), dict(T=-1), dict(H=0), dict(D=0),
    dict(H=1 << 20), dict(x=P + 1), dict(out=2 * P + 1), dict(pos_bytes=2), dict(positions=P + 2), dict(pos_bytes=8, positions=P + 4),
    dict(freqs=P + 4), dict(rot=0), dict(rot=63), dict(rot=66), dict(rot=4098, D=8192, x_head=8192, x_row=1 << 17, o_head=8192, o_row=1 << 17),
    dict(start=-1), dict(start=2), dict(interleaved=2), dict(grad=2), dict(magnitude=math.inf), dict(magnitude=math.nan),
    dict(x_head=63), dict(x_row=511), dict(o_head=63), dict(o_row=100), dict(x_row=-512), dict(out=P + 128), dict(out=P, o_row=1024),
    dict(out=P + 64 * 2), dict(x_row=1 << 40), dict(freqs=2 * P + 1024), dict(positions=2 * P - 8)])
def test_rope_refuses(change):
    _refused("rope_rotate", ROPE, change)


@pytest.mark.parametrize("change", [
    dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(k_cache=None), dict(v_cache=None), dict(page_table=None),
    dict(lengths=None), dict(starts=None), dict(T=-2), dict(B=0), dict(Hkv=0), dict(Hkv=3), dict(Hq=0), dict(D=48), dict(D=0),
    dict(D=288), dict(page=8), dict(page=24), dict(page=2048), dict(pages=0), dict(cols=0), dict(ld_table=4), dict(fp8=2),
    dict(k_scale=P), dict(v_scale=P), dict(fp8=1, k_scale=P + 2), dict(k_cache=4 * P + 8), dict(v_cache=8 * P + 2), dict(k=P + 1),
    dict(rot=66), dict(rot=7), dict(start=1), dict(interleaved=-1), dict(magnitude=math.nan), dict(positions=P, pos_bytes=3),
    dict(positions=P + 4, pos_bytes=8), dict(k_row=64), dict(v_head=32), dict(q_row=64), dict(qo_row=64), dict(page_table=P + 2),
    dict(q_out=P + 128, qo_row=1024), dict(q_out=P + 1024, qo_row=1024), dict(q_out=4 * P), dict(k_cache=P - 1024), dict(v_cache=4 * P + 64),
    dict(k=8 * P + 256), dict(freqs=2 * P + 512), dict(positions=4 * P + 4, pos_bytes=4), dict(page_table=8 * P - 4), dict(lengths=2 * P),
    dict(starts=4 * P + 16), dict(fp8=1, k_scale=8 * P + 4)])
def test_append_refuses(change):
    _refused("kv_cache_append", APPEND, change)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(out=None), dict(k_cache=None), dict(v_cache=None), dict(page_table=None), dict(lengths=None), dict(starts=None),
    dict(T=-1), dict(B=0), dict(Hq=7), dict(Hq=0), dict(Hkv=0), dict(D=40), dict(D=512), dict(page=10), dict(page=8), dict(pages=-1),
    dict(cols=0), dict(ld_table=1), dict(fp8=-1), dict(k_scale=P), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
    dict(scale=math.inf), dict(window=-1), dict(q=P + 8), dict(out=2 * P + 2), dict(q_row=516), dict(q_head=68), dict(o_head=68, o_row=552),
    dict(q_row=448), dict(out=P), dict(out=P + 128), dict(out=4 * P), dict(out=8 * P + 16), dict(T=1 << 28), dict(B=1 << 27),
    dict(ws=None), dict(ws=16 * P + 8), dict(ws_bytes=1000), dict(ws=P + 256), dict(ws=2 * P + 4080), dict(ws=8 * P), dict(page_table=16 * P + 4),
    dict(lengths=2 * P + 4), dict(starts=2 * P - 4), dict(fp8=1, v_scale=2 * P + 8), dict(T=1 << 24)])
def test_attention_refuses(change):
    _refused("kv_cache_attention", ATTEND, change)


def test_workspace_sizes():
    size = _lib.load().kv_cache_attention_workspace_size
    assert size(64, 64, 64, 8, 128) > 0 and size(4096, 1, 64, 8, 128) > size(64, 64, 64, 8, 128)
    for bad in ((0, 1, 8, 2, 64), (1, 0, 8, 2, 64), (1, 1, 7, 2, 64), (1, 1, 8, 0, 64), (1, 1, 8, 2, 65), (1, 1, 8, 2, 512), (1 << 30, 1, 8, 2, 64)):
        assert size(*bad) == 0
    assert _call("kv_cache_attention", **{**ATTEND, "ws_bytes": size(4, 2, 8, 2, 64) - 1})[0] == _lib.ERR_WORKSPACE


def test_nothing_to_do_is_no_call():
    for name, base in (("rope_rotate", ROPE), ("kv_cache_append", APPEND), ("kv_cache_attention", ATTEND)):
        assert _call(name, **{**base, "T": 0})[0] == _lib.OK


def _cache(dtype=BF, pages=3, heads=2, page=16, D=64, **kw):
    return ops.kv_cache(pages, heads, page, D, dtype, device="cpu", **kw)


def _batch(B=2, cols=3):
    i = dict(dtype=torch.int32)
    return ops.CacheBatch(torch.zeros((B, cols), **i), torch.ones((B,), **i), torch.arange(B + 1, **i))


def test_handles_are_checked_when_made():
    f64 = torch.ones(8, dtype=torch.float64)
    for bad in (f64.float(), f64.view(2, 4), torch.ones(16, dtype=torch.float64)[::2], f64[:0]):
        with pytest.raises(ValueError, match="Rope"):
            ops.Rope(bad)
    with pytest.raises(ValueError, match="Rope"):
        ops.Rope(f64, start=-1)
    with pytest.raises(ValueError, match="Rope"):
        ops.Rope(f64, magnitude=math.nan)
    assert ops.Rope(f64).rot == 16
    c = _cache()
    for k, v in ((c.k.float(), c.v.float()), (c.k, c.v.float()), (c.k, c.k), (c.k[0], c.v), (c.k.transpose(0, 1), c.v),
                 (c.k, c.v.transpose(2, 3).contiguous().transpose(2, 3)), (c.k.to(F8), c.v)):
        with pytest.raises(ValueError, match="KVCache"):
            ops.KVCache(k, v)
    scale = torch.ones(2)
    for kw in (dict(k_scale=scale), dict(dtype=F8, k_scale=scale.double()), dict(dtype=F8, v_scale=torch.ones(3)),
               dict(dtype=F8, v_scale=torch.ones(4)[::2])):
        with pytest.raises(ValueError, match="KVCache"):
            _cache(**kw)
    assert _cache(F8, k_scale=scale, v_scale=scale).k.dtype == F8
    b = _batch()
    for t, n, s in ((b.page_table.long(), b.lengths, b.starts), (b.page_table, b.lengths[:1], b.starts), (b.page_table, b.lengths, b.starts[:2]),
                    (b.page_table[:, :0], b.lengths, b.starts), (b.page_table.t().contiguous().t(), b.lengths, b.starts),
                    (b.page_table, torch.ones(4, dtype=torch.int32)[::2], b.starts), (b.page_table[:0], b.lengths[:0], b.starts[:1])):
        with pytest.raises(ValueError, match="CacheBatch"):
            ops.CacheBatch(t, n, s)
    with pytest.raises(AttributeError):
        c.k = None


def test_calls_refuse_what_is_not_on_a_gpu():
    x = torch.zeros((2, 4, 64), dtype=BF)
    with pytest.raises(ValueError, match="one GPU"):
        ops.rope_rotate(x, torch.zeros(2, dtype=torch.int32), ops.Rope(torch.ones(32, dtype=torch.float64)))
    with pytest.raises(ValueError, match="one GPU"):
        ops.kv_cache_append(_cache(), _batch(), x[:, :2], x[:, 2:])
    with pytest.raises(ValueError, match="one GPU"):
        ops.kv_cache_attention(x, _cache(), _batch())


def _tiled(R, C, B=1, mx=False):
    lib = _lib.load()
    u8 = dict(dtype=torch.uint8)
    codes = torch.zeros((B, lib.nvfp4_tiled_codes_bytes(R, C)), **u8)
    if mx:
        return ops.MxTiledWeights(codes, torch.zeros((B, lib.mxfp4_tiled_scales_bytes(R, C)), **u8), R, C)
    return ops.TiledWeights(codes, torch.zeros((B, lib.nvfp4_tiled_scales_bytes(R, C)), **u8), torch.ones(B), R, C)


def test_attention_block_refuses_what_does_not_fit():
    """Four heads of 64 over two key heads: a projection to 8 heads, one from 4."""
    x, r = torch.zeros((3, 128), dtype=BF), torch.zeros((3, 128))
    good = dict(qkv=_tiled(512, 128), o=_tiled(128, 256), heads=4)
    for change in (dict(qkv=_tiled(512, 128, mx=True)), dict(qkv=_tiled(448, 128)), dict(qkv=_tiled(512, 192)), dict(o=_tiled(128, 192)),
                   dict(o=_tiled(192, 256)), dict(heads=2), dict(qkv=_tiled(512, 128, 2)), dict(o=_tiled(128, 256, 2))):
        with pytest.raises(ValueError, match="one matrix"):
            layer.attention_block_forward(r, x, layer.AttentionWeights(**{**good, **change}), _cache(), _batch())
    for y in (x.float(), x[:, :64], x[0]):
        with pytest.raises(ValueError, match="x must be bf16"):
            layer.attention_block_forward(r, y, layer.AttentionWeights(**good), _cache(), _batch())
    with pytest.raises(ValueError, match="few goes up to 16"):
        layer.attention_block_forward(r, torch.zeros((17, 128), dtype=BF), layer.AttentionWeights(**good), _cache(), _batch(), few=True)


def test_frequencies():
    f, m = ops.rope_frequencies(64, device="cpu")
    assert m == 1.0 and f.dtype == torch.float64 and torch.allclose(f, 10000.0 ** (-torch.arange(32).double() / 32), rtol=1e-14)
    lin, m = ops.rope_frequencies(64, scaling="linear", factor=8.0, device="cpu")
    assert m == 1.0 and torch.equal(lin, f / 8.0)
    base, _ = ops.rope_frequencies(64, scaling="base", factor=8.0, device="cpu")
    assert base[0] == 1.0 and abs(float(base[-1] / f[-1]) - 1.0 / 8.0) < 1e-12     # the fastest stays, the slowest is divided
    for kind in ("ramp", "bands"):
        g, m = ops.rope_frequencies(128, scaling=kind, factor=16.0, original=4096, fast=32.0, slow=1.0, device="cpu")
        f128, _ = ops.rope_frequencies(128, device="cpu")
        turns = 4096 * f128 / (2 * math.pi)
        assert m == (0.1 * math.log(16.0) + 1.0 if kind == "ramp" else 1.0)
        assert torch.equal(g[turns > 33.0], f128[turns > 33.0])
        assert torch.allclose(g[turns < 0.8], f128[turns < 0.8] / 16.0, rtol=1e-14)
        ratio = f128 / g
        assert (ratio.diff() >= -1e-12).all() and (ratio >= 1.0 - 1e-12).all() and (ratio <= 16.0 + 1e-12).all()
        one, m = ops.rope_frequencies(128, scaling=kind, factor=1.0, original=4096, device="cpu")
        assert m == 1.0 and torch.allclose(one, f128, rtol=1e-15)
    for bad in (dict(rot=0), dict(rot=7), dict(rot=8, base=1.0), dict(rot=8, factor=0.5), dict(rot=8, scaling="other"), dict(rot=8, scaling="ramp"),
                dict(rot=8, scaling="bands", original=10, fast=1.0, slow=1.0), dict(rot=2, scaling="base"), dict(rot=8, base=math.inf)):
        with pytest.raises(ValueError, match="rope_frequencies"):
            ops.rope_frequencies(**bad, device="cpu")


def test_numbers_that_a_call_cannot_hold():
    """Sizes past 31 bits are refused, not cut. (Tensors of stride 0 on the meta device: nothing is held.)"""
    one = torch.zeros((1,), dtype=torch.int32)
    with pytest.raises(ValueError, match="2\\^31"):
        ops.CacheBatch(torch.empty((1, 1 << 31), dtype=torch.int32, device="meta"), one, torch.zeros((2,), dtype=torch.int32))
    big = torch.empty((1 << 31, 1, 64), dtype=BF, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        ops._heads("f", "x", big, 1, 64, 1 << 31)
    with pytest.raises(ValueError, match="2\\^24"):
        ops._heads("f", "x", torch.empty((1, 1 << 20, 16), dtype=BF, device="meta"), 1 << 20, 16, 1)


def test_window_is_refused_before_it_is_cut(monkeypatch):
    monkeypatch.setattr(ops, "_gpu", lambda fn, *ts: 0)
    x = torch.zeros((2, 4, 64), dtype=BF)
    for window in (-1, 1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError, match="window"):
            ops.kv_cache_attention(x, _cache(), _batch(), window=window)
