"""What the few-row calls and the block's functions refuse before they reach the device, on the CPU:
each of these would otherwise read past a tensor or take its bytes for something else."""
import pytest
import torch

from nvfp4_block_scaled_moe_amd import _lib, layer, ops

BF = torch.bfloat16


def _weights(R, C, B=1, mx=False):
    lib = _lib.load()
    u8 = dict(dtype=torch.uint8)
    codes = torch.zeros((B, lib.nvfp4_tiled_codes_bytes(R, C)), **u8)
    if mx:
        return ops.MxTiledWeights(codes, torch.zeros((B, lib.mxfp4_tiled_scales_bytes(R, C)), **u8), R, C)
    return ops.TiledWeights(codes, torch.zeros((B, lib.nvfp4_tiled_scales_bytes(R, C)), **u8), torch.ones(B), R, C)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [3, 17])
def test_shared_expert_refuses_what_does_not_fit(mx, T):
    """Above 16 rows the expert is a grouped GEMM of one matrix, which takes its sizes from the weights."""
    x = torch.zeros((T, 64), dtype=BF)
    w13, w2 = _weights(128, 64, mx=mx), _weights(64, 64, mx=mx)
    for bad in (layer.SharedExpert(_weights(128, 64, 2, mx), w2), layer.SharedExpert(w13, _weights(64, 64, 2, mx)),
                layer.SharedExpert(w13, _weights(64, 96, mx=mx)), layer.SharedExpert(w13, _weights(64, 64, mx=not mx))):
        with pytest.raises(ValueError, match="one matrix"):
            layer.shared_expert_forward(x, bad)
    for y in (x[:, :32], x.float(), x[0], torch.zeros((T, 96), dtype=BF)):
        with pytest.raises(ValueError, match="x must be bf16"):
            layer.shared_expert_forward(y, layer.SharedExpert(w13, w2))


def test_few_row_calls_refuse_weights_of_another_format():
    """Also MXFP8 weights, which share MXFP4's class, and storage that is not what its sizes say."""
    lib = _lib.load()
    x, lg = torch.zeros((3, 64), dtype=BF), torch.zeros((3, 2))
    nv, mx = _weights(64, 64), _weights(64, 64, mx=True)
    mx8 = ops.MxTiledWeights(torch.zeros((1, lib.mxfp8_tiled_codes_bytes(64, 64)), dtype=torch.uint8), mx.scales, 64, 64)
    short = ops.TiledWeights(nv.codes, nv.scales, nv.g, 128, 64)
    apart = ops.TiledWeights(torch.zeros((2,) + nv.codes.shape[1:], dtype=torch.uint8)[::2].expand(2, -1), nv.scales, nv.g, 64, 64)
    for call, bad in ((ops.nvfp4_matvec, (mx, mx8, short, apart)), (ops.mxfp4_matvec, (nv, mx8))):
        for w in bad:
            with pytest.raises(ValueError, match="weights must be"):
                call(x, w)
    for g in (nv.g.to(BF), torch.ones(2)):
        with pytest.raises(ValueError, match="global scales"):
            ops.nvfp4_matvec(x, ops.TiledWeights(nv.codes, nv.scales, g, 64, 64))
    e13, e2 = _weights(64, 64, 2), _weights(64, 32, 2)
    m13, m2 = _weights(64, 64, 2, mx=True), _weights(64, 32, 2, mx=True)
    for call, pairs in ((ops.moe_layer_few_nvfp4, ((m13, e2), (e13, m2), (m13, m2))),
                        (ops.moe_layer_few_mxfp4, ((m13, e2), (e13, m2), (e13, e2)))):
        for a, b in pairs:
            with pytest.raises(ValueError, match="weights must be"):
                call(x, lg, 1, a, b)


def _touched(at, ld, t, n):
    return {at + r * ld + i for r in range(t) for i in range(n)}


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_matvec_refuses_an_output_that_shares_bytes(fmt):
    """Addresses that are never dereferenced: every layout in which out has a byte of x, or of add
    without being add, is refused."""
    lib = _lib.load()
    at, far, seen = 1 << 30, 1 << 34, 0
    g = (far,) if fmt == "nvfp4" else ()
    call = getattr(lib, fmt + "_matvec")
    for T, ldx, ld_out, od in ((1, 32, 16, _lib.F32), (3, 48, 24, _lib.F32), (3, 64, 64, _lib.BF16), (2, 32, 80, _lib.BF16)):
        size = 4 if od == _lib.F32 else 2
        for off in range(-192, 400, 16):
            share = _touched(0, 2 * ldx, T, 64) & _touched(off, size * ld_out, T, 16 * size)
            if share:
                assert call(_lib.EPI_NONE, at, ldx, T, far, far, *g, 16, 32, None, _lib.F32, 16, at + off, od, ld_out,
                            None) == _lib.ERR_INVALID_ARG, (T, ldx, ld_out, off)
                assert b"overlap x" in lib.nvfp4moe_last_error()
                seen += 1
            for ad, ld_add in ((_lib.F32, ld_out), (_lib.BF16, ld_out), (od, ld_out + 8)):
                asize = 4 if ad == _lib.F32 else 2
                same = off == 0 and ad == od and (T == 1 or ld_add == ld_out)
                if not same and _touched(0, asize * ld_add, T, 16 * asize) & _touched(off, size * ld_out, T, 16 * size):
                    assert call(_lib.EPI_NONE, far, ldx, T, far, far, *g, 16, 32, at, ad, ld_add, at + off, od, ld_out,
                                None) == _lib.ERR_INVALID_ARG, (T, ad, ld_add, ld_out, off)
                    assert b"overlap add" in lib.nvfp4moe_last_error()
                    seen += 1
    assert seen > 100


def test_block_norm_refuses_outputs_that_share_bytes():
    lib = _lib.load()
    far = [1 << 34 | i << 28 for i in range(12)]
    at, H = 1 << 30, 16
    names = ["resid", "y", "ya", "post", "pre", "gate"]
    F, B = _lib.F32, _lib.BF16

    def norm(T, k, place, gr, gc, out, nxt, ld_ro=24, ld_n=24):
        p = dict(zip(names, far))
        p.update(place)
        rows = (far[8], far[9], k) if k else (None, None, 0)
        return lib.moe_block_norm(p["resid"], F, 24, p["y"], F, 24, p["ya"], F, 24, *rows, p["post"], p["pre"], F, 0.0,
                                  1e-6, p["gate"], F, gr, gc, 1.0, T, H, out, ld_ro, nxt, ld_n, None)

    for T, k in ((1, 0), (3, 0), (3, 2)):
        n = dict(resid=T, y=T * max(k, 1), ya=T, post=1, pre=1)
        for gr, gc in ((24, 1), (0, 1), (8, 0)):
            n["gate"] = T if gr else 1
            for name in names:
                wide = 4 * (1 if name == "gate" and not gc else H)
                ld = 4 * (gr if name == "gate" else 24)
                for off in range(-64, 256, 16):
                    mine = _touched(0, ld, n[name], wide)
                    own = name in ("resid", "ya") or (name == "y" and not k) or (name == "gate" and gc and (gr or T == 1))
                    if mine & _touched(off, 96, T, 4 * H) and not (own and off == 0):
                        assert norm(T, k, {name: at}, gr, gc, at + off, far[10]) == _lib.ERR_INVALID_ARG, (T, k, name, off)
                        assert b"overlaps what is read" in lib.nvfp4moe_last_error()
                    if mine & _touched(off, 48, T, 2 * H):
                        assert norm(T, k, {name: at}, gr, gc, far[10], at + off) == _lib.ERR_INVALID_ARG, (T, k, name, off)
                        assert b"overlaps what is read" in lib.nvfp4moe_last_error()
        for off in range(-32, 64, 16):
            if _touched(0, 96, T, 64) & _touched(off, 48, T, 32):
                assert norm(T, k, {}, 24, 1, at, at + off) == _lib.ERR_INVALID_ARG
                assert b"resid_out and next overlap" in lib.nvfp4moe_last_error()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_layer_few_float32_output_is_checked(fmt):
    lib, at, nv = _lib.load(), 1 << 30, fmt == "nvfp4"
    call = getattr(lib, f"moe_layer_few_{fmt}_f32")
    size = getattr(lib, f"moe_layer_few_{fmt}_workspace_size")(4, 8, 2, 64, 32)

    def status(out=at, ws=at, n=size, T=4):
        w = (0, at, at, at, at, at, at) if nv else (at,) * 4
        return call(at, at, T, 8, 2, 64, 32, *w, out, ws, n, None)

    for kw, want in ((dict(out=at + 2), _lib.ERR_INVALID_ARG), (dict(out=None), _lib.ERR_INVALID_ARG),
                     (dict(T=17), _lib.ERR_INVALID_ARG), (dict(n=size - 1), _lib.ERR_WORKSPACE)):
        assert status(**kw) == want and lib.nvfp4moe_last_error().startswith(f"moe_layer_few_{fmt}_f32".encode()), kw


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [3, 40])
def test_block_refuses_what_does_not_fit(mx, T):
    """At every number of tokens: above the few-row calls the GEMMs take their sizes from the weights."""
    def experts(a, b):
        w = object.__new__(layer.MXFP4Experts if mx else layer.NVFP4Experts)
        w.w13_t, w.w2_t = a, b
        return w

    x, lg, resid = torch.zeros((T, 64), dtype=BF), torch.zeros((T, 4)), torch.zeros((T, 64))
    good = experts(_weights(64, 64, 4, mx), _weights(64, 32, 4, mx))
    for w, y, logits in ((good, x.float(), lg), (good, x[:, :32], lg), (good, x[0], lg), (good, x, lg[:, :3]),
                         (good, x, lg[1:]), (experts(good.w13_t, _weights(64, 32, 3, mx)), x, lg),
                         (experts(good.w13_t, _weights(64, 64, 4, mx)), x, lg),
                         (experts(good.w13_t, _weights(96, 32, 4, mx)), x, lg)):
        with pytest.raises(ValueError, match=r"fit|bf16 \[T|contiguous tiled"):
            layer.moe_block_forward(resid, y, 2, w, lambda _: logits)


@pytest.mark.parametrize("mx", [False, True])
def test_calls_above_the_few_rows_run_on_the_tensors_gpu(mx, monkeypatch):
    """shared_expert_forward and moe_block_forward make the tensors' GPU current for the layer's
    calls, which launch on the current one (as the few-row calls do for theirs)."""
    import contextlib
    current, used = [0], []

    @contextlib.contextmanager
    def on(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    monkeypatch.setattr(ops, "_gpu", lambda fn, *ts: 3)
    monkeypatch.setattr(ops, "_on", on)

    def call(result):
        return lambda *a, **kw: used.append(current[0]) or result

    x, t = torch.zeros((20, 64), dtype=BF), torch.zeros((20, 64))
    for name, result in (("moe_grouped_gemm_nvfp4", t), ("moe_grouped_gemm_mxfp4", t), ("mxfp4_quantize", (t, t)),
                         ("moe_grouped_gemm_mxfp4_swiglu_q", (t, t)), ("moe_block_norm", (t, t))):
        monkeypatch.setattr(ops, name, call(result))
    for name in ("moe_forward", "moe_forward_mxfp4"):
        monkeypatch.setattr(layer, name, call((t, t, t)))
    layer.shared_expert_forward(x, layer.SharedExpert(_weights(128, 64, 1, mx), _weights(64, 64, 1, mx)))
    assert used == [3] * (3 if mx else 2) and current == [0]
    used.clear()
    w = object.__new__(layer.MXFP4Experts if mx else layer.NVFP4Experts)
    w.w13_t, w.w2_t = _weights(128, 64, 4, mx), _weights(64, 64, 4, mx)
    layer.moe_block_forward(t, x, 2, w, lambda _: torch.zeros((20, 4)))
    assert used[0] == 3 and current == [0]
