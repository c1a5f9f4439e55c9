"""CPU-only argument checks of the few-row calls and of the block norm: refused on the host
before any HIP call, each with its status and a message."""
import ctypes

import pytest
import torch

from nvfp4_block_scaled_moe_amd import _lib, layer, ops

FAKE = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 2)


def _err(st):
    return st, _lib.load().nvfp4moe_last_error().decode()


def _matvec(fmt, **kw):
    a = dict(epi=_lib.EPI_NONE, x=FAKE, ldx=64, T=3, codes=FAKE, scales=FAKE, g=FAKE, Nw=32, K=64, add=None,
             add_dtype=_lib.F32, ld_add=32, out=FAKE, out_dtype=_lib.BF16, ld_out=32)
    a.update(kw)
    g = (a["g"],) if fmt == "nvfp4" else ()
    return getattr(_lib.load(), fmt + "_matvec")(
        a["epi"], a["x"], a["ldx"], a["T"], a["codes"], a["scales"], *g, a["Nw"], a["K"], a["add"], a["add_dtype"],
        a["ld_add"], a["out"], a["out_dtype"], a["ld_out"], None)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_matvec_rejects_bad_arguments(fmt):
    bad = [dict(epi=2), dict(x=None), dict(out=None), dict(codes=None), dict(scales=None), dict(T=0), dict(T=17),
           dict(Nw=24), dict(Nw=0), dict(Nw=48, epi=_lib.EPI_SWIGLU), dict(K=48, ldx=64), dict(K=0), dict(ldx=56),
           dict(ldx=68), dict(ldx=1 << 26), dict(x=ODD), dict(codes=ODD), dict(scales=ODD), dict(out_dtype=5),
           dict(out_dtype=_lib.F32, out=ODD), dict(ld_out=31), dict(add=FAKE, ld_add=31), dict(add=FAKE, add_dtype=7),
           dict(add=ODD), dict(Nw=1 << 26, K=64, ld_out=1 << 26)]
    if fmt == "nvfp4":
        bad.append(dict(g=None))
    for kw in bad:
        st, msg = _err(_matvec(fmt, **kw))
        assert st == _lib.ERR_INVALID_ARG and msg.startswith(fmt + "_matvec"), kw


def _layer(fmt, **kw):
    a = dict(logits=FAKE, x=FAKE, T=4, E=8, k=2, H=64, F=32, fp8=0, c13=FAKE, s13=FAKE, g13=FAKE, c2=FAKE, s2=FAKE,
             g2=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    lib = _lib.load()
    head = (a["logits"], a["x"], a["T"], a["E"], a["k"], a["H"], a["F"])
    tail = (a["out"], a["ws"], a["ws_bytes"], None)
    if fmt == "nvfp4":
        return lib.moe_layer_few_nvfp4(*head, a["fp8"], a["c13"], a["s13"], a["g13"], a["c2"], a["s2"], a["g2"], *tail)
    return lib.moe_layer_few_mxfp4(*head, a["c13"], a["s13"], a["c2"], a["s2"], *tail)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_layer_few_rejects_bad_arguments(fmt):
    lib = _lib.load()
    size = getattr(lib, f"moe_layer_few_{fmt}_workspace_size")
    bad = [dict(logits=None), dict(x=None), dict(out=None), dict(T=0), dict(T=17), dict(E=0), dict(E=1025), dict(k=0),
           dict(k=9), dict(E=128, k=65), dict(H=48), dict(H=0), dict(H=32800), dict(F=40), dict(F=0), dict(c13=None),
           dict(s2=None), dict(c2=ODD), dict(x=ODD), dict(ws=ODD)]
    if fmt == "nvfp4":
        bad += [dict(g13=None), dict(g2=None), dict(fp8=2)]
    for kw in bad:
        st, msg = _err(_layer(fmt, **kw))
        assert st == _lib.ERR_INVALID_ARG and msg.startswith(f"moe_layer_few_{fmt}"), kw
        sizes = {n: kw.get(n, d) for n, d in (("T", 4), ("E", 8), ("k", 2), ("H", 64), ("F", 32))}
        if any(n in kw for n in sizes):
            assert size(*sizes.values()) == 0, kw
    need = size(4, 8, 2, 64, 32)
    assert need >= 4 * 2 * 32 * 2
    for ws, n in ((None, 1 << 30), (FAKE, need - 1)):
        st, msg = _err(_layer(fmt, ws=ws, ws_bytes=n))
        assert st == _lib.ERR_WORKSPACE and "workspace" in msg


def _norm(**kw):
    a = dict(resid=FAKE, r=_lib.F32, ld_r=64, y=FAKE, yd=_lib.BF16, ld_y=64, ya=None, yad=_lib.F32, ld_ya=64, s2r=None,
             tw=None, k=0, post=FAKE, pre=FAKE, wd=_lib.F32, off=0.0, eps=1e-6, gate=None, gd=_lib.F32, gr=0, gc=1,
             scale=1.0, T=3, H=64, out=FAKE, ld_ro=64, nxt=FAKE, ld_n=64)
    a.update(kw)
    return _lib.load().moe_block_norm(
        a["resid"], a["r"], a["ld_r"], a["y"], a["yd"], a["ld_y"], a["ya"], a["yad"], a["ld_ya"], a["s2r"], a["tw"],
        a["k"], a["post"], a["pre"], a["wd"], a["off"], a["eps"], a["gate"], a["gd"], a["gr"], a["gc"], a["scale"],
        a["T"], a["H"], a["out"], a["ld_ro"], a["nxt"], a["ld_n"], None)


def test_block_norm_rejects_bad_arguments():
    bad = [dict(resid=None), dict(out=None), dict(nxt=None), dict(y=None, pre=None), dict(y=None), dict(s2r=FAKE),
           dict(tw=FAKE), dict(s2r=FAKE, tw=FAKE, k=0), dict(s2r=FAKE, tw=FAKE, k=65), dict(T=0), dict(H=12), dict(H=0),
           dict(H=32776), dict(ld_r=56), dict(ld_y=68), dict(ld_ro=60), dict(ld_n=60), dict(resid=ODD), dict(y=ODD),
           dict(post=ODD), dict(pre=ODD), dict(out=ODD), dict(nxt=ODD), dict(ya=ODD), dict(ya=FAKE, ld_ya=60),
           dict(r=3), dict(yd=3), dict(wd=3), dict(ya=FAKE, yad=3), dict(gate=FAKE, gd=3), dict(gate=FAKE, gc=2),
           dict(gate=FAKE, gr=-8), dict(gate=FAKE, gr=60), dict(gate=FAKE, gr=56), dict(gate=ODD),
           dict(gate=ctypes.c_void_p((1 << 20) + 1), gc=0), dict(y=None, post=None, ya=FAKE)]
    for kw in bad:
        st, msg = _err(_norm(**kw))
        assert st == _lib.ERR_INVALID_ARG and msg.startswith("moe_block_norm"), kw


def _weights(R, C, B=1):
    lib = _lib.load()
    u8 = dict(dtype=torch.uint8)
    return ops.TiledWeights(torch.zeros((B, lib.nvfp4_tiled_codes_bytes(R, C)), **u8),
                            torch.zeros((B, lib.nvfp4_tiled_scales_bytes(R, C)), **u8), torch.ones(B), R, C)


def test_binding_refuses_cpu_tensors_shapes_and_types():
    """The binding's own checks (types and shapes before the device, so they run here)."""
    bf = torch.bfloat16
    x = torch.zeros((3, 64), dtype=bf)
    for call in [lambda: ops.nvfp4_matvec(x.float(), _weights(32, 64)), lambda: ops.nvfp4_matvec(x, _weights(32, 64, 2)),
                 lambda: ops.nvfp4_matvec(x, _weights(32, 64), out_dtype=torch.float16),
                 lambda: ops.nvfp4_matvec(x, _weights(32, 64)),
                 lambda: ops.moe_layer_few_nvfp4(x, torch.zeros((2, 4)), 1, _weights(64, 64, 4), _weights(64, 32, 4)),
                 lambda: ops.moe_layer_few_nvfp4(x, torch.zeros((3, 5)), 1, _weights(64, 64, 4), _weights(64, 32, 4)),
                 lambda: ops.moe_layer_few_nvfp4(x, torch.zeros((3, 4)), 1, _weights(64, 64, 4), _weights(64, 32, 4)),
                 lambda: ops.moe_block_norm(x, x)]:
        with pytest.raises(ValueError):
            call()


def test_few_paths_refuse_fp8_rows_with_mxfp4_experts():
    w = layer.MXFP4Experts(*(torch.zeros((1, 1, 1), dtype=torch.uint8),) * 4)
    with pytest.raises(ValueError, match="fp8_acts"):
        layer.moe_forward_few(torch.zeros((1, 32), dtype=torch.bfloat16), torch.zeros((1, 1)), 1, w, fp8_acts=True)
