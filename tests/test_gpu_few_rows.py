"""Products of a few rows with FP4 weights (nvfp4_matvec, mxfp4_matvec) and the whole MoE layer
of up to 16 tokens in two launches (moe_layer_few_*), against float64 products of the weights
that the oracle dequantizes from the codes.

Tolerances. The operands are exact (FP4 codes times their scales, bf16 rows), so the only
errors are the float32 sums and the final rounding. A sum of K products in any order is off by
at most K 2^-24 sum |x w| to first order; with rounding errors of random sign sqrt(K) 2^-24 is
typical, and 16 sqrt(K) 2^-24 sum |x w| is held to here, plus eps/2 of the result (2^-8 for
bf16, 2^-24 for float32). SwiGLU's gate error is multiplied by at most |u| (1 + |g| / 4) and up's by
|silu(g)|; its own exp2 and reciprocal add 2^-20 (|g| < 16). In the layer, h is rounded once to
f16 relative to its block (2^-11) or to bf16 (2^-8), errors that add up over F and the experts
to at most that share of sum |w h W2|.
"""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_moe_amd import inputs, layer, ops
from oracle import moe as omoe
from oracle import mxfp4, nvfp4
from tests.gpu_util import np_, say

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _matrices(fmt, E, R, C, seed, std=0.02):
    """(tiled weights, float64 [E, R, C]) of E quantized matrices."""
    wf = torch.stack([inputs.random_fp32((R, C), seed + 7 * e, std=std * (1 + e % 3)) for e in range(E)]).to(DEV)
    if fmt == "nvfp4":
        p, s, g = ops.nvfp4_quantize(wf)
        deq = np.stack([nvfp4.dequantize(np_(p[e]), np_(s[e]), np_(g[e])) for e in range(E)])
        return ops.nvfp4_weights_tile(p, s, g), deq
    p, s = ops.mxfp4_quantize(wf)
    return ops.mxfp4_weights_tile(p, s), np.stack([mxfp4.dequantize(np_(p[e]), np_(s[e])) for e in range(E)])


def _call(fmt):
    return ops.nvfp4_matvec if fmt == "nvfp4" else ops.mxfp4_matvec


def _rows(T, K, seed):
    x = inputs.random_fp32((T, K), seed) * torch.exp(0.5 * inputs.random_fp32((K,), seed + 1))
    return x.to(torch.bfloat16)


def _product(x, W):
    """(x W^T, bound on the float32 sums' error) in float64."""
    K = x.shape[1]
    return x @ W.T, 16 * np.sqrt(K) * 2.0 ** -24 * (np.abs(x) @ np.abs(W).T)


def _swiglu(P, err):
    """(silu(g) u, error bound) from the product and the bound on its error."""
    F = P.shape[1] // 2
    g, u, eg, eu = P[:, :F], P[:, F:], err[:, :F], err[:, F:]
    h = omoe.silu(g) * u
    return h, eg * np.abs(u) * (1 + np.abs(g) / 4) + eu * np.abs(omoe.silu(g)) + 2.0 ** -20 * np.abs(h)


def _check(got, want, err, dtype):
    got = np.asarray(got, np.float64)
    tol = err + torch.finfo(dtype).eps / 2 * (np.abs(want) + err) + 1e-38
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) / tol):.2f} of the bound"


MATVEC = [
    # T, Nw, K
    (1, 16, 32), (1, 32, 128), (2, 48, 160), (3, 64, 288), (4, 1024, 256), (5, 2064, 1184), (1, 2048, 6144),
    (7, 96, 544), (8, 80, 1056), (13, 160, 2080), (16, 512, 6144), (16, 16, 96), (9, 4112, 416), (16, 33024, 64),
    (2, 16384, 1152),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,Nw,K", MATVEC)
def test_matvec(fmt, T, Nw, K):
    say("matvec", fmt, T, Nw, K)
    w, W = _matrices(fmt, 1, Nw, K, 11)
    x = _rows(T, K, 5 + T)
    P, err = _product(x.double().numpy(), W[0])
    for dt in (torch.float32, torch.bfloat16):
        got = _call(fmt)(x.to(DEV), w, out_dtype=dt)
        torch.cuda.synchronize()
        assert got.shape == (T, Nw) and got.dtype == dt
        _check(np_(got), P, err, dt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,Nw,K", [(1, 32, 32), (1, 1024, 256), (3, 96, 416), (6, 4128, 1184), (16, 1088, 2304),
                                    (1, 4096, 6144), (2, 35072, 128)])
def test_matvec_swiglu_add(fmt, T, Nw, K):
    say("matvec swiglu", fmt, T, Nw, K)
    w, W = _matrices(fmt, 1, Nw, K, 13, std=0.05)
    x = _rows(T, K, 50 + T)
    h, err = _swiglu(*_product(x.double().numpy(), W[0]))
    n = Nw // 2
    for add_dt in (None, torch.float32, torch.bfloat16):
        add = None if add_dt is None else inputs.random_fp32((T, n), 77).to(add_dt)
        want = h if add is None else h + add.double().numpy()
        got = _call(fmt)(x.to(DEV), w, ops.EPI_SWIGLU, add=None if add is None else add.to(DEV),
                         out_dtype=torch.float32)
        torch.cuda.synchronize()
        _check(np_(got), want, err, torch.float32)


# Rows that do not fit in a CU's LDS beside each other (T * K too large): the waves of a workgroup
# take parts of K, or, with more row blocks than such workgroups, row blocks of their own.
LONG = [
    # T, Nw, K, SwiGLU
    (16, 16, 4096, False), (16, 80, 16416, False), (5, 2080, 12064, False), (9, 64, 7200, True), (2, 48, 40992, False),
    (1, 64, 65568, True), (16, 16448, 3616, False), (11, 16624, 5152, False), (4, 16400, 14368, False),
    (16, 32832, 3616, True), (7, 32896, 8320, True),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,Nw,K,swiglu", LONG)
def test_matvec_long_rows(fmt, T, Nw, K, swiglu):
    """A sample of the weight rows, the first and the last 40 among them, against float64."""
    say("matvec long", fmt, T, Nw, K, swiglu)
    gen = torch.Generator(device=DEV).manual_seed(K + T)
    wf = torch.randn((1, Nw, K), generator=gen, device=DEV, dtype=torch.bfloat16) * 0.03
    q = ops.nvfp4_quantize(wf) if fmt == "nvfp4" else ops.mxfp4_quantize(wf)
    w = ops.nvfp4_weights_tile(*q) if fmt == "nvfp4" else ops.mxfp4_weights_tile(*q)
    n = Nw // 2 if swiglu else Nw
    rows = np.unique(np.concatenate([np.arange(min(40, n)), np.arange(max(0, n - 40), n),
                                     np.random.default_rng(K).integers(0, n, 60)]))
    sel = np.concatenate([rows, rows + n]) if swiglu else rows
    part = [np_(t[0][torch.from_numpy(sel).to(DEV)]) for t in q[:2]]
    W = nvfp4.dequantize(*part, np_(q[2][0])) if fmt == "nvfp4" else mxfp4.dequantize(*part)
    x = _rows(T, K, 6 + T)
    P, err = _product(x.double().numpy(), W)
    if swiglu:
        P, err = _swiglu(P, err)
    add = inputs.random_fp32((T, n), 78).to(DEV)
    got = _call(fmt)(x.to(DEV), w, ops.EPI_SWIGLU if swiglu else ops.EPI_NONE, add=add, out_dtype=torch.float32)
    again = _call(fmt)(x.to(DEV), w, ops.EPI_SWIGLU if swiglu else ops.EPI_NONE, add=add, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(got, again)
    _check(np_(got)[:, rows], P + np_(add)[:, rows].astype(np.float64), err, torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("Nw", [64, 16448])
def test_matvec_long_nonfinite_and_extreme_rows(fmt, Nw):
    """As for short rows: NaN and Inf stay in their row, zero, tiny and huge rows keep their precision."""
    T, K = 14, 4128
    gen = torch.Generator(device=DEV).manual_seed(3)
    q = (ops.nvfp4_quantize if fmt == "nvfp4" else ops.mxfp4_quantize)(
        torch.randn((1, Nw, K), generator=gen, device=DEV, dtype=torch.bfloat16) * 0.03)
    w = (ops.nvfp4_weights_tile if fmt == "nvfp4" else ops.mxfp4_weights_tile)(*q)
    part = [np_(t[0][-48:]) for t in q[:2]]
    W = nvfp4.dequantize(*part, np_(q[2][0])) if fmt == "nvfp4" else mxfp4.dequantize(*part)
    x = _rows(T, K, 8)
    x[0, 4003] = float("nan")
    x[1] = 0.0
    x[2] = x[2] * 2.0 ** 100
    x[3] = x[3] * 2.0 ** -100
    x[5, 200] = float("inf")
    x[6, ::2] = x[6, ::2] * 2.0 ** 20
    got = np_(_call(fmt)(x.to(DEV), w, out_dtype=torch.float32))[:, -48:]
    with np.errstate(invalid="ignore"):
        P, err = _product(x.double().numpy(), W)
    assert np.isnan(got[0]).all() and (got[1] == 0).all()
    nz = W[:, 200] != 0
    assert np.array_equal(got[5][nz], P[5][nz])
    for t in range(2, T):
        if t != 5:
            _check(got[t], P[t], err[t], torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_matvec_strided_rows_and_in_place_add(fmt):
    """Rows of x, add and out that lie apart; add in place; nothing between the rows is written."""
    T, Nw, K = 5, 112, 224
    w, W = _matrices(fmt, 1, Nw, K, 17)
    big = torch.zeros((T, K + 40), dtype=torch.bfloat16)
    big[:, :] = float("nan")
    x = _rows(T, K, 3)
    big[:, 8:8 + K] = x
    base = inputs.random_fp32((T, Nw + 24), 4).to(DEV)
    before = base.clone()
    view = base[:, 5:5 + Nw]
    got = _call(fmt)(big.to(DEV)[:, 8:8 + K], w, add=view, out=view)
    torch.cuda.synchronize()
    assert got.data_ptr() == view.data_ptr()
    P, err = _product(x.double().numpy(), W[0])
    _check(np_(view), P + np_(before[:, 5:5 + Nw]).astype(np.float64), err, torch.float32)
    assert torch.equal(base[:, :5], before[:, :5]) and torch.equal(base[:, 5 + Nw:], before[:, 5 + Nw:])
    # a column-major x and one with a row distance that is no multiple of 8 are copied
    for y in (x.t().contiguous().t(), torch.nn.functional.pad(x, (0, 3))[:, :K]):
        got = _call(fmt)(y.to(DEV), w, out_dtype=torch.float32)
        torch.cuda.synchronize()
        _check(np_(got), P, err, torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [2, 4, 11])
def test_matvec_nonfinite_and_extreme_rows(fmt, T):
    """NaN and Inf stay in their row; zero rows give zeros; tiny and huge rows keep their precision."""
    Nw, K = 64, 416
    w, W = _matrices(fmt, 1, Nw, K, 19)
    x = _rows(T, K, 8)
    x[0, 3] = float("nan")
    x[1] = 0.0
    if T > 2:
        x[2] = x[2] * 2.0 ** 100
        x[3] = x[3] * 2.0 ** -100
    if T > 4:
        x[4, 200] = float("inf")
        x[5, ::2] = x[5, ::2] * 2.0 ** 20     # a row that spans many binades
        x[6] = 0.0
        x[6, 1] = float("-inf")
    got = np_(_call(fmt)(x.to(DEV), w, out_dtype=torch.float32))
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        P, err = _product(x.double().numpy(), W[0])
    assert np.isnan(got[0]).all()
    assert (got[1] == 0).all()
    for t in range(1, T):
        if t in (4, 6) and T > 4:
            assert not np.isfinite(got[t]).all() or (W[0][:, 200] == 0).any()
            nz = (W[0][:, 200 if t == 4 else 1] != 0)
            assert np.array_equal(got[t][nz], P[t][nz])
        else:
            _check(got[t], P[t], err[t], torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_matvec_nan_scale(fmt):
    """A NaN weight group (its scale is NaN) gives NaN in its column alone."""
    T, Nw, K = 3, 48, 256
    wf = inputs.random_fp32((Nw, K), 23, std=0.02)
    wf[17, 130] = float("nan")
    if fmt == "nvfp4":
        p, s, g = ops.nvfp4_quantize(wf.to(DEV))
        w = ops.nvfp4_weights_tile(p, s, g)
    else:
        w = ops.mxfp4_weights_tile(*ops.mxfp4_quantize(wf.to(DEV)))
    got = np_(_call(fmt)(_rows(T, K, 4).to(DEV), w, out_dtype=torch.float32))
    assert np.isnan(got[:, 17]).all() and np.isfinite(np.delete(got, 17, 1)).all()


def test_mxfp4_scale_range():
    """Scales over E8M0's whole range (0 and 254 among them) decode exactly."""
    R, K = 256, 32
    codes = torch.full((1, R, K // 2), 0x22, dtype=torch.uint8, device=DEV)     # every element 1.0
    scales = torch.arange(R, dtype=torch.uint8, device=DEV).view(1, R, 1)
    w = ops.mxfp4_weights_tile(codes, scales)
    x = torch.zeros((2, K), dtype=torch.bfloat16)
    x[0, 0], x[1, 5] = 1.0, 2.0 ** 60
    got = np_(ops.mxfp4_matvec(x.to(DEV), w, out_dtype=torch.float32)).astype(np.float64)
    sc = mxfp4.E8M0_TABLE
    for s in range(255):
        for t, v in ((0, 1.0), (1, 2.0 ** 60)):
            want = np.float64(np.float32(sc[s] * v)) if sc[s] * v < 2.0 ** 128 else np.inf
            # results below float32's normal range may be flushed
            assert got[t, s] == want or want < 2.0 ** -126, (s, t, got[t, s], want)
    assert np.isnan(got[:, 255]).all()


# ------------------------------------------------------------------ the layer
def _layer_want(x, logits, k, W13, W2, h_eps):
    """(out, bound on its error) of the layer in float64; h_eps: half a step of h's rounding."""
    ids, wt = omoe.route(logits, k)
    T, H = x.shape
    out, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            h, eh = _swiglu(*_product(x[t:t + 1], W13[e]))
            eh = eh + h_eps * (np.abs(h) + eh)
            y, ey = _product(h, W2[e])
            out[t] += wt[t, j] * y[0]
            # the rounded routing weight and the sums over the experts: 2^-22 of every addend
            err[t] += wt[t, j] * (ey[0] + (eh @ np.abs(W2[e]).T)[0] + 2.0 ** -22 * (np.abs(h) @ np.abs(W2[e]).T)[0])
    return out, err


def _layer_call(fmt, x, lg, k, w13, w2, **kw):
    call = ops.moe_layer_few_nvfp4 if fmt == "nvfp4" else ops.moe_layer_few_mxfp4
    return call(x, lg, k, w13, w2, **kw)


LAYER = [
    # T, E, k, H, F
    (1, 8, 2, 256, 512), (16, 8, 2, 256, 512), (1, 1, 1, 32, 32), (16, 1, 1, 160, 96), (3, 60, 4, 416, 288),
    (5, 4, 4, 128, 64), (16, 5, 3, 544, 160), (2, 300, 22, 64, 64), (7, 1000, 17, 96, 32), (16, 1024, 64, 32, 32),
    (4, 16, 6, 1184, 1056), (1, 16, 8, 2080, 128),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,F", LAYER)
def test_layer_few(fmt, T, E, k, H, F):
    say("layer few", fmt, T, E, k, H, F)
    w13, W13 = _matrices(fmt, E, 2 * F, H, 100, std=0.05)
    w2, W2 = _matrices(fmt, E, H, F, 200, std=0.05)
    x = _rows(T, H, 9)
    lg = inputs.random_fp32((T, E), 31)
    got = _layer_call(fmt, x.to(DEV), lg.to(DEV), k, w13, w2)
    again = _layer_call(fmt, x.to(DEV), lg.to(DEV), k, w13, w2)
    torch.cuda.synchronize()
    assert got.dtype == torch.bfloat16 and got.shape == (T, H) and torch.equal(got, again)
    want, err = _layer_want(x.double().numpy(), lg.numpy(), k, W13, W2, 2.0 ** -11 if fmt == "nvfp4" else 2.0 ** -8)
    _check(np_(got), want, err, torch.bfloat16)


# Wide layers, whose second launch has tiles of two row blocks (more than 256 blocks, or long lists),
# whole and shared by several workgroups.
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,F", [(3, 8, 2, 4128, 96), (1, 4, 2, 6176, 160), (16, 24, 8, 4128, 416),
                                       (16, 64, 32, 2080, 256), (4, 40, 16, 4096, 544), (2, 6, 3, 9248, 32)])
def test_layer_few_wide(fmt, T, E, k, H, F):
    test_layer_few(fmt, T, E, k, H, F)


# Long rows, of which three, two and one fit in LDS: so many tokens an item.
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,F", [(8, 4, 2, 16384, 32), (5, 3, 2, 24576, 32), (3, 4, 2, 32768, 32), (1, 2, 1, 32768, 64)])
def test_layer_few_long_rows(fmt, T, E, k, H, F):
    test_layer_few(fmt, T, E, k, H, F)


def test_layer_few_fp8_long_rows():
    """The FP8 scale over all rows where the rows are staged an item at a time."""
    T, E, k, H, F = 7, 3, 2, 16416, 32
    w13, _ = _matrices("nvfp4", E, 2 * F, H, 510, std=0.05)
    w2, _ = _matrices("nvfp4", E, H, F, 610, std=0.05)
    x, lg = _rows(T, H, 13).to(DEV), inputs.random_fp32((T, E), 34).to(DEV)
    got = ops.moe_layer_few_nvfp4(x, lg, k, w13, w2, fp8_acts=True)
    same = ops.moe_layer_few_nvfp4(ops.act_fp8_e4m3_roundtrip(x), lg, k, w13, w2)
    torch.cuda.synchronize()
    assert torch.equal(got, same)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [4, 5, 16])
def test_layer_few_one_expert_for_all_and_ties(fmt, T):
    """Every token to the same experts (several items an expert), equal logits (lowest ids win)."""
    E, k, H, F = 12, 3, 160, 96
    w13, W13 = _matrices(fmt, E, 2 * F, H, 300, std=0.05)
    w2, W2 = _matrices(fmt, E, H, F, 400, std=0.05)
    x = _rows(T, H, 10)
    for lg in (torch.zeros((T, E)), (torch.arange(E) == 7).float().expand(T, E).contiguous() * 30.0):
        got = _layer_call(fmt, x.to(DEV), lg.to(DEV), k, w13, w2)
        torch.cuda.synchronize()
        want, err = _layer_want(x.double().numpy(), lg.numpy(), k, W13, W2,
                                2.0 ** -11 if fmt == "nvfp4" else 2.0 ** -8)
        _check(np_(got), want, err, torch.bfloat16)


@pytest.mark.parametrize("T", [1, 6, 16])
def test_layer_few_fp8_rows(T):
    """fp8_acts: the rows take the FP8 round trip with one scale for all of them first."""
    E, k, H, F = 20, 5, 288, 128
    w13, W13 = _matrices("nvfp4", E, 2 * F, H, 500, std=0.05)
    w2, W2 = _matrices("nvfp4", E, H, F, 600, std=0.05)
    x = _rows(T, H, 12)
    lg = inputs.random_fp32((T, E), 33)
    got = ops.moe_layer_few_nvfp4(x.to(DEV), lg.to(DEV), k, w13, w2, fp8_acts=True)
    rows = ops.act_fp8_e4m3_roundtrip(x.to(DEV))
    same = ops.moe_layer_few_nvfp4(rows, lg.to(DEV), k, w13, w2)
    torch.cuda.synchronize()
    assert torch.equal(got, same)
    want, err = _layer_want(omoe.fp8_roundtrip_bf16(x.float().numpy()), lg.numpy(), k, W13, W2, 2.0 ** -11)
    _check(np_(got), want, err, torch.bfloat16)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_layer_few_nan_row_and_nan_expert(fmt):
    """A NaN row spoils its own output only; a NaN weight only the tokens sent to that expert."""
    T, E, k, H, F = 6, 10, 2, 128, 64
    wf = torch.stack([inputs.random_fp32((2 * F, H), 700 + e, std=0.05) for e in range(E)])
    wd = torch.stack([inputs.random_fp32((H, F), 800 + e, std=0.05) for e in range(E)])
    lg = inputs.random_fp32((T, E), 35)
    ids, _ = omoe.route(lg.numpy(), k)
    bad_up, bad_down = int(ids[1, 0]), int(ids[2, 1])
    wf[bad_up, 5, 7] = float("nan")
    wd[bad_down, 9, 3] = float("inf")
    if fmt == "nvfp4":
        w13, w2 = (ops.nvfp4_quantize(w.to(DEV), tiled=True) for w in (wf, wd))
    else:
        w13, w2 = (ops.mxfp4_weights_tile(*ops.mxfp4_quantize(w.to(DEV))) for w in (wf, wd))
    x = _rows(T, H, 14)
    x[4, 11] = float("nan")
    got = np_(_layer_call(fmt, x.to(DEV), lg.to(DEV), k, w13, w2))
    for t in range(T):
        up, down = bad_up in ids[t], bad_down in ids[t]
        if t == 4 or up:
            assert np.isnan(got[t]).all(), t
        elif down:
            assert np.isnan(got[t, 9]) and np.isfinite(np.delete(got[t], 9)).all(), t
        else:
            assert np.isfinite(got[t]).all(), t


def test_layer_few_agrees_with_the_separate_calls():
    """The tiny layer at 1, 5 and 16 tokens against layer.moe_forward: same routing and operands;
    they differ by the rounding of h (bf16 there) and the final one."""
    wl = inputs.WORKLOADS["tiny"]
    w = layer.quantize_experts(wl, DEV)
    for T in (1, 5, 16):
        x, lg = inputs.activations_bf16(wl, T).to(DEV), inputs.router_logits(wl, T).to(DEV)
        a = np_(layer.moe_forward(x, lg, wl.k, w)).astype(np.float64)
        b = np_(ops.moe_layer_few_nvfp4(x, lg, wl.k, w.w13_t, w.w2_t)).astype(np.float64)
        assert np.linalg.norm(a - b) <= 2.0 ** -7 * np.linalg.norm(a)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_few_rows_in_a_graph_and_on_another_stream(fmt):
    """Captured and replayed with other inputs in the same buffers, eager work between the replays;
    and issued on a stream of its own beside the same call on the current one."""
    T, E, k, H, F = 7, 24, 4, 256, 128
    w13, _ = _matrices(fmt, E, 2 * F, H, 900, std=0.05)
    w2, _ = _matrices(fmt, E, H, F, 950, std=0.05)
    wd, _ = _matrices(fmt, 1, 2 * F, H, 970, std=0.05)
    xs = [_rows(T, H, 40 + i).to(DEV) for i in range(3)]
    lgs = [inputs.random_fp32((T, E), 60 + i).to(DEV) for i in range(3)]

    def both(x, lg):
        return _layer_call(fmt, x, lg, k, w13, w2), _call(fmt)(x, wd, ops.EPI_SWIGLU, out_dtype=torch.float32)

    want = [tuple(t.clone() for t in both(x, lg)) for x, lg in zip(xs, lgs)]
    x, lg = xs[0].clone(), lgs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = both(xs[1], lgs[1])
    here = both(xs[2], lgs[2])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(on_side + here, want[1] + want[2]):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both(x, lg)
    for i in (0, 1, 2, 0):
        x.copy_(xs[i])
        lg.copy_(lgs[i])
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b), f"replay on inputs {i}"
        both(xs[1], lgs[1])
        torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_few_rows_refusals(fmt):
    """What the calls do not take is refused before anything is launched, with nothing written."""
    E, k, H, F = 4, 2, 64, 32
    w13, _ = _matrices(fmt, E, 2 * F, H, 21)
    w2, _ = _matrices(fmt, E, H, F, 22)
    w, _ = _matrices(fmt, 1, 48, H, 23)
    x = _rows(3, H, 1).to(DEV)
    lg = torch.zeros((3, E), device=DEV)
    call = _call(fmt)
    out = torch.full((3, 48), 7.0, device=DEV)
    for bad in (lambda: call(x.float(), w), lambda: call(x.cpu(), w), lambda: call(x[0], w), lambda: call(x[:, :32], w),
                lambda: call(x, w13), lambda: call(x, w, out_dtype=torch.float16),
                lambda: call(x, w, add=torch.zeros((2, 48), device=DEV)), lambda: call(x, w, add=torch.zeros(48, device=DEV)),
                lambda: call(x, w, add=out.half()), lambda: call(x, w, out=out[:2]), lambda: call(x, w, out=out.t()),
                lambda: _layer_call(fmt, x, lg[:2], k, w13, w2), lambda: _layer_call(fmt, x, lg, k, w13, w13),
                lambda: _layer_call(fmt, x.float(), lg, k, w13, w2), lambda: _layer_call(fmt, x, lg.cpu(), k, w13, w2),
                lambda: _layer_call(fmt, x, lg[:, :3], k, w13, w2),
                lambda: _layer_call(fmt, x, lg, k, w13, w2, out=torch.zeros((3, H), device=DEV))):
        with pytest.raises(ValueError):
            bad()
    many = _rows(17, H, 2).to(DEV)
    for bad in (lambda: call(many, w), lambda: call(x[:0], w), lambda: call(x, w, ops.EPI_SWIGLU), lambda: call(x, w, 7),
                lambda: _layer_call(fmt, many, torch.zeros((17, E), device=DEV), k, w13, w2),
                lambda: _layer_call(fmt, x, lg, 0, w13, w2), lambda: _layer_call(fmt, x, lg, E + 1, w13, w2),
                lambda: _layer_call(fmt, x[:0], lg[:0], k, w13, w2)):
        with pytest.raises(RuntimeError):
            bad()
    torch.cuda.synchronize()
    assert (out == 7.0).all()
