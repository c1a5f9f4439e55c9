"""The block around the MoE layer (layer.moe_block_forward: router, routed and shared experts, the
norms, gate and residual in a few calls) and the shared expert by itself.

Tolerances. A few tokens (up to 8; MXFP4: 16) against float64 from the dequantized weights: the bounds of the
products are those of the few-row tests (float32 sums, h of the routed experts rounded once, h of
the shared one to bf16: 2^-8 of sum |h W2|), y's bf16 rounding is 2^-8 of it, and the norms pass
an error on through its element and through their mean of squares. With more tokens the routed
rows are the layer's own (tested by themselves), so that what is checked here is how they are
joined, and the shared expert is held against the same expert as a layer of one: both round the
same h to the same codes but may add in another order, which moves single roundings of h, each
2^-8 (bf16) of its own value.
"""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_moe_amd import inputs, layer, ops
from tests.gpu_util import np_, rel_fro, say
from tests.test_gpu_block_norm import _check as check_norm
from tests.test_gpu_block_norm import _want as want_norm
from tests.test_gpu_few_rows import _layer_want, _matrices, _product, _rows, _swiglu

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _experts(fmt, E, H, F, Fs, seed):
    """(experts, shared expert, their float64 matrices)"""
    w13, W13 = _matrices(fmt, E, 2 * F, H, seed, std=0.05)
    w2, W2 = _matrices(fmt, E, H, F, seed + 1000, std=0.05)
    s13, S13 = _matrices(fmt, 1, 2 * Fs, H, seed + 2000, std=0.05)
    s2, S2 = _matrices(fmt, 1, H, Fs, seed + 3000, std=0.05)
    kind = layer.NVFP4Experts if fmt == "nvfp4" else layer.MXFP4Experts
    w = object.__new__(kind)
    w.w13_t, w.w2_t = w13, w2
    return w, layer.SharedExpert(s13, s2), W13, W2, S13[0], S2[0]


def _shared_want(x, S13, S2):
    h, eh = _swiglu(*_product(x, S13))
    eh = eh + 2.0 ** -8 * (np.abs(h) + eh)
    y, ey = _product(h, S2)
    return y, ey + eh @ np.abs(S2).T


def _normed(v, err, w, eps):
    """(rms(v) * w, bound on its error) for v known to err."""
    H = v.shape[1]
    inv = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    u = v * inv * w
    return u, np.abs(w) * inv * err + np.abs(u) * (inv * np.sqrt((err * err).sum(-1, keepdims=True) / H) + 2.0 ** -18)


def _close(got, want, err, eps_out, what):
    got = np_(got).astype(np.float64)
    tol = err + eps_out * (np.abs(want) + err)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) / tol):.2f}"


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,Fs", [(1, 64), (6, 160), (16, 96)])
def test_shared_expert_of_a_few_rows(fmt, T, Fs):
    say("shared", fmt, T, Fs)
    _, sh, _, _, S13, S2 = _experts(fmt, 1, 288, 32, Fs, 40)
    x = _rows(T, 288, 3)
    want, err = _shared_want(x.double().numpy(), S13, S2)
    _close(layer.shared_expert_forward(x.to(DEV), sh), want, err, 2.0 ** -24, "shared")
    add = inputs.random_fp32((T, 288), 5).to(torch.bfloat16)
    _close(layer.shared_expert_forward(x.to(DEV), sh, add=add.to(DEV)), want + add.double().numpy(), err, 2.0 ** -24,
           "shared + add")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [17, 40, 300])
def test_shared_expert_of_many_rows_is_a_layer_of_one(fmt, T):
    say("shared many", fmt, T)
    H, F = 512, 256
    w13, _ = _matrices(fmt, 1, 2 * F, H, 60, std=0.05)
    w2, _ = _matrices(fmt, 1, H, F, 61, std=0.05)
    x = _rows(T, H, 4).to(DEV)
    got = layer.shared_expert_forward(x, layer.SharedExpert(w13, w2))
    kind = layer.NVFP4Experts if fmt == "nvfp4" else layer.MXFP4Experts
    w = object.__new__(kind)
    w.w13_t, w.w2_t = w13, w2
    forward = layer.moe_forward if fmt == "nvfp4" else layer.moe_forward_mxfp4
    one = forward(x, torch.zeros((T, 1), device=DEV), 1, w)
    torch.cuda.synchronize()
    assert got.dtype == torch.float32 and rel_fro(np_(got), np_(one)) <= 2.0 ** -8
    with pytest.raises(ValueError):
        layer.shared_expert_forward(x, layer.SharedExpert(w13, w2), add=got)


@pytest.mark.parametrize("fmt,T", [("nvfp4", 1), ("nvfp4", 5), ("nvfp4", 8), ("mxfp4", 1), ("mxfp4", 5), ("mxfp4", 16)])
@pytest.mark.parametrize("shared", [False, True])
def test_block_of_a_few_tokens(fmt, T, shared):
    say("block", fmt, T, shared)
    E, k, H, F = 12, 3, 288, 96
    w, sh, W13, W2, S13, S2 = _experts(fmt, E, H, F, 64, 70)
    resid = 2.0 * inputs.random_fp32((T, H), 1)
    pre0, post, pre = (1 + inputs.random_fp32((H,), s, std=0.1) for s in (2, 3, 4))
    wr = inputs.random_fp32((H, E), 6, std=0.2)
    lg = {}

    def router(x):
        lg["x"] = x
        lg["l"] = x.float() @ wr.to(DEV)
        return lg["l"]

    x = ops.moe_block_norm(resid.to(DEV), pre_w=pre0.to(DEV))[1]
    got = layer.moe_block_forward(resid.to(DEV), x, k, w, router, shared=sh if shared else None, post_w=post.to(DEV),
                                  scale=0.5, pre_w=pre.to(DEV))
    torch.cuda.synchronize()
    assert lg["x"] is x
    xd = x.double().cpu().numpy()
    y, ey = _layer_want(xd, np_(lg["l"]), k, W13, W2, 2.0 ** -11 if fmt == "nvfp4" else 2.0 ** -8)
    ey = ey + 2.0 ** -8 * (np.abs(y) + ey)
    if shared:
        s, es = _shared_want(xd, S13, S2)
        y, ey = y + s, ey + es + 2.0 ** -24 * np.abs(y + s)
    u, eu = _normed(y, ey, post.double().numpy(), 1e-6)
    r = resid.double().numpy() + 0.5 * u
    er = 0.5 * eu + 2.0 ** -22 * np.abs(r)
    _close(got[0], r, er, 2.0 ** -24, "resid")
    n, en = _normed(r, er, pre.double().numpy(), 1e-6)
    _close(got[1], n, en, 2.0 ** -8, "next")


@pytest.mark.parametrize("fmt,T", [("nvfp4", 9), ("nvfp4", 16), ("nvfp4", 17), ("nvfp4", 130), ("mxfp4", 17), ("mxfp4", 130)])
@pytest.mark.parametrize("shared", [False, True])
def test_block_of_many_tokens_joins_the_rows(fmt, T, shared):
    say("block many", fmt, T, shared)
    E, k, H, F = 8, 2, 512, 256
    w, sh, *_ = _experts(fmt, E, H, F, 256, 80)
    resid = (2.0 * inputs.random_fp32((T, H), 1)).to(torch.bfloat16).to(DEV)
    pre = (1 + inputs.random_fp32((H,), 4, std=0.1)).to(DEV)
    gate = torch.sigmoid(inputs.random_fp32((T, 1), 5)).to(DEV)
    x = ops.moe_block_norm(resid, pre_w=pre)[1]
    lg = inputs.random_fp32((T, E), 31).to(DEV)
    got = layer.moe_block_forward(resid, x, k, w, lambda _: lg, shared=sh if shared else None, gate=gate, pre_w=pre)
    forward = layer.moe_forward if fmt == "nvfp4" else layer.moe_forward_mxfp4
    y, s2r, tw = forward(x, lg, k, w, reduce=False)
    assert rel_fro(np_(ops.moe_unpermute_reduce(y, s2r, tw)), np_(forward(x, lg, k, w))) == 0.0
    if shared:
        y = torch.cat([y, layer.shared_expert_forward(x, sh)])
        own = T * k + torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1)
        s2r = torch.cat([s2r.view(T, k), own], 1)
        tw = torch.cat([tw.view(T, k), torch.ones((T, 1), device=DEV)], 1)
    torch.cuda.synchronize()
    check_norm(resid, got, want_norm(resid, y, None, gate, 1.0, pre, 0.0, 1e-6, s2r, tw.view(T, -1)), pre, 0.0, 1e-6)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [4, 16, 24])
def test_two_blocks_in_a_graph(fmt, T):
    """Two blocks, the second on the first's outputs, captured once and replayed on other inputs
    with eager calls between: the bits of the eager calls."""
    E, k, H, F = 8, 2, 256, 128
    blocks = [_experts(fmt, E, H, F, 128, 90 + 7 * i)[:2] for i in range(2)]
    ws = [(1 + inputs.random_fp32((H,), s, std=0.1)).to(DEV) for s in (2, 3, 4)]
    lgs = [inputs.random_fp32((T, E), 50 + i).to(DEV) for i in range(2)]
    ins = [inputs.random_fp32((T, H), 10 + i).to(DEV) for i in range(3)]

    def both(resid):
        x = ops.moe_block_norm(resid, pre_w=ws[0])[1]
        for i, (w, sh) in enumerate(blocks):
            resid, x = layer.moe_block_forward(resid, x, k, w, lambda _: lgs[i], shared=sh, post_w=ws[2],
                                               pre_w=ws[1])
        return resid, x

    want = [tuple(t.clone() for t in both(r)) for r in ins]
    torch.cuda.synchronize()
    r = ins[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both(r)
    for i in (0, 1, 2, 0):
        r.copy_(ins[i])
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b), f"replay on inputs {i}"
        both(ins[(i + 1) % 3])
        torch.cuda.synchronize()


def test_block_refusals():
    w, sh, *_ = _experts("mxfp4", 4, 64, 32, 32, 20)
    x = _rows(2, 64, 1).to(DEV)
    resid, lg = torch.zeros((2, 64), device=DEV), torch.zeros((2, 4), device=DEV)
    with pytest.raises(ValueError):
        layer.moe_block_forward(resid, x, 2, w, lambda _: lg, fp8_acts=True)
    with pytest.raises(ValueError):
        layer.moe_block_forward(resid[:1], x, 2, w, lambda _: lg)
    with pytest.raises(RuntimeError):
        layer.moe_block_forward(resid, x, 5, w, lambda _: lg)   # k > E
    for forward in (layer.moe_forward, layer.moe_forward_mxfp4):
        for other in (dict(combine=True), dict(keep=True)):
            with pytest.raises(ValueError):
                forward(x, lg, 2, w, reduce=False, **other)
