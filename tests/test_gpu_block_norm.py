"""moe_block_norm (the norms before and after a block with its gate and residual scale) against
the formula in float64.

Tolerances, relative to each element's own terms: a float32 sum of H squares of one sign is off
by at most (H / 64 + 12) 2^-24 of itself (a thread adds at most 32 squares, then lanes, waves),
a root of it by half that; products, the residual sum and rsqrt add a few 2^-24 each. 2^-18 of
the element's addends covers them for every H here; the stored roundings add 2^-8 (bf16) or
2^-24 (float32) of the value, and next also what its r' was off by.
"""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_moe_amd import inputs, ops
from tests.gpu_util import np_, say

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _rms(v, eps):
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def _want(resid, y, post_w, gate, scale, pre_w, off, eps, s2r=None, tw=None):
    """(r', bound of its addends, next) in float64; None for what is absent."""
    d = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    r, y, post_w, gate, pre_w, tw = (d(t) for t in (resid, y, post_w, gate, pre_w, tw))
    mag = np.abs(r)
    if y is not None:
        if s2r is not None:
            T, k = tw.shape
            rows = y[s2r.cpu().numpy().reshape(T, k)]
            y, ymag = (tw[..., None] * rows).sum(1), (np.abs(tw)[..., None] * np.abs(rows)).sum(1)
        else:
            ymag = np.abs(y)
        f = 1.0 if gate is None else gate
        f = f * scale
        if post_w is not None:
            inv = 1.0 / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
            f = f * inv * (off + post_w)
        r, mag = r + f * y, mag + np.abs(f) * ymag
    nxt = None if pre_w is None else _rms(r, eps) * (off + pre_w)
    return r, mag, nxt


def _close(got, want, tol, what):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / tol):.2f}"


def _check(resid, got, want, pre_w, off, eps):
    r, mag, nxt = want
    err = 2.0 ** -18 * mag
    if got[0] is not None:
        assert got[0].dtype == resid.dtype
        _close(np_(got[0]), r, err + torch.finfo(resid.dtype).eps / 2 * (np.abs(r) + err), "resid")
    if nxt is not None:
        assert got[1].dtype == BF
        per = np.abs(off + pre_w.double().cpu().numpy()) / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
        # an error of r' reaches next through its element and through the mean of squares
        through = per * err + np.abs(nxt) * (np.sqrt((err * err).mean(-1, keepdims=True)) /
                                             np.sqrt((r * r).mean(-1, keepdims=True) + eps) + 2.0 ** -18)
        _close(np_(got[1]), nxt, through + 2.0 ** -8 * (np.abs(nxt) + through), "next")


def _gate(kind, T, H, dt, seed):
    if kind is None:
        return None
    shape = {"h": (H,), "t": (T, 1), "th": (T, H)}[kind]
    return inputs.random_fp32(shape, seed).to(dt).to(DEV)


SHAPES = [(1, 8), (1, 64), (3, 72), (1, 1000), (5, 2048), (37, 1000), (2, 6144), (1, 8192), (7, 8200), (1, 16392),
          (2, 32768), (300, 136), (257, 2056), (256, 8192), (260, 12296)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("rdt", [F32, BF])
def test_block_norm(T, H, rdt):
    """Every combination of post-norm, gate and next norm on rows of every launch shape."""
    say("block norm", T, H, rdt)
    resid = (3.0 * inputs.random_fp32((T, H), 1)).to(rdt).to(DEV)
    for i, (ydt, post, gate, pre, off, scale, wdt) in enumerate([
            (BF, True, None, True, 0.0, 1.0, F32), (F32, False, "h", True, 1.0, 0.25, BF),
            (BF, True, "t", False, 1.0, -0.5, BF), (F32, True, "th", True, 0.0, 2.0, F32)]):
        y = inputs.random_fp32((T, H), 2 + i).to(ydt).to(DEV)
        w = lambda s: (inputs.random_fp32((H,), s, std=0.3) + (0 if off else 1)).to(wdt).to(DEV)  # noqa: E731
        post_w, pre_w = (w(10) if post else None), (w(11) if pre else None)
        g = _gate(gate, T, H, ydt, 12)
        eps = 1e-5
        got = ops.moe_block_norm(resid, y, post_w=post_w, gate=g, scale=scale, pre_w=pre_w, w_offset=off, eps=eps)
        torch.cuda.synchronize()
        assert (got[1] is None) == (not pre)
        _check(resid, got, _want(resid, y, post_w, g, scale, pre_w, off, eps), pre_w, off, eps)
    pre_w = inputs.random_fp32((H,), 13).to(DEV)
    got = ops.moe_block_norm(resid, pre_w=pre_w, eps=0.0)
    torch.cuda.synchronize()
    assert got[0] is None
    _check(resid, got, _want(resid, None, None, None, 1.0, pre_w, 0.0, 0.0), pre_w, 0.0, 0.0)


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 6144), (5, 3, 1000), (16, 22, 4096), (300, 5, 264), (257, 2, 12296),
                                   (2, 64, 72)])
@pytest.mark.parametrize("ydt", [F32, BF])
def test_block_norm_of_the_experts_rows(T, k, H, ydt):
    say("block norm rows", T, k, H, ydt)
    y = inputs.random_fp32((T * k, H), 3).to(ydt).to(DEV)
    gen = torch.Generator().manual_seed(5)
    s2r = torch.randperm(T * k, generator=gen).to(torch.int32).to(DEV)
    tw = torch.softmax(inputs.random_fp32((T, k), 6), -1).to(DEV)
    post_w, pre_w = (1 + inputs.random_fp32((H,), s, std=0.1).to(DEV) for s in (7, 8))
    for rdt in (F32, BF):
        resid = inputs.random_fp32((T, H), 1).to(rdt).to(DEV)
        for pw in (post_w, None):
            got = ops.moe_block_norm(resid, y, post_w=pw, scale=0.7, pre_w=pre_w, slot_to_row=s2r, topk_w=tw)
            torch.cuda.synchronize()
            _check(resid, got, _want(resid, y, pw, None, 0.7, pre_w, 0.0, 1e-6, s2r, tw), pre_w, 0.0, 1e-6)


@pytest.mark.parametrize("T,k,H", [(1, 0, 64), (5, 0, 1000), (260, 0, 2056), (2, 0, 32768), (1, 8, 6144), (7, 3, 264),
                                   (300, 2, 8200)])
@pytest.mark.parametrize("adt", [F32, BF])
def test_block_norm_with_a_second_addend(T, k, H, adt):
    """y_add beside y, and beside the experts' rows (k > 0); rows of it that lie apart."""
    say("block norm y_add", T, k, H, adt)
    y = inputs.random_fp32((T * max(k, 1), H), 3).to(BF).to(DEV)
    base = torch.full((T, H + 16), float("nan"), dtype=adt, device=DEV)
    base[:, 8:8 + H] = inputs.random_fp32((T, H), 4).to(adt).to(DEV)
    y_add = base[:, 8:8 + H]
    rows = {}
    if k:
        rows = dict(slot_to_row=torch.randperm(T * k, generator=torch.Generator().manual_seed(5)).to(torch.int32).to(DEV),
                    topk_w=torch.softmax(inputs.random_fp32((T, k), 6), -1).to(DEV))
    # in the formula y_add is one more row of every token, with weight 1
    both = torch.cat([y.float(), y_add.float()])
    own = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1)
    s2r = torch.cat([rows["slot_to_row"].view(T, k) if k else own, own + y.shape[0]], 1)
    tw = torch.cat([rows["topk_w"] if k else torch.ones((T, 1), device=DEV), torch.ones((T, 1), device=DEV)], 1)
    post_w, pre_w = (1 + inputs.random_fp32((H,), s, std=0.1).to(DEV) for s in (7, 8))
    for rdt in (F32, BF):
        resid = inputs.random_fp32((T, H), 1).to(rdt).to(DEV)
        for pw in (post_w, None):
            got = ops.moe_block_norm(resid, y, y_add=y_add, post_w=pw, scale=0.7, pre_w=pre_w, **rows)
            torch.cuda.synchronize()
            _check(resid, got, _want(resid, both, pw, None, 0.7, pre_w, 0.0, 1e-6, s2r, tw), pre_w, 0.0, 1e-6)


def test_block_norm_strides_in_place_and_expanded_gates():
    """Rows apart, outputs into views (nothing between the rows is written), resid updated in
    place, gates expanded or with columns apart, an address that 16-byte reads do not allow."""
    T, H = 6, 264
    big = inputs.random_fp32((T, H + 40), 1).to(DEV)
    resid, before = big[:, 16:16 + H], big.clone()
    ybig = inputs.random_fp32((T, 2 * H), 2).to(BF).to(DEV)
    y = ybig[:, H:]
    pre_w = inputs.random_fp32((H + 1,), 3).to(DEV)[1:]          # not 16-byte aligned: copied
    gates = [torch.full((1, 1), 0.5, device=DEV).expand(T, H), inputs.random_fp32((1, H), 4).to(DEV).expand(T, H),
             inputs.random_fp32((T, 1), 5).to(DEV).expand(T, H), inputs.random_fp32((H, T), 6).to(DEV).t(),
             inputs.random_fp32((T, 3), 7).to(DEV)[:, 1:2]]
    for g in gates:
        want = _want(resid, y, None, g, 1.5, pre_w, 0.0, 1e-6)
        nxt = torch.full((T, H + 8), 7.0, dtype=BF, device=DEV)
        got = ops.moe_block_norm(resid, y, gate=g, scale=1.5, pre_w=pre_w, next_out=nxt[:, :H])
        torch.cuda.synchronize()
        _check(resid, got, want, pre_w, 0.0, 1e-6)
        assert (nxt[:, H:] == 7.0).all()
    want = _want(resid, y, None, None, 1.0, pre_w, 0.0, 1e-6)
    got = ops.moe_block_norm(resid, y, pre_w=pre_w, resid_out=resid)
    torch.cuda.synchronize()
    assert got[0].data_ptr() == resid.data_ptr()
    _check(before[:, 16:16 + H], got, want, pre_w, 0.0, 1e-6)
    assert torch.equal(big[:, :16], before[:, :16]) and torch.equal(big[:, 16 + H:], before[:, 16 + H:])


def test_block_norm_zero_and_nonfinite_rows():
    """Zero rows stay finite through eps; a NaN or Inf row spoils itself only."""
    T, H = 5, 640
    resid = inputs.random_fp32((T, H), 1)
    y = inputs.random_fp32((T, H), 2)
    resid[0], y[0] = 0.0, 0.0
    y[1, 3] = float("nan")
    y[2, 5] = float("inf")
    w = torch.ones(H, device=DEV)
    r, n = ops.moe_block_norm(resid.to(DEV), y.to(DEV), post_w=w, pre_w=w)
    torch.cuda.synchronize()
    assert (r[0] == 0).all() and (n[0] == 0).all()
    assert torch.isnan(r[1]).all() and torch.isnan(n[1]).all()
    assert torch.isnan(r[2, 5]) and not torch.isfinite(n[2]).all()
    assert torch.isfinite(r[3:]).all() and torch.isfinite(n[3:]).all()


def test_block_norm_in_a_graph_and_on_another_stream():
    T, H, k = 9, 1032, 4
    pre_w = inputs.random_fp32((H,), 3).to(DEV)
    s2r = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
    tw = torch.rand((T, k), generator=torch.Generator().manual_seed(2)).to(DEV)
    ins = [(inputs.random_fp32((T, H), 10 + i).to(DEV), inputs.random_fp32((T * k, H), 20 + i).to(DEV)) for i in range(3)]
    call = lambda r, y: ops.moe_block_norm(r, y, post_w=pre_w, pre_w=pre_w, slot_to_row=s2r, topk_w=tw)  # noqa: E731
    want = [tuple(t.clone() for t in call(*a)) for a in ins]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(*ins[1])
    here = call(*ins[2])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(other + here, want[1] + want[2]):
        assert torch.equal(a, b)
    r, y = ins[0][0].clone(), ins[0][1].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(r, y)
    for i in (0, 1, 2, 0):
        r.copy_(ins[i][0])
        y.copy_(ins[i][1])
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)
        call(*ins[1])
        torch.cuda.synchronize()


def test_block_norm_refusals():
    T, H, k = 3, 64, 2
    r, y = torch.zeros((T, H), device=DEV), torch.zeros((T, H), dtype=BF, device=DEV)
    w = torch.ones(H, device=DEV)
    rows, s2r, tw = torch.zeros((T * k, H), device=DEV), torch.zeros(T * k, dtype=torch.int32, device=DEV), torch.ones((T, k), device=DEV)
    f = ops.moe_block_norm
    for bad in (lambda: f(r.cpu(), y), lambda: f(r[0], y), lambda: f(r, y.half()), lambda: f(r, y[:2]), lambda: f(r, y[:, :32]),
                lambda: f(r, y, post_w=w[:32]), lambda: f(r, pre_w=w.cpu()), lambda: f(r, y, gate=w[:32]),
                lambda: f(r, y, gate=w.cpu()), lambda: f(r, y, y_add=r[:2]), lambda: f(r, y, resid_out=torch.zeros_like(y)),
                lambda: f(r, pre_w=w, next_out=torch.zeros_like(r)), lambda: f(r, rows[:5], slot_to_row=s2r, topk_w=tw),
                lambda: f(r, rows, slot_to_row=s2r.long(), topk_w=tw), lambda: f(r, rows, slot_to_row=s2r, topk_w=tw[:2]),
                lambda: f(r, rows, slot_to_row=s2r.cpu(), topk_w=tw)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(r), lambda: f(r, post_w=w, pre_w=w), lambda: f(r, gate=w, pre_w=w), lambda: f(r, y_add=y, pre_w=w),
                lambda: f(r, y, topk_w=tw), lambda: f(r[:0], y[:0]), lambda: f(r[:, :12].contiguous(), y[:, :12].contiguous())):
        with pytest.raises(RuntimeError):
            bad()
