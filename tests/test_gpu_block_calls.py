"""Calls of the few-row products, the few-token layer, the norms and the block that their documentation
allows and that take ways of their own: rows that lie apart, outputs in place, types, several ways
to the same result. Where two ways compute the same thing, their bits are compared.
"""
import pytest
import torch

from nvfp4_block_scaled_moe_amd import inputs, layer, ops
from tests.gpu_util import say
from tests.test_gpu_few_rows import _matrices, _rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _shared(fmt, H, F, seed):
    return layer.SharedExpert(_matrices(fmt, 1, 2 * F, H, seed, std=0.05)[0], _matrices(fmt, 1, H, F, seed + 1, std=0.05)[0])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [5, 16, 17, 40])
def test_shared_expert_of_rows_that_lie_apart(fmt, T):
    say("shared apart", fmt, T)
    H, F = 256, 128
    sh = _shared(fmt, H, F, 40)
    x = _rows(T, H, 3).to(DEV)
    base = torch.full((T, H + 24), float("nan"), dtype=BF, device=DEV)
    base[:, 8:8 + H] = x
    odd = torch.full((T * H + 1,), float("nan"), dtype=BF, device=DEV)
    odd[1:] = x.view(-1)
    want = layer.shared_expert_forward(x, sh)
    for y in (base[:, 8:8 + H], x.t().contiguous().t(), odd[1:].view(T, H)):
        got = layer.shared_expert_forward(y, sh)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("dt", [torch.float32, BF])
def test_block_norm_of_resid_alone_reads_it_as_it_lies(T, dt):
    """Without y resid is only read, also where the caller names it as the output."""
    say("norm resid alone", T, dt)
    H = 64
    buf = inputs.random_fp32((T, 2 * H), 1).to(dt).to(DEV)
    w = (1 + inputs.random_fp32((H,), 2, std=0.1)).to(DEV)
    odd = inputs.random_fp32((T * H + 1,), 3).to(dt).to(DEV)[1:].view(T, H)
    for resid in (buf[:, ::2], buf[:, 4:4 + H], buf.t().contiguous().t()[:, :H], odd):
        want = ops.moe_block_norm(resid.contiguous().clone(), pre_w=w)[1]
        before = resid.clone()
        r, got = ops.moe_block_norm(resid, pre_w=w, resid_out=resid)
        torch.cuda.synchronize()
        assert r is None and torch.equal(got, want) and torch.equal(resid, before)


def test_block_norm_refuses_other_types_of_weights():
    r, w = torch.zeros((2, 64), device=DEV), torch.ones(64, device=DEV)
    for a, b in ((w.half(), w), (w, w.half()), (w.double(), w.to(BF)), (w.half(), w.half())):
        with pytest.raises(ValueError, match="float32 or bf16"):
            ops.moe_block_norm(r, r, post_w=a, pre_w=b)
    both = ops.moe_block_norm(r + 1, r + 2, post_w=w, pre_w=w)
    for a, b in ((w.to(BF), w), (w, w.to(BF))):   # one of each: as float32
        for x, y in zip(ops.moe_block_norm(r + 1, r + 2, post_w=a, pre_w=b), both):
            assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 5])
def test_matvec_refuses_an_output_over_its_rows(fmt, T):
    """out over x, or over add in another place: workgroups would read what others have written."""
    say("matvec out over x", fmt, T)
    H = 128
    w, _ = _matrices(fmt, 1, H, H, 17)
    call = ops.nvfp4_matvec if fmt == "nvfp4" else ops.mxfp4_matvec
    buf = torch.zeros((T, 3 * H), dtype=BF, device=DEV)
    buf[:, :H] = _rows(T, H, 3).to(DEV)
    x, before = buf[:, :H], buf.clone()
    flat = inputs.random_fp32((T * H + 8,), 4).to(DEV)
    add, shifted = flat[:T * H].view(T, H), flat[8:].view(T, H)
    for bad in (dict(out=x), dict(out=buf[:, 8:8 + H]), dict(add=add, out=shifted), dict(add=add.view(BF)[:, :H], out=add)):
        with pytest.raises(RuntimeError, match="overlap"):
            call(x, w, **bad)
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    want = call(x, w)
    got = call(x, w, out=buf[:, H:2 * H])     # beside x in the same rows
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(buf[:, :H], before[:, :H]) and (buf[:, 2 * H:] == 0).all()


@pytest.mark.parametrize("T,H", [(1, 64), (5, 1000), (260, 12296)])
def test_block_norm_outputs_over_inputs(T, H):
    """Outputs in the very rows of an input give the same bits; other overlaps are refused."""
    say("norm outputs over inputs", T, H)
    r, y, a = (inputs.random_fp32((T, H), s).to(BF).to(DEV) for s in (1, 2, 3))
    gate = inputs.random_fp32((T, H), 4).to(BF).to(DEV)
    post, pre = ((1 + inputs.random_fp32((H,), s, std=0.1)).to(DEV) for s in (5, 6))
    kw = dict(post_w=post, pre_w=pre, scale=0.5)
    want = ops.moe_block_norm(r, y, y_add=a, gate=gate, **kw)
    for names in (("r", "y"), ("y", "r"), ("a", "g"), ("g", "a"), (None, "r"), ("y", None)):
        t = dict(r=r.clone(), y=y.clone(), a=a.clone(), g=gate.clone())
        got = ops.moe_block_norm(t["r"], t["y"], y_add=t["a"], gate=t["g"], resid_out=t.get(names[0]),
                                 next_out=t.get(names[1]), **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want)), names
    t = r.clone()
    assert torch.equal(ops.moe_block_norm(t, pre_w=pre, next_out=t)[1], ops.moe_block_norm(r, pre_w=pre)[1])
    big = torch.zeros((T + 1, H), dtype=BF, device=DEV)
    rows = torch.zeros((2 * T, H), dtype=BF, device=DEV)
    s2r = torch.arange(2 * T, dtype=torch.int32, device=DEV)
    tw = torch.ones((T, 2), device=DEV)
    bad = [(r, y, dict(resid_out=big[:T], next_out=big[:T], **kw)),
           (r, rows, dict(slot_to_row=s2r, topk_w=tw, resid_out=rows[:T], **kw)),
           (r, rows, dict(slot_to_row=s2r, topk_w=tw, next_out=rows[T:], **kw)),
           (r, y, dict(post_w=big[0], pre_w=pre.to(BF), next_out=big[:T]))]
    if T > 1:
        bad += [(big[1:], y, dict(resid_out=big[:T], **kw)), (r, y, dict(gate=big[:1].expand(T, H), next_out=big[:T], **kw))]
    for x, z, other in bad:
        with pytest.raises(RuntimeError, match="overlap"):
            ops.moe_block_norm(x, z, **other)


def _layer(fmt, x, lg, k, w13, w2, **kw):
    return (ops.moe_layer_few_nvfp4 if fmt == "nvfp4" else ops.moe_layer_few_mxfp4)(x, lg, k, w13, w2, **kw)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 256, 512), (5, 12, 3, 288, 96), (16, 24, 8, 4128, 416), (16, 64, 32, 2080, 256)])
def test_layer_few_float32_sums(fmt, T, E, k, H, F):
    """The float32 output is what the bf16 one rounds; tiles of one and two row blocks, whole and shared."""
    say("layer few f32", fmt, T, E, k, H, F)
    w13, w2 = _matrices(fmt, E, 2 * F, H, 100, std=0.05)[0], _matrices(fmt, E, H, F, 200, std=0.05)[0]
    x, lg = _rows(T, H, 9).to(DEV), inputs.random_fp32((T, E), 31).to(DEV)
    half = _layer(fmt, x, lg, k, w13, w2)
    out = torch.full((T, H), 7.0, device=DEV)
    for full in (_layer(fmt, x, lg, k, w13, w2, out_dtype=torch.float32),
                 _layer(fmt, x, lg, k, w13, w2, out_dtype=torch.float32, out=out)):
        torch.cuda.synchronize()
        assert full.dtype == torch.float32 and torch.equal(full.to(BF), half)
    assert full is out and (full.view(torch.int32) & 0xffff).bool().any()
    for bad in (dict(out_dtype=torch.float16), dict(out=out), dict(out_dtype=torch.float32, out=half)):
        with pytest.raises(ValueError):
            _layer(fmt, x, lg, k, w13, w2, **bad)


def _experts(fmt, E, H, F, seed):
    w = object.__new__(layer.NVFP4Experts if fmt == "nvfp4" else layer.MXFP4Experts)
    w.w13_t, w.w2_t = _matrices(fmt, E, 2 * F, H, seed, std=0.05)[0], _matrices(fmt, E, H, F, seed + 1000, std=0.05)[0]
    return w


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("shared", [False, True])
def test_block_of_a_few_tokens_keeps_the_experts_sum_in_float32(fmt, shared):
    """The routed experts' sum goes into the shared expert's, the norm and the residual unrounded."""
    T, E, k, H, F = 6, 12, 3, 288, 96
    w, sh = _experts(fmt, E, H, F, 70), _shared(fmt, H, 64, 75) if shared else None
    x, resid = _rows(T, H, 9).to(DEV), inputs.random_fp32((T, H), 1).to(DEV)
    lg, post = inputs.random_fp32((T, E), 31).to(DEV), (1 + inputs.random_fp32((H,), 2, std=0.1)).to(DEV)
    got = layer.moe_block_forward(resid, x, k, w, lambda _: lg, shared=sh, post_w=post, pre_w=post)
    y = layer.moe_forward_few(x, lg, k, w, out_dtype=torch.float32)
    if shared:
        y = layer.shared_expert_forward(x, sh, add=y)
    want = ops.moe_block_norm(resid, y, post_w=post, pre_w=post)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(layer.moe_forward_few(x, lg, k, w), layer.moe_forward_few(x, lg, k, w, out_dtype=torch.float32).to(BF))


def _block(fmt, T, seed=70, E=12, k=3, H=256, F=128):
    w, sh = _experts(fmt, E, H, F, seed), _shared(fmt, H, 128, seed + 5)
    x, resid = _rows(T, H, 9).to(DEV), inputs.random_fp32((T, H), 1).to(DEV)
    return w, sh, x, resid, inputs.random_fp32((T, E), 31).to(DEV), (1 + inputs.random_fp32((H,), 2, std=0.1)).to(DEV), k


@pytest.mark.parametrize("fmt,T", [("nvfp4", 3), ("nvfp4", 8), ("nvfp4", 12), ("nvfp4", 16), ("nvfp4", 20), ("mxfp4", 3),
                                   ("mxfp4", 16), ("mxfp4", 20)])
@pytest.mark.parametrize("few", [None, True, False])
def test_block_by_the_way_asked_for(fmt, T, few):
    """few: two launches and products, or the separate calls, at every number of tokens that they take."""
    say("block few", fmt, T, few)
    w, sh, x, resid, lg, post, k = _block(fmt, T)
    run = lambda **kw: layer.moe_block_forward(resid, x, k, w, lambda _: lg, shared=sh, post_w=post, pre_w=post, **kw)  # noqa: E731
    if few and T > 16:
        with pytest.raises(ValueError, match="up to 16"):
            run(few=True)
        return
    got = run(few=few)
    if T <= (8 if fmt == "nvfp4" else 16) if few is None else few:
        y = layer.shared_expert_forward(x, sh, add=layer.moe_forward_few(x, lg, k, w, out_dtype=torch.float32))
        want = ops.moe_block_norm(resid, y, post_w=post, pre_w=post)
    else:
        forward = layer.moe_forward if fmt == "nvfp4" else layer.moe_forward_mxfp4
        y, s2r, tw = forward(x, lg, k, w, reduce=False)
        want = ops.moe_block_norm(resid, y, post_w=post, pre_w=post, slot_to_row=s2r, topk_w=tw,
                                  y_add=layer.shared_expert_forward(x, sh, few=few))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_block_of_mxfp4_experts_that_the_separate_calls_do_not_take():
    """F off the multiples of 128: two launches take it, the separate calls refuse it."""
    w, sh, x, resid, lg, _, k = _block("mxfp4", 5, F=96)
    run = lambda **kw: layer.moe_block_forward(resid, x, k, w, lambda _: lg, shared=sh, **kw)  # noqa: E731
    assert torch.isfinite(run()[0]).all()
    with pytest.raises(RuntimeError, match="Nw"):
        run(few=False)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [1, 7, 16])
def test_shared_expert_by_the_way_asked_for(fmt, T):
    """few=False at a few rows: the GEMMs that more rows take, a row's result the same in both batches
    but for the order of its sums (MXFP4 quantizes each row by itself)."""
    say("shared few", fmt, T)
    H, F = 512, 256
    sh = _shared(fmt, H, F, 60)
    x = _rows(24, H, 4).to(DEV)
    many = layer.shared_expert_forward(x, sh)
    got = layer.shared_expert_forward(x[:T], sh, few=False)
    products = layer.shared_expert_forward(x[:T], sh, few=True)
    torch.cuda.synchronize()
    # float32 sums of 512 and 256 products in another order may move single roundings of h, each to
    # bf16 by 2^-8, or to its MXFP4 code by half of its distance to the next (at most a third) of itself
    assert (got - many[:T]).norm() <= (2.0 ** -8 if fmt == "nvfp4" else 2.0 ** -5) * many[:T].norm()
    assert torch.equal(products, layer.shared_expert_forward(x[:T], sh)) and not torch.equal(products, got)
    with pytest.raises(ValueError, match="few-row products"):
        layer.shared_expert_forward(x[:T], sh, add=got, few=False)
    with pytest.raises(ValueError, match="up to 16"):
        layer.shared_expert_forward(x, sh, few=True)


@pytest.mark.parametrize("T", [1, 5, 8, 12, 16, 40])
@pytest.mark.parametrize("shared", [False, True])
def test_block_with_fp8_rows(T, shared):
    """fp8_acts reaches the routed experts' rows, in two launches and in the separate calls, and not
    the shared expert's: the block on rows that took the round trip before, the shared expert on x."""
    say("block fp8", T, shared)
    w, sh, x, resid, lg, post, k = _block("nvfp4", T)
    got = layer.moe_block_forward(resid, x, k, w, lambda _: lg, shared=sh if shared else None, post_w=post, pre_w=post,
                                  fp8_acts=True)
    rows = ops.act_fp8_e4m3_roundtrip(x)
    if T <= 8:
        y = layer.moe_forward_few(rows, lg, k, w, out_dtype=torch.float32)
        if shared:
            y = layer.shared_expert_forward(x, sh, add=y)
        want = ops.moe_block_norm(resid, y, post_w=post, pre_w=post)
    else:
        y, s2r, tw = layer.moe_forward(rows, lg, k, w, reduce=False)
        ys = layer.shared_expert_forward(x, sh) if shared else None
        want = ops.moe_block_norm(resid, y, post_w=post, pre_w=post, slot_to_row=s2r, topk_w=tw, y_add=ys)
    plain = layer.moe_block_forward(resid, x, k, w, lambda _: lg, shared=sh if shared else None, post_w=post, pre_w=post)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not torch.equal(got[0], plain[0])


@pytest.mark.parametrize("T", [2, 13])
def test_layer_few_with_fp8_rows_by_the_layer(T):
    w, _, x, _, lg, _, k = _block("nvfp4", T)
    got = layer.moe_forward_few(x, lg, k, w, fp8_acts=True)
    want = layer.moe_forward_few(ops.act_fp8_e4m3_roundtrip(x), lg, k, w)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and not torch.equal(got, layer.moe_forward_few(x, lg, k, w))
