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
