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
