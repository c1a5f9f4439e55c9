"""How precisely the few-token layer holds h between its two launches, seen in its float32 output.

Tolerances: those of tests/test_gpu_few_rows.py (float32 sums, 16 sqrt(K) 2^-24 sum |x w|), and for h
half a step of what holds it: f16, 2^-11 (NVFP4); two bf16 values, the second within 2^-8 of the first
and rounded by 2^-8 of itself, 2^-16 (MXFP4). No rounding of the output's but float32's.
"""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_moe_amd import inputs
from tests.gpu_util import np_, say
from tests.test_gpu_few_rows import _check, _layer_call, _layer_want, _matrices, _rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
H_EPS = {"nvfp4": 2.0 ** -11, "mxfp4": 2.0 ** -16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 256, 512), (2, 60, 4, 416, 288), (16, 1, 1, 160, 96), (3, 1, 1, 64, 1056),
                                       (5, 4, 4, 128, 64), (16, 5, 3, 544, 160), (16, 24, 8, 4128, 416), (7, 9, 5, 9248, 32),
                                       (16, 64, 32, 288, 1024)])
def test_layer_few_in_float32(fmt, T, E, k, H, F):
    """Items of one to four tokens, tiles of one and two row blocks, whole and shared, ragged chunks."""
    say("layer few precision", fmt, T, E, k, H, F)
    w13, W13 = _matrices(fmt, E, 2 * F, H, 100, std=0.05)
    w2, W2 = _matrices(fmt, E, H, F, 200, std=0.05)
    x, lg = _rows(T, H, 9), inputs.random_fp32((T, E), 31)
    got = _layer_call(fmt, x.to(DEV), lg.to(DEV), k, w13, w2, out_dtype=torch.float32)
    again = _layer_call(fmt, x.to(DEV), lg.to(DEV), k, w13, w2, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(got, again)
    want, err = _layer_want(x.double().numpy(), lg.numpy(), k, W13, W2, H_EPS[fmt])
    _check(np_(got), want, err, torch.float32)
    # the bound adds up worst cases; in the norm, roundings of random sign leave h's own relative error
    rel = np.linalg.norm(np_(got) - want) / np.linalg.norm(want)
    assert rel <= (2.0 ** -11 if fmt == "nvfp4" else 2.0 ** -15), rel


@pytest.mark.parametrize("T", [1, 4, 16])
def test_mxfp4_layer_few_keeps_infinities_in_h(T):
    """An h that overflows is infinite and has no rest: Inf or NaN only where its expert's product is."""
    E, k, H, F = 6, 2, 64, 64
    w13, W13 = _matrices("mxfp4", E, 2 * F, H, 100, std=0.05)
    w2, W2 = _matrices("mxfp4", E, H, F, 200, std=0.05)
    x, lg = _rows(T, H, 9), inputs.random_fp32((T, E), 31)
    x[0] = x[0].float().sign().to(torch.bfloat16) * 2.0 ** 70     # up and gate near 2^67: the product overflows
    got = np_(_layer_call("mxfp4", x.to(DEV), lg.to(DEV), k, w13, w2, out_dtype=torch.float32))
    assert not np.isfinite(got[0]).all() and np.isfinite(got[1:]).all()
    if T > 1:
        want, err = _layer_want(x[1:].double().numpy(), lg[1:].numpy(), k, W13, W2, H_EPS["mxfp4"])
        _check(got[1:], want, err, torch.float32)
