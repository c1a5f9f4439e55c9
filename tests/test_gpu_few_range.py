"""The range of magnitudes that the products of a few rows keep (nvfp4_matvec, mxfp4_matvec):
rows whose products come near float32's largest and smallest values, with as many rows as fit in
LDS and with more (9 and 10 of 6144 columns), in each kernel.

Tolerances as in the tests of the products: exact operands, so that the float32 sums
(16 sqrt(K) 2^-24 sum |x w|) and the output's rounding are all there is, and 2^-126 for what
float32 cannot hold normally.
"""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_moe_amd import inputs, ops
from oracle import mxfp4, nvfp4
from tests.gpu_util import np_, say
from tests.test_gpu_few_rows import _call, _check, _product, _rows, _swiglu

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _matrix(fmt, Nw, K, std, seed, clear=None):
    """(tiled weights, function: float64 rows of the matrix). clear: (rows, columns) set to zero."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    wf = torch.randn((1, Nw, K), generator=gen, device=DEV, dtype=torch.float32) * std
    if clear is not None:
        wf[0, :clear[0], :clear[1]] = 0.0
    q = ops.nvfp4_quantize(wf) if fmt == "nvfp4" else ops.mxfp4_quantize(wf)
    w = ops.nvfp4_weights_tile(*q) if fmt == "nvfp4" else ops.mxfp4_weights_tile(*q)

    def rows(sel):
        part = [np_(t[0][torch.from_numpy(sel).to(DEV)]) for t in q[:2]]
        return nvfp4.dequantize(*part, np_(q[2][0])) if fmt == "nvfp4" else mxfp4.dequantize(*part)

    return w, rows


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [9, 10])
@pytest.mark.parametrize("Nw", [64, 4160, 16448])
@pytest.mark.parametrize("std,power", [(0.03, 118), (0.03, 121), (4.0, 113), (0.03, -112), (1e-5, -100), (1e-9, -90)])
def test_matvec_rows_near_the_ends_of_the_range(fmt, T, Nw, std, power):
    """Rows of 6144 columns around 2^power beside ordinary ones: finite, and as precise."""
    say("matvec range", fmt, T, Nw, std, power)
    K = 6144
    w, rows = _matrix(fmt, Nw, K, std, 7)
    x = _rows(T, K, 8)
    x[2] = (inputs.random_fp32((K,), 9) * 2.0 ** power).to(torch.bfloat16)
    x[T - 1, :128] = (inputs.random_fp32((128,), 10) * 2.0 ** power).to(torch.bfloat16)   # one chunk of it
    sel = np.unique(np.concatenate([np.arange(32), np.arange(Nw - 32, Nw)]))
    got = _call(fmt)(x.to(DEV), w, out_dtype=torch.float32)
    torch.cuda.synchronize()
    P, err = _product(x.double().numpy(), rows(sel))
    assert (np.abs(P) < 2.0 ** 128).all()
    _check(np_(got)[:, sel], P, err, torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("Nw", [64, 4160, 33024])
def test_matvec_swiglu_rows_near_the_end_of_the_range(fmt, Nw):
    """SwiGLU of 10 such rows: up near 2^118, gate of ordinary size (its weights are zero where the
    row is large)."""
    say("matvec swiglu range", fmt, Nw)
    T, K, n = 10, 6144, Nw // 2
    w, rows = _matrix(fmt, Nw, K, 0.03, 11, clear=(n, 128))
    x = _rows(T, K, 12)
    x[3, :128] = (inputs.random_fp32((128,), 13) * 2.0 ** 118).to(torch.bfloat16)
    sel = np.unique(np.concatenate([np.arange(16), np.arange(n - 16, n)]))
    got = _call(fmt)(x.to(DEV), w, ops.EPI_SWIGLU, out_dtype=torch.float32)
    torch.cuda.synchronize()
    h, err = _swiglu(*_product(x.double().numpy(), rows(np.concatenate([sel, sel + n]))))
    assert (np.abs(h) < 2.0 ** 128).all()
    _check(np_(got)[:, sel], h, err, torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,Nw,K", [(1, 64, 544), (9, 48, 6144), (10, 48, 6144), (12, 16448, 5152)])
@pytest.mark.parametrize("down", [20, 31, 36, 45])
def test_matvec_small_elements_beside_a_large_one(fmt, T, Nw, K, down):
    """A large element that meets zero weights, the others 2^-down of it: NVFP4 products are exact down to
    2^-31 (of the row's largest magnitude, or of the chunk's where the rows do not fit); below, each
    element is off by at most half a step, 2^-39 of that magnitude's power of two. MXFP4 is exact."""
    say("matvec small beside large", fmt, T, Nw, K, down)
    w, rows = _matrix(fmt, Nw, K, 0.03, 15, clear=(Nw, 32))
    # magnitudes from 2^(60 - down) up to twice that, with all eight bits in use
    x = ((1 + torch.rand((T, K), generator=torch.Generator().manual_seed(4))) * 2.0 ** (60 - down)).to(torch.bfloat16)
    x[:, ::3] *= -1
    x[:, 5] = 1.5 * 2.0 ** 60
    sel = np.unique(np.concatenate([np.arange(16), np.arange(Nw - 16, Nw)]))
    got = _call(fmt)(x.to(DEV), w, out_dtype=torch.float32)
    torch.cuda.synchronize()
    W = rows(sel)
    assert (W[:, 5] == 0).all()
    P, err = _product(x.double().numpy(), W)
    if fmt == "nvfp4" and down > 31:
        fits = T * ((K + 127) // 128 * 128) <= 57344
        err = err + 2.0 ** (60 - 39) * np.abs(W if fits else W[:, :128]).sum(1)
    _check(np_(got)[:, sel], P, err, torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,K", [(2, 416), (11, 416), (11, 6144)])
def test_matvec_infinite_elements(fmt, T, K):
    """An infinite element gives its row Inf of the product's sign where the weight it meets is not
    zero, NaN where it is, and leaves the other rows as they are."""
    say("matvec infinite", fmt, T, K)
    w, rows = _matrix(fmt, 64, K, 0.03, 19)
    W = rows(np.arange(64))
    x = _rows(T, K, 8)
    at = {0: (200, float("inf")), T - 1: (1, float("-inf"))}
    for t, (c, v) in at.items():
        x[t, c] = v
        assert (W[:, c] != 0).sum() >= 32 and (W[:, c] == 0).any()
    got = np_(_call(fmt)(x.to(DEV), w, out_dtype=torch.float32))
    with np.errstate(invalid="ignore"):
        P, err = _product(x.double().numpy(), W)
    for t in range(T):
        if t in at:
            c, v = at[t]
            nz = W[:, c] != 0
            assert np.array_equal(got[t][nz], np.sign(W[nz, c]) * v) and np.isnan(got[t][~nz]).all()
        else:
            _check(got[t], P[t], err[t], torch.float32)
