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
