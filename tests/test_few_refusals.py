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
