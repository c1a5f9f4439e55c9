"""Thin PyTorch binding of libnvfp4moe: one function per C ABI call, same names.

Only argument marshalling happens here: tensors are checked for device/dtype/shape,
outputs and workspaces are allocated with torch (device memory and streams are all torch
is used for), and the C call is made on the current HIP stream. Every step of the
computation runs in the library's HIP kernels; a failed call raises NVFP4MoEError.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import (BF16, EPI_NONE, EPI_SWIGLU, F32, PATH_MFMA, PATH_NONE, PATH_STREAM,  # noqa: F401
                   W4A4, W4A16, W4A16_PREPARED)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be on the GPU")


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


_DT = {torch.float32: F32, torch.bfloat16: BF16}


def nvfp4_quantize(x: torch.Tensor, g: torch.Tensor | None = None, amax: torch.Tensor | None = None,
                   out: tuple | None = None, tiled: bool = False):
    """Quantize [R, C] or [B, R, C] float32/bf16 to NVFP4.

    Row-major (default) -> (packed [B, R, C/2], scales [B, R, C/16], g [B]) (the batch dim
    dropped for a 2-D x); ``tiled`` -> a TiledWeights in the storage moe_grouped_gemm_nvfp4
    reads, written by the same call (R % 16 == 0).
    ``g``: optional device float[B] global scales; ``amax``: optional device float[B]
    finite max |x| per matrix (used when ``g`` is None); ``out``: optional preallocated
    (packed, scales, g) to write into (contiguous; row-major shapes, or the tiled byte counts).
    """
    _dev(x, g, amax)
    squeeze = x.dim() == 2
    x3 = x.unsqueeze(0) if squeeze else x
    x3 = x3.contiguous()
    B, R, C = x3.shape
    lib = _lib.load()
    if tiled:
        ncb, nsb = lib.nvfp4_tiled_codes_bytes(R, C), lib.nvfp4_tiled_scales_bytes(R, C)
        shapes = ((B, ncb), (B, nsb))
    else:
        shapes = ((B, R, C // 2), (B, R, C // 16))
    if out is not None:
        packed, scales, g_out = out
        assert packed.is_contiguous() and scales.is_contiguous() and g_out.is_contiguous()
        assert packed.numel() == math.prod(shapes[0]) and scales.numel() == math.prod(shapes[1])
        assert g_out.numel() == B
    else:
        packed = torch.empty(shapes[0], dtype=torch.uint8, device=x.device)
        scales = torch.empty(shapes[1], dtype=torch.uint8, device=x.device)
        g_out = torch.empty((B,), dtype=torch.float32, device=x.device)
    ws = _ws(lib.nvfp4_quantize_workspace_size(B, R, C), x.device)
    layout = _lib.LAYOUT_TILED if tiled else _lib.LAYOUT_ROW_MAJOR
    st = lib.nvfp4_quantize(_ptr(x3), _DT[x3.dtype], B, R, C, _ptr(g), _ptr(amax), layout, _ptr(packed),
                            _ptr(scales), _ptr(g_out), _ptr(ws), ws.numel(), _stream())
    _lib.check("nvfp4_quantize", st)
    if tiled:
        return TiledWeights(packed, scales, g_out, R, C)
    if squeeze and out is None:
        return packed[0], scales[0], g_out
    return packed, scales, g_out


@dataclass
class TiledWeights:
    """B NVFP4 matrices [R, C] in the tiled storage of nvfp4_weights_tile, with their
    per-matrix global scales: what moe_grouped_gemm_nvfp4 takes as expert weights."""
    codes: torch.Tensor    # uint8 [B, nvfp4_tiled_codes_bytes(R, C)]
    scales: torch.Tensor   # uint8 [B, nvfp4_tiled_scales_bytes(R, C)]
    g: torch.Tensor        # float32 [B]
    R: int
    C: int

    @property
    def B(self):
        return self.codes.shape[0]


def nvfp4_weights_tile(packed: torch.Tensor, scales: torch.Tensor, g: torch.Tensor) -> TiledWeights:
    """Reorder NVFP4 weights packed [B, R, C/2] + scales [B, R, C/16] (or one [R, ...]
    matrix) into the tiled storage the grouped GEMM reads; a byte permutation with zero
    padding (include/nvfp4moe.h). ``g`` float32 [B] is carried along unchanged."""
    _dev(packed, scales, g)
    p3 = (packed.unsqueeze(0) if packed.dim() == 2 else packed).contiguous()
    s3 = (scales.unsqueeze(0) if scales.dim() == 2 else scales).contiguous()
    B, R, Ch = p3.shape
    C = 2 * Ch
    assert s3.shape == (B, R, C // 16), (s3.shape, p3.shape)
    lib = _lib.load()
    cb, sb = lib.nvfp4_tiled_codes_bytes(R, C), lib.nvfp4_tiled_scales_bytes(R, C)
    if cb == 0 or sb == 0:
        raise _lib.NVFP4MoEError("nvfp4_weights_tile", _lib.ERR_INVALID_ARG, f"unsupported shape R={R} C={C}")
    codes = torch.empty((B, cb), dtype=torch.uint8, device=packed.device)
    sc = torch.empty((B, sb), dtype=torch.uint8, device=packed.device)
    st = lib.nvfp4_weights_tile(_ptr(p3), _ptr(s3), B, R, C, _ptr(codes), _ptr(sc), _stream())
    _lib.check("nvfp4_weights_tile", st)
    g = g.reshape(-1).float().contiguous()
    assert g.numel() == B
    return TiledWeights(codes, sc, g, R, C)


def moe_route_permute(logits: torch.Tensor, k: int):
    """Router + permutation. Returns a dict of device tensors (see include/nvfp4moe.h)."""
    _dev(logits)
    logits = logits.contiguous().float()
    T, E = logits.shape
    dev = logits.device
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(
        topk_ids=torch.empty((T, k), **i32),
        topk_w=torch.empty((T, k), dtype=torch.float32, device=dev),
        expert_offsets=torch.empty((E + 1,), **i32),
        sorted_slot=torch.empty((T * k,), **i32),
        slot_to_row=torch.empty((T * k,), **i32),
        active_experts=torch.empty((E,), **i32),
        n_active=torch.empty((1,), **i32),
    )
    lib = _lib.load()
    ws = _ws(lib.moe_route_permute_workspace_size(T, E, k), dev)
    st = lib.moe_route_permute(_ptr(logits), T, E, k, _ptr(out["topk_ids"]), _ptr(out["topk_w"]),
                               _ptr(out["expert_offsets"]), _ptr(out["sorted_slot"]),
                               _ptr(out["slot_to_row"]), _ptr(out["active_experts"]),
                               _ptr(out["n_active"]), _ptr(ws), ws.numel(), _stream())
    _lib.check("moe_route_permute", st)
    return out


def moe_grouped_gemm_nvfp4(mode: int, epi: int, a: torch.Tensor, w: TiledWeights,
                           expert_offsets: torch.Tensor, active_experts: torch.Tensor,
                           n_active: torch.Tensor, *,
                           a_scales: torch.Tensor | None = None, a_g: torch.Tensor | None = None,
                           gather_index: torch.Tensor | None = None, gather_div: int = 1,
                           rows: int | None = None, out_dtype=torch.bfloat16,
                           want_amax: bool = False, out: torch.Tensor | None = None,
                           a_rows: int | None = None):
    """Grouped NVFP4 GEMM (+ SwiGLU). ``w``: E expert matrices [Nw, K] (tiled); ``a`` bf16
    [a_rows, K] (W4A16), packed uint8 [a_rows, K/2] (W4A4), or the ``x_prep`` bytes of
    moe_dispatch_w4a16 (W4A16_PREPARED, with ``a_rows`` = its T). Returns out (and amax)."""
    _dev(a, w.codes, w.scales, w.g, expert_offsets, active_experts, n_active, a_scales, a_g, gather_index)
    E, Nw, K = w.B, w.R, w.C
    if a_rows is None:
        if mode == W4A16_PREPARED:
            raise ValueError("W4A16_PREPARED needs a_rows (the T of moe_dispatch_w4a16)")
        a_rows = a.shape[0]
    if rows is None:
        rows = gather_index.numel() if gather_index is not None else a_rows
    ncol = Nw // 2 if epi == EPI_SWIGLU else Nw
    if out is None:
        out = torch.empty((rows, ncol), dtype=out_dtype, device=a.device)
    amax = torch.empty((1,), dtype=torch.float32, device=a.device) if want_amax else None
    lib = _lib.load()
    ws = _ws(lib.moe_grouped_gemm_workspace_size(mode, a_rows, rows, E, Nw, K), a.device)
    st = lib.moe_grouped_gemm_nvfp4(
        mode, epi, _ptr(a), _ptr(a_scales), _ptr(a_g), a_rows, _ptr(gather_index), int(gather_div),
        _ptr(w.codes), _ptr(w.scales), _ptr(w.g), _ptr(expert_offsets), _ptr(active_experts),
        _ptr(n_active), E, rows, Nw, K, _ptr(out), _DT[out.dtype], _ptr(amax), _ptr(ws), ws.numel(),
        _stream())
    _lib.check("moe_grouped_gemm_nvfp4", st)
    return (out, amax) if want_amax else out


def moe_dispatch_w4a16(logits: torch.Tensor, x: torch.Tensor, k: int, fp8_act: bool = False):
    """moe_route_permute of ``logits`` [T, E] plus the W4A16 preparation of the token rows
    ``x`` [T, H] bf16 (after the FP8 E4M3 round trip with ``fp8_act``). Returns the routing
    dict of moe_route_permute with ``x_prep``: the bytes moe_grouped_gemm_nvfp4 reads in mode
    W4A16_PREPARED (a_rows = T, K = H)."""
    _dev(logits, x)
    logits = logits.contiguous().float()
    x = x.contiguous()
    T, E = logits.shape
    H = x.shape[1]
    dev = logits.device
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(
        topk_ids=torch.empty((T, k), **i32),
        topk_w=torch.empty((T, k), dtype=torch.float32, device=dev),
        expert_offsets=torch.empty((E + 1,), **i32),
        sorted_slot=torch.empty((T * k,), **i32),
        slot_to_row=torch.empty((T * k,), **i32),
        active_experts=torch.empty((E,), **i32),
        n_active=torch.empty((1,), **i32),
    )
    lib = _lib.load()
    out["x_prep"] = torch.empty((lib.moe_prepared_act_bytes(T, H),), dtype=torch.uint8, device=dev)
    ws = _ws(lib.moe_dispatch_w4a16_workspace_size(T, E, k, H, int(fp8_act)), dev)
    st = lib.moe_dispatch_w4a16(_ptr(logits), _ptr(x), T, E, k, H, int(fp8_act), _ptr(out["topk_ids"]),
                                _ptr(out["topk_w"]), _ptr(out["expert_offsets"]), _ptr(out["sorted_slot"]),
                                _ptr(out["slot_to_row"]), _ptr(out["active_experts"]), _ptr(out["n_active"]),
                                _ptr(out["x_prep"]), _ptr(ws), ws.numel(), _stream())
    _lib.check("moe_dispatch_w4a16", st)
    return out


def moe_grouped_gemm_nvfp4_combine(mode: int, a: torch.Tensor, w: TiledWeights, expert_offsets: torch.Tensor,
                                   active_experts: torch.Tensor, n_active: torch.Tensor, sorted_slot: torch.Tensor,
                                   slot_to_row: torch.Tensor, topk_w: torch.Tensor, *,
                                   a_scales: torch.Tensor | None = None, a_g: torch.Tensor | None = None,
                                   out: torch.Tensor | None = None):
    """Down GEMM + weighted unpermute-reduce in one call: ``a`` [T*k, K] (bf16, or NVFP4
    packed for W4A4) in permuted row order, ``w`` E matrices [H, K] (tiled), routing of
    ``topk_w`` [T, k] tokens -> bf16 out [T, H]."""
    _dev(a, w.codes, w.scales, w.g, expert_offsets, active_experts, n_active, sorted_slot, slot_to_row, topk_w,
         a_scales, a_g)
    E, Nw, K = w.B, w.R, w.C
    T, k = topk_w.shape
    if out is None:
        out = torch.empty((T, Nw), dtype=torch.bfloat16, device=a.device)
    lib = _lib.load()
    ws = _ws(lib.moe_grouped_gemm_nvfp4_combine_workspace_size(mode, T, k, E, Nw, K), a.device)
    st = lib.moe_grouped_gemm_nvfp4_combine(
        mode, _ptr(a), _ptr(a_scales), _ptr(a_g), _ptr(w.codes), _ptr(w.scales), _ptr(w.g), _ptr(expert_offsets),
        _ptr(active_experts), _ptr(n_active), _ptr(sorted_slot), _ptr(slot_to_row), _ptr(topk_w.contiguous()),
        E, T, k, Nw, K, _ptr(out), _ptr(ws), ws.numel(), _stream())
    _lib.check("moe_grouped_gemm_nvfp4_combine", st)
    return out


def moe_unpermute_reduce(y: torch.Tensor, slot_to_row: torch.Tensor, topk_w: torch.Tensor,
                         out: torch.Tensor | None = None):
    """out[t] = bf16(sum_j topk_w[t, j] * y[slot_to_row[t*k + j]])."""
    _dev(y, slot_to_row, topk_w)
    T, k = topk_w.shape
    H = y.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    lib = _lib.load()
    st = lib.moe_unpermute_reduce(_ptr(y), _DT[y.dtype], _ptr(slot_to_row), _ptr(topk_w), T, k, H,
                                  _ptr(out), _stream())
    _lib.check("moe_unpermute_reduce", st)
    return out


def act_fp8_e4m3_roundtrip(x: torch.Tensor, out: torch.Tensor | None = None):
    """FP8 E4M3 (per-tensor scale) round trip of bf16 activations, returned as bf16."""
    _dev(x)
    x = x.contiguous()
    if out is None:
        out = torch.empty_like(x)
    lib = _lib.load()
    n = x.numel()
    ws = _ws(lib.act_fp8_e4m3_roundtrip_workspace_size(n), x.device)
    st = lib.act_fp8_e4m3_roundtrip(_ptr(x), n, _ptr(out), _ptr(ws), ws.numel(), _stream())
    _lib.check("act_fp8_e4m3_roundtrip", st)
    return out


# ------------------------------------------------------------------ MXFP4 variant
def mxfp4_quantize(x: torch.Tensor):
    """Float rows [..., C] (C % 32 == 0) -> MXFP4 (packed uint8 [..., C/2], UE8M0 scales
    uint8 [..., C/32]); one scale per 32 elements, no per-tensor scale."""
    _dev(x)
    x = x.contiguous()
    C = x.shape[-1]
    R = x.numel() // C
    packed = torch.empty(x.shape[:-1] + (C // 2,), dtype=torch.uint8, device=x.device)
    scales = torch.empty(x.shape[:-1] + (C // 32,), dtype=torch.uint8, device=x.device)
    lib = _lib.load()
    st = lib.mxfp4_quantize(_ptr(x), _DT[x.dtype], R, C, _ptr(packed), _ptr(scales), _stream())
    _lib.check("mxfp4_quantize", st)
    return packed, scales


@dataclass
class MxTiledWeights:
    """B MXFP4 matrices [R, C] in the tiled storage moe_grouped_gemm_mxfp4 reads."""
    codes: torch.Tensor    # uint8 [B, nvfp4_tiled_codes_bytes(R, C)]
    scales: torch.Tensor   # uint8 [B, mxfp4_tiled_scales_bytes(R, C)]
    R: int
    C: int

    @property
    def B(self) -> int:
        return self.codes.shape[0]


def mxfp4_weights_tile(packed: torch.Tensor, scales: torch.Tensor) -> MxTiledWeights:
    """Reorder MXFP4 weights packed [B, R, C/2] + scales [B, R, C/32] (or one matrix) into
    the tiled storage; a byte permutation with zero padding (include/nvfp4moe.h)."""
    _dev(packed, scales)
    p3 = (packed.unsqueeze(0) if packed.dim() == 2 else packed).contiguous()
    s3 = (scales.unsqueeze(0) if scales.dim() == 2 else scales).contiguous()
    B, R, Ch = p3.shape
    C = 2 * Ch
    assert s3.shape == (B, R, C // 32), (s3.shape, p3.shape)
    lib = _lib.load()
    cb, sb = lib.nvfp4_tiled_codes_bytes(R, C), lib.mxfp4_tiled_scales_bytes(R, C)
    if cb == 0 or sb == 0:
        raise _lib.NVFP4MoEError("mxfp4_weights_tile", _lib.ERR_INVALID_ARG, f"unsupported shape R={R} C={C}")
    codes = torch.empty((B, cb), dtype=torch.uint8, device=packed.device)
    sc = torch.empty((B, sb), dtype=torch.uint8, device=packed.device)
    st = lib.mxfp4_weights_tile(_ptr(p3), _ptr(s3), B, R, C, _ptr(codes), _ptr(sc), _stream())
    _lib.check("mxfp4_weights_tile", st)
    return MxTiledWeights(codes, sc, R, C)


def moe_grouped_gemm_mxfp4(epi: int, a: torch.Tensor, a_scales: torch.Tensor, w: MxTiledWeights,
                           expert_offsets: torch.Tensor, active_experts: torch.Tensor,
                           n_active: torch.Tensor, *, gather_index: torch.Tensor | None = None,
                           gather_div: int = 1, rows: int | None = None, out_dtype=torch.bfloat16,
                           want_amax: bool = False, out: torch.Tensor | None = None):
    """W4A4 grouped GEMM with MXFP4 weights ``w`` (E matrices [Nw, K], tiled) and MXFP4
    activations ``a`` [a_rows, K/2] + ``a_scales`` [a_rows, K/32] (+ SwiGLU)."""
    _dev(a, a_scales, w.codes, w.scales, expert_offsets, active_experts, n_active, gather_index)
    E, Nw, K = w.B, w.R, w.C
    a_rows = a.shape[0]
    if rows is None:
        rows = gather_index.numel() if gather_index is not None else a_rows
    ncol = Nw // 2 if epi == EPI_SWIGLU else Nw
    if out is None:
        out = torch.empty((rows, ncol), dtype=out_dtype, device=a.device)
    amax = torch.empty((1,), dtype=torch.float32, device=a.device) if want_amax else None
    lib = _lib.load()
    ws = _ws(lib.moe_grouped_gemm_mxfp4_workspace_size(rows, E, Nw, K), a.device)
    st = lib.moe_grouped_gemm_mxfp4(
        epi, _ptr(a), _ptr(a_scales), a_rows, _ptr(gather_index), int(gather_div), _ptr(w.codes),
        _ptr(w.scales), _ptr(expert_offsets), _ptr(active_experts), _ptr(n_active), E, rows, Nw, K,
        _ptr(out), _DT[out.dtype], _ptr(amax), _ptr(ws), ws.numel(), _stream())
    _lib.check("moe_grouped_gemm_mxfp4", st)
    return (out, amax) if want_amax else out


def moe_grouped_gemm_mxfp4_combine(a: torch.Tensor, a_scales: torch.Tensor, w: MxTiledWeights,
                                   expert_offsets: torch.Tensor, active_experts: torch.Tensor, n_active: torch.Tensor,
                                   sorted_slot: torch.Tensor, slot_to_row: torch.Tensor, topk_w: torch.Tensor, *,
                                   out: torch.Tensor | None = None):
    """MXFP4 down GEMM + weighted unpermute-reduce in one call -> bf16 out [T, H]."""
    _dev(a, a_scales, w.codes, w.scales, expert_offsets, active_experts, n_active, sorted_slot, slot_to_row, topk_w)
    E, Nw, K = w.B, w.R, w.C
    T, k = topk_w.shape
    if out is None:
        out = torch.empty((T, Nw), dtype=torch.bfloat16, device=a.device)
    lib = _lib.load()
    ws = _ws(lib.moe_grouped_gemm_mxfp4_combine_workspace_size(T, k, E, Nw, K), a.device)
    st = lib.moe_grouped_gemm_mxfp4_combine(
        _ptr(a), _ptr(a_scales), _ptr(w.codes), _ptr(w.scales), _ptr(expert_offsets), _ptr(active_experts),
        _ptr(n_active), _ptr(sorted_slot), _ptr(slot_to_row), _ptr(topk_w.contiguous()), E, T, k, Nw, K, _ptr(out),
        _ptr(ws), ws.numel(), _stream())
    _lib.check("moe_grouped_gemm_mxfp4_combine", st)
    return out


def moe_grouped_gemm_mxfp4_swiglu_q(a: torch.Tensor, a_scales: torch.Tensor, w: MxTiledWeights,
                                    expert_offsets: torch.Tensor, active_experts: torch.Tensor,
                                    n_active: torch.Tensor, *, gather_index: torch.Tensor | None = None,
                                    gather_div: int = 1, rows: int | None = None):
    """MXFP4 up/gate GEMM + SwiGLU with h written as MXFP4 by the epilogue: returns
    (h_packed uint8 [rows, Nw/4], h_scales uint8 [rows, Nw/64])."""
    _dev(a, a_scales, w.codes, w.scales, expert_offsets, active_experts, n_active, gather_index)
    E, Nw, K = w.B, w.R, w.C
    a_rows = a.shape[0]
    if rows is None:
        rows = gather_index.numel() if gather_index is not None else a_rows
    F = Nw // 2
    hp = torch.empty((rows, F // 2), dtype=torch.uint8, device=a.device)
    hs = torch.empty((rows, F // 32), dtype=torch.uint8, device=a.device)
    lib = _lib.load()
    ws = _ws(lib.moe_grouped_gemm_mxfp4_workspace_size(rows, E, Nw, K), a.device)
    st = lib.moe_grouped_gemm_mxfp4_swiglu_q(
        _ptr(a), _ptr(a_scales), a_rows, _ptr(gather_index), int(gather_div), _ptr(w.codes), _ptr(w.scales),
        _ptr(expert_offsets), _ptr(active_experts), _ptr(n_active), E, rows, Nw, K, _ptr(hp), _ptr(hs),
        _ptr(ws), ws.numel(), _stream())
    _lib.check("moe_grouped_gemm_mxfp4_swiglu_q", st)
    return hp, hs


def mxfp8_quantize(x: torch.Tensor):
    """Float rows [..., C] (C % 32 == 0) -> MXFP8 (E4M3 codes uint8 [..., C], UE8M0 scales
    uint8 [..., C/32]); one scale per 32 elements, no per-tensor scale."""
    _dev(x)
    x = x.contiguous()
    C = x.shape[-1]
    R = x.numel() // C
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty(x.shape[:-1] + (C // 32,), dtype=torch.uint8, device=x.device)
    st = _lib.load().mxfp8_quantize(_ptr(x), _DT[x.dtype], R, C, _ptr(codes), _ptr(scales), _stream())
    _lib.check("mxfp8_quantize", st)
    return codes, scales


def mxfp8_weights_tile(codes: torch.Tensor, scales: torch.Tensor) -> MxTiledWeights:
    """Reorder MXFP8 weights codes [B, R, C] + scales [B, R, C/32] (or one matrix) into the
    tiled storage moe_grouped_gemm_mxfp8 reads (include/nvfp4moe.h)."""
    _dev(codes, scales)
    c3 = (codes.unsqueeze(0) if codes.dim() == 2 else codes).contiguous()
    s3 = (scales.unsqueeze(0) if scales.dim() == 2 else scales).contiguous()
    B, R, C = c3.shape
    assert s3.shape == (B, R, C // 32), (s3.shape, c3.shape)
    lib = _lib.load()
    cb, sb = lib.mxfp8_tiled_codes_bytes(R, C), lib.mxfp4_tiled_scales_bytes(R, C)
    if cb == 0 or sb == 0:
        raise _lib.NVFP4MoEError("mxfp8_weights_tile", _lib.ERR_INVALID_ARG, f"unsupported shape R={R} C={C}")
    tc = torch.empty((B, cb), dtype=torch.uint8, device=codes.device)
    ts = torch.empty((B, sb), dtype=torch.uint8, device=codes.device)
    st = lib.mxfp8_weights_tile(_ptr(c3), _ptr(s3), B, R, C, _ptr(tc), _ptr(ts), _stream())
    _lib.check("mxfp8_weights_tile", st)
    return MxTiledWeights(tc, ts, R, C)


def moe_grouped_gemm_mxfp8(epi: int, a: torch.Tensor, a_scales: torch.Tensor, w: MxTiledWeights,
                           expert_offsets: torch.Tensor, active_experts: torch.Tensor,
                           n_active: torch.Tensor, *, gather_index: torch.Tensor | None = None,
                           gather_div: int = 1, rows: int | None = None, out_dtype=torch.bfloat16,
                           want_amax: bool = False, out: torch.Tensor | None = None):
    """W8A8 grouped GEMM with MXFP8 weights ``w`` (E matrices [Nw, K], tiled) and MXFP8
    activations ``a`` [a_rows, K] + ``a_scales`` [a_rows, K/32] (+ SwiGLU)."""
    _dev(a, a_scales, w.codes, w.scales, expert_offsets, active_experts, n_active, gather_index)
    E, Nw, K = w.B, w.R, w.C
    a_rows = a.shape[0]
    if rows is None:
        rows = gather_index.numel() if gather_index is not None else a_rows
    ncol = Nw // 2 if epi == EPI_SWIGLU else Nw
    if out is None:
        out = torch.empty((rows, ncol), dtype=out_dtype, device=a.device)
    amax = torch.empty((1,), dtype=torch.float32, device=a.device) if want_amax else None
    lib = _lib.load()
    ws = _ws(lib.moe_grouped_gemm_mxfp8_workspace_size(rows, E, Nw, K), a.device)
    st = lib.moe_grouped_gemm_mxfp8(
        epi, _ptr(a), _ptr(a_scales), a_rows, _ptr(gather_index), int(gather_div), _ptr(w.codes),
        _ptr(w.scales), _ptr(expert_offsets), _ptr(active_experts), _ptr(n_active), E, rows, Nw, K,
        _ptr(out), _DT[out.dtype], _ptr(amax), _ptr(ws), ws.numel(), _stream())
    _lib.check("moe_grouped_gemm_mxfp8", st)
    return (out, amax) if want_amax else out


# ------------------------------------------------------------------ a few rows
# These calls run for a few microseconds each, so what the binding does around them counts: the
# stream comes as a raw handle (2.5 us less than the Stream object) and pointers go as integers.
_NO_GUARD = contextlib.nullcontext()


def _gpu(fn: str, *ts) -> int:
    """Index of the GPU that holds every given tensor (None entries aside)."""
    index = first = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != first:
            index = -1
    if index < 0:
        raise ValueError(f"{fn}: all tensors must be on one GPU")
    return index


def _on(index: int):
    """The tensors' GPU made current for the call (launches go to the current one)."""
    return _NO_GUARD if torch._C._cuda_getDevice() == index else torch.cuda.device(index)


def _raw_stream(index: int) -> int:
    """Handle of the GPU's current stream."""
    return torch._C._cuda_getCurrentRawStream(index)


def _rows(fn: str, what: str, t: torch.Tensor, n: int, align: int = 1):
    """(t, row distance): a 2-D tensor [rows, n] whose rows are contiguous, in place if its
    row distance and address allow, else as a contiguous copy."""
    if t.dim() != 2 or t.shape[1] != n:
        raise ValueError(f"{fn}: {what} must be [rows, {n}], got {tuple(t.shape)}")
    if t.is_contiguous() and t.data_ptr() % (align * t.element_size()) == 0:
        return t, n
    one = t.shape[0] <= 1
    if t.stride(1) != 1 or (not one and (t.stride(0) < n or t.stride(0) % align)) or \
            t.data_ptr() % (align * t.element_size()):
        t = t.contiguous()
        if t.data_ptr() % (align * t.element_size()):   # a view with an offset that was contiguous already
            t = t.clone()
    return t, (n if one or t.is_contiguous() else t.stride(0))


def _out_rows(fn: str, out, T: int, n: int, dtype, like):
    """(out, row distance) of an output [T, n]: allocated where ``like`` is, or the caller's
    with contiguous rows."""
    if out is None:
        if like.shape == (T, n):
            return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format), n
        return like.new_empty((T, n), dtype=dtype), n
    if out.shape != (T, n) or out.dtype not in _DT or (n > 1 and out.stride(1) != 1) or \
            (T > 1 and out.stride(0) < n):
        raise ValueError(f"{fn}: out must be float32 or bf16 [{T}, {n}] with contiguous rows")
    return out, (out.stride(0) if T > 1 else n)


def _tiled(fn: str, w, mx: bool, n: int):
    """(codes, scales, global scales or None) of the weights. Refuses those that are not ``n``
    matrices of the format, or whose bytes are not what their sizes say (a kilobyte holds 16 rows'
    codes of 128 columns, or scales of 1024, MXFP4 2048)."""
    if not isinstance(w, MxTiledWeights if mx else TiledWeights):
        raise ValueError(f"{fn}: weights must be {'MX' if mx else 'NV'}FP4, got {type(w).__name__}")
    codes, scales, rows, cols = w.codes, w.scales, 64 * n * w.R, w.C
    if codes.numel() != rows * (cols + 127 >> 7) or \
            scales.numel() != rows * (cols + 2047 >> 11 if mx else cols + 1023 >> 10) or \
            (n > 1 and not (codes.is_contiguous() and scales.is_contiguous())):
        raise ValueError(f"{fn}: weights must be {n} contiguous tiled matrices [{w.R}, {cols}], got codes "
                         f"{tuple(codes.shape)} and scales {tuple(scales.shape)}")
    if mx:
        return codes, scales, None
    g = w.g
    if g.numel() != n or g.dtype != torch.float32 or (n > 1 and not g.is_contiguous()):
        raise ValueError(f"{fn}: the global scales must be contiguous float32 [{n}]")
    return codes, scales, g


def _matvec(fn: str, mx: bool, x, w, epi, add, out_dtype, out):
    if x.dtype != torch.bfloat16:
        raise ValueError(f"{fn}: x must be bf16, got {x.dtype}")
    codes, scales, g = _tiled(fn, w, mx, 1)
    out_dt = _DT.get(out_dtype)
    if out_dt is None or (add is not None and add.dtype not in _DT):
        raise ValueError(f"{fn}: out_dtype and add must be float32 or bf16")
    idx = _gpu(fn, x, codes, scales, g, add, out)
    Nw, K = w.R, w.C
    shape, p_x, ldx = x.shape, x.data_ptr(), K
    if len(shape) != 2 or shape[1] != K or p_x & 15 or not x.is_contiguous():
        x, ldx = _rows(fn, "x", x, K, 8)
        shape, p_x = x.shape, x.data_ptr()
    T = shape[0]
    n = Nw // 2 if epi == EPI_SWIGLU else Nw
    p_add, add_dt, ld_add = None, F32, n
    if add is not None:
        add, ld_add = _rows(fn, "add", add, n)
        if add.shape[0] != T:
            raise ValueError(f"{fn}: add must be [{T}, {n}], got {tuple(add.shape)}")
        p_add, add_dt = add.data_ptr(), _DT[add.dtype]
    with _on(idx):
        if out is None:
            out, ld_out = x.new_empty((T, n), dtype=out_dtype), n
        else:
            out, ld_out = _out_rows(fn, out, T, n, out_dtype, x)
            out_dt = _DT[out.dtype]
        lib = _lib.load()
        if not mx:
            st = lib.nvfp4_matvec(epi, p_x, ldx, T, codes.data_ptr(), scales.data_ptr(), g.data_ptr(), Nw, K,
                                  p_add, add_dt, ld_add, out.data_ptr(), out_dt, ld_out, _raw_stream(idx))
        else:
            st = lib.mxfp4_matvec(epi, p_x, ldx, T, codes.data_ptr(), scales.data_ptr(), Nw, K, p_add, add_dt,
                                  ld_add, out.data_ptr(), out_dt, ld_out, _raw_stream(idx))
    if st:
        _lib.check(fn, st)
    return out


def nvfp4_matvec(x: torch.Tensor, w: TiledWeights, epi: int = EPI_NONE, *, add: torch.Tensor | None = None,
                 out_dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """Up to 16 bf16 rows ``x`` [T, K] times one NVFP4 matrix ``w`` [Nw, K] (tiled):
    x W^T (+ add), or with EPI_SWIGLU silu(gate) * up (+ add), in one launch. ``add`` [T, n]
    float32 or bf16 (may be ``out``); rows of x, add and out may lie apart. ``out`` must not
    overlap x."""
    return _matvec("nvfp4_matvec", False, x, w, epi, add, out_dtype, out)


def mxfp4_matvec(x: torch.Tensor, w: MxTiledWeights, epi: int = EPI_NONE, *, add: torch.Tensor | None = None,
                 out_dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """nvfp4_matvec with one MXFP4 matrix ``w`` (mxfp4_weights_tile)."""
    return _matvec("mxfp4_matvec", True, x, w, epi, add, out_dtype, out)


@functools.lru_cache(maxsize=1024)
def _few_workspace(mx: bool, T: int, E: int, k: int, H: int, F: int) -> int:
    lib = _lib.load()
    size = lib.moe_layer_few_mxfp4_workspace_size if mx else lib.moe_layer_few_nvfp4_workspace_size
    return size(T, E, k, H, F)


def _layer_few(fn: str, mx: bool, x, logits, k, w13, w2, fp8_acts, out_dtype, out):
    shape, lshape, p_x = x.shape, logits.shape, x.data_ptr()
    if x.dtype != torch.bfloat16 or len(shape) != 2 or len(lshape) != 2 or lshape[0] != shape[0]:
        raise ValueError(f"{fn}: x must be bf16 [T, H] and logits [T, E]")
    (T, H), E, F = shape, lshape[1], w2.C
    c13, s13, g13 = _tiled(fn, w13, mx, E)
    c2, s2, g2 = _tiled(fn, w2, mx, E)
    if w13.C != H or w2.R != H or w13.R != 2 * F:
        raise ValueError(f"{fn}: weights [{w13.R}, {w13.C}] and [{w2.R}, {w2.C}] do not fit x [T, {H}]")
    idx = _gpu(fn, x, logits, c13, s13, c2, s2, g13, g2, out)
    if logits.dtype != torch.float32 or not logits.is_contiguous():
        logits = logits.contiguous().float()
    if p_x & 15 or not x.is_contiguous():
        x, ldx = _rows(fn, "x", x, H, 8)
        if ldx != H:
            x = x.contiguous()
        p_x = x.data_ptr()
    if out_dtype not in _DT:
        raise ValueError(f"{fn}: out_dtype must be float32 or bf16")
    if out is not None and (out.shape != shape or out.dtype != out_dtype or not out.is_contiguous()):
        raise ValueError(f"{fn}: out must be contiguous {out_dtype} [{T}, {H}]")
    lib = _lib.load()
    with _on(idx):
        if out is None:
            out = x.new_empty(shape, dtype=out_dtype)
        nbytes = _few_workspace(mx, T, E, k, H, F)
        ws = x.new_empty((nbytes,), dtype=torch.uint8)
        if not mx:
            call = lib.moe_layer_few_nvfp4 if out_dtype == torch.bfloat16 else lib.moe_layer_few_nvfp4_f32
            st = call(logits.data_ptr(), p_x, T, E, k, H, F, int(fp8_acts), c13.data_ptr(), s13.data_ptr(), g13.data_ptr(),
                      c2.data_ptr(), s2.data_ptr(), g2.data_ptr(), out.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(idx))
        else:
            call = lib.moe_layer_few_mxfp4 if out_dtype == torch.bfloat16 else lib.moe_layer_few_mxfp4_f32
            st = call(logits.data_ptr(), p_x, T, E, k, H, F, c13.data_ptr(), s13.data_ptr(), c2.data_ptr(), s2.data_ptr(),
                      out.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(idx))
    if st:
        _lib.check(fn, st)
    return out


def moe_layer_few_nvfp4(x: torch.Tensor, logits: torch.Tensor, k: int, w13: TiledWeights, w2: TiledWeights, *,
                        fp8_acts: bool = False, out_dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """The whole MoE layer of up to 16 tokens in two launches: top-``k`` of ``logits`` [T, E],
    SwiGLU experts ``w13`` (E matrices [2F, H]) and ``w2`` (E matrices [H, F]), weighted sum.
    ``x`` bf16 [T, H] (after the FP8 E4M3 round trip with ``fp8_acts``) -> bf16 [T, H], or with
    ``out_dtype`` float32 the sums before that rounding."""
    return _layer_few("moe_layer_few_nvfp4", False, x, logits, k, w13, w2, fp8_acts, out_dtype, out)


def moe_layer_few_mxfp4(x: torch.Tensor, logits: torch.Tensor, k: int, w13: MxTiledWeights, w2: MxTiledWeights, *,
                        out_dtype=torch.bfloat16, out: torch.Tensor | None = None):
    """moe_layer_few_nvfp4 with MXFP4 experts (16-bit activations)."""
    return _layer_few("moe_layer_few_mxfp4", True, x, logits, k, w13, w2, False, out_dtype, out)


# ------------------------------------------------------------------ the norms around a block
def moe_block_norm(resid: torch.Tensor, y: torch.Tensor | None = None, *, post_w: torch.Tensor | None = None,
                   gate: torch.Tensor | None = None, scale: float = 1.0, pre_w: torch.Tensor | None = None,
                   w_offset: float = 0.0, eps: float = 1e-6, slot_to_row: torch.Tensor | None = None,
                   topk_w: torch.Tensor | None = None, y_add: torch.Tensor | None = None,
                   resid_out: torch.Tensor | None = None, next_out: torch.Tensor | None = None):
    """The norms after and before a block with its gate and residual scale, in one launch:
    r' = resid + scale * gate * (rms(y) * (w_offset + post_w), or y), next = bf16(rms(r') *
    (w_offset + pre_w)). Returns (r', next), with None for what is not asked for (without ``y``
    only next, of ``resid``; without ``pre_w`` only r').

    ``resid`` float32 or bf16 [T, H]; ``y`` [T, H], or with ``slot_to_row`` and ``topk_w`` the
    experts' rows [T*k, H]; ``y_add`` [T, H] is added to it (a shared expert); ``post_w``,
    ``pre_w`` [H]; ``gate`` [H], [T, 1] or [T, H]. ``resid_out`` may be ``resid``; an output may be
    any of resid, y [T, H], y_add and a full gate, of its type, and must not overlap the rest."""
    fn = "moe_block_norm"
    idx = resid.get_device()
    if idx < 0 or (resid_out is not None and resid_out.get_device() != idx) or \
            (next_out is not None and next_out.get_device() != idx):
        raise ValueError(f"{fn}: all tensors must be on one GPU")
    if resid.dim() != 2:
        raise ValueError(f"{fn}: resid must be [T, H], got {tuple(resid.shape)}")
    T, H = resid.shape
    if post_w is not None and pre_w is not None and post_w.dtype != pre_w.dtype:
        _float_type(fn, post_w), _float_type(fn, pre_w)
        post_w, pre_w = post_w.float(), pre_w.float()
    p_y = p_add = p_rows = p_topk = p_post = p_pre = p_gate = p_ro = p_next = None
    y_dt = add_dt = w_dt = gate_dt = F32
    ld_y = ld_add = k = gate_row = gate_col = ld_ro = ld_next = 0
    with _on(idx):
        if y is None or resid_out is not resid:   # (without y resid_out is not used)
            resid, p_resid, r_dt, ld_r = _operand(fn, "resid", resid, T, H, idx)
        else:
            p_resid, r_dt, ld_r = resid.data_ptr(), _float_type(fn, resid), resid.stride(0) if T > 1 else H
        if post_w is not None:
            post_w, p_post, w_dt, _ = _operand(fn, "post_w", post_w, None, H, idx)
        if pre_w is not None:
            pre_w, p_pre, w_dt, _ = _operand(fn, "pre_w", pre_w, None, H, idx)
            if next_out is None:
                next_out, ld_next = torch.empty_like(resid, dtype=torch.bfloat16, memory_format=torch.contiguous_format), H
            else:
                next_out, ld_next = _out_rows(fn, next_out, T, H, torch.bfloat16, resid)
                if next_out.dtype != torch.bfloat16:
                    raise ValueError(f"{fn}: next_out must be bf16")
            p_next = next_out.data_ptr()
        if y_add is not None:
            y_add, p_add, add_dt, ld_add = _operand(fn, "y_add", y_add, T, H, idx)
        if y is not None:
            rows = T
            if topk_w is not None and slot_to_row is not None:
                _gpu(fn, resid, slot_to_row, topk_w)
                if topk_w.dtype != torch.float32 or not topk_w.is_contiguous():
                    topk_w = topk_w.float().contiguous()
                slot_to_row = slot_to_row.contiguous()
                rows = topk_w.numel()
                if topk_w.dim() != 2 or topk_w.shape[0] != T or slot_to_row.dtype != torch.int32 or \
                        slot_to_row.numel() != rows:
                    raise ValueError(f"{fn}: topk_w must be [{T}, k], slot_to_row int32 [{T} * k] and y [{T} * k, {H}]")
                k = topk_w.shape[1]
            y, p_y, y_dt, ld_y = _operand(fn, "y", y, rows, H, idx)
            if resid_out is None:
                resid_out, ld_ro = torch.empty_like(resid, memory_format=torch.contiguous_format), H
            else:
                resid_out, ld_ro = _out_rows(fn, resid_out, T, H, resid.dtype, resid)
                if resid_out.dtype != resid.dtype:
                    raise ValueError(f"{fn}: resid_out must have resid's type")
            p_ro = resid_out.data_ptr()
        if slot_to_row is not None:
            p_rows = slot_to_row.data_ptr()
        if topk_w is not None:
            p_topk = topk_w.data_ptr()
        if gate is not None:
            if gate.get_device() != idx or gate.shape not in ((H,), (T, 1), (T, H)):
                raise ValueError(f"{fn}: gate must be [{H}], [{T}, 1] or [{T}, {H}] on resid's GPU, got {tuple(gate.shape)}")
            gate_dt = _float_type(fn, gate)
            gate, gate_row, gate_col = _gate(gate, T, H)
            p_gate = gate.data_ptr()
        st = _lib.load().moe_block_norm(
            p_resid, r_dt, ld_r, p_y, y_dt, ld_y, p_add, add_dt, ld_add, p_rows, p_topk, k, p_post, p_pre,
            w_dt, w_offset, eps, p_gate, gate_dt, gate_row, gate_col, scale, T, H, p_ro, ld_ro, p_next, ld_next,
            _raw_stream(idx))
    if st:
        _lib.check(fn, st)
    return (None if y is None else resid_out), (None if pre_w is None else next_out)


def _operand(fn: str, what: str, t, rows, n: int, idx: int):
    """(t, address, type, row distance) of an input [rows, n], or [n] where rows is None, as
    moe_block_norm reads it: in place, or a copy whose addresses allow 16-byte reads."""
    dt = _DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{fn}: {what} must be float32 or bf16, got {t.dtype}")
    if t.get_device() != idx:
        raise ValueError(f"{fn}: all tensors must be on one GPU")
    shape = (n,) if rows is None else (rows, n)
    if t.shape != shape:
        raise ValueError(f"{fn}: {what} must be {list(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        p = t.data_ptr()
        if p % 16 == 0:
            return t, p, dt, n
    if rows is None:
        t, ld = _aligned(t), n
    else:
        t, ld = _rows(fn, what, t, n, 8)
    return t, t.data_ptr(), dt, ld


def _float_type(fn: str, t) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{fn}: resid, y, y_add, gate and the weights must be float32 or bf16, got {t.dtype}")
    return dt


def _aligned(t):
    """A contiguous 16-byte-aligned vector (the tensor itself if it is one)."""
    if t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _gate(gate: torch.Tensor, T: int, H: int):
    """(gate, row distance, column distance 0 or 1) for moe_block_norm; a copy where columns lie
    apart or an address does not allow 16-byte reads."""
    if gate.dim() == 1:
        return _aligned(gate), 0, 1
    if gate.shape[1] == 1 and H != 1:
        return gate, (gate.stride(0) if T > 1 else 0), 0
    row, col = gate.stride()
    row = 0 if T == 1 else row
    if col == 0:                        # a row's value, expanded over the columns
        return gate, row, 0
    if col != 1 or gate.data_ptr() % 16 or row % 8 or (row != 0 and row < H):
        gate = gate.clone(memory_format=torch.contiguous_format)
        row = H
    return gate, row, 1


def last_dispatch() -> int:
    return _lib.load().nvfp4moe_last_dispatch()
