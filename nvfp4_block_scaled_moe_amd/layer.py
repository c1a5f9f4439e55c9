"""The MoE layer as a sequence of C ABI calls (route -> up/gate + SwiGLU -> down -> reduce), the
layer of a few tokens as one call, the block around it (shared expert, norms, residual), and the
attention block before it (projections, rotary positions, paged cache, attention, norms).

This module only sequences the library calls and allocates their outputs with torch; all
arithmetic runs in the HIP kernels behind include/nvfp4moe.h.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import inputs, ops


@dataclass
class NVFP4Experts:
    """NVFP4 expert weights: W13_e = [2F, H] (gate rows first), W2_e = [H, F], in the pages'
    row-major storage and, for the GEMMs, in the library's tiled storage."""
    w13_packed: torch.Tensor   # uint8 [E, 2F, H/2]
    w13_scales: torch.Tensor   # uint8 [E, 2F, H/16]
    w13_g: torch.Tensor        # f32 [E]
    w2_packed: torch.Tensor    # uint8 [E, H, F/2]
    w2_scales: torch.Tensor    # uint8 [E, H, F/16]
    w2_g: torch.Tensor         # f32 [E]
    w13_t: ops.TiledWeights = None
    w2_t: ops.TiledWeights = None

    @property
    def E(self):
        return self.w13_packed.shape[0]

    def w13(self, e):
        return self.w13_packed[e], self.w13_scales[e], self.w13_g[e]

    def w2(self, e):
        return self.w2_packed[e], self.w2_scales[e], self.w2_g[e]


def quantize_experts(wl: inputs.Workload, device="cuda", experts=None) -> NVFP4Experts:
    """Generate the workload's seeded FP32 expert weights one expert at a time on ``device``
    and quantize each with the library's nvfp4_quantize twice: into the row-major storage
    (kept for users and checks) and straight into the tiled storage the GEMMs read."""
    E, H, F = wl.E, wl.H, wl.F
    experts = range(E) if experts is None else experts
    u8 = dict(dtype=torch.uint8, device=device)
    w = NVFP4Experts(
        torch.zeros((E, 2 * F, H // 2), **u8), torch.zeros((E, 2 * F, H // 16), **u8),
        torch.ones((E,), dtype=torch.float32, device=device),
        torch.zeros((E, H, F // 2), **u8), torch.zeros((E, H, F // 16), **u8),
        torch.ones((E,), dtype=torch.float32, device=device))
    lib = ops._lib.load()
    w.w13_t = ops.TiledWeights(torch.zeros((E, lib.nvfp4_tiled_codes_bytes(2 * F, H)), **u8),
                               torch.zeros((E, lib.nvfp4_tiled_scales_bytes(2 * F, H)), **u8), w.w13_g, 2 * F, H)
    w.w2_t = ops.TiledWeights(torch.zeros((E, lib.nvfp4_tiled_codes_bytes(H, F)), **u8),
                              torch.zeros((E, lib.nvfp4_tiled_scales_bytes(H, F)), **u8), w.w2_g, H, F)
    for e in experts:
        for name, rm, t, gg in (("w13", (w.w13_packed, w.w13_scales), w.w13_t, w.w13_g),
                                ("w2", (w.w2_packed, w.w2_scales), w.w2_t, w.w2_g)):
            wf = inputs.expert_weight_fp32(wl, name, e, device)
            ops.nvfp4_quantize(wf, out=(rm[0][e], rm[1][e], gg[e:e + 1]))
            ops.nvfp4_quantize(wf, out=(t.codes[e], t.scales[e], gg[e:e + 1]), tiled=True)
    return w


def moe_forward(x: torch.Tensor, logits: torch.Tensor, k: int, w: NVFP4Experts, mode: int = ops.W4A16,
                fp8_acts: bool = False, keep: bool = False, combine: bool = False, reduce: bool = True):
    """One MoE layer forward. ``x`` bf16 [T, H]; ``logits`` f32 [T, E].

    Returns the bf16 output [T, H]; with ``keep`` a dict of every stage's tensors. With
    ``combine`` the down GEMM and the weighted reduce run as one call
    (moe_grouped_gemm_nvfp4_combine; same output bits, no Y in the stages). Without ``reduce``
    the experts' rows are returned unsummed: (Y f32 [T*k, H], slot_to_row, topk_w).
    """
    if not reduce and (combine or keep):
        raise ValueError("moe_forward: reduce=False goes without combine and keep")
    st = {}
    T = x.shape[0]
    S = T * k
    if mode == ops.W4A16:
        # routing, permutation and the token rows' preparation (after the FP8 round trip when
        # asked): one launch for up to 16 tokens
        r = ops.moe_dispatch_w4a16(logits, x, k, fp8_act=fp8_acts)
        if keep and fp8_acts:   # the rows the GEMM sees, for inspection only
            st["x_fp8"] = ops.act_fp8_e4m3_roundtrip(x)
    else:
        if fp8_acts:
            x = ops.act_fp8_e4m3_roundtrip(x)
            st["x_fp8"] = x
        r = ops.moe_route_permute(logits, k)
    st.update(r)
    common = dict(expert_offsets=r["expert_offsets"], active_experts=r["active_experts"],
                  n_active=r["n_active"])
    if mode == ops.W4A16:
        h = ops.moe_grouped_gemm_nvfp4(ops.W4A16_PREPARED, ops.EPI_SWIGLU, r["x_prep"], w.w13_t,
                                       gather_index=r["sorted_slot"], gather_div=k, rows=S, a_rows=T,
                                       out_dtype=torch.bfloat16, **common)
        if combine:
            out = ops.moe_grouped_gemm_nvfp4_combine(ops.W4A16, h, w.w2_t, sorted_slot=r["sorted_slot"],
                                                     slot_to_row=r["slot_to_row"], topk_w=r["topk_w"], **common)
        else:
            y = ops.moe_grouped_gemm_nvfp4(ops.W4A16, ops.EPI_NONE, h, w.w2_t,
                                           rows=S, out_dtype=torch.float32, **common)
    else:
        xq, xs, xg = ops.nvfp4_quantize(x)
        st.update(xq=xq, xs=xs, xg=xg)
        h, amax = ops.moe_grouped_gemm_nvfp4(ops.W4A4, ops.EPI_SWIGLU, xq, w.w13_t,
                                             a_scales=xs, a_g=xg, gather_index=r["sorted_slot"],
                                             gather_div=k, rows=S, out_dtype=torch.float32,
                                             want_amax=True, **common)
        hq, hs, hg = ops.nvfp4_quantize(h, amax=amax)
        st.update(h_amax=amax, hq=hq, hs=hs, hg=hg)
        if combine:
            out = ops.moe_grouped_gemm_nvfp4_combine(ops.W4A4, hq, w.w2_t, sorted_slot=r["sorted_slot"],
                                                     slot_to_row=r["slot_to_row"], topk_w=r["topk_w"],
                                                     a_scales=hs, a_g=hg, **common)
        else:
            y = ops.moe_grouped_gemm_nvfp4(ops.W4A4, ops.EPI_NONE, hq, w.w2_t,
                                           a_scales=hs, a_g=hg, rows=S, out_dtype=torch.float32, **common)
    if not reduce:
        return y, r["slot_to_row"], r["topk_w"]
    if not combine:
        out = ops.moe_unpermute_reduce(y, r["slot_to_row"], r["topk_w"])
    if keep:
        st.update(h=h, out=out, **({} if combine else dict(y=y)))
        return out, st
    return out


@dataclass
class MXFP4Experts:
    """MXFP4 expert weights (group-32 UE8M0 scales, no per-tensor scale), same shapes as
    NVFP4Experts: row-major as quantized, and tiled for the GEMM."""
    w13_packed: torch.Tensor   # uint8 [E, 2F, H/2]
    w13_scales: torch.Tensor   # uint8 [E, 2F, H/32]
    w2_packed: torch.Tensor    # uint8 [E, H, F/2]
    w2_scales: torch.Tensor    # uint8 [E, H, F/32]
    w13_t: ops.MxTiledWeights = None
    w2_t: ops.MxTiledWeights = None

    @property
    def E(self):
        return self.w13_packed.shape[0]


def quantize_experts_mxfp4(wl: inputs.Workload, device="cuda") -> MXFP4Experts:
    """The workload's seeded FP32 expert weights (the same values quantize_experts starts
    from), quantized one expert at a time with mxfp4_quantize, then tiled."""
    E, H, F = wl.E, wl.H, wl.F
    u8 = dict(dtype=torch.uint8, device=device)
    w = MXFP4Experts(torch.empty((E, 2 * F, H // 2), **u8), torch.empty((E, 2 * F, H // 32), **u8),
                     torch.empty((E, H, F // 2), **u8), torch.empty((E, H, F // 32), **u8))
    for e in range(E):
        p, sc = ops.mxfp4_quantize(inputs.expert_weight_fp32(wl, "w13", e, device))
        w.w13_packed[e].copy_(p)
        w.w13_scales[e].copy_(sc)
        p, sc = ops.mxfp4_quantize(inputs.expert_weight_fp32(wl, "w2", e, device))
        w.w2_packed[e].copy_(p)
        w.w2_scales[e].copy_(sc)
    w.w13_t = ops.mxfp4_weights_tile(w.w13_packed, w.w13_scales)
    w.w2_t = ops.mxfp4_weights_tile(w.w2_packed, w.w2_scales)
    return w


def moe_forward_mxfp4(x: torch.Tensor, logits: torch.Tensor, k: int, w: MXFP4Experts,
                      keep: bool = False, combine: bool = False, reduce: bool = True):
    """One MoE layer forward in MXFP4 W4A4: token rows and h are MXFP4-quantized (one UE8M0
    scale per 32 elements, no per-tensor scale, so the up/gate GEMM's epilogue writes h as
    MXFP4 directly); both GEMMs run on the scaled FP4 matrix cores. ``x`` bf16 [T, H];
    ``logits`` f32 [T, E]. ``reduce`` as for moe_forward."""
    if not reduce and (combine or keep):
        raise ValueError("moe_forward_mxfp4: reduce=False goes without combine and keep")
    st = {}
    r = ops.moe_route_permute(logits, k)
    st.update(r)
    S = x.shape[0] * k
    common = dict(expert_offsets=r["expert_offsets"], active_experts=r["active_experts"],
                  n_active=r["n_active"])
    xq, xs = ops.mxfp4_quantize(x)
    hq, hs = ops.moe_grouped_gemm_mxfp4_swiglu_q(xq, xs, w.w13_t, gather_index=r["sorted_slot"],
                                                 gather_div=k, rows=S, **common)
    if combine:
        out = ops.moe_grouped_gemm_mxfp4_combine(hq, hs, w.w2_t, sorted_slot=r["sorted_slot"],
                                                 slot_to_row=r["slot_to_row"], topk_w=r["topk_w"], **common)
    else:
        y = ops.moe_grouped_gemm_mxfp4(ops.EPI_NONE, hq, hs, w.w2_t, rows=S, out_dtype=torch.float32, **common)
        if not reduce:
            return y, r["slot_to_row"], r["topk_w"]
        out = ops.moe_unpermute_reduce(y, r["slot_to_row"], r["topk_w"])
    if keep:
        st.update(xq=xq, xs=xs, hq=hq, hs=hs, out=out, **({} if combine else dict(y=y)))
        return out, st
    return out


# ------------------------------------------------------------------ a few tokens, and the block
#: rows up to which the few-row calls run (nvfp4_matvec, moe_layer_few_nvfp4 and their MXFP4 forms)
FEW_TOKENS = 16
#: tokens up to which the block takes NVFP4 layers as two launches, set by layers of gigabytes. Cold
#: weights in a graph, two launches / the separate calls, 256 experts of 6144 x 2048 top-8 and 512 of
#: 4096 x 1024 top-22, us: 1 token 46 / 54 and 48 / 55, 8 tokens 237 / 238 and 210 / 208, 12 tokens
#: 312 / 304 and 285 / 273, 16 tokens 390 / 381 and 346 / 328. Layers whose touched weights stay below a
#: gigabyte are the faster in two launches up to FEW_TOKENS, and a caller with those passes few=True:
#: 8 experts of 256 x 512 top-2, 16 tokens 17 / 26; 60 of 2080 x 1376 top-4 63 / 85; 128 of 2048 x 768
#: top-8 60 / 67; 64 of 4096 x 1024 top-8 89 / 95; 128 of 4096 x 1536 top-8 (0.88 GB) 168 / 177.
#: (MXFP4 is the faster at every size, 44 / 76, 225 / 258 and 364 / 402 at 1, 8 and 16 tokens of the first
#: layer, with 16-bit activations: two launches up to FEW_TOKENS.)
FEW_TOKENS_NVFP4_BLOCK = 8


def _few(fn: str, few: bool | None, T: int, limit: int) -> bool:
    """Whether T rows take the few-row calls: as asked, or up to ``limit``."""
    if few and T > FEW_TOKENS:
        raise ValueError(f"{fn}: few goes up to {FEW_TOKENS} rows, got {T}")
    return T <= limit if few is None else few


def moe_forward_few(x: torch.Tensor, logits: torch.Tensor, k: int, w: NVFP4Experts | MXFP4Experts,
                    fp8_acts: bool = False, out_dtype=torch.bfloat16):
    """The MoE layer of up to 16 tokens in two launches, with 16-bit activations (after the FP8
    round trip with ``fp8_acts``, NVFP4 only) for either weight format -> bf16 [T, H], or with
    ``out_dtype`` float32 the experts' sums before that rounding."""
    if isinstance(w, MXFP4Experts):
        if fp8_acts:
            raise ValueError("moe_forward_few: fp8_acts goes with NVFP4 experts")
        return ops.moe_layer_few_mxfp4(x, logits, k, w.w13_t, w.w2_t, out_dtype=out_dtype)
    return ops.moe_layer_few_nvfp4(x, logits, k, w.w13_t, w.w2_t, fp8_acts=fp8_acts, out_dtype=out_dtype)


@dataclass
class SharedExpert:
    """A SwiGLU expert that every token goes through: one tiled matrix [2F, H] (gate rows first)
    and one [H, F], both NVFP4 or both MXFP4."""
    w13: ops.TiledWeights | ops.MxTiledWeights
    w2: ops.TiledWeights | ops.MxTiledWeights


def shared_expert_forward(x: torch.Tensor, w: SharedExpert, add: torch.Tensor | None = None, few: bool | None = None):
    """f32 [T, H] of the shared expert for bf16 rows ``x`` [T, H]: two few-row products up to 16
    rows, the second adding ``add`` (the routed experts' output); dense grouped GEMMs above,
    where ``add`` is not taken. ``few`` asks for one of the two.

    With NVFP4 weights both take 16-bit activations and round h to bf16. With MXFP4 weights the
    products do, but the GEMMs quantize x and h to MXFP4: their result is a few percent off the
    products', and a caller that needs every batch size to round alike passes few=False."""
    nv = isinstance(w.w13, ops.TiledWeights)
    if type(w.w13) is not type(w.w2) or w.w13.B != 1 or w.w2.B != 1 or w.w13.R != 2 * w.w2.C:
        raise ValueError("shared_expert_forward: w13 must be one matrix [2F, H] and w2 one [H, F] of the same format")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != w.w13.C:
        raise ValueError(f"shared_expert_forward: x must be bf16 [T, {w.w13.C}], got {x.dtype} {tuple(x.shape)}")
    T = x.shape[0]
    few = _few("shared_expert_forward", few, T, FEW_TOKENS)
    if few:
        mv = ops.nvfp4_matvec if nv else ops.mxfp4_matvec
        return mv(mv(x, w.w13, ops.EPI_SWIGLU), w.w2, add=add, out_dtype=torch.float32)
    if add is not None:
        raise ValueError(f"shared_expert_forward: add is taken by the few-row products, up to {FEW_TOKENS} rows")
    x, ldx = ops._rows("shared_expert_forward", "x", x, w.w13.C, 8)
    x = x if ldx == w.w13.C else x.contiguous()   # (the grouped GEMM takes rows beside each other)
    with ops._on(ops._gpu("shared_expert_forward", x, w.w13.codes, w.w2.codes)):   # (the GEMMs launch on the current GPU)
        i32 = dict(dtype=torch.int32, device=x.device)
        dense = dict(expert_offsets=torch.arange(0, 2 * T, T, **i32), active_experts=torch.zeros((1,), **i32),
                     n_active=torch.ones((1,), **i32))
        if nv:
            h = ops.moe_grouped_gemm_nvfp4(ops.W4A16, ops.EPI_SWIGLU, x, w.w13, **dense)
            return ops.moe_grouped_gemm_nvfp4(ops.W4A16, ops.EPI_NONE, h, w.w2, out_dtype=torch.float32, **dense)
        hq, hs = ops.moe_grouped_gemm_mxfp4_swiglu_q(*ops.mxfp4_quantize(x), w.w13, **dense)
        return ops.moe_grouped_gemm_mxfp4(ops.EPI_NONE, hq, hs, w.w2, out_dtype=torch.float32, **dense)


def moe_block_forward(resid: torch.Tensor, x: torch.Tensor, k: int, w: NVFP4Experts | MXFP4Experts, router, *,
                      shared: SharedExpert | None = None, post_w: torch.Tensor | None = None,
                      gate: torch.Tensor | None = None, scale: float = 1.0, pre_w: torch.Tensor | None = None,
                      w_offset: float = 0.0, eps: float = 1e-6, fp8_acts: bool = False, few: bool | None = None):
    """One MoE block and the norms around it: logits = ``router``(x), y = the routed experts (and
    the ``shared`` one), then moe_block_norm's r' = resid + scale * gate * (post-norm of y) and
    the next block's normed input. ``x`` bf16 [T, H] is this block's normed input: the next
    of the call before, or ``ops.moe_block_norm(resid, pre_w=...)[1]`` at the start.

    Up to 8 tokens (MXFP4: 16) the layer runs as two launches (moe_forward_few) and the shared
    expert, up to 16, as two more; above, the separate calls' rows (moe_forward, W4A16, or
    moe_forward_mxfp4) go unsummed into the norm, which adds the shared expert's output. ``few``
    asks for one of the two for both: True goes up to 16 tokens. y stays float32 either way, but
    what is rounded before it differs: with NVFP4 experts h (to 11 bits in two launches, to bf16
    in the separate calls); with MXFP4 experts x and h, which the separate calls quantize to MXFP4
    while two launches take x as it is and hold h in 16 bits. A caller that needs a request's
    numbers not to change that way with the batch it is in passes few=False. (The separate calls
    take MXFP4 experts, and an MXFP4 shared one, with H a multiple of 256 and F of 128; two
    launches with any multiples of 32.)

    ``fp8_acts``: the routed experts' rows take the FP8 round trip first (NVFP4 only); the shared
    expert's do not. Returns (r', next); next is None without ``pre_w``."""
    T = x.shape[0]
    mx = isinstance(w, MXFP4Experts)
    limit = FEW_TOKENS if mx else FEW_TOKENS_NVFP4_BLOCK
    two_launches = _few("moe_block_forward", few, T, limit)
    logits = router(x)
    norm = dict(post_w=post_w, gate=gate, scale=scale, pre_w=pre_w, w_offset=w_offset, eps=eps)
    if two_launches:
        y = moe_forward_few(x, logits, k, w, fp8_acts, torch.float32)   # (not rounded before the norm)
        if shared is not None:
            y = shared_expert_forward(x, shared, add=y)
        return ops.moe_block_norm(resid, y, **norm)
    # (the separate calls take their sizes from the weights alone)
    w13, w2 = w.w13_t, w.w2_t
    if x.dtype != torch.bfloat16 or x.shape != (T, w13.C) or logits.shape != (T, w13.B) or \
            (w2.B, w2.R, w13.R) != (w13.B, w13.C, 2 * w2.C):
        raise ValueError(f"moe_block_forward: weights {w13.B} x [{w13.R}, {w13.C}] and {w2.B} x [{w2.R}, {w2.C}], x "
                         f"{x.dtype} {tuple(x.shape)} (bf16 [T, H]) and logits {tuple(logits.shape)} do not fit together")
    if mx and fp8_acts:
        raise ValueError("moe_block_forward: fp8_acts goes with NVFP4 experts")
    with ops._on(ops._gpu("moe_block_forward", x, logits, w13.codes, w2.codes)):
        if mx:
            y, slot_to_row, topk_w = moe_forward_mxfp4(x, logits, k, w, reduce=False)
        else:
            y, slot_to_row, topk_w = moe_forward(x, logits, k, w, fp8_acts=fp8_acts, reduce=False)
    ys = None if shared is None else shared_expert_forward(x, shared, few=few)
    return ops.moe_block_norm(resid, y, slot_to_row=slot_to_row, topk_w=topk_w, y_add=ys, **norm)


# ------------------------------------------------------------------ the attention block
@dataclass
class AttentionWeights:
    """An attention block's projections, each one tiled matrix, both NVFP4 or both MXFP4: qkv
    [(heads + 2 * key heads) * D, H] (queries' heads first, then the keys', then the values') and o
    [H, heads * D]. The cache says how many key heads there are and their D. A layer that reads the cache of
    an earlier one, and brings no keys of its own, has queries alone: qkv [heads * D, H]."""
    qkv: ops.TiledWeights | ops.MxTiledWeights
    o: ops.TiledWeights | ops.MxTiledWeights
    heads: int


def _projection(x: torch.Tensor, w, out_dtype, few: bool):
    """x W^T of rows [T, K]: a few-row product, or a grouped GEMM of one matrix."""
    nv = isinstance(w, ops.TiledWeights)
    if few:
        return (ops.nvfp4_matvec if nv else ops.mxfp4_matvec)(x, w, out_dtype=out_dtype)
    T = x.shape[0]
    i32 = dict(dtype=torch.int32, device=x.device)
    dense = dict(expert_offsets=torch.arange(0, 2 * T, T, **i32), active_experts=torch.zeros((1,), **i32),
                 n_active=torch.ones((1,), **i32), out_dtype=out_dtype)
    if nv:
        return ops.moe_grouped_gemm_nvfp4(ops.W4A16, ops.EPI_NONE, x, w, **dense)
    return ops.moe_grouped_gemm_mxfp4(ops.EPI_NONE, *ops.mxfp4_quantize(x), w, **dense)


def attention_block_forward(resid: torch.Tensor, x: torch.Tensor, w: AttentionWeights, cache: ops.KVCache,
                            batch: ops.CacheBatch, *, rope: ops.Rope | None = None, positions: torch.Tensor | None = None,
                            attention_scale: float | None = None, window: int = 0, post_w: torch.Tensor | None = None,
                            gate: torch.Tensor | None = None, scale: float = 1.0, pre_w: torch.Tensor | None = None,
                            w_offset: float = 0.0, eps: float = 1e-6, few: bool | None = None):
    """One attention block and the norms around it, the other half of the decoder layer that
    moe_block_forward ends: queries, keys and values of the new tokens ``x`` bf16 [T, H] (this block's
    normed input) by one projection, kv_cache_append with ``rope``, kv_cache_attention, the output
    projection to float32, and moe_block_norm's r' = resid + scale * gate * (post-norm of it) with the
    next block's normed input. Returns (r', next): what moe_block_forward takes as ``resid`` and ``x``.

    Up to 16 rows the projections are few-row products, above grouped GEMMs of one matrix; ``few`` asks
    for one of the two, as in shared_expert_forward (MXFP4 GEMMs quantize their rows, products do not).
    Queries, keys, values and the attention's output are bf16. With queries alone (AttentionWeights) nothing is
    appended and the queries are turned by rope_rotate, at ``positions``, which it needs then. Rows behind the batch's last sequence
    (a padded batch) give no keys, and what comes back in them is of no meaning."""
    fn = "attention_block_forward"
    heads, D = cache.k.shape[1], cache.k.shape[3]
    H, Hq = w.o.R, w.heads
    queries_alone = w.qkv.R == Hq * D
    if type(w.qkv) is not type(w.o) or w.qkv.B != 1 or w.o.B != 1 or w.qkv.C != H or w.o.C != Hq * D or \
            not (queries_alone or w.qkv.R == (Hq + 2 * heads) * D):
        raise ValueError(f"{fn}: qkv must be one matrix [{(Hq + 2 * heads) * D}, H] (or [{Hq * D}, H]) and o one [H, {Hq * D}] "
                         f"of the same format, got [{w.qkv.R}, {w.qkv.C}] and [{w.o.R}, {w.o.C}]")
    if queries_alone and rope is not None and positions is None:
        raise ValueError(f"{fn}: a layer with queries alone needs their positions")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != H:
        raise ValueError(f"{fn}: x must be bf16 [T, {H}], got {x.dtype} {tuple(x.shape)}")
    T = x.shape[0]
    few = _few(fn, few, T, FEW_TOKENS)
    x, ldx = ops._rows(fn, "x", x, H, 8)
    x = x if few or ldx == H else x.contiguous()   # (the grouped GEMM takes rows beside each other)
    with ops._on(ops._gpu(fn, x, w.qkv.codes, w.o.codes)):   # (the GEMMs launch on the current GPU)
        qkv = _projection(x, w.qkv, torch.bfloat16, few).view(T, -1, D)
        q = qkv[:, :Hq]
        if queries_alone and rope is not None:
            ops.rope_rotate(q, positions, rope, out=q)
        elif not queries_alone:
            ops.kv_cache_append(cache, batch, qkv[:, Hq:Hq + heads], qkv[:, Hq + heads:], q=q, rope=rope,
                                positions=positions, q_out=q)
        a = ops.kv_cache_attention(q, cache, batch, scale=attention_scale, window=window)
        y = _projection(a.view(T, Hq * D), w.o, torch.float32, few)
    return ops.moe_block_norm(resid, y, post_w=post_w, gate=gate, scale=scale, pre_w=pre_w, w_offset=w_offset, eps=eps)
