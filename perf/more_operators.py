"""What is measured of the attention half of a decoder block: rotary positions, appending keys and values to a paged
cache with the rotation applied on the way, and the attention of new tokens over that cache.

`run` computes them plainly with torch in float32 (angles in float64), or, where `own` is true, through the library's
calls. The cache holds keys as [pages, heads, page, D] and values as [pages, heads, D, page], in bf16 or in FP8 E4M3
with a float32 scale for each head; a batch is a page table [B, n], the lengths of its sequences with their new tokens,
and the row at which each one's new tokens start.
"""
import math
import random

import torch

own = False

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
TABLE_SPARE = 3   # columns of the page table behind the longest sequence's pages


# ---------------------------------------------------------------------------- cases
def _rope(name, T, H, D, rot, start=0, interleaved=False, grad=False, f32=False, scaled=False, far=4096):
    return dict(name=name, op="rope", T=T, H=H, D=D, rot=rot, start=start, interleaved=interleaved, grad=grad, f32=f32,
                scaled=scaled, far=far)


def _append(name, B, new, ctx, Hq, Hkv, D, rot, page, fp8=False, start=0, interleaved=False, scaled=False, lens=1):
    return dict(name=name, op="append", B=B, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1], ones=0, Hq=Hq,
                Hkv=Hkv, D=D, rot=rot, page=page, fp8=fp8, start=start, interleaved=interleaved, scaled=scaled, lens=lens)


def _attend(name, B, new, ctx, Hq, Hkv, D, page, fp8=False, window=0, ones=0, lens=1):
    return dict(name=name, op="attend", B=B, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1], ones=ones, Hq=Hq,
                Hkv=Hkv, D=D, page=page, fp8=fp8, window=window, lens=lens)


def listed():
    return [
        # One token of a small model: all latency.
        _rope("rope one token", 1, 8, 64, 64),
        # The gradient for a training step in float32: an odd number of rows, adjacent pairs, the second half of the
        # head alone, far positions of a stretched context.
        _rope("rope odd gradient", 1021, 24, 128, 64, start=64, interleaved=True, grad=True, f32=True, scaled=True, far=500_000),
        # A prompt's queries.
        _rope("rope prompt", 8192, 64, 128, 128),
        # One request decoding: its query, key and value.
        _append("append one token", 1, (1, 1), (700, 700), 64, 8, 128, 128, 64),
        # Requests that bring a few tokens each, small pages, part of the head in adjacent pairs, FP8.
        _append("append odd few", 37, (1, 9), (0, 900), 20, 4, 96, 32, 16, fp8=True, interleaved=True),
        # Prompts of different lengths.
        _append("append prompts", 6, (300, 5000), (0, 64), 64, 8, 128, 128, 64, scaled=True),
        # A short conversation's next token: all latency.
        _attend("attend one short", 1, (1, 1), (180, 180), 16, 2, 64, 16),
        # A serving batch decoding at very different lengths.
        _attend("attend decode batch", 64, (1, 1), (500, 8100), 64, 8, 128, 64),
        # Two long documents, FP8 cache, one of them four tokens ahead (drafted tokens to be checked).
        _attend("attend long fp8", 2, (1, 4), (90_000, 130_000), 64, 8, 128, 64, fp8=True),
        # A chunk of a long prompt.
        _attend("attend chunk", 1, (2048, 2048), (14_000, 14_000), 64, 8, 128, 64),
        # Whole prompts of odd lengths in one batch, a sliding window, another head size.
        _attend("attend prompts window", 7, (33, 2900), (0, 200), 24, 4, 96, 32, window=1000),
        # A chunk of one prompt beside requests that decode, FP8, small pages.
        _attend("attend mixed fp8", 33, (500, 500), (200, 3500), 32, 8, 128, 16, fp8=True, ones=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "attend"))
    D = rng.choice((32, 64, 64, 96, 128, 128, 128, 160, 192, 224, 256))
    rot = rng.choice((D, D, D // 2, 8 * rng.randint(1, D // 8)))
    start = rng.choice((0, D - rot))
    interleaved = rng.random() < 0.5
    if op == "rope":
        H = rng.randint(1, 64)
        T = _log(rng, 1, max(2, min(8192, 60_000_000 // (H * D))))
        return dict(op=op, T=T, H=H, D=D, rot=rot, start=start, interleaved=interleaved, grad=rng.random() < 0.4,
                    f32=rng.random() < 0.4, scaled=rng.random() < 0.4, far=_log(rng, 16, 1_000_000))
    Hkv = rng.choice((1, 2, 4, 8, 8, 3, 5))
    G = rng.choice((1, 2, 4, 6, 8, 8, 16))
    page, fp8, lens = rng.choice((16, 32, 64, 64, 128, 256)), rng.random() < 0.4, rng.randint(1, 1 << 20)
    if op == "append":
        B = _log(rng, 1, 64)
        most = max(1, min(4096, 80_000_000 // (Hkv * (G + 2) * D * B)))
        new = sorted((_log(rng, 1, most), _log(rng, 1, most)))
        ctx = sorted((rng.randint(0, 1000), rng.randint(0, 1000)))
        return dict(op=op, B=B, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1], ones=rng.choice((0, 0, B - 1)),
                    Hq=G * Hkv, Hkv=Hkv, D=D, rot=rot, page=page, fp8=fp8, start=start, interleaved=interleaved,
                    scaled=rng.random() < 0.4, lens=lens)
    kind = rng.choice(("decode", "decode", "drafts", "chunk", "mixed"))
    B = 1 if kind == "chunk" and rng.random() < 0.4 else _log(rng, 1, 8 if kind == "chunk" else 96)
    most = {"decode": 1, "drafts": 8}.get(kind) or max(16, min(2048, 2000 * 128 // (B * D)))
    new = sorted((_log(rng, 1, most), _log(rng, 1, most)))
    # what a pass reads and, in the plain form, holds: at most about that of the largest listed cases
    far = min(100_000, 150_000_000 // (B * Hkv * D), 1_200_000_000 * 128 // (B * G * Hkv * new[1] * max(D, 128)))
    ctx = sorted((_log(rng, 1, max(2, far)) - 1, _log(rng, 1, max(2, far)) - 1))
    return dict(op=op, B=B, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1], ones=B - 1 if kind == "mixed" else 0,
                Hq=G * Hkv, Hkv=Hkv, D=D, page=page, fp8=fp8, window=_log(rng, 16, 8000) if rng.random() < 0.25 else 0, lens=lens)


def _lengths(case):
    """([new tokens], [tokens before them]) of the case's sequences; the last one takes the upper ends."""
    rng = random.Random(case["lens"])
    B = case["B"]
    pick = lambda lo, hi: lo if lo == hi else max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1))  # noqa: E731
    new = [1 if b < case["ones"] else pick(case["new_lo"], case["new_hi"]) for b in range(B)]
    ctx = [pick(case["ctx_lo"], case["ctx_hi"]) for b in range(B)]
    new[-1], ctx[-1] = case["new_hi"], case["ctx_hi"]
    return new, ctx


# ---------------------------------------------------------------------------- inputs
def _frequencies(rot, scaled, dev):
    """Radians a position of each pair (base 10000) and the magnitude; stretched 32-fold: the pairs that turn fewer
    than once in 4096 positions 32 times slower, those of 32 turns and more as they were, a ramp between."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    f = 10000.0 ** (-2.0 * i / rot)
    if not scaled:
        return f, 1.0
    at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    low, high = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return f / 32.0 * ramp + f * (1.0 - ramp), 0.1 * math.log(32.0) + 1.0


def _rows(gen, T, H, D, dev):
    """bf16 [T, H, D]: N(0, 1) with a spread between channels."""
    spread = torch.exp(0.4 * torch.randn((H, D), generator=gen, device=dev))
    return (torch.randn((T, H, D), generator=gen, device=dev) * spread).to(BF)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case=case)
    D = case["D"]
    if case["op"] == "rope":
        T, H = case["T"], case["H"]
        s["x"] = _rows(gen, T, H, D, dev)
        if case["f32"]:
            s["x"] = torch.randn((T, H, D), generator=gen, device=dev)
        s["positions"] = torch.randint(case["far"], (T,), generator=gen, device=dev).to(torch.int32)
        s["freqs"], s["magnitude"] = _frequencies(case["rot"], case["scaled"], dev)
        return s
    new, ctx = _lengths(case)
    B, Hq, Hkv, page = case["B"], case["Hq"], case["Hkv"], case["page"]
    T = sum(new)
    i32 = dict(dtype=torch.int32, device=dev)
    s["lengths"] = torch.tensor([n + c for n, c in zip(new, ctx)], **i32)
    s["starts"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], **i32)
    used = [-(-(n + c) // page) for n, c in zip(new, ctx)]
    pages = sum(used) + 5
    table = torch.full((B, max(used) + TABLE_SPARE), -1, dtype=torch.int32)
    places = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).cpu()
    at = 0
    for b in range(B):
        table[b, :used[b]] = places[at:at + used[b]]
        at += used[b]
    s["page_table"] = table.to(dev)
    s["max_new"], s["max_length"] = max(new), max(n + c for n, c in zip(new, ctx))
    k = torch.randn((pages, Hkv, page, D), generator=gen, device=dev, dtype=BF)
    k *= torch.exp(0.4 * torch.randn((Hkv, 1, D), generator=gen, device=dev)).to(BF)
    v = torch.randn((pages, Hkv, D, page), generator=gen, device=dev, dtype=BF)
    s["k_scale"] = s["v_scale"] = None
    if case["fp8"]:
        s["k_scale"] = 0.01 + 0.02 * torch.rand((Hkv,), generator=gen, device=dev)
        s["v_scale"] = 0.01 + 0.02 * torch.rand((Hkv,), generator=gen, device=dev)
        k = (k / s["k_scale"].to(BF).view(-1, 1, 1)).clamp(-448.0, 448.0).to(F8)
        v = (v / s["v_scale"].to(BF).view(-1, 1, 1)).clamp(-448.0, 448.0).to(F8)
    s["k_cache"], s["v_cache"] = k, v
    if case["op"] == "append":
        # queries, keys and values as a projection leaves them: beside each other in one row
        s["qkv"] = _rows(gen, T, Hq + 2 * Hkv, D, dev)
        s["freqs"], s["magnitude"] = _frequencies(case["rot"], case["scaled"], dev)
    else:
        s["q"] = _rows(gen, T, Hq, D, dev)
    return s


# ---------------------------------------------------------------------------- the plain forms
def _rotated(x, positions, s, grad=False):
    """float32 rows x [T, H, D] with the case's part of each head turned by its position's angles."""
    c = s["case"]
    a, r = c["start"], c["rot"]
    angle = positions.double().unsqueeze(-1) * s["freqs"]
    cos = (torch.cos(angle) * s["magnitude"]).float().unsqueeze(1)
    sin = (torch.sin(angle) * (-s["magnitude"] if grad else s["magnitude"])).float().unsqueeze(1)
    part = x[..., a:a + r]
    if c["interleaved"]:
        u, w = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2)
    else:
        u, w = part[..., :r // 2], part[..., r // 2:]
        turned = torch.cat((u * cos - w * sin, w * cos + u * sin), -1)
    return torch.cat((x[..., :a], turned, x[..., a + r:]), -1)


def _row_places(s):
    """(sequence, index among its new tokens, position) of every row."""
    starts, T = s["starts"].long(), int(s["T"])
    t = torch.arange(T, device=starts.device)
    b = torch.searchsorted(starts, t, right=True) - 1
    i = t - starts[b]
    return b, i, s["lengths"].long()[b] - (starts[b + 1] - starts[b]) + i


def _to_cache(x, cache, scale):
    if scale is None:
        return x.to(BF)
    return (x / scale.view(-1, 1)).clamp(-448.0, 448.0).to(F8).view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    Hq, Hkv, page = c["Hq"], c["Hkv"], c["page"]
    s["T"] = s["qkv"].shape[0]
    b, _, position = _row_places(s)
    x = s["qkv"].float()
    q = _rotated(x[:, :Hq], position, s).to(BF)
    k = _to_cache(_rotated(x[:, Hq:Hq + Hkv], position, s), s["k_cache"], s["k_scale"])
    v = _to_cache(x[:, Hq + Hkv:], s["v_cache"], s["v_scale"])
    at, slot = s["page_table"].long()[b, position // page], position % page
    kc, vc = (s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)) if c["fp8"] else (s["k_cache"], s["v_cache"])
    kc[at, :, slot] = k
    vc[at, :, :, slot] = v
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _cache_values(cache, table, scale):
    """float32 [B, heads, n, ., .] of the pages of a table [B, n]."""
    if scale is None:
        x = cache[table].float()
    else:
        x = cache.view(torch.uint8)[table].view(F8).float() * scale.view(-1, 1, 1)
    return x.transpose(1, 2)


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, D, page, n = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"], s["max_new"]
    s["T"] = s["q"].shape[0]
    b, i, _ = _row_places(s)
    dev = s["q"].device
    cols = -(-s["max_length"] // page)
    table = s["page_table"][:, :cols].long().clamp(min=0)
    k = _cache_values(s["k_cache"], table, s["k_scale"]).reshape(B, Hkv, cols * page, D)
    v = _cache_values(s["v_cache"], table, s["v_scale"]).transpose(-1, -2).reshape(B, Hkv, cols * page, D)
    rows = (s["starts"][:-1].long().unsqueeze(1) + torch.arange(n, device=dev)).clamp(max=s["T"] - 1)
    q = s["q"].float()[rows].view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5).view(B, Hkv, Hq // Hkv, n, -1)
    last = (s["lengths"] - (s["starts"][1:] - s["starts"][:-1])).view(B, 1) + torch.arange(n, device=dev)
    key = torch.arange(cols * page, device=dev)
    hidden = key > last.unsqueeze(-1)
    if c["window"]:
        hidden = hidden | (key <= last.unsqueeze(-1) - c["window"])
    score.masked_fill_(hidden.view(B, 1, 1, n, -1), -math.inf)
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1)
    out = torch.matmul(score.view(B, Hkv, -1, cols * page), v).view(B, Hkv, Hq // Hkv, n, D) / total.unsqueeze(-1)
    return out.permute(0, 3, 1, 2, 4)[b, i].reshape(s["T"], Hq, D).to(BF)


# ---------------------------------------------------------------------------- the library's calls
def _handles(s):
    """What a program makes once and keeps: the rotation, the cache and the batch, of the tensors it has."""
    from nvfp4_block_scaled_moe_amd import ops
    c = s["case"]
    h = {}
    if "freqs" in s:
        h["rope"] = ops.Rope(s["freqs"], start=c["start"], interleaved=c["interleaved"], magnitude=s["magnitude"])
    if "k_cache" in s:
        h["cache"] = ops.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        h["batch"] = ops.CacheBatch(s["page_table"], s["lengths"], s["starts"])
    s["handles"] = h
    return h


def _own(s):
    from nvfp4_block_scaled_moe_amd import ops
    c = s["case"]
    h = s.get("handles") or _handles(s)
    if c["op"] == "rope":
        return ops.rope_rotate(s["x"], s["positions"], h["rope"], grad=c["grad"])
    if c["op"] == "append":
        Hq, Hkv = c["Hq"], c["Hkv"]
        x = s["qkv"]
        q = ops.kv_cache_append(h["cache"], h["batch"], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q=x[:, :Hq], rope=h["rope"])
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    return ops.kv_cache_attention(s["q"], h["cache"], h["batch"], window=c["window"])


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "rope":
        x = state["x"]
        return _rotated(x.float(), state["positions"], state, c["grad"]).to(x.dtype)
    return _plain_append(state) if c["op"] == "append" else _plain_attend(state)


# ---------------------------------------------------------------------------- work
def work(case):
    D = case["D"]
    if case["op"] == "rope":
        n = case["T"] * case["H"] * D
        return dict(bytes=2 * n * (4 if case["f32"] else 2) + 4 * case["T"] + 4 * case["rot"],
                    flops=3 * case["T"] * case["H"] * case["rot"])
    new, ctx = _lengths(case)
    T, Hq, Hkv, size = sum(new), case["Hq"], case["Hkv"], 1 if case["fp8"] else 2
    plan = 8 * case["B"] + 4
    if case["op"] == "append":
        return dict(bytes=T * D * (4 * Hq + 2 * (2 + size) * Hkv) + plan + 4 * T + 4 * case["rot"],
                    flops=3 * T * (Hq + Hkv) * case["rot"])
    W = case["window"]
    keys = [n + c - (max(0, c + 1 - W) if W else 0) for n, c in zip(new, ctx)]   # that any of the new tokens sees
    # a new token of position p sees p + 1 keys, or the window's
    full = lambda n, c: n * c + n * (n + 1) // 2  # noqa: E731  (sum of p + 1 over p = c .. c + n - 1)
    seen = [full(n, c) - (full(n, c) - full(min(n, max(0, W - c)), c) - W * (n - min(n, max(0, W - c))) if W else 0)
            for n, c in zip(new, ctx)]
    pages = sum(-(-k // case["page"]) for k in keys)
    return dict(bytes=2 * size * sum(keys) * Hkv * D + 4 * T * Hq * D + plan + 4 * pages, flops=4 * sum(seen) * Hq * D)


# ---------------------------------------------------------------------------- exact values
def _turned(x, positions, case, s, sign):
    """float64: each pair as a complex number times magnitude * exp(+-i angle)."""
    a, r = case["start"], case["rot"]
    x = x.double().clone()
    part = x[..., a:a + r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
    axis = -1 if case["interleaved"] else -2
    z = torch.complex(*(part.select(axis, j) for j in (0, 1)))
    angle = sign * torch.outer(positions.double(), s["freqs"])
    z = z * torch.polar(torch.full_like(angle, s["magnitude"]), angle)[:, None]
    x[..., a:a + r] = torch.stack((z.real, z.imag), axis).flatten(-2)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(s["x"], s["positions"], case, s, -1.0 if case["grad"] else 1.0)
    new, ctx = _lengths(case)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    kc, vc = s["k_cache"], s["v_cache"]
    first = 0
    if case["op"] == "append":
        q, kc, vc = [], kc.double(), vc.double()
        ks, vs = (s["k_scale"].double().view(-1, 1), s["v_scale"].double().view(-1, 1)) if case["fp8"] else (1.0, 1.0)
        top = 448.0 if case["fp8"] else math.inf
        for b, (n, c) in enumerate(zip(new, ctx)):
            p = torch.arange(c, c + n, device=kc.device)
            x = s["qkv"][first:first + n]
            first += n
            q.append(_turned(x[:, :Hq], p, case, s, 1.0))
            k = (_turned(x[:, Hq:Hq + Hkv], p, case, s, 1.0) / ks).clamp(-top, top)
            v = (x[:, Hq + Hkv:].double() / vs).clamp(-top, top)
            at = s["page_table"][b, torch.div(p, page, rounding_mode="floor")].long()
            kc.transpose(1, 2)[at, p % page] = k
            vc.permute(0, 3, 1, 2)[at, p % page] = v
        return dict(q=torch.cat(q), k_cache=kc, v_cache=vc)
    out = []
    for b, (n, c) in enumerate(zip(new, ctx)):
        at = s["page_table"][b, :-(-(n + c) // page)].long()
        take = lambda t: (t.view(torch.uint8)[at].view(F8) if case["fp8"] else t[at]).double()  # noqa: E731
        k = take(kc).permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n + c]
        v = take(vc).permute(1, 0, 3, 2).reshape(Hkv, -1, D)[:, :n + c]
        if case["fp8"]:
            k, v = k * s["k_scale"].double().view(-1, 1, 1), v * s["v_scale"].double().view(-1, 1, 1)
        far = torch.arange(c, c + n, device=k.device).unsqueeze(1) - torch.arange(n + c, device=k.device)
        seen = (far >= 0) & (far < (case["window"] or n + c))
        bias = torch.zeros_like(far, dtype=torch.float64).masked_fill_(~seen, -math.inf)
        rows = s["q"][first:first + n].double().unflatten(1, (Hkv, -1))
        first += n
        heads = [torch.softmax(torch.matmul(rows[:, h].transpose(0, 1), k[h].t()) / math.sqrt(D) + bias, -1) @ v[h]
                 for h in range(Hkv)]
        out.append(torch.stack(heads, 0).permute(2, 0, 1, 3).reshape(n, Hq, D))
    return torch.cat(out)
