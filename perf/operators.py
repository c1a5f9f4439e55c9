"""What is measured of the decode block's operators: products of a few rows with 4-bit weights, a whole
mixture-of-experts layer for a few tokens, and the norms around it with their gate and residual scale.

`run` computes them plainly with torch in float32, or, where `own` is true, through the library's calls.
Weights are NVFP4 (E2M1 codes, an E4M3 scale for 16 columns, a float32 scale a matrix) or MXFP4 (a power-of-two
scale for 32 columns); they are laid out once, row-major and in the library's tiled storage, as a program that
serves them keeps them.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDPOINTS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
POOL_ROWS = 768
EPS = 1e-6


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # The smallest product: a gate/up projection of a small model, one token; all latency.
        dict(name="matvec small one row", op="matvec", fmt="nvfp4", T=1, N=1024, K=256, swiglu=True, add=False, f32=False),
        # A dense projection beside the experts while one request decodes.
        dict(name="matvec one row", op="matvec", fmt="nvfp4", T=1, N=2048, K=6144, swiglu=False, add=False, f32=True),
        # Sizes off the powers of two, a ragged last chunk, MXFP4 weights, added to another branch's output.
        dict(name="matvec odd rows", op="matvec", fmt="mxfp4", T=5, N=2064, K=1184, swiglu=False, add=True, f32=False),
        # A wide output projection for a batch of 16 requests.
        dict(name="matvec wide 16 rows", op="matvec", fmt="nvfp4", T=16, N=65536, K=6144, swiglu=False, add=False, f32=False),
        # A small layer, a few tokens: latency of routing and both products.
        dict(name="layer small", op="layer", fmt="nvfp4", T=3, E=8, k=2, H=256, F=512, fp8=False),
        # One request decoding through a large layer: 8 of 256 experts are read.
        dict(name="layer one token", op="layer", fmt="nvfp4", T=1, E=256, k=8, H=6144, F=2048, fp8=False),
        # Many small experts with FP8 activations, four requests.
        dict(name="layer many small", op="layer", fmt="nvfp4", T=4, E=512, k=22, H=4096, F=1024, fp8=True),
        # MXFP4 experts at odd sizes, two requests.
        dict(name="layer odd", op="layer", fmt="mxfp4", T=2, E=60, k=4, H=2080, F=1376, fp8=False),
        # Sixteen requests: most of the large layer's experts are touched.
        dict(name="layer 16 tokens", op="layer", fmt="nvfp4", T=16, E=256, k=8, H=6144, F=2048, fp8=False),
        # One token after the experts: weighted sum of their rows, post-norm, residual, next pre-norm.
        dict(name="norm experts one token", op="norm", T=1, H=6144, k=8, rows=True, post=True, gate="none", scale=1.0, pre=True, f32=False),
        # A batch with an odd width and a gate for every element.
        dict(name="norm odd", op="norm", T=37, H=1000, k=0, rows=False, post=True, gate="full", scale=0.25, pre=True, f32=True),
        # A long prompt: residual in float32, a learned gate for each channel.
        dict(name="norm prompt", op="norm", T=8192, H=7168, k=0, rows=False, post=True, gate="channel", scale=0.5, pre=True, f32=True),
    ]


def _log(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread evenly over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step))


def draw(rng):
    op = rng.choice(("matvec", "layer", "norm"))
    fmt = rng.choice(("nvfp4", "mxfp4"))
    if op == "matvec":
        swiglu = rng.random() < 0.4
        return dict(op=op, fmt=fmt, T=rng.randint(1, 16), N=_log(rng, 64, 32768, 32 if swiglu else 16),
                    K=_log(rng, 64, 12288, 32), swiglu=swiglu, add=rng.random() < 0.4, f32=rng.random() < 0.5)
    if op == "layer":
        E = rng.randint(4, 160)
        return dict(op=op, fmt=fmt, T=rng.randint(1, 16), E=E, k=rng.randint(1, min(10, E)), H=_log(rng, 128, 6144, 32),
                    F=_log(rng, 64, 2048, 32), fp8=fmt == "nvfp4" and rng.random() < 0.3)
    rows = rng.random() < 0.5
    H = _log(rng, 64, 12288, 8)
    k = rng.randint(1, 12) if rows else 0
    return dict(op=op, T=_log(rng, 1, max(2, min(8192, 40_000_000 // (H * max(1, k)))), 1), H=H, k=k, rows=rows,
                post=rng.random() < 0.8, gate=rng.choice(("none", "channel", "token", "full")),
                scale=rng.choice((1.0, 0.5, 0.22)), pre=rng.random() < 0.8, f32=rng.random() < 0.5)


# ---------------------------------------------------------------------------- inputs
def _quantized_rows(gen, rows, C, fmt, device):
    """Codes and scales of `rows` rows of N(0, 0.02) weights, rounded to the format."""
    group = 16 if fmt == "nvfp4" else 32
    w = (torch.randn((rows, C), generator=gen, device=device) * 0.02).view(rows, C // group, group)
    top = w.abs().amax(-1)
    if fmt == "nvfp4":
        g = float(top.max()) / 2688.0
        scales = (top / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        step = scales.float() * g
        scales = scales.view(torch.uint8)
    else:
        g = 1.0
        e = torch.floor(torch.log2(top)) - 2.0
        step = torch.exp2(e)
        scales = (e + 127.0).to(torch.uint8)
    edges = torch.tensor(MIDPOINTS, device=device)
    mag = torch.bucketize((w.abs() / step.unsqueeze(-1)).contiguous(), edges)
    codes = (mag + 8 * (w < 0)).to(torch.uint8).view(rows, C // 2, 2)
    return codes[..., 0] | (codes[..., 1] << 4), scales, g


def _weights(gen, E, R, C, fmt, device):
    """E matrices [R, C]: rows taken from a pool of quantized ones, a scale of its own for each matrix; row-major
    and in the tiled storage (16 rows x 128 columns of codes a kilobyte; the scales of 8 or 16 such tiles a kilobyte)."""
    pc, ps, g = _quantized_rows(gen, POOL_ROWS, C, fmt, device)
    pick = torch.randint(POOL_ROWS, (E * R,), generator=gen, device=device)
    codes, scales = pc[pick], ps[pick]
    gs = g * (0.5 + torch.rand((E,), generator=gen, device=device)) if fmt == "nvfp4" else None
    nch = -(-C // 128)
    t = torch.nn.functional.pad(codes, (0, 64 * nch - C // 2)) if C % 128 else codes
    tc = t.view(E, R // 16, 16, nch, 4, 16).permute(0, 1, 3, 4, 2, 5).reshape(E, -1)
    if fmt == "nvfp4":
        nwin = -(-C // 1024)
        t = torch.nn.functional.pad(scales, (0, 64 * nwin - C // 16))
        ts = t.view(E, R // 16, 16, nwin, 8, 4, 2).permute(0, 1, 3, 5, 2, 4, 6).reshape(E, -1)
    else:
        nwin = -(-C // 2048)
        t = torch.nn.functional.pad(scales, (0, 64 * nwin - C // 32))
        ts = t.view(E, R // 16, 16, nwin, 16, 4).permute(0, 1, 3, 5, 2, 4).reshape(E, -1)
    return dict(fmt=fmt, R=R, C=C, codes=codes.view(E, R, C // 2), scales=scales.view(E, R, -1), g=gs,
                tiled_codes=tc.contiguous(), tiled_scales=ts.contiguous())


def _rows(gen, T, H, device):
    """bf16 activations: N(0, 1) with a spread between channels."""
    spread = torch.exp(0.5 * torch.randn((H,), generator=gen, device=device))
    return (torch.randn((T, H), generator=gen, device=device) * spread).to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "matvec":
        s["w"] = _weights(gen, 1, case["N"], case["K"], case["fmt"], dev)
        s["x"] = _rows(gen, case["T"], case["K"], dev)
        n = case["N"] // 2 if case["swiglu"] else case["N"]
        s["add"] = torch.randn((case["T"], n), generator=gen, device=dev) if case["add"] else None
    elif case["op"] == "layer":
        s["w13"] = _weights(gen, case["E"], 2 * case["F"], case["H"], case["fmt"], dev)
        s["w2"] = _weights(gen, case["E"], case["H"], case["F"], case["fmt"], dev)
        s["x"] = _rows(gen, case["T"], case["H"], dev)
        s["logits"] = torch.randn((case["T"], case["E"]), generator=gen, device=dev)
    else:
        T, H, k = case["T"], case["H"], case["k"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        s["resid"] = (4.0 * _rows(gen, T, H, dev).float()).to(dt)
        if case["rows"]:
            s["y"] = torch.randn((T * k, H), generator=gen, device=dev)
            s["slot_to_row"] = torch.randperm(T * k, generator=gen, device=dev).to(torch.int32)
            s["topk_w"] = torch.softmax(torch.randn((T, k), generator=gen, device=dev), -1)
        else:
            s["y"] = _rows(gen, T, H, dev)
            s["slot_to_row"] = s["topk_w"] = None
        weight = lambda: 1.0 + 0.1 * torch.randn((H,), generator=gen, device=dev)  # noqa: E731
        s["post_w"] = weight() if case["post"] else None
        s["pre_w"] = weight() if case["pre"] else None
        shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[case["gate"]]
        s["gate"] = None if shape is None else torch.randn(shape, generator=gen, device=dev)
    return s


# ---------------------------------------------------------------------------- the plain forms
def _dequantized(w, which):
    """float32 values [n, R, C] of the matrices `which` of w."""
    codes, scales = w["codes"][which], w["scales"][which]
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pairs = torch.stack((one.repeat(16), one.repeat_interleave(16)), -1)   # byte -> (low nibble, high nibble)
    v = torch.nn.functional.embedding(codes.int(), pairs)
    if w["fmt"] == "nvfp4":
        sc = scales.view(torch.float8_e4m3fn).float() * w["g"][which].view(-1, 1, 1)
    else:
        sc = torch.exp2(scales.float() - 127.0)
    n, R, C = codes.shape[0], w["R"], w["C"]
    return v.view(n, R, sc.shape[-1], -1).mul_(sc.unsqueeze(-1)).view(n, R, C)


def _swiglu(p):
    gate, up = p.chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_matvec(s):
    c = s["case"]
    w = _dequantized(s["w"], torch.zeros((1,), dtype=torch.long, device=s["x"].device))[0]
    out = s["x"].float() @ w.t()
    out = _swiglu(out) if c["swiglu"] else out
    out = out + s["add"] if c["add"] else out
    return out if c["f32"] else out.to(torch.bfloat16)


def _fp8_rows(x):
    """bf16 rows through FP8 with one scale for all of them."""
    amax = x.float().abs().max()
    sc = torch.where(amax == 0, torch.ones_like(amax), amax / 448.0)
    return ((x.float() / sc).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float() * sc).to(torch.bfloat16)


def _plain_layer(s):
    c = s["case"]
    T, k = c["T"], c["k"]
    kept, ids = torch.sort(s["logits"], dim=-1, descending=True, stable=True)
    p = torch.softmax(kept[:, :k].double(), -1).float()
    slots = ids[:, :k].reshape(-1)
    x = _fp8_rows(s["x"]) if c["fp8"] else s["x"]
    rows = x.float().repeat_interleave(k, 0).unsqueeze(-1)
    h = _swiglu(torch.bmm(_dequantized(s["w13"], slots), rows).squeeze(-1))
    y = torch.bmm(_dequantized(s["w2"], slots), h.unsqueeze(-1)).view(T, k, -1)
    return (y * p.unsqueeze(-1)).sum(1).to(torch.bfloat16)


def _rms(v, w):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w


def _plain_norm(s):
    c = s["case"]
    if c["rows"]:
        y = (s["y"][s["slot_to_row"].long()].view(c["T"], c["k"], -1) * s["topk_w"].unsqueeze(-1)).sum(1)
    else:
        y = s["y"].float()
    u = _rms(y, s["post_w"]) if c["post"] else y
    u = u * s["gate"] if s["gate"] is not None else u
    r = s["resid"].float() + c["scale"] * u
    out = dict(resid=r.to(s["resid"].dtype))
    if c["pre"]:
        out["next"] = _rms(r, s["pre_w"]).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------- the library's calls
def _own_weights(w):
    from nvfp4_block_scaled_moe_amd import ops
    if w["fmt"] == "nvfp4":
        return ops.TiledWeights(w["tiled_codes"], w["tiled_scales"], w["g"], w["R"], w["C"])
    return ops.MxTiledWeights(w["tiled_codes"], w["tiled_scales"], w["R"], w["C"])


def _own_run(s):
    from nvfp4_block_scaled_moe_amd import ops
    c = s["case"]
    if c["op"] == "norm":
        r, nxt = ops.moe_block_norm(s["resid"], s["y"], post_w=s["post_w"], gate=s["gate"], scale=c["scale"],
                                    pre_w=s["pre_w"], eps=EPS, slot_to_row=s["slot_to_row"], topk_w=s["topk_w"])
        return dict(resid=r, next=nxt) if c["pre"] else dict(resid=r)
    if c["op"] == "matvec":
        dt = torch.float32 if c["f32"] else torch.bfloat16
        call = ops.nvfp4_matvec if c["fmt"] == "nvfp4" else ops.mxfp4_matvec
        return call(s["x"], _own_weights(s["w"]), ops.EPI_SWIGLU if c["swiglu"] else ops.EPI_NONE, add=s["add"],
                    out_dtype=dt)
    w13, w2 = _own_weights(s["w13"]), _own_weights(s["w2"])
    if c["fmt"] == "nvfp4":
        return ops.moe_layer_few_nvfp4(s["x"], s["logits"], c["k"], w13, w2, fp8_acts=c["fp8"])
    return ops.moe_layer_few_mxfp4(s["x"], s["logits"], c["k"], w13, w2)


def run(state):
    if own:
        return _own_run(state)
    return {"matvec": _plain_matvec, "layer": _plain_layer, "norm": _plain_norm}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- work and exact values
def work(case):
    if case["op"] == "norm":
        T, H, k = case["T"], case["H"], case["k"]
        r = 4 if case["f32"] else 2
        gate = {"none": 0, "channel": 4 * H, "token": 4 * T, "full": 4 * T * H}[case["gate"]]
        y = T * k * (4 * H + 8) if case["rows"] else 2 * T * H
        nbytes = y + gate + 2 * r * T * H + 4 * H * (case["post"] + case["pre"]) + 2 * T * H * case["pre"]
        return dict(bytes=nbytes, flops=T * H * (2 * k + 4 * case["post"] + 3 + 4 * case["pre"]))
    weight = 9 / 16 if case["fmt"] == "nvfp4" else 17 / 32
    if case["op"] == "matvec":
        out = 4 if case["f32"] else 2
        T, N, K = case["T"], case["N"], case["K"]
        n = N // 2 if case["swiglu"] else N
        return dict(bytes=N * K * weight + 2 * T * K + T * n * (out + 4 * case["add"]), flops=2 * T * N * K)
    T, E, k, H, F = case["T"], case["E"], case["k"], case["H"], case["F"]
    active = E * (1.0 - (1.0 - k / E) ** T)   # expected number of experts that some token is sent to
    return dict(bytes=active * 3 * F * H * weight + T * (2 * H + 4 * E + 2 * H), flops=2 * T * k * 3 * F * H)


def _exact_matrix(w, e):
    """float64 [R, C] of matrix e, from the bits: sign, two exponent bits and one mantissa bit a code."""
    b = w["codes"][e]
    q = torch.stack((b & 15, b >> 4), -1).view(w["R"], w["C"])
    exponent, mantissa = ((q >> 1) & 3).double(), (q & 1).double()
    mag = torch.where(exponent == 0, 0.5 * mantissa, torch.ldexp(1.0 + 0.5 * mantissa, exponent - 1.0))
    v = torch.where(q >= 8, -mag, mag)
    sb = w["scales"][e]
    if w["fmt"] == "nvfp4":
        se, sm = (sb >> 3).double(), (sb & 7).double()
        sc = torch.where(se == 0, sm * 2.0 ** -9, torch.ldexp(1.0 + sm / 8.0, se - 7.0)) * w["g"][e].double()
        return v * sc.repeat_interleave(16, -1)
    return v * torch.ldexp(torch.ones((), dtype=torch.float64, device=b.device), sb.double() - 127.0).repeat_interleave(32, -1)


def _exact_gated(p):
    half = p.shape[-1] // 2
    return p[..., :half] * torch.sigmoid(p[..., :half]) * p[..., half:]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        out = s["x"].double() @ _exact_matrix(s["w"], 0).t()
        out = _exact_gated(out) if case["swiglu"] else out
        return out + s["add"].double() if case["add"] else out
    if case["op"] == "layer":
        x = (_fp8_rows(s["x"]) if case["fp8"] else s["x"]).double()
        lg = s["logits"].double().cpu()
        out = torch.zeros_like(x)
        members = {}
        for t in range(case["T"]):
            order = sorted(range(case["E"]), key=lambda e: (-float(lg[t, e]), e))[: case["k"]]
            z = [math.exp(float(lg[t, e]) - float(lg[t, order[0]])) for e in order]
            for e, v in zip(order, z):
                members.setdefault(e, []).append((t, v / math.fsum(z)))
        for e, who in members.items():
            rows = torch.tensor([t for t, _ in who], device=x.device)
            p = torch.tensor([v for _, v in who], dtype=torch.float64, device=x.device)
            h = _exact_gated(x[rows] @ _exact_matrix(s["w13"], e).t())
            out[rows] += p.unsqueeze(-1) * (h @ _exact_matrix(s["w2"], e).t())
        return out
    if case["rows"]:
        y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device=s["y"].device)
        where = s["slot_to_row"].long().view(case["T"], case["k"])
        for j in range(case["k"]):
            y += s["topk_w"][:, j:j + 1].double() * s["y"][where[:, j]].double()
    else:
        y = s["y"].double()
    if case["post"]:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["H"] + EPS) * s["post_w"].double()
    if s["gate"] is not None:
        y = y * s["gate"].double()
    r = s["resid"].double() + case["scale"] * y
    out = dict(resid=r)
    if case["pre"]:
        out["next"] = r / torch.sqrt((r * r).sum(-1, keepdim=True) / case["H"] + EPS) * s["pre_w"].double()
    return out
