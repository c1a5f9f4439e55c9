"""Cases of the paged cache's calls and their float64 references, for the GPU tests."""
import math

import torch

from nvfp4_block_scaled_moe_amd import ops

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
HALF = {torch.float32: 2.0 ** -24, BF: 2.0 ** -8}   # half a step, relative to the value


def frequencies(rot, base=10000.0):
    return base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)


def rotated(x, positions, freqs, start=0, interleaved=False, magnitude=1.0, sign=1.0):
    """float64 of x [T, H, D] (CPU) turned, and for each element the sum of magnitudes that its pair brings."""
    x = x.double().clone()
    r = 2 * freqs.shape[0]
    part = x[..., start:start + r].unflatten(-1, (r // 2, 2) if interleaved else (2, r // 2))
    axis = -1 if interleaved else -2
    u, w = part.select(axis, 0), part.select(axis, 1)
    a = positions.double()[:, None, None] * freqs * sign
    c, s = torch.cos(a), torch.sin(a)
    y = torch.stack((u * c - w * s, w * c + u * s), axis).flatten(-2) * magnitude
    both = torch.stack((u.abs() + w.abs(),) * 2, axis).flatten(-2) * abs(magnitude)
    size = torch.zeros_like(x)
    x[..., start:start + r] = y
    size[..., start:start + r] = both
    return x, size


class Case:
    """Sequences with ``new[b]`` new tokens after ``ctx[b]`` others, their pages dealt at random. Pages and places that
    hold no token are NaN; what the page table holds behind a sequence's pages is -1 or a page too many."""

    def __init__(self, new, ctx, Hq, Hkv, D, page, fp8=False, seed=0, spare_rows=0, v_spread=1.0, dev="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.new, self.ctx, self.Hq, self.Hkv, self.D, self.page, self.fp8 = new, ctx, Hq, Hkv, D, page, fp8
        B = len(new)
        total = [n + c for n, c in zip(new, ctx)]
        used = [-(-t // page) for t in total]
        pages = sum(used) + 3
        order = torch.randperm(pages, generator=g).to(torch.int32)
        cols = max(max(used), 1) + 2
        table = torch.full((B, cols), -1, dtype=torch.int32)
        table[:, -1] = pages
        at = 0
        for b in range(B):
            table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
        self.T = sum(new)
        rows = self.T + spare_rows
        k = torch.full((pages, Hkv, page, D), math.nan)
        v = torch.full((pages, Hkv, D, page), math.nan)
        self.keys, self.values = [], []
        self.k_scale = self.v_scale = None
        if fp8:
            self.k_scale, self.v_scale = 0.01 + 0.02 * torch.rand(Hkv, generator=g), 0.01 + 0.02 * torch.rand(Hkv, generator=g)
        cast = (lambda x, s: (x / s.view(-1, 1)).clamp(-448, 448).to(F8)) if fp8 else (lambda x, s: x.to(BF))
        for b in range(B):
            kb = cast(torch.randn((total[b], Hkv, D), generator=g), self.k_scale)
            vb = cast(v_spread * torch.randn((total[b], Hkv, D), generator=g), self.v_scale)
            p = torch.arange(total[b])
            pg = table[b].long()[p // page]
            k[pg, :, p % page] = kb.float()
            v[pg, :, :, p % page] = vb.float()
            self.keys.append(kb.double() * (self.k_scale.double().view(-1, 1) if fp8 else 1.0))
            self.values.append(vb.double() * (self.v_scale.double().view(-1, 1) if fp8 else 1.0))
        self.table, self.total, self.pages = table, total, pages
        self.q = torch.randn((rows, Hq, D), generator=g).to(BF)
        dt = F8 if fp8 else BF
        dv = lambda t: None if t is None else t.to(dev)  # noqa: E731
        self.cache = ops.KVCache(dv(k.to(dt)), dv(v.to(dt)), dv(self.k_scale), dv(self.v_scale))
        starts = [sum(new[:b]) for b in range(B + 1)]
        self.starts = starts
        self.batch = ops.CacheBatch(dv(table), dv(torch.tensor(total, dtype=torch.int32)), dv(torch.tensor(starts, dtype=torch.int32)))

    def rows(self):
        """Rows (token, head of the group) of a sequence, on average."""
        return self.q.shape[0] * (self.Hq // self.Hkv) / len(self.new)

    def attention(self, scale=None, window=0):
        """float64 outputs of the new tokens' rows, and how far each may be off."""
        scale = self.D ** -0.5 if scale is None else scale
        G = self.Hq // self.Hkv
        out = torch.zeros((self.T, self.Hq, self.D), dtype=torch.float64)
        tol = torch.zeros_like(out)
        weight_step = 2.0 ** -15 if self.rows() <= 16 else 2.0 ** -8
        for b, (n, c) in enumerate(zip(self.new, self.ctx)):
            if n == 0 or self.total[b] == 0:
                continue
            q = self.q[self.starts[b]:self.starts[b] + n].double()
            far = (c + torch.arange(n))[:, None] - torch.arange(n + c)
            sees = (far >= 0) & ((far < window) if window else True)
            for h in range(self.Hq):
                k, v = self.keys[b][:, h // G], self.values[b][:, h // G]
                # (values that no new token sees may be NaN)
                v = torch.where(sees.any(0)[:, None], v, torch.zeros(()).double())
                s = torch.where(sees, (q[:, h] @ k.t()) * scale, -math.inf)
                p = torch.softmax(s, -1)
                o = p @ v
                a = p @ v.abs()                                       # what roundings of the weights scale with
                d = torch.where(sees, (q[:, h].abs() @ k.abs().t()) * scale, 0.0).amax(-1, keepdim=True)
                # a score is off by its float32 sum of D products, a weight by twice that (its own and the sum's),
                # the exponential and the sums over the keys
                rel = 2.0 * d * (self.D + 8) * 2.0 ** -24 + (n + c + 64) * 2.0 ** -23 + weight_step
                rows = slice(self.starts[b], self.starts[b] + n)
                out[rows, h] = o
                tol[rows, h] = HALF[BF] * (o.abs() + rel * a) + rel * a
        return out, tol


def check(got, want, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - tol
    i = int(over.argmax())
    assert over.flatten()[i] <= 0, f"{what}: {got.flatten()[i]} for {want.flatten()[i]}, allowed {tol.flatten()[i]} at {i}"
