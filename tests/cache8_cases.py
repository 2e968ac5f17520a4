"""Inputs and 64-bit references for the 8-bit paged cache's operators (test
infrastructure), on top of cache_cases.py.

Tolerances count roundings, with the terms of cache_cases.py and these:
 - q goes into the product in e4m3 pieces under one power of two per row: what
   is left over is at most half of e4m3's smallest subnormal, 2^-10, where the
   row's largest element is over 224, so 2^-17.8 of that element.  A score is
   off by that times scale * s_k * sum |k8| more;
 - a weight times its scale of v goes into the product with v as an fp16 number
   in e5m2 pieces: half a step of fp16 and what the third piece leaves, 2^-11
   each, and nothing below half of e5m2's least number, 2^-17, where the row's
   largest is 2^7 at least (2^7 when its maximum is taken, 2^15 before it is
   taken again): 2^-24 of that one;
 - an element of the cache is off by half a step of e4m3, 2^-4 of it, or half of
   the smallest subnormal, 2^-10 times its scale.
"""
import math

import numpy as np
import torch

from cache_cases import E32, CacheCase, half_step, half_subnormal

E4M3 = torch.float8_e4m3fn
Q_LEFT = 2.0 ** -17.8
WEIGHT = 2.0 ** -10
WEIGHT_FLOOR = 2.0 ** -24


def least_scale(top):
    """The least power of two from 2^-100 to 2^100 with top <= 448 times it (top in 64 bits)."""
    top = torch.as_tensor(top, dtype=torch.float64)
    t = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448))
    t = torch.where(top <= 448 * torch.exp2(t - 1), t - 1, t)  # log2's own rounding
    t = torch.where(top > 448 * torch.exp2(t), t + 1, t)
    return torch.exp2(t.clamp(-100, 100))


def rounded(x):
    """64-bit values on e4m3's grid: to nearest, ties to even, past 448 to 448."""
    m, e = torch.frexp(x.abs().clamp(max=448.0))
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.copysign(torch.round(x.abs().clamp(max=448.0) / step) * step, x).clamp(-448, 448)


def bits(x):
    return x.view(torch.uint8)


class Cache8Case(CacheCase):
    """A CacheCase whose cache is held in 8 bits: k, v in e4m3, ks, vs their scales.  spread: how far blocks' scales
    lie apart (powers of two)."""

    def __init__(self, ctx, new, poison=False, spread=1, odd_scales=False, seed=0, strided=False, order="nhd", **kw):
        super().__init__(ctx, new, seed=seed, strided=strided, order=order, **kw)
        g = torch.Generator().manual_seed(seed + 1)
        dev = self.device
        layers, blocks = self.k.shape[0], self.k.shape[1]
        made = []
        for x in (self.k, self.v):
            size = torch.exp2(spread * torch.randn((layers, blocks, self.kv_heads), generator=g)).to(dev)
            y = x.double() * size[:, :, None, :, None]
            scale = least_scale(y.abs().amax(dim=(2, 4))).float()
            if odd_scales:  # as another program may have chosen them
                scale = scale * (0.6 + torch.rand(scale.shape, generator=g).to(dev))
            y = (y / scale[:, :, None, :, None]).float().clamp(-448, 448).to(E4M3)
            if strided:  # K and V of a block side by side, rows padded
                made.append(y)
            elif order == "hnd":
                made.append(bits(y).transpose(2, 3).contiguous().view(E4M3).transpose(2, 3))
            else:
                made.append(bits(y).contiguous().view(E4M3))
            made.append(scale)
        k, self.ks, v, self.vs = made
        if strided:
            shape = (layers, blocks, 2, self.kv_heads, self.block, self.dim + 16) if order == "hnd" else \
                (layers, blocks, 2, self.block, self.kv_heads, self.dim + 16)
            both = torch.zeros(shape, dtype=torch.uint8, device=dev)
            a, b = (both[:, :, i, ..., :self.dim] for i in range(2))
            if order == "hnd":
                a, b = a.transpose(2, 3), b.transpose(2, 3)
            a.copy_(bits(k))
            b.copy_(bits(v))
            k, v = a.view(E4M3), b.view(E4M3)
        self.k, self.v = k, v
        if strided:  # scales of K and V side by side
            s = torch.stack([self.ks, self.vs], dim=-1)
            self.ks, self.vs = s[..., 0], s[..., 1]
        if poison:
            unused = torch.ones(blocks, self.block, dtype=torch.bool)
            for i, n in enumerate(self.lengths):
                for p in range(n):
                    unused[self.tables[i, p // self.block], p % self.block] = False
            bad = unused[None, :, :, None, None].to(dev)
            bits(self.k).masked_fill_(bad, 0x7f)
            bits(self.v).masked_fill_(bad, 0xff)
            free = unused.all(dim=1)
            self.ks[:, free] = float("nan")
            self.vs[:, free] = float("inf")

    def cache(self, smcsd):
        return smcsd.make_cache8(self.k, self.v, self.ks, self.vs)

    def value(self, which, layer, block, token):
        """Elements [kv_heads, dim] in 64 bits."""
        x, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        return x[layer, block, token].double() * s[layer, block].double()[:, None]

    def gather(self, s, head):
        n = self.lengths[s]
        blocks = self.tables[s, :-(-n // self.block)].long()
        return ((x[self.layer][blocks][:, :, head].double() * y[self.layer, blocks, head].double()[:, None, None])
                .reshape(-1, self.dim)[:n] for x, y in ((self.k, self.ks), (self.v, self.vs)))

    def reference(self):
        """out, lse in 64 bits, and the elementwise bounds of their errors."""
        dev = self.device
        out = torch.zeros((self.rows, self.heads, self.dim), dtype=torch.float64, device=dev)
        lse = torch.full((self.rows, self.heads), -math.inf, dtype=torch.float64, device=dev)
        tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        rep, u, d = self.heads // self.kv_heads, half_step(self.dtype), half_subnormal(self.dtype)
        for s in range(len(self.ctx)):
            m = self.new[s]
            if not m:
                continue
            r0 = int(self.starts[s])
            sees = torch.zeros((m, self.lengths[s]), dtype=torch.bool)
            sees[:, :self.ctx[s]] = True
            for i in range(m):
                for j in (range(i + 1) if self.seen is None else self.seen[r0 + i]):
                    sees[i, self.ctx[s] + j] = True
            sees = sees.repeat_interleave(rep, 0).to(dev)
            some = sees.any(dim=1)
            n = self.lengths[s]
            blocks = self.tables[s, :-(-n // self.block)].long()
            for g in range(self.kv_heads):
                k, v = (torch.nan_to_num(x) for x in self.gather(s, g))
                sv = self.vs[self.layer, blocks, g].double().repeat_interleave(self.block)[:n]
                hs = slice(g * rep, (g + 1) * rep)
                x = self.q[r0:r0 + m, hs].double().reshape(-1, self.dim)
                z = (x @ k.T * self.scale).masked_fill(~sees, -math.inf)
                a = self.scale * ((self.dim + 2) * E32 * (x.abs() @ k.abs().T) +
                                  Q_LEFT * x.abs().amax(1, keepdim=True) * k.abs().sum(1)).masked_fill(~sees, 0).amax(1)
                top = torch.where(some, z.amax(1), 0.0)[:, None]
                w = torch.exp(z - top)
                total = w.sum(1, keepdim=True)
                p = torch.where(some[:, None], w / total, 0.0)
                o, mag = p @ v, p @ v.abs()
                l = torch.where(some, top[:, 0] + total[:, 0].log(), -math.inf)
                rel = 2 * a + 2.0 ** -19 + 2 * n * E32
                # a weight's floor counts against the largest weight times scale
                floor = WEIGHT_FLOOR * (p * sv).amax(1, keepdim=True) * (sees.double() @ (v.abs() / sv[:, None]))
                t = (rel + WEIGHT)[:, None] * 1.01 * mag + u * o.abs() * 1.01 + d + floor
                out[r0:r0 + m, hs] = o.view(m, rep, -1)
                tol[r0:r0 + m, hs] = t.view(m, rep, -1)
                lse[r0:r0 + m, hs] = l.view(m, rep)
                tol_lse[r0:r0 + m, hs] = (rel + 4 * E32 * (1 + torch.where(some, l, 0.0).abs())).view(m, rep)
        return out, lse, tol, tol_lse


def checked_scale(got, amax, off, old=None):
    """Whether scales [heads] are those of new tokens whose largest element is amax [heads], off by at most `off`;
    old: the block's scale where it holds earlier tokens."""
    lo, hi = (least_scale((amax + s * off).clamp(min=0)).to(got.device) for s in (-1, 1))
    if old is not None:
        lo, hi = torch.maximum(lo, old), torch.maximum(hi, old)
    return bool(((got >= lo) & (got <= hi)).all()) and bool(((got == lo) | (got == hi)).all())


def np_path(rng, m, most):
    return sorted(rng.choice(m, int(rng.integers(0, min(m, most) + 1)), replace=False).tolist()) if m else []


def compacted(c, path):
    """Cache and scales after kv_compact_tokens8, by loops: {name: (values in e4m3's grid, scales)} in 64 bits."""
    out = {}
    block = c.block
    for name, x, s in (("k", c.k, c.ks), ("v", c.v, c.vs)):
        data, scale = x.double().clone(), s.double().clone()
        before, old = data.clone(), scale.clone()
        for q, p in enumerate(path):
            moves, last = [], -1
            for i, j in enumerate(p):
                if not 0 <= j < c.new[q]:
                    continue
                if j > last and j > i:
                    moves.append((c.ctx[q] + j, c.ctx[q] + i))
                last = max(last, j)
            for slot in sorted({b // block for _, b in moves}):
                d = int(c.tables[q, slot])
                into = [m for m in moves if m[1] // block == slot]
                new = old[:, d].clone()
                for a, _ in into:
                    new = torch.maximum(new, old[:, int(c.tables[q, a // block])])
                scale[:, d] = new
                f = (old[:, d] / new)[:, None, :, None]
                held = min(block, c.lengths[q] - slot * block)
                again = rounded((before[:, d, :held] * f).float().double())
                data[:, d, :held] = torch.where(f == 1, before[:, d, :held], again)
                for a, b in into:
                    src = int(c.tables[q, a // block])
                    g = (old[:, src] / new)[..., None]
                    x8 = before[:, src, a % block]
                    data[:, d, b % block] = torch.where(g == 1, x8, rounded((x8 * g).float().double()))
        out[name] = (data, scale)
    return out
