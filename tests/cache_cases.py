"""Inputs and 64-bit references for the paged cache's operators (test
infrastructure): plain loops over sequences, rows and heads.

Tolerances count roundings.  With u = finfo(dtype).eps / 2 of the cache's
dtype and e = 2^-24 of fp32, a score z = scale * <q, k> is off by at most
a = (D + 2) e scale sum |q k|, its weight by a relative 2a + 2^-20 (the exp2
of a scaled difference, in fp32) plus u (the weight's rounding for the product
with v), sums over n tokens by n e, the result by u once more.  Below the
smallest normal value the rounding is off by half of the smallest subnormal
instead (d): the result's, and each fp16 weight's beside a largest of 1.
"""
import math

import numpy as np
import torch

E32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def half_subnormal(dtype):
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


class CacheCase:
    """Sequences with `ctx` committed and `new` new tokens in a shuffled pool."""

    def __init__(self, ctx, new, heads=8, kv_heads=2, dim=128, block=16, dtype=torch.bfloat16,
                 order="nhd", layers=1, layer=0, group=1, shared=0, mask="chain", seed=0,
                 device="cuda", poison=False, strided=False, max_new=None, sigma=1.0, slots=0):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.new, self.lengths = ctx, new, [a + b for a, b in zip(ctx, new)]
        self.heads, self.kv_heads, self.dim, self.block = heads, kv_heads, dim, block
        self.dtype, self.layer, self.group, self.device = dtype, layer, group, device
        self.max_new = max(1, max(new)) if max_new is None else max_new
        S = len(ctx)
        need = [-(-n // block) for n in self.lengths]
        common = shared // block
        T = max(max(need) + 1, 2, slots)
        count = sum(need) + 3
        order_ids = torch.randperm(count, generator=g).tolist()
        tables = torch.full((S, T), -1, dtype=torch.int32)
        used = 0
        for i, n in enumerate(need):
            first = i - i % group
            skip = common if i != first else 0
            tables[i, :skip] = tables[first, :skip]
            for t in range(skip, n):
                tables[i, t] = order_ids[used]
                used += 1
        self.blocks = count
        shape = ((layers, count, kv_heads, block, dim) if order == "hnd"
                 else (layers, count, block, kv_heads, dim))
        if strided:  # K and V of a block side by side in one array, rows padded
            both = torch.randn((*shape[:2], 2, *shape[2:4], dim + 8), generator=g) * sigma
            both = both.to(dtype).to(device)
            k, v = both[:, :, 0, ..., :dim], both[:, :, 1, ..., :dim]
        else:
            k, v = ((torch.randn(shape, generator=g) * sigma).to(dtype).to(device) for _ in range(2))
        if order == "hnd":
            k, v = k.transpose(2, 3), v.transpose(2, 3)
        self.k, self.v = k, v
        if poison:  # slots that hold no token
            unused = torch.ones(count, block, dtype=torch.bool)
            for i, n in enumerate(self.lengths):
                for p in range(n):
                    unused[tables[i, p // block], p % block] = False
            bad = unused[None, :, :, None, None].to(device)
            k.masked_fill_(bad, float("nan"))
            v.masked_fill_(bad, float("inf"))
        starts = np.concatenate([[0], np.cumsum(new)])
        self.rows = int(starts[-1])
        self.starts = starts
        self.tables = tables.to(device)
        self.seq_len = torch.tensor(self.lengths, dtype=torch.int32, device=device)
        self.row_start = torch.tensor(starts, dtype=torch.int32, device=device)
        row = heads * dim + 16 if strided else heads * dim
        self.q = torch.randn((self.rows, row), generator=g).to(dtype).to(device)[:, :heads * dim]
        self.q = self.q.unflatten(1, (heads, dim))
        self.seen = None if mask == "chain" else self._trees(g, mask)
        self.mask = None if self.seen is None else self._packed()
        self.scale = dim ** -0.5

    def _trees(self, g, mask):
        """Per row, the list of new tokens that it sees."""
        out = []
        for m in self.new:
            rows = []
            for i in range(m):
                if mask == "none" or (mask == "holes" and i % 3 == 2):
                    rows.append([])
                    continue
                parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
                rows.append((rows[parent] if parent >= 0 else []) + [i])
            out += rows
        return out

    def _packed(self):
        words = -(-self.max_new // 32)
        a = np.zeros((self.rows, words), dtype=np.uint32)
        for r, seen in enumerate(self.seen):
            for j in seen:
                a[r, j // 32] |= np.uint32(1 << (j % 32))
        return torch.from_numpy(a.view(np.int32)).to(self.device)

    def cache(self, smcsd):
        return smcsd.make_cache(self.k, self.v)

    def batch(self, smcsd, uniform=False):
        if uniform:
            return smcsd.make_batch(self.tables, self.seq_len, self.max_new, group=self.group)
        return smcsd.make_batch(self.tables, self.seq_len, self.max_new, row_start=self.row_start,
                                rows=self.rows, group=self.group)

    def gather(self, s, head):
        """Keys and values [len, dim] of sequence s, in 64 bits."""
        n = self.lengths[s]
        blocks = self.tables[s, :-(-n // self.block)].long()
        return (c[self.layer, blocks, :, head].double().reshape(-1, self.dim)[:n]
                for c in (self.k, self.v))

    def reference(self):
        """out, lse in 64 bits, and the elementwise bounds of their errors."""
        dev = self.device
        out = torch.zeros((self.rows, self.heads, self.dim), dtype=torch.float64, device=dev)
        lse = torch.full((self.rows, self.heads), -math.inf, dtype=torch.float64, device=dev)
        tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        rep, u, d = self.heads // self.kv_heads, half_step(self.dtype), half_subnormal(self.dtype)
        for s in range(len(self.ctx)):
            for g in range(self.kv_heads):
                k, v = self.gather(s, g)
                for i in range(self.new[s]):
                    r = int(self.starts[s]) + i
                    seen = range(i + 1) if self.seen is None else self.seen[r]
                    cols = torch.tensor([*range(self.ctx[s]), *(self.ctx[s] + j for j in seen)],
                                        dtype=torch.long, device=dev)
                    if not len(cols):
                        continue
                    hs = slice(g * rep, (g + 1) * rep)
                    x, kk, vv = self.q[r, hs].double(), k[cols], v[cols]
                    z = x @ kk.T * self.scale
                    a = (self.dim + 2) * E32 * self.scale * (x.abs() @ kk.abs().T).amax(-1)
                    top = z.amax(-1, keepdim=True)
                    w = torch.exp(z - top)
                    total = w.sum(-1, keepdim=True)
                    p = w / total
                    out[r, hs] = p @ vv
                    lse[r, hs] = (top + total.log()).squeeze(-1)
                    rel = 2 * a + 2.0 ** -20 + 2 * len(cols) * E32
                    tol[r, hs] = ((rel + u)[:, None] * 1.01 * (p @ vv.abs())
                                  + u * out[r, hs].abs() * 1.01 + d
                                  + d / total * vv.abs().sum(0))
                    tol_lse[r, hs] = rel + 4 * E32 * (1 + lse[r, hs].abs())
        return out, lse, tol, tol_lse


def rope_table(max_pos, rot, device="cuda", base=10000.0):
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    angle = torch.outer(torch.arange(max_pos, dtype=torch.float64), freq)
    return torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32).to(device)


def qk_reference(x, weight, table, positions, rot, interleaved, eps, offset):
    """Norm and rotation of x [rows, heads, dim] in 64 bits, and the bound of
    an fp32 evaluation rounded once to x's dtype."""
    y = x.double()
    dim = y.shape[-1]
    mag = y.abs()
    if weight is not None:
        r = torch.rsqrt(y.square().mean(-1, keepdim=True) + eps)
        w = weight.double() + offset
        y, mag = y * r * w, mag * r * w.abs()
    half = rot // 2
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    t = table.double()[positions.long()][:, None]
    c, s = t[..., :half], t[..., half:]
    out, bound = y.clone(), mag.clone()
    a, b = y[..., first], y[..., second]
    out[..., first], out[..., second] = a * c - b * s, a * s + b * c
    ma, mb = mag[..., first], mag[..., second]
    bound[..., first] = ma * c.abs() + mb * s.abs()
    bound[..., second] = ma * s.abs() + mb * c.abs()
    # the mean's sum, rsqrt and the products: dim / 2 + 10 roundings of fp32
    tol = (dim / 2 + 10) * E32 * bound + half_step(x.dtype) * out.abs() * 1.01
    return out, tol + half_subnormal(x.dtype)
