"""Workloads of the operators on a paged key/value cache held in 8 bits, with their plain forms.

Three operators around one cache [layers, blocks, block_size, kv_heads, head_dim] of 8-bit floating-point numbers (e4m3)
and one scale for each layer, block and key head, [layers, blocks, kv_heads]: an element is its number times its scale.

  attend   attention of the new (drafted) tokens of each sequence over its blocks, under a tree mask
  append   per-head RMS norms of queries and keys with the position rotation; keys and values quantised into the cache,
           each block under the least power of two that holds its new tokens (and what it held before)
  compact  the accepted path of a drafted tree moved to the front of the new tokens, in every layer, values that meet
           another block's scale quantised again

A sequence's new tokens are the last ones that it holds: seq_len counts them.  Plain forms: elementary torch
operations in 32 bits, rounded once at the end.  Outputs in 8 bits are float8 tensors, with their blocks' scales beside
them.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
LEAST = -100  # exponent of the least scale


# ---- cases -----------------------------------------------------------------

def _attend(name, dtype, prompts, group, new, heads, kv_heads, dim, block, ctx, ragged, shared, mask, order="nhd"):
    """prompts * group sequences of up to ctx committed tokens; the first `shared` tokens of a prompt's sequences are
    the same blocks.  ragged: share of the length by which sequences differ (0: none)."""
    return {"name": name, "op": "attend", "dtype": dtype, "prompts": prompts, "group": group, "new": new,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "block": block, "ctx": ctx, "ragged": ragged,
            "shared": shared, "mask": mask, "order": order}


def _append(name, dtype, seqs, new, heads, kv_heads, dim, rot, interleaved, norm, block, ctx, ragged, order="nhd"):
    return {"name": name, "op": "append", "dtype": dtype, "seqs": seqs, "new": new, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rot": rot, "interleaved": interleaved, "norm": norm, "block": block,
            "ctx": ctx, "ragged": ragged, "order": order}


def _compact(name, seqs, new, path, layers, kv_heads, dim, block, ctx, order="nhd"):
    return {"name": name, "op": "compact", "dtype": "bf16", "seqs": seqs, "new": new, "path": path, "layers": layers,
            "kv_heads": kv_heads, "dim": dim, "block": block, "ctx": ctx, "order": order}


def listed():
    return [
        # one sequence decodes one token behind the single-prompt workload's 512-token prefix: latency
        _attend("attend8_one_token", "bf16", 1, 1, 1, 32, 8, 128, 16, 513, 0.0, 0, "chain"),
        # the serving workload: 16 prompts x 16 particles, K = 4, prefix 2048 shared, tails of up to 640 tokens
        _attend("attend8_serving_particles", "bf16", 16, 16, 5, 32, 8, 128, 16, 2688, 0.2, 2048, "chain"),
        # drafted trees of 64 tokens verified for 16 requests: many rows for each key
        _attend("attend8_tree_64", "bf16", 16, 1, 64, 32, 8, 128, 64, 4096, 0.3, 0, "tree"),
        # one request with a long document, a small tree: the split over the length
        _attend("attend8_long_context", "bf16", 1, 1, 8, 64, 8, 128, 64, 131072, 0.0, 0, "tree"),
        # odd sizes: fp16, as many key heads as heads, 64 wide, blocks of 24 tokens in head-major order, some
        # sequences with no committed token, rows of padding that see nothing
        _attend("attend8_ragged_f16", "f16", 5, 1, 7, 12, 12, 64, 24, 777, 1.0, 0, "tree_padded", "hnd"),
        # a full batch with trees of 16 tokens and contexts of up to 8192: the largest
        _attend("attend8_batch_8k", "bf16", 64, 1, 16, 32, 8, 128, 32, 8192, 0.5, 0, "tree"),
        # one token of one sequence on its way into the attention: latency
        _append("append8_one_token", "bf16", 1, 1, 32, 8, 128, 128, False, True, 16, 513, 0.0),
        # the serving workload's 1280 rows, behind tails that end inside a block
        _append("append8_serving_rows", "bf16", 256, 5, 32, 8, 128, 128, False, True, 16, 200, 0.2),
        # a prompt's rows, in fp16, 96 wide heads rotated in part, neighbouring pairs
        _append("append8_prompt_rows", "f16", 3, 5000, 40, 8, 96, 64, True, True, 16, 0, 0.3),
        # a short path of one request's tree in a few layers: latency
        _compact("compact8_one_request", 1, 8, 3, 4, 8, 128, 16, 150),
        # accepted paths of the trees of 64 requests, all layers
        _compact("compact8_tree_paths", 64, 64, 9, 32, 8, 128, 16, 150),
        # odd sizes: long paths over small blocks, head-major
        _compact("compact8_odd_paths", 23, 100, 37, 7, 5, 80, 20, 91, "hnd"),
    ]


def _cost(c):
    """Bytes that the plain form handles, to keep drawn cases below the largest listed one."""
    if c["op"] == "attend":
        n = c["prompts"] * c["group"]
        length = c["ctx"] + c["new"]
        return n * length * (12.0 * c["kv_heads"] * c["dim"] + c["heads"] * c["new"] * 8)
    if c["op"] == "append":
        return c["seqs"] * (c["new"] + c["ctx"]) * (c["heads"] + 2 * c["kv_heads"]) * c["dim"] * 8.0
    blocks = c["seqs"] * (-(-(c["ctx"] + c["new"]) // c["block"]) + 1)
    return 4.0 * c["layers"] * c["block"] * c["kv_heads"] * c["dim"] * blocks


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {"attend": 5.0e9, "append": 5.0e8, "compact": 4.0e9}
    while True:
        op = rng.choice(["attend", "attend", "attend", "append", "append", "compact"])
        kv, rep = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 8])
        block = rng.choice([8, 16, 16, 32, 48, 64, 128, 20])
        order = rng.choice(["nhd", "hnd"])
        if op == "attend":
            group = rng.choice([1, 1, 1, 2, 5, 8, 16])
            ctx = _log(rng, 1, 60000)
            c = _attend("", rng.choice(["bf16", "bf16", "f16"]), _log(rng, 1, 64), group, _log(rng, 1, 128), kv * rep,
                        kv, rng.choice([64, 128, 128, 80, 96]), block, ctx, rng.choice([0.0, 0.3, 1.0]),
                        int(ctx * rng.random()) if group > 1 else 0, rng.choice(["chain", "tree", "tree_padded"]), order)
        elif op == "append":
            dim = rng.choice([64, 128, 96, 80])
            c = _append("", rng.choice(["bf16", "f16", "f32"]), _log(rng, 1, 300), _log(rng, 1, 2000), kv * rep, kv, dim,
                        rng.choice([dim, dim // 2]), rng.random() < 0.5, rng.random() < 0.8, block, _log(rng, 1, 2000),
                        rng.choice([0.0, 0.5]), order)
        else:
            new = _log(rng, 2, 100)
            c = _compact("", _log(rng, 1, 64), new, rng.randint(1, min(40, new)), rng.choice([1, 7, 24, 32]), kv,
                         rng.choice([64, 128, 80]), block, _log(rng, 1, 300), order)
        del c["name"]
        if _cost(c) <= top[op]:
            return c


# ---- lengths: from the case alone ------------------------------------------

def _lengths(c):
    """(committed, new) tokens of each sequence."""
    rng = random.Random("%s %s %s %s" % (c["op"], c["ctx"], c["new"], c.get("prompts", c.get("seqs"))))
    n = c["prompts"] * c["group"] if c["op"] == "attend" else c["seqs"]
    ragged = c.get("ragged", 0.3)
    ctx = [c["ctx"] - int(ragged * c["ctx"] * rng.random()) for _ in range(n)]
    new = [c["new"] - int(0.5 * ragged * c["new"] * rng.random()) for _ in range(n)]
    if c["op"] == "attend":
        ctx = [max(v, c["shared"]) for v in ctx]
    if ragged == 1.0:  # some sequences have committed nothing yet
        ctx = [0 if i % 5 == 3 else v for i, v in enumerate(ctx)] if not c["shared"] else ctx
    if c["op"] == "append" and ragged == 0.0 or c.get("mask") == "chain":
        new = [c["new"]] * n  # particles always draft the same number
    ctx[0], new[0] = c["ctx"], c["new"]
    return ctx, new


def work(case):
    c = case
    bs = c["block"]
    token = 2 * c["kv_heads"] * c["dim"]  # bytes of a token's keys and values in one layer
    scales = 8 * c["kv_heads"]            # bytes of a block's scales
    ctx, new = _lengths(c)
    if c["op"] == "compact":
        # the path's tokens, the scales of the blocks that they come from and go to
        moved = sum(min(c["path"], m) for m in new)
        blocks = sum(1 + (v + min(c["path"], m) - 1) // bs - v // bs for v, m in zip(ctx, new))
        return {"bytes": c["layers"] * (2 * moved * token + 2 * blocks * scales), "flops": 0}
    s = 4 if c["dtype"] == "f32" else 2
    rows = sum(new)
    if c["op"] == "append":
        q = c["heads"] * c["dim"] * s
        blocks = sum((v + m - 1) // bs - v // bs + 1 for v, m in zip(ctx, new))
        return {"bytes": rows * (2 * q + token * s + token + 4 * c["rot"]) + blocks * scales,
                "flops": 10 * rows * (c["heads"] + 2 * c["kv_heads"]) * c["dim"]}
    common = c["shared"] // bs * bs
    kept = c["prompts"] * common + sum(v - common + m for v, m in zip(ctx, new))
    flops = sum(4 * c["heads"] * c["dim"] * m * (v + m) for v, m in zip(ctx, new))
    return {"bytes": kept * (token + scales / bs) + 2 * rows * c["heads"] * c["dim"] * s + 4 * rows * c["heads"],
            "flops": flops}


# ---- inputs ----------------------------------------------------------------

def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _least_scale(top):
    """The least power of two s, 2^LEAST at least, with top <= 448 s: 448 s = 0.875 * 2^(t + 9)."""
    m, e = torch.frexp(top.float())
    t = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.ldexp(torch.ones_like(m), torch.where(top > 0, t, LEAST).clamp(min=LEAST))


def _quantised(c, layers, blocks, g):
    """A cache's numbers [layers, blocks, block, kv_heads, dim] (a view where the memory order is head-major) and scales
    [layers, blocks, kv_heads]: heads and blocks of different magnitudes, as trained models have them."""
    kv, bs, dim = c["kv_heads"], c["block"], c["dim"]
    x = torch.randn((layers, blocks, kv, bs, dim), generator=g, device="cuda", dtype=torch.bfloat16)
    size = torch.exp(0.4 * torch.randn((layers, 1, kv), generator=g, device="cuda") +
                     0.3 * torch.randn((layers, blocks, kv), generator=g, device="cuda"))
    scale = _least_scale(x.abs().amax(dim=(3, 4)).float() * size)
    x = (x * (size / scale)[..., None, None]).clamp(-448, 448).to(E4M3)
    if c["order"] == "nhd":
        x = x.view(torch.uint8).transpose(2, 3).contiguous().view(E4M3)
    else:
        x = x.transpose(2, 3)
    return x, scale.contiguous()


def _tables(c, lengths, group, shared, g):
    """Block tables [S, T] over a shuffled pool; a group's first shared // block slots name the same blocks."""
    bs = c["block"]
    need = [-(-v // bs) for v in lengths]
    common = shared // bs
    slots = max(need) + 1
    count = sum(need) + 8
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    at = torch.full((len(lengths), slots), -1, dtype=torch.int64)
    k = 0
    for i, n in enumerate(need):
        first = i % group != 0
        skip = common if first else 0
        if first:
            at[i, :skip] = at[i - i % group, :skip]
        at[i, skip:n] = torch.arange(k, k + n - skip)
        k += n - skip
    at = at.cuda()
    return torch.where(at >= 0, order[at.clamp(min=0)], -1).to(torch.int32).contiguous(), count


def _rows(new):
    start = [0]
    for m in new:
        start.append(start[-1] + m)
    return torch.tensor(start, dtype=torch.int32, device="cuda")


def _masks(c, new, rng):
    """Packed ancestor bits [rows, words]: bit j of word j // 32 says that the row sees its sequence's new token j."""
    words = -(-c["new"] // 32)
    out = []
    for m in new:
        seen = []
        for i in range(m):
            parent = rng.randint(max(-1, i - 8), i - 1) if i else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        if c["mask"] == "tree_padded":  # the last rows of a tree that came out smaller
            seen[m - m // 4:] = [0] * (m // 4)
        out += [[(v >> 32 * w & 0xFFFFFFFF) for w in range(words)] for v in seen]
    t = torch.tensor(out, dtype=torch.int64)
    return torch.where(t >= 1 << 31, t - (1 << 32), t).to(torch.int32).cuda()


def prepare(case, seed):
    c = case
    g = _generator(c, seed)
    rng = random.Random(seed)
    ctx, new = _lengths(c)
    lengths = [a + b for a, b in zip(ctx, new)]
    group, shared = c.get("group", 1), c.get("shared", 0)
    tables, blocks = _tables(c, lengths, group, shared, g)
    (k, ks), (v, vs) = (_quantised(c, c.get("layers", 1), blocks, g) for _ in range(2))
    state = {"case": c, "k": k, "v": v, "ks": ks, "vs": vs, "tables": tables, "group": group, "max_new": c["new"],
             "seq_len": torch.tensor(lengths, dtype=torch.int32, device="cuda"), "row_start": _rows(new)}
    rows = sum(new)
    if c["op"] == "compact":
        path = [sorted(rng.sample(range(m), min(c["path"], m))) for m in new]
        state["n_path"] = torch.tensor([len(p) for p in path], dtype=torch.int32, device="cuda")
        state["path"] = torch.tensor([p + [-1] * (c["path"] - len(p)) for p in path], dtype=torch.int32, device="cuda")
        return state
    dt = DTYPES[c["dtype"]]
    heads, kv, dim = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        # the projection's one output row holds the heads of q, k and v side by side
        qkv = torch.randn((rows, (heads + 2 * kv) * dim), generator=g, device="cuda", dtype=dt)
        state["q"], state["kn"], state["vn"] = (t.unflatten(1, (-1, dim)) for t in qkv.split([heads * dim, kv * dim, kv * dim], dim=1))
        pos = torch.cat([torch.arange(a, a + m) for a, m in zip(ctx, new)]).to(torch.int32)
        state["positions"] = pos.cuda()
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
        angle = torch.outer(torch.arange(max(lengths), dtype=torch.float64), freq)
        state["rope"] = torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32).cuda()
        for w in ("q_weight", "k_weight"):
            state[w] = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(dt) if c["norm"] else None
        state["q_out"] = torch.empty((rows, heads, dim), dtype=dt, device="cuda")
        return state
    state["q"] = (1.5 * torch.randn((rows, heads, dim), generator=g, device="cuda")).to(dt)
    state["out"] = torch.empty_like(state["q"])
    state["lse"] = torch.empty((rows, heads), dtype=torch.float32, device="cuda")
    state["mask"] = None if c["mask"] == "chain" else _masks(c, new, rng)
    state["scale"] = 1 / math.sqrt(dim)
    if c["mask"] == "tree_padded":  # what no sequence has written yet is whatever the memory held
        unused = torch.ones(blocks * c["block"], dtype=torch.bool, device="cuda")
        used = _slots(state, torch.arange(max(lengths), device="cuda")[None].expand(len(lengths), -1))
        inside = torch.arange(max(lengths), device="cuda")[None] < state["seq_len"][:, None]
        unused[used[inside]] = False
        bad = unused.view(blocks, c["block"])[None, :, :, None, None]
        k.view(torch.uint8).masked_fill_(bad, 0x7F)
        v.view(torch.uint8).masked_fill_(bad, 0x7F)
    return state


def _slots(state, at):
    """Cache slots (block * block_size + offset) of token positions [S, n]."""
    bs = state["case"]["block"]
    col = (at // bs).clamp(max=state["tables"].shape[1] - 1)
    return state["tables"].long().gather(1, col).clamp(min=0) * bs + at % bs


# ---- plain forms -----------------------------------------------------------

def _held(x, scale, slot, held, block):
    """Values [S, n, kv_heads, dim] in 32 bits of the slots [S, n] of one layer; 0 where nothing is held."""
    y = x[slot // block, slot % block].float() * scale[slot // block][..., None]
    return torch.where(held[..., None, None], y, 0)


def _plain_attend(state):
    c, q = state["case"], state["q"]
    heads, kv, dim, new = c["heads"], c["kv_heads"], c["dim"], c["new"]
    start, lengths = state["row_start"].long(), state["seq_len"].long()
    seqs, longest = lengths.numel(), state["tables"].shape[1] * c["block"]
    count = start[1:] - start[:-1]
    ctx = lengths - count
    # the rows of each sequence, padded to the longest
    i = torch.arange(new, device="cuda")
    live = i[None] < count[:, None]
    row = torch.where(live, start[:-1, None] + i[None], 0)
    qs = q.float()[row].view(seqs, new, kv, heads // kv, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, dim)
    # keys and values of each sequence by its table, and which of them each row sees
    at = torch.arange(longest, device="cuda")[None].expand(seqs, -1)
    slot = _slots(state, at)
    held = at < lengths[:, None]
    ks = _held(state["k"][0], state["ks"][0], slot, held, c["block"]).permute(0, 2, 1, 3)
    vs = _held(state["v"][0], state["vs"][0], slot, held, c["block"]).permute(0, 2, 1, 3)
    j = at - ctx[:, None]
    if state["mask"] is None:
        sees = j[:, None, :] <= i[None, :, None]
    else:
        word = state["mask"][row]
        col = j.clamp(min=0, max=new - 1)
        bit = word.gather(2, (col // 32)[:, None].expand(-1, new, -1)) >> (col % 32).to(torch.int32)[:, None]
        sees = (j < 0)[:, None] | (bit & 1).bool()
    sees = sees & held[:, None]
    scores = (qs @ ks.transpose(2, 3)) * state["scale"]
    scores = scores.view(seqs, kv, heads // kv, new, longest).masked_fill(~sees[:, None, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = weights.sum(dim=-1, keepdim=True)
    o = (weights.view(seqs, kv, -1, longest) @ vs).view(seqs, kv, heads // kv, new, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(seqs, new, heads, dim)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(seqs, new, heads)
    return {"out": o[live].to(q.dtype), "lse": lse[live]}


def _rotated(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = (a * cos - b * sin, a * sin + b * cos)
    y = torch.stack(y, dim=-1).flatten(-2) if interleaved else torch.cat(y, dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * w.float()


def _store(cache, scale, rows, block, offset, first_block, first):
    """Rows [n, kv_heads, dim] in 32 bits into (block, offset) of one layer's cache; each sequence's first new token goes
    to offset `first` of first_block, behind what that block keeps."""
    row_top = rows.abs().amax(dim=-1)
    top = torch.zeros_like(scale).scatter_reduce(0, block[:, None].expand_as(row_top), row_top, "amax")
    written = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill(0, block, True)
    kept = torch.zeros_like(written).index_put((first_block,), first > 0)
    new = torch.maximum(_least_scale(top), torch.where(kept[:, None], scale, 0.0))
    new = torch.where(written[:, None], new, scale)
    # what the first blocks keep, under their new scales
    old = cache[first_block].float()
    again = (old * (scale / new)[first_block][:, None, :, None]).to(E4M3).view(torch.uint8)
    before = torch.arange(cache.shape[1], device="cuda")[None] < first[:, None]
    bits = cache.view(torch.uint8)
    bits[first_block] = torch.where(before[..., None, None], again, bits[first_block])
    bits[block, offset] = (rows / new[block][..., None]).to(E4M3).view(torch.uint8)
    scale.copy_(new)


def _plain_append(state):
    c = state["case"]
    rot, rows = c["rot"], state["q"].shape[0]
    start, lengths = state["row_start"].long(), state["seq_len"].long()
    seq = torch.bucketize(torch.arange(rows, device="cuda"), start[1:], right=True)
    at = lengths[seq] - start[seq + 1] + torch.arange(rows, device="cuda")
    bs = c["block"]
    block, offset = state["tables"].long()[seq, at // bs], at % bs
    head = lengths - start[1:] + start[:-1]
    first_block = state["tables"].long().gather(1, (head // bs)[:, None])[:, 0]
    cs = state["rope"][state["positions"].long()][:, None]
    q, k = (_rotated(_normed(x, w), cs[..., :rot // 2], cs[..., rot // 2:], rot, c["interleaved"])
            for x, w in ((state["q"], state["q_weight"]), (state["kn"], state["k_weight"])))
    _store(state["k"][0], state["ks"][0], k, block, offset, first_block, head % bs)
    _store(state["v"][0], state["vs"][0], state["vn"].float(), block, offset, first_block, head % bs)
    return {"q": q.to(state["q"].dtype), "k": state["k"], "v": state["v"], "ks": state["ks"], "vs": state["vs"]}


def _plain_compact(state):
    c = state["case"]
    bs = c["block"]
    start, lengths, path = state["row_start"].long(), state["seq_len"].long(), state["path"].long()
    ctx = (lengths - start[1:] + start[:-1])[:, None]
    n = state["n_path"].long()[:, None]
    i = torch.arange(path.shape[1], device="cuda")[None]
    live = i < n
    # the places past a path's end write again what its first place gets
    to = _slots(state, ctx + torch.where(live, i, 0)).reshape(-1)
    source = _slots(state, ctx + torch.where(live, path, path[:, :1])).reshape(-1)
    # the blocks that a path's places lie in, and which of their tokens the sequence holds
    reach = (path.shape[1] - 1) // bs + 1
    col = torch.minimum(ctx // bs + torch.arange(reach + 1, device="cuda")[None], (ctx + n - 1) // bs)
    there = state["tables"].long().gather(1, col)
    at = col[..., None] * bs + torch.arange(bs, device="cuda")
    held = (at < lengths[:, None, None])[None, ..., None, None]
    for x, scale in ((state["k"], state["ks"]), (state["v"], state["vs"])):
        layers, _, _, kv, dim = x.shape
        index = (to // bs)[None, :, None].expand(layers, -1, kv)
        new = scale.scatter_reduce(1, index, scale[:, source // bs], "amax")
        bits = x.view(torch.uint8)
        moved = x[:, source // bs, source % bs].float() * (scale[:, source // bs] / new[:, to // bs])[..., None]
        again = (x[:, there].float() * (scale / new)[:, there][:, :, :, None, :, None]).to(E4M3).view(torch.uint8)
        bits[:, there] = torch.where(held, again, bits[:, there])
        bits[:, to // bs, to % bs] = moved.to(E4M3).view(torch.uint8)
        scale.copy_(new)
    return {"k": state["k"], "v": state["v"], "ks": state["ks"], "vs": state["vs"]}


# ---- the framework's calls -------------------------------------------------

def _plan(state):
    """What a program keeps between calls: descriptors of the cache and of the batch, a workspace."""
    import smc_speculative_decoding_gb300 as smcsd
    plan = {"smcsd": smcsd, "cache": smcsd.make_cache8(state["k"], state["v"], state["ks"], state["vs"])}
    plan["batch"] = smcsd.make_batch(state["tables"], state["seq_len"], state["max_new"], row_start=state["row_start"],
                                     rows=state["q"].shape[0] if "q" in state else None, group=state["group"])
    heads = state["case"].get("heads", state["case"]["kv_heads"])
    plan["workspace"] = smcsd.alloc_cache8_workspace(plan["cache"], plan["batch"], heads)
    state["plan"] = plan
    return plan


def _own(state):
    plan = state.get("plan") or _plan(state)
    smcsd, cache, ws, op = plan["smcsd"], plan["cache"], plan["workspace"], state["case"]["op"]
    if op == "attend":
        smcsd.smc_tree_attention8(cache, 0, plan["batch"], state["q"], state["out"], ws, mask=state["mask"],
                                  lse=state["lse"], scale=state["scale"])
        return {"out": state["out"], "lse": state["lse"]}
    kept = {"k": state["k"], "v": state["v"], "ks": state["ks"], "vs": state["vs"]}
    if op == "append":
        smcsd.smc_qk_norm_rope8(cache, 0, plan["batch"], state["q"], state["kn"], state["vn"], state["rope"],
                                state["q_out"], ws, positions=state["positions"], q_weight=state["q_weight"],
                                k_weight=state["k_weight"], eps=1e-6, interleaved=state["case"]["interleaved"])
        return {"q": state["q_out"], **kept}
    smcsd.kv_compact_tokens8(cache, plan["batch"], state["path"], state["n_path"], ws)
    return kept


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "append": _plain_append, "compact": _plain_compact}[state["case"]["op"]](state)


# ---- in 64 bits, from the definitions --------------------------------------

def _exact_attend(s):
    c = s["case"]
    rep, bs = c["heads"] // c["kv_heads"], c["block"]
    start, lengths = s["row_start"].tolist(), s["seq_len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lengths):
        r0, r1 = start[b], start[b + 1]
        new = r1 - r0
        blocks = s["tables"][b, :-(-n // bs)].long()
        if s["mask"] is None:
            sees = torch.ones((new, new), dtype=torch.bool, device="cuda").tril()
        else:
            words = s["mask"][r0:r1].long()
            sees = torch.stack([words[:, j // 32] >> j % 32 & 1 for j in range(new)], dim=1).bool()
        sees = torch.cat([torch.ones((new, n - new), dtype=torch.bool, device="cuda"), sees], dim=1).repeat_interleave(rep, 0)
        some = sees.any(dim=1)
        for h in range(c["kv_heads"]):
            k = (s["k"][0][blocks][:, :, h].double() * s["ks"][0, blocks, h].double()[:, None, None]).reshape(-1, c["dim"])[:n]
            v = (s["v"][0][blocks][:, :, h].double() * s["vs"][0, blocks, h].double()[:, None, None]).reshape(-1, c["dim"])[:n]
            x = s["q"][r0:r1, h * rep:(h + 1) * rep].reshape(-1, c["dim"]).double()
            z = (s["scale"] * (x @ k.T)).masked_fill(~sees, -math.inf)
            p = torch.softmax(z, dim=1) @ v
            out[r0:r1, h * rep:(h + 1) * rep] = torch.where(some[:, None], p, 0.0).view(new, rep, -1)
            lse[r0:r1, h * rep:(h + 1) * rep] = torch.logsumexp(z, dim=1).view(new, rep)
    return {"out": out, "lse": lse}


def _power(top):
    """The least power of two from 2^LEAST with top <= 448 times it, by counting up."""
    return next(2.0 ** t for t in range(LEAST, 128) if top <= 448 * 2.0 ** t)


def _exact_append(s):
    c = s["case"]
    rot, dim, bs = c["rot"], c["dim"], c["block"]
    half = rot // 2
    a = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    b = a + (1 if c["interleaved"] else half)
    t = s["rope"].double()[s["positions"].long()]
    turn = torch.complex(t[:, :half], t[:, half:])[:, None]
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["kn"], s["k_weight"])):
        y = x.double()
        if w is not None:
            y = y / ((y * y).sum(-1, keepdim=True) / dim + 1e-6).sqrt() * w.double()
        z = torch.complex(y[..., a], y[..., b]) * turn
        y[..., a], y[..., b] = z.real, z.imag
        got.append(y)
    start, lengths, tables = s["row_start"].tolist(), s["seq_len"].tolist(), s["tables"].tolist()
    where = []  # (block, rows from, to, offset of the first)
    for q, n in enumerate(lengths):
        row, p = start[q], n - (start[q + 1] - start[q])
        while p < n:
            m = min(bs - p % bs, n - p)
            where.append((tables[q][p // bs], row, row + m, p % bs))
            row, p = row + m, p + m
    out = {"q": got[0]}
    for name, x, y in (("k", s["k"], got[1]), ("v", s["v"], s["vn"].double())):
        cache, scale = x.double(), s[name + "s"].double()
        tops = torch.stack([y[r0:r1].abs().amax(dim=(0, 2)) for _, r0, r1, _ in where]).tolist()
        for (block, r0, r1, first), top in zip(where, tops):
            need = torch.tensor([_power(v) for v in top], dtype=torch.float64, device="cuda")
            if first:
                need = torch.maximum(need, scale[0, block])
                cache[0, block, :first] *= (scale[0, block] / need)[None, :, None]
            scale[0, block] = need
            cache[0, block, first:first + r1 - r0] = y[r0:r1] / need[None, :, None]
        out[name], out[name + "s"] = cache, scale
    return out


def _exact_compact(s):
    bs = s["case"]["block"]
    start, lengths, tables = s["row_start"].tolist(), s["seq_len"].tolist(), s["tables"].tolist()
    paths, counts = s["path"].tolist(), s["n_path"].tolist()
    out = {}
    for name in ("k", "v"):
        cache, scale = s[name].double(), s[name + "s"].double()
        before, old = cache.clone(), scale.clone()
        for q, n in enumerate(lengths):
            ctx = n - (start[q + 1] - start[q])
            moves = [(tables[q][(ctx + j) // bs], (ctx + j) % bs, (ctx + i) // bs, (ctx + i) % bs)
                     for i, j in enumerate(paths[q][:counts[q]])]
            for slot in sorted({m[2] for m in moves}):
                block = tables[q][slot]
                into = [m for m in moves if m[2] == slot]
                scale[:, block] = torch.stack([old[:, block]] + [old[:, m[0]] for m in into]).amax(dim=0)
                kept = min(bs, n - slot * bs)
                cache[:, block, :kept] = before[:, block, :kept] * (old[:, block] / scale[:, block])[:, None, :, None]
                for src, at, _, dst in into:
                    cache[:, block, dst] = before[:, src, at] * (old[:, src] / scale[:, block])[..., None]
        out[name], out[name + "s"] = cache, scale
    return out


def exact(case, seed):
    c = case
    if c["op"] == "attend" and c["prompts"] * c["group"] * c["kv_heads"] > 4000:
        return None
    if c["op"] == "append" and c["seqs"] * (c["new"] / c["block"] + 2) > 20000:
        return None
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "compact": _exact_compact}[c["op"]](s)
