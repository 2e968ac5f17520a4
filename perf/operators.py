"""Workloads of the paged key/value cache's operators, with their plain forms.

Three operators around one paged cache [layers, blocks, block_size, kv_heads, head_dim]:

  qk         per-head RMS norms of queries and keys with the position rotation, K and V written to the cache
  attention  attention of the new (drafted) tokens of each sequence over its blocks, under a tree mask
  copy       copy-on-write pairs of blocks copied in every layer
  compact    the accepted path of a drafted tree moved to the front of the new tokens, in every layer

A sequence's new tokens are the last ones that it holds: seq_len counts them.  Plain forms: elementary torch
operations in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------

def _attention(name, dtype, prompts, group, new, heads, kv_heads, dim, block, ctx, ragged, shared, mask, order="nhd"):
    """prompts * group sequences of up to ctx committed tokens; the first `shared` tokens of a prompt's sequences are
    the same blocks.  ragged: share of the length by which sequences differ (0: none)."""
    return {"name": name, "op": "attention", "dtype": dtype, "prompts": prompts, "group": group, "new": new,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "block": block, "ctx": ctx, "ragged": ragged,
            "shared": shared, "mask": mask, "order": order}


def _qk(name, dtype, seqs, new, heads, kv_heads, dim, rot, interleaved, norm, block, ctx, ragged):
    return {"name": name, "op": "qk", "dtype": dtype, "seqs": seqs, "new": new, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "rot": rot, "interleaved": interleaved, "norm": norm, "block": block, "ctx": ctx,
            "ragged": ragged}


def _copy(name, dtype, prompts, group, layers, blocks, kv_heads, dim, block, filled):
    return {"name": name, "op": "copy", "dtype": dtype, "prompts": prompts, "group": group, "layers": layers,
            "blocks": blocks, "kv_heads": kv_heads, "dim": dim, "block": block, "filled": filled}


def _compact(name, dtype, seqs, new, path, layers, kv_heads, dim, block, ctx):
    return {"name": name, "op": "compact", "dtype": dtype, "seqs": seqs, "new": new, "path": path, "layers": layers,
            "kv_heads": kv_heads, "dim": dim, "block": block, "ctx": ctx}


def listed():
    return [
        # one sequence decodes one token behind the single-prompt workload's 512-token prefix: latency
        _attention("attend_one_token", "bf16", 1, 1, 1, 32, 8, 128, 16, 513, 0.0, 0, "chain"),
        # the single-prompt workload: 8 particles x (K = 4 drafted + 1) tokens, prefix 512 shared, own tails
        _attention("attend_single_prompt", "bf16", 1, 8, 5, 32, 8, 128, 16, 700, 0.1, 512, "chain"),
        # the serving workload: 16 prompts x 16 particles, K = 4, prefix 2048 shared, tails of up to 640 tokens
        _attention("attend_serving_particles", "bf16", 16, 16, 5, 32, 8, 128, 16, 2688, 0.2, 2048, "chain"),
        # drafted trees of 64 tokens verified for 16 requests: many rows for each key
        _attention("attend_tree_64", "bf16", 16, 1, 64, 32, 8, 128, 64, 4096, 0.3, 0, "tree"),
        # one request with a long document, a small tree: the split over the length
        _attention("attend_long_context", "bf16", 1, 1, 8, 64, 8, 128, 64, 131072, 0.0, 0, "tree"),
        # odd sizes: fp16, as many key heads as heads, 64 wide, blocks of 24 tokens in head-major order, some
        # sequences with no committed token, rows of padding that see nothing
        _attention("attend_ragged_f16", "f16", 5, 1, 7, 12, 12, 64, 24, 777, 1.0, 0, "tree_padded", "hnd"),
        # a full batch with trees of 16 tokens and contexts of up to 8192: the largest
        _attention("attend_batch_8k", "bf16", 64, 1, 16, 32, 8, 128, 32, 8192, 0.5, 0, "tree"),
        # one token of one sequence on its way into the attention: latency
        _qk("qk_one_token", "bf16", 1, 1, 32, 8, 128, 128, False, True, 16, 513, 0.0),
        # the serving workload's 1280 rows
        _qk("qk_serving_rows", "bf16", 256, 5, 32, 8, 128, 128, False, True, 16, 512, 0.2),
        # a prompt's rows, in fp16, 96 wide heads rotated in part, neighbouring pairs
        _qk("qk_prompt_rows", "f16", 3, 5000, 40, 8, 96, 64, True, True, 16, 0, 0.3),
        # the serving workload's copy-on-write pairs after a resampling step, all layers of the cache
        _copy("copy_cow_serving", "bf16", 16, 16, 32, 1024, 8, 128, 16, 0.6),
        # accepted paths of the trees of 64 requests, all layers
        _compact("compact_tree_paths", "bf16", 64, 64, 9, 32, 8, 128, 16, 150),
    ]


def _cost(c):
    """Bytes that the plain form handles, to keep drawn cases below the largest listed one."""
    s = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "attention":
        n = c["prompts"] * c["group"]
        length = c["ctx"] + c["new"]
        return n * length * (2 * c["kv_heads"] * c["dim"] * (s + 4) + c["heads"] * c["new"] * 8) * 1.0
    if c["op"] == "qk":
        return c["seqs"] * (c["new"] + c["ctx"]) * (c["heads"] + 2 * c["kv_heads"]) * c["dim"] * 8.0
    return 4.0 * c["layers"] * c["block"] * c["kv_heads"] * c["dim"] * s * (
        c["blocks"] if c["op"] == "copy" else c["seqs"] * (-(-(c["ctx"] + c["new"]) // c["block"]) + 1))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {"attention": 5.0e9, "qk": 5.0e8, "copy": 4.0e9, "compact": 4.0e9}
    while True:
        op = rng.choice(["attention", "attention", "attention", "qk", "qk", "copy", "compact"])
        kv, rep = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 8])
        block = rng.choice([8, 16, 16, 32, 48, 64, 128, 20])
        if op == "attention":
            group = rng.choice([1, 1, 1, 2, 5, 8, 16])
            new = _log(rng, 1, 128)
            ctx = _log(rng, 1, 60000)
            c = _attention("", rng.choice(["bf16", "bf16", "f16"]), _log(rng, 1, 64), group, new, kv * rep, kv,
                           rng.choice([64, 128, 128, 80, 96]), block, ctx, rng.choice([0.0, 0.3, 1.0]),
                           int(ctx * rng.random()) if group > 1 else 0,
                           rng.choice(["chain", "tree", "tree_padded"]), rng.choice(["nhd", "hnd"]))
        elif op == "qk":
            dim = rng.choice([64, 128, 96, 80])
            c = _qk("", rng.choice(["bf16", "f16", "f32"]), _log(rng, 1, 300), _log(rng, 1, 2000), kv * rep, kv, dim,
                    rng.choice([dim, dim // 2]), rng.random() < 0.5, rng.random() < 0.8, block, _log(rng, 1, 2000),
                    rng.choice([0.0, 0.5]))
        elif op == "copy":
            c = _copy("", rng.choice(["bf16", "f32"]), _log(rng, 1, 16), rng.choice([1, 3, 8, 16]),
                      rng.choice([1, 7, 24, 32]), _log(rng, 40, 1024), kv, rng.choice([64, 128, 80]), block, rng.random())
            if c["blocks"] < 2 * c["prompts"] * c["group"]:
                continue
        else:
            new = _log(rng, 2, 100)
            c = _compact("", rng.choice(["bf16", "f32"]), _log(rng, 1, 64), new, rng.randint(1, min(12, new)),
                         rng.choice([1, 7, 24, 32]), kv, rng.choice([64, 128, 80]), block, _log(rng, 1, 300))
        del c["name"]
        widths = [h * c["dim"] for h in (kv, kv * rep, kv * rep + 2 * kv)]
        if _cost(c) <= top[op] and 3072 not in widths + [v for v in c.values() if not isinstance(v, str)]:
            return c


# ---- lengths: from the case alone ------------------------------------------

def _lengths(c):
    """(committed, new) tokens of each sequence."""
    rng = random.Random("%s %s %s %s" % (c["op"], c["ctx"], c["new"], c.get("prompts", c.get("seqs"))))
    n = c["prompts"] * c["group"] if c["op"] == "attention" else c["seqs"]
    ragged = c.get("ragged", 0.3)
    ctx = [c["ctx"] - int(ragged * c["ctx"] * rng.random()) for _ in range(n)]
    new = [c["new"] - int(0.5 * ragged * c["new"] * rng.random()) for _ in range(n)]
    if c["op"] == "attention":
        ctx = [max(v, c["shared"]) for v in ctx]
    if ragged == 1.0:  # some sequences have committed nothing yet
        ctx = [0 if i % 5 == 3 else v for i, v in enumerate(ctx)] if not c["shared"] else ctx
    if c["op"] == "qk" and ragged == 0.0 or c.get("mask") == "chain":
        new = [c["new"]] * n  # particles always draft the same number
    ctx[0], new[0] = c["ctx"], c["new"]
    return ctx, new


def work(case):
    c = case
    s = 4 if c["dtype"] == "f32" else 2
    token = 2 * c["kv_heads"] * c["dim"] * s
    if c["op"] == "copy":
        pairs = sum(_pairs(c))
        return {"bytes": 2 * pairs * c["layers"] * c["block"] * token, "flops": 0}
    ctx, new = _lengths(c)
    if c["op"] == "compact":
        moved = sum(min(c["path"], m) for m in new)
        return {"bytes": 2 * moved * c["layers"] * token, "flops": 0}
    rows = sum(new)
    if c["op"] == "qk":
        io = (c["heads"] + 2 * c["kv_heads"]) * c["dim"] * s
        return {"bytes": rows * (2 * io + 4 * c["rot"]), "flops": 10 * rows * (c["heads"] + c["kv_heads"]) * c["dim"]}
    common = c["shared"] // c["block"] * c["block"]
    kept = c["prompts"] * common + sum(v - common + m for v, m in zip(ctx, new))
    flops = sum(4 * c["heads"] * c["dim"] * m * (v + m) for v, m in zip(ctx, new))
    return {"bytes": kept * token + 2 * rows * c["heads"] * c["dim"] * s, "flops": flops}


# ---- inputs ----------------------------------------------------------------

def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cache(c, layers, blocks, g):
    """Keys and values [layers, blocks, block, kv_heads, dim], as views where the memory order is head-major."""
    dt = DTYPES[c["dtype"]]
    hnd = c.get("order") == "hnd"
    shape = (layers, blocks, c["kv_heads"], c["block"], c["dim"]) if hnd else (layers, blocks, c["block"], c["kv_heads"], c["dim"])
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=dt) for _ in range(2))
    return (k.transpose(2, 3), v.transpose(2, 3)) if hnd else (k, v)


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


def _masks(c, new, g, rng):
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


def _pairs(c):
    """How many copy-on-write pairs each prompt has: at most group - 1."""
    rng = random.Random("%s %s" % (c["prompts"], c["filled"]))
    return [min(c["group"], max(1, int(round(c["group"] * c["filled"] * rng.uniform(0.7, 1.3))))) for _ in range(c["prompts"])]


def prepare(case, seed):
    c = case
    g = _generator(c, seed)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "copy":
        k, v = _cache(c, c["layers"], c["blocks"], g)
        ids = torch.randperm(c["blocks"], generator=g, device="cuda").to(torch.int32)
        half = c["prompts"] * c["group"]
        pairs = torch.stack([ids[:half], ids[half:2 * half]], dim=1).view(c["prompts"], c["group"], 2).contiguous()
        return {"case": c, "k": k, "v": v, "pairs": pairs,
                "counts": torch.tensor(_pairs(c), dtype=torch.int32, device="cuda")}
    ctx, new = _lengths(c)
    lengths = [a + b for a, b in zip(ctx, new)]
    group, shared = c.get("group", 1), c.get("shared", 0)
    tables, blocks = _tables(c, lengths, group, shared, g)
    k, v = _cache(c, c.get("layers", 1), blocks, g)
    state = {"case": c, "k": k, "v": v, "tables": tables, "group": group, "max_new": c["new"],
             "seq_len": torch.tensor(lengths, dtype=torch.int32, device="cuda"), "row_start": _rows(new)}
    rows = sum(new)
    rng = random.Random(seed)
    if c["op"] == "compact":
        path = [sorted(rng.sample(range(m), min(c["path"], m))) for m in new]
        state["n_path"] = torch.tensor([len(p) for p in path], dtype=torch.int32, device="cuda")
        state["path"] = torch.tensor([p + [-1] * (c["path"] - len(p)) for p in path], dtype=torch.int32, device="cuda")
        return state
    heads, kv, dim = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "qk":
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
    state["mask"] = None if c["mask"] == "chain" else _masks(c, new, g, rng)
    state["scale"] = 1 / math.sqrt(dim)
    if c["mask"] == "tree_padded":  # what no sequence has written yet is whatever the memory held
        unused = torch.ones(blocks * c["block"], dtype=torch.bool, device="cuda")
        used = _slots(state, torch.arange(max(lengths), device="cuda")[None].expand(len(lengths), -1))
        inside = torch.arange(max(lengths), device="cuda")[None] < state["seq_len"][:, None]
        unused[used[inside]] = False
        bad = unused.view(blocks, c["block"])[None, :, :, None, None]
        k.masked_fill_(bad, float("nan"))
        v.masked_fill_(bad, float("nan"))
    return state


def _slots(state, at):
    """Cache slots (block * block_size + offset) of token positions [S, n]."""
    bs = state["case"]["block"]
    col = (at // bs).clamp(max=state["tables"].shape[1] - 1)
    return state["tables"].long().gather(1, col).clamp(min=0) * bs + at % bs


# ---- plain forms -----------------------------------------------------------

def _flat(cache):
    """[layers, slots, kv_heads, dim] of a cache, as a copy where the memory order is another."""
    return cache.reshape(cache.shape[0], -1, *cache.shape[3:])


def _plain_attention(state):
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
    ks = torch.where(held[..., None, None], state["k"][0].flatten(0, 1)[slot].float(), 0).permute(0, 2, 1, 3)
    vs = torch.where(held[..., None, None], state["v"][0].flatten(0, 1)[slot].float(), 0).permute(0, 2, 1, 3)
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


def _plain_qk(state):
    c = state["case"]
    rot, rows = c["rot"], state["q"].shape[0]
    start, lengths = state["row_start"].long(), state["seq_len"].long()
    seq = torch.bucketize(torch.arange(rows, device="cuda"), start[1:], right=True)
    at = lengths[seq] - start[seq + 1] + torch.arange(rows, device="cuda")
    bs = c["block"]
    block, offset = state["tables"].long()[seq, at // bs], at % bs
    cs = state["rope"][state["positions"].long()][:, None]
    done = []
    for x, w in ((state["q"], state["q_weight"]), (state["kn"], state["k_weight"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * w.float()
        done.append(_rotated(x, cs[..., :rot // 2], cs[..., rot // 2:], rot, c["interleaved"]).to(state["q"].dtype))
    state["k"][0].index_put_((block, offset), done[1])
    state["v"][0].index_put_((block, offset), state["vn"])
    return {"q": done[0], "k": state["k"], "v": state["v"]}


def _plain_copy(state):
    pairs, counts = state["pairs"].long(), state["counts"]
    live = torch.arange(pairs.shape[1], device="cuda")[None] < counts[:, None]
    src, dst = pairs[..., 0].reshape(-1), pairs[..., 1].reshape(-1)
    src = torch.where(live.reshape(-1), src, dst)  # a pair past the count copies a block onto itself
    state["k"][:, dst] = state["k"][:, src]
    state["v"][:, dst] = state["v"][:, src]
    return {"k": state["k"], "v": state["v"]}


def _plain_compact(state):
    start, lengths, path = state["row_start"].long(), state["seq_len"].long(), state["path"].long()
    ctx = (lengths - start[1:] + start[:-1])[:, None]
    i = torch.arange(path.shape[1], device="cuda")[None]
    live = i < state["n_path"][:, None]
    to = _slots(state, ctx + torch.where(live, i, 0)).reshape(-1)
    # the places past a path's end write again what its first place gets
    source = torch.where(live, path, path[:, :1])
    source = _slots(state, ctx + source).reshape(-1)
    for cache in (state["k"], state["v"]):
        flat = cache.view(cache.shape[0], -1, *cache.shape[3:])
        flat[:, to] = flat[:, source]
    return {"k": state["k"], "v": state["v"]}


# ---- the framework's calls -------------------------------------------------

def _plan(state):
    """What a program keeps between calls: descriptors of the cache and of the batch, a workspace."""
    import smc_speculative_decoding_gb300 as smcsd
    plan = {"smcsd": smcsd, "cache": smcsd.make_cache(state["k"], state["v"])}
    if "tables" in state:
        plan["batch"] = smcsd.make_batch(state["tables"], state["seq_len"], state["max_new"], row_start=state["row_start"],
                                         rows=state["q"].shape[0] if "q" in state else None, group=state["group"])
        heads = state["case"].get("heads", state["case"]["kv_heads"])
        plan["workspace"] = smcsd.alloc_cache_workspace(plan["cache"], plan["batch"], heads)
    else:
        plan["workspace"] = smcsd.alloc_cache_workspace(plan["cache"])
    state["plan"] = plan
    return plan


def _own(state):
    plan = state.get("plan") or _plan(state)
    smcsd, cache, ws, op = plan["smcsd"], plan["cache"], plan["workspace"], state["case"]["op"]
    if op == "attention":
        smcsd.smc_tree_attention(cache, 0, plan["batch"], state["q"], state["out"], ws, mask=state["mask"],
                                 lse=state["lse"], scale=state["scale"])
        return {"out": state["out"], "lse": state["lse"]}
    if op == "qk":
        smcsd.smc_qk_norm_rope(cache, 0, plan["batch"], state["q"], state["kn"], state["vn"], state["rope"],
                               state["q_out"], ws, positions=state["positions"], q_weight=state["q_weight"],
                               k_weight=state["k_weight"], eps=1e-6, interleaved=state["case"]["interleaved"])
        return {"q": state["q_out"], "k": state["k"], "v": state["v"]}
    if op == "copy":
        smcsd.kv_copy_blocks(cache, state["pairs"], state["counts"], ws)
    else:
        smcsd.kv_compact_tokens(cache, plan["batch"], state["path"], state["n_path"], ws)
    return {"k": state["k"], "v": state["v"]}


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "qk": _plain_qk, "copy": _plain_copy, "compact": _plain_compact}[state["case"]["op"]](state)


# ---- in 64 bits, from the definitions --------------------------------------

def _exact_attention(s):
    c = s["case"]
    rep, bs = c["heads"] // c["kv_heads"], c["block"]
    start, lengths = s["row_start"].tolist(), s["seq_len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lengths):
        r0, r1 = start[b], start[b + 1]
        blocks = s["tables"][b, :-(-n // bs)].long()
        committed = n - (r1 - r0)
        for h in range(c["kv_heads"]):
            k = s["k"][0, blocks, :, h].double().reshape(-1, c["dim"])[:n]
            v = s["v"][0, blocks, :, h].double().reshape(-1, c["dim"])[:n]
            for r in range(r0, r1):
                if s["mask"] is None:
                    seen = list(range(r - r0 + 1))
                else:
                    bits = sum((w & 0xFFFFFFFF) << 32 * i for i, w in enumerate(s["masks"][r]))
                    seen = [j for j in range(r1 - r0) if bits >> j & 1]
                cols = torch.tensor(list(range(committed, n)) if len(seen) == r1 - r0 else [committed + j for j in seen], device="cuda", dtype=torch.long)
                if committed + len(seen) == 0:
                    continue
                x = s["q"][r, h * rep:(h + 1) * rep].double()
                z = torch.cat([k[:committed] @ x.T, k[cols] @ x.T]) * s["scale"]
                lse[r, h * rep:(h + 1) * rep] = torch.logsumexp(z, dim=0)
                p = torch.softmax(z, dim=0)
                out[r, h * rep:(h + 1) * rep] = p[:committed].T @ v[:committed] + p[committed:].T @ v[cols]
    return {"out": out, "lse": lse}


def _exact_qk(s):
    c = s["case"]
    rot, dim, bs = c["rot"], c["dim"], c["block"]
    half = rot // 2
    first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)
    t = s["rope"].double()[s["positions"].long()]
    turn = torch.complex(t[:, :half], t[:, half:])[:, None]
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["kn"], s["k_weight"])):
        y = x.double()
        if w is not None:
            y = y / ((y * y).sum(-1, keepdim=True) / dim + 1e-6).sqrt() * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        got.append(y)
    k, v = s["k"].double(), s["v"].double()
    start, lengths, tables = s["row_start"].tolist(), s["seq_len"].tolist(), s["tables"].tolist()
    block, offset = [], []
    for b, n in enumerate(lengths):
        for p in range(n - (start[b + 1] - start[b]), n):
            block.append(tables[b][p // bs])
            offset.append(p % bs)
    k[0, block, offset], v[0, block, offset] = got[1], s["vn"].double()
    return {"q": got[0], "k": k, "v": v}


def exact(case, seed):
    c = case
    if c["op"] == "attention" and sum(_lengths(c)[1]) * c["kv_heads"] > 12000:
        return None
    s = prepare(case, seed)
    if c["op"] == "attention":
        if s["mask"] is not None:
            s["masks"] = s["mask"].tolist()
        return _exact_attention(s)
    if c["op"] == "qk":
        return _exact_qk(s)
    out = {}
    for name in ("k", "v"):  # moved values are their own 64-bit values
        cache = s[name]
        new = cache.clone()
        if c["op"] == "copy":
            for b, n in enumerate(s["counts"].tolist()):
                for src, dst in s["pairs"][b, :n].tolist():
                    new[:, dst] = cache[:, src]
        else:
            start, lengths, tables = s["row_start"].tolist(), s["seq_len"].tolist(), s["tables"].tolist()
            for b, n in enumerate(s["n_path"].tolist()):
                ctx = lengths[b] - (start[b + 1] - start[b])
                for i, j in enumerate(s["path"][b, :n].tolist()):
                    a, z = ctx + j, ctx + i
                    new[:, tables[b][z // c["block"]], z % c["block"]] = cache[:, tables[b][a // c["block"]], a % c["block"]]
        out[name] = new.double()
    return out
