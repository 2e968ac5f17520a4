"""Particles and drafted trees through a paged cache, with a small random model.

Shows how the entry points fit together around one decoding step:

  particles(...)  B prompts x N particles.  Each step, every layer norms and
                  rotates the queries and keys of the K + 1 new tokens of every
                  particle and writes keys and values to the cache
                  (smc_qk_norm_rope), attends them over the particle's blocks,
                  reading the blocks that a prompt's particles share once
                  (smc_tree_attention); smc_step reweights and resamples, remaps
                  the block tables and makes room for the next K + 1 tokens; the
                  copy-on-write pairs it leaves are copied (kv_copy_blocks).
  tree(...)       one sequence per prompt verifies a drafted tree: room for its
                  tokens (kv_blocktable_remap), attention under the tree's mask,
                  the accepted path moved to the front (kv_compact_tokens), the
                  rest of the room given back (kv_truncate).

    python examples/draft_scoring.py [--prompts 4] [--particles 8] [--steps 6] [--bits 8]

With --bits 8 the cache is one of 8-bit numbers with a scale per block and key
head: the same calls with an 8 behind their names.

The model's weights are random and its logits mean nothing; a real one puts its
projections where `Model` has two matrix products.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import smc_speculative_decoding_gb300 as smcsd  # noqa: E402
from smc_speculative_decoding_gb300.workloads import make_kv_state  # noqa: E402


class Cache:
    """A zero-filled paged cache of `bits` bits an element, and its entry points."""

    def __init__(self, model, blocks, block_size, bits=16, device="cuda"):
        shape = (len(model.qkv), blocks, block_size, model.kv_heads, model.dim)
        if bits == 8:
            self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
            self.k_scale, self.v_scale = (torch.ones((shape[0], blocks, model.kv_heads), device=device) for _ in range(2))
            self.args = smcsd.make_cache8(self.k, self.v, self.k_scale, self.v_scale)
            self.alloc_workspace, self.copy_blocks = smcsd.alloc_cache8_workspace, smcsd.kv_copy_blocks8
            self.qk_norm_rope, self.attention = smcsd.smc_qk_norm_rope8, smcsd.smc_tree_attention8
            self.compact_tokens = smcsd.kv_compact_tokens8
        else:
            self.k, self.v = (torch.zeros(shape, dtype=model.dtype, device=device) for _ in range(2))
            self.args = smcsd.make_cache(self.k, self.v)
            self.alloc_workspace, self.copy_blocks = smcsd.alloc_cache_workspace, smcsd.kv_copy_blocks
            self.qk_norm_rope, self.attention = smcsd.smc_qk_norm_rope, smcsd.smc_tree_attention
            self.compact_tokens = smcsd.kv_compact_tokens


class Model:
    """`layers` attention layers of random weights over a paged cache."""

    def __init__(self, vocab, layers=2, heads=8, kv_heads=2, dim=64, dtype=torch.bfloat16, seed=0,
                 max_pos=4096, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.dtype = heads, kv_heads, dim, dtype
        width = heads * dim

        def rand(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device=device) * scale).to(dtype)

        self.embedding = rand(vocab, width)
        self.qkv = [rand(width, (heads + 2 * kv_heads) * dim, scale=width ** -0.5) for _ in range(layers)]
        self.out = [rand(width, width, scale=width ** -0.5) for _ in range(layers)]
        self.q_weight = [1 + rand(dim, scale=0.1) for _ in range(layers)]
        self.k_weight = [1 + rand(dim, scale=0.1) for _ in range(layers)]
        freq = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
        angle = torch.outer(torch.arange(max_pos, dtype=torch.float64), freq)
        self.rope = torch.cat([angle.cos(), angle.sin()], dim=1).float().to(device)

    def forward(self, tokens, cache, batch, workspace, positions=None, mask=None, seen=None):
        """Logits of the new tokens [rows]; their keys and values go to the
        cache.  `seen` collects each layer's (q, attention output)."""
        x = self.embedding[tokens.long()]
        h, kv, d = self.heads, self.kv_heads, self.dim
        for i in range(len(self.qkv)):
            q, k, v = (t.unflatten(1, (-1, d)) for t in (x @ self.qkv[i]).split([h * d, kv * d, kv * d], dim=1))
            turned = torch.empty((x.shape[0], h, d), dtype=self.dtype, device=x.device)
            cache.qk_norm_rope(cache.args, i, batch, q, k, v, self.rope, turned, workspace, positions=positions,
                               q_weight=self.q_weight[i], k_weight=self.k_weight[i])
            o = torch.empty_like(turned)
            cache.attention(cache.args, i, batch, turned, o, workspace, mask=mask)
            if seen is not None:
                seen.append((turned, o))
            x = x + o.flatten(1) @ self.out[i]
        return (x @ self.embedding.T).float() * x.shape[1] ** -0.5


def particles(prompts=4, n=8, K=4, vocab=512, steps=6, prefix=40, block_size=16, seed=0, observe=None, bits=16):
    """Runs `steps` SMC steps; returns the tokens that each particle emitted
    [B, N, steps * (K + 1)] and the share of blocks that sharing saves.
    observe(step, state) sees the state after each forward pass."""
    dev, T = "cuda", K + 1
    model = Model(vocab, seed=seed)
    slots = -(-(prefix + (steps + 2) * T) // block_size) + 1
    pool = n * slots + 1
    kv = make_kv_state(prompts, n, prefix, block_size, slots, pool, device=dev)
    cache = Cache(model, prompts * pool, block_size, bits)
    k, v = cache.k, cache.v
    params = smcsd.make_params(prompts, n, K, vocab, "f32", ess_frac=0.6, seed=seed)
    kvs = smcsd.make_kv(params, kv, block_size)
    step_ws = smcsd.alloc_workspace(params, kvs)
    g = torch.Generator(device=dev).manual_seed(seed + 1)

    # the prompt: its keys and values once, by the first particle of each prompt
    first = smcsd.make_batch(kv["tables"][:, :1].reshape(prompts, -1).contiguous(),
                             kv["seq_len"][:, :1].reshape(-1).contiguous(), prefix)
    ws0 = cache.alloc_workspace(cache.args, first, model.heads)
    prompt_tokens = torch.randint(0, vocab, (prompts * prefix,), generator=g, device=dev)
    model.forward(prompt_tokens, cache, first, ws0)

    # room for the first K + 1 tokens of every particle
    log_weights = torch.zeros(prompts * n, device=dev)
    ancestors = torch.arange(n, dtype=torch.int32, device=dev).repeat(prompts)
    resampled = torch.zeros(prompts, dtype=torch.int32, device=dev)
    smcsd.kv_blocktable_remap(params, kvs, ancestors, resampled, T, step_ws)
    batch = smcsd.make_batch(kv["tables"], kv["seq_len"], T, group=n)
    ws = cache.alloc_workspace(cache.args, batch, model.heads)
    cache.copy_blocks(cache.args, kv["cow_pairs"], kv["n_cow"], ws)
    last = torch.randint(0, vocab, (prompts, n, 1), generator=g, device=dev, dtype=torch.int32)
    emitted = []
    ess = torch.empty(prompts, device=dev)
    tokens_out = torch.empty((prompts, n, T), dtype=torch.int32, device=dev)
    for step in range(steps):
        # a draft model would extend each particle; here its logits are a noisy copy of random ones
        draft = torch.randn((prompts, n, K, vocab), generator=g, device=dev)
        drafted = torch.multinomial(torch.softmax(draft, -1).view(-1, vocab), 1, generator=g)
        drafted = drafted.view(prompts, n, K).to(torch.int32)
        new = torch.cat([last, drafted], dim=2)
        seen = []
        logits = model.forward(new.reshape(-1), cache, batch, ws, seen=seen)
        target = (draft.mean() + logits).view(prompts, n, T, vocab).contiguous()
        if observe:
            observe(step, dict(kv=kv, k=k, v=v, seen=seen, new=new, block_size=block_size, model=model, cache=cache))
        params.step = step
        smcsd.smc_step(params, target, draft, drafted, log_weights, tokens_out, ancestors, ess, resampled, kv=kvs,
                       workspace=step_ws)
        cache.copy_blocks(cache.args, kv["cow_pairs"], kv["n_cow"], ws)
        if observe:
            observe(step, dict(ancestors=ancestors.view(prompts, n), resampled=resampled))
        last = tokens_out[:, :, K:].clone()
        # each particle's history goes with it through the resampling
        pick = torch.where(resampled[:, None] != 0, ancestors.view(prompts, n), torch.arange(n, device=dev)).long()
        emitted = [e.gather(1, pick[:, :, None].expand_as(e)) for e in emitted] + [tokens_out.clone()]
    for w in (step_ws, ws, ws0):
        if bits := smcsd.smc_device_status(w):
            raise RuntimeError(f"device status {smcsd.status_names(bits)}")
    used, unshared = (torch.empty(prompts, dtype=torch.int32, device=dev) for _ in range(2))
    smcsd.smc_kv_usage(params, kvs, used, unshared)
    return torch.cat(emitted, dim=2), 1 - used.sum().item() / unshared.sum().item()


def ancestor_masks(parents):
    """Packed masks [rows, words] and depths [rows] of trees given by parents
    [S, M] (-1: a child of the committed text)."""
    S, M = parents.shape
    words = -(-M // 32)
    masks, depths = [], []
    for tree in parents.tolist():
        bits, depth = [], []
        for i, p in enumerate(tree):
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        masks += [[b >> 32 * w & 0xFFFFFFFF for w in range(words)] for b in bits]
        depths += depth
    m = torch.tensor(masks, dtype=torch.int64)
    return torch.where(m >= 1 << 31, m - (1 << 32), m).to(torch.int32).cuda(), torch.tensor(depths, dtype=torch.int32).cuda()


def tree(prompts=3, M=12, vocab=512, prefix=37, rounds=4, block_size=16, seed=0, observe=None, bits=16):
    """Verifies `rounds` drafted trees of M tokens per prompt by greedy
    decoding; returns the token counts [prompts] at the end."""
    dev = "cuda"
    model = Model(vocab, seed=seed)
    slots = -(-(prefix + rounds * M + M) // block_size) + 1
    kv = make_kv_state(prompts, 1, prefix, block_size, slots, slots + 1, device=dev)
    cache = Cache(model, prompts * (slots + 1), block_size, bits)
    k, v = cache.k, cache.v
    params = smcsd.make_params(prompts, 1, 1, vocab, "f32")
    kvs = smcsd.make_kv(params, kv, block_size)
    step_ws = smcsd.alloc_workspace(params, kvs)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    batch = smcsd.make_batch(kv["tables"], kv["seq_len"], prefix)
    ws = cache.alloc_workspace(cache.args, batch, model.heads)
    model.forward(torch.randint(0, vocab, (prompts * prefix,), generator=g, device=dev), cache, batch, ws)
    batch = smcsd.make_batch(kv["tables"], kv["seq_len"], M)
    ws = cache.alloc_workspace(cache.args, batch, model.heads)
    nobody = torch.zeros(prompts, dtype=torch.int32, device=dev)
    for round_ in range(rounds):
        # a drafted tree: token i continues a random earlier one
        parents = torch.tensor([[-1 if i == 0 else int(torch.randint(0, i, (1,), generator=g, device=dev))
                                 for i in range(M)] for _ in range(prompts)])
        drafted = torch.randint(0, vocab, (prompts, M), generator=g, device=dev, dtype=torch.int32)
        committed = kv["seq_len"].view(-1).clone()
        smcsd.kv_blocktable_remap(params, kvs, nobody, nobody, M, step_ws)
        mask, depth = ancestor_masks(parents)
        positions = (committed[:, None] + depth.view(prompts, M)).reshape(-1).to(torch.int32)
        logits = model.forward(drafted.reshape(-1), cache, batch, ws, positions=positions, mask=mask)
        # an accepted path: from the first token on, a child by the logits' preference, up to 4 tokens
        path = torch.zeros((prompts, 4), dtype=torch.int32)
        n_path = torch.zeros(prompts, dtype=torch.int32)
        scores = logits.view(prompts, M, vocab).cpu()
        for s in range(prompts):
            at, taken = 0, [0]
            while len(taken) < 4:
                children = [i for i in range(M) if parents[s, i] == at]
                if not children:
                    break
                at = max(children, key=lambda i: scores[s, at, drafted[s, i].item()].item())
                taken.append(at)
            path[s, :len(taken)], n_path[s] = torch.tensor(taken, dtype=torch.int32), len(taken)
        path, n_path = path.to(dev), n_path.to(dev)
        if observe:
            observe(round_, dict(kv=kv, k=k, v=v, committed=committed, path=path, n_path=n_path, block_size=block_size,
                                 cache=cache))
        cache.compact_tokens(cache.args, batch, path, n_path, ws)
        smcsd.kv_truncate(params, kvs, committed + n_path, step_ws)
        if observe:
            observe(round_, dict(kv=kv, k=k, v=v, committed=committed, n_path=n_path, block_size=block_size, cache=cache,
                                 after=True))
    for w in (step_ws, ws):
        if bits := smcsd.smc_device_status(w):
            raise RuntimeError(f"device status {smcsd.status_names(bits)}")
    return kv["seq_len"].view(-1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompts", type=int, default=4)
    ap.add_argument("--particles", type=int, default=8)
    ap.add_argument("--steps", type=int, default=6)
    ap.add_argument("--bits", type=int, default=16, choices=(8, 16))
    a = ap.parse_args()
    tokens, saved = particles(a.prompts, a.particles, steps=a.steps, bits=a.bits)
    print(f"{a.prompts} prompts x {a.particles} particles: {tokens.shape[2]} tokens each, "
          f"{100 * saved:.0f} % fewer cache blocks than unshared copies")
    print("tokens held after four drafted trees:", tree(a.prompts, bits=a.bits).tolist())


if __name__ == "__main__":
    main()
