"""The 8-bit paged cache's operators at the edges of what their calls may say,
against 64-bit references."""
import math

import numpy as np
import pytest
import torch

import smc_speculative_decoding_gb300 as smcsd

from cache8_cases import E4M3, WEIGHT, Cache8Case, bits, compacted
from cache_cases import E32, CacheCase, half_step, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from smc_speculative_decoding_gb300 import build
    build.build()


@pytest.mark.parametrize("block,new,n", [(16, [5, 2], 90), (16, [5, 0], 90), (4, [7, 3], 100), (1, [2, 2], 100),
                                         (20, [9, 20], 64)])
def test_compact_of_a_path_longer_than_its_new_tokens(block, new, n):
    """Counts past a sequence's new tokens, in full tables: the entries past them are refused, and the table's end is
    the last slot that is looked up, whatever lies behind it (here blocks of the cache)."""
    c = Cache8Case([block, 4 * block - new[1]], new, dim=64, block=block, layers=2, spread=3)
    S, T = 2, -(-max(c.lengths) // block)
    assert c.lengths[1] == T * block  # the last sequence's table is full
    behind = torch.randint(0, c.blocks, (S * T + 200,), dtype=torch.int32, device="cuda")
    behind[:S * T] = c.tables[:, :T].reshape(-1)
    c.tables = behind[:S * T].view(S, T)
    path = [[1, 4] + [0] * (n - 2), ([1] if new[1] > 1 else [0]) + list(range(5, n + 4))]
    want = compacted(c, path)
    n_path = torch.tensor([len(p) for p in path], dtype=torch.int32, device="cuda")
    cache = c.cache(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache)
    smcsd.kv_compact_tokens8(cache, c.batch(smcsd), torch.tensor(path, dtype=torch.int32, device="cuda"), n_path, ws)
    assert smcsd.status_names(smcsd.smc_device_status(ws)) == ["bad_rows"]
    for name, x, s in (("k", c.k, c.ks), ("v", c.v, c.vs)):
        data, scale = want[name]
        assert torch.equal(s.double(), scale) and torch.equal(x.double(), data)


# ---- attention ------------------------------------------------------------------

def _beside_a_heavy_token(n, gap, dtype, noise=0.0, sequences=304, dim=64):
    """`sequences` sequences of one new token over the same n + 1 tokens: the first of them `gap` nats over the others
    and of no value, the others' scores alike (or spread by `noise`), their values positive and alike in each dim.  So
    many sequences that a multiprocessor takes whole ones: every weight has the first token's beside it."""
    g = torch.Generator().manual_seed(n)
    block, blocks = 16, -(-(n + 1) // 16)
    k, v = torch.zeros((1, blocks, block, 1, dim)), torch.zeros((1, blocks, block, 1, dim))
    k[0, 0, 0, 0, 0] = 448
    k[..., 1] = torch.randn((1, blocks, block, 1), generator=g) * 64 if noise else 0
    k[0, 0, 0, 0, 1] = 0
    grid = torch.arange(0x38, 0x38 + 46, dtype=torch.uint8).view(E4M3).float()  # 1 to 52
    v[:] = grid[torch.arange(dim) % 46]
    v[0, 0, 0] = 0
    # blocks' scales: one for all, or powers of two with the heavy token's the least of them
    size = torch.exp2(torch.randint(-3, 4, (1, blocks, 1), generator=g).float()) if noise else torch.full((1, blocks, 1), 0.25)
    size[0, 0, 0] = size.min()
    v = (v / size[..., None, None]).to(E4M3)
    k = k.to(E4M3)
    c = dict(k=k.cuda(), v=v.cuda(), ks=torch.ones_like(size).cuda(), vs=size.cuda())
    scale = 2.0 ** -12
    q = torch.zeros((sequences, 1, dim), dtype=dtype)
    q[..., 0] = gap / (448 * scale)
    q[..., 1] = noise / (64 * scale)
    table = torch.arange(blocks, dtype=torch.int32).expand(sequences, -1).contiguous()
    c.update(q=q.cuda(), scale=scale, tables=table.cuda(), seq_len=torch.full((sequences,), n + 1, dtype=torch.int32).cuda())
    kk = k.double().reshape(-1, dim)[:n + 1]
    vv = (v.double() * size.double()[..., None, None]).reshape(-1, dim)[:n + 1]
    z = scale * (kk @ q[0, 0].double())
    w = torch.exp(z - z[0])
    c.update(want=(w[1:] @ vv[1:] / w.sum()).cuda(), lse=(z[0] + w.sum().log()).item(), w=w)
    return c


# 131072 tokens are a gap of 11.8 nats' mass beside the heavy one
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,gap,noise", [(20000, 11.0, 0), (20000, 14.0, 0), (20000, 15.0, 0), (20000, 16.5, 0),
                                         (20000, 17.0, 0), (20000, 18.0, 0), (20000, 20.0, 0), (20000, 17.0, 0.5),
                                         (3000, 16.5, 0), (3000, 15.0, 1.0)])
def test_many_small_weights_beside_a_heavy_token(n, gap, noise, dtype):
    """What falls to the many keeps its size, however small each one's share.

    The output is the small weights' sum alone.  A weight is off by half of fp16's step: 2^-11 of it, or half of
    2^-24 where the heavy one is 2^8; by WEIGHT for its pieces while it is over 2^-6 there.  Less of it is a multiple
    of 2^-16, up or down by the token's place: over consecutive places these are off by a few steps in all (a golden
    ratio's multiples: at most two for each of the 26 Fibonacci numbers below 131072, so 52), not by half a step each."""
    c = _beside_a_heavy_token(n, gap, dtype, noise)
    w = c["w"][1:] * 2.0 ** 8
    small = w.clamp(max=2.0 ** -6)
    half = torch.maximum(2.0 ** -11 * w, torch.full_like(w, 2.0 ** -25)).sum() / w.sum()
    steps = 52 * 2.0 ** -16 / w.sum() if small.min() < 2.0 ** -6 else 0.0
    if noise:  # (weights of all sizes: their steps are as good as independent, 6 standard deviations of half a step)
        steps = 6 * 0.5 * 2.0 ** -16 * math.sqrt(n) / w.sum()
    score = 2 * (66 * E32 + 2.0 ** -17.8) * gap * 1.01 + 2.0 ** -19 + 2 * n * E32
    rel = (half + steps + WEIGHT + score + half_step(dtype)).item() * 1.01
    assert rel < 0.5  # an output without the small weights is off by 1
    cache = smcsd.make_cache8(c["k"], c["v"], c["ks"], c["vs"])
    batch = smcsd.make_batch(c["tables"], c["seq_len"], 1)
    ws = smcsd.alloc_cache8_workspace(cache, batch, 1)
    out, lse = torch.empty_like(c["q"]), torch.empty(c["q"].shape[:2], device="cuda")
    smcsd.smc_tree_attention8(cache, 0, batch, c["q"], out, ws, lse=lse, scale=c["scale"])
    assert smcsd.smc_device_status(ws) == 0
    off = ((out.double() - c["want"]) / c["want"]).abs().max().item()
    assert off <= rel, (off, rel)
    assert (lse.double() - c["lse"]).abs().max().item() <= score + 4 * E32 * (1 + c["lse"])


@pytest.mark.parametrize("group,sequences", [(1, 300), (4, 320)])
def test_calls_on_caches_of_both_widths_share_a_workspace(group, sequences):
    """A draft in 16 bits and a target in 8, by turns, in one workspace: each call's parts are joined whatever the
    calls before it left there."""
    wide = CacheCase([150] * sequences, [1] * sequences, heads=8, kv_heads=2, group=group,
                     shared=128 if group > 1 else 0, slots=2000 if group > 1 else 0)
    long16 = CacheCase([20000], [1], heads=8, kv_heads=8, dim=64)
    long8 = Cache8Case([20000], [1], heads=8, kv_heads=8, dim=64)
    wide8 = Cache8Case([150] * sequences, [1] * sequences, heads=8, kv_heads=2, group=group,
                       shared=128 if group > 1 else 0, slots=4000 if group > 1 else 0)
    calls = []
    for c, eight in ((wide, False), (long8, True), (long16, False), (wide8, True), (long8, True), (wide, False)):
        sizes, call = (smcsd.smc_cache8_workspace_bytes, smcsd.smc_tree_attention8) if eight else \
            (smcsd.smc_cache_workspace_bytes, smcsd.smc_tree_attention)
        cache, batch = c.cache(smcsd), c.batch(smcsd)
        out = torch.full((c.rows, c.heads, c.dim), 7.0, dtype=c.dtype, device="cuda")
        calls.append((c, call, cache, batch, out, sizes(cache, batch, c.heads)))
    ws = torch.zeros(max(call[-1] for call in calls), dtype=torch.uint8, device="cuda")
    for c, call, cache, batch, out, _ in calls:
        call(cache, 0, batch, c.q, out, ws, scale=c.scale)
    assert smcsd.smc_device_status(ws) == 0
    for c, _, _, _, out, _ in calls:
        ref, _, tol, _ = c.reference()
        assert ((out.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("q,k,scale", [(110, -90, -20), (-110, 90, 20), (118, -90, -28), (0, 60, -60)])
def test_attention_of_rows_of_any_size(q, k, scale):
    """Rows of q, scales of k and the scores' scale by powers of two that make up for one another."""
    c = Cache8Case([300, 40], [5, 9], mask="tree", spread=0)
    want = c.reference()
    c.q = c.q * 2.0 ** q
    c.ks *= 2.0 ** k
    c.scale *= 2.0 ** scale
    assert torch.isfinite(c.q).all() and c.ks.max() < 2.0 ** 100 and c.ks.min() > 2.0 ** -100
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache, batch, c.heads)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    smcsd.smc_tree_attention8(cache, 0, batch, c.q, out, ws, mask=c.mask, lse=lse, scale=c.scale)
    assert smcsd.smc_device_status(ws) == 0
    ref, ref_lse, tol, tol_lse = want
    assert ((out.double() - ref).abs() <= tol).all()
    assert ((lse.double() - ref_lse).abs() <= tol_lse).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", [-1.0, -1e20, -1e33, -1e37, 1e37])
def test_attention_of_scores_of_any_size(score, dtype):
    """Scores that are all alike, however far below or above zero: the mean of what a row sees.  Some rows see nothing
    in the first 128 tokens."""
    c = Cache8Case([0, 140], [200, 5], mask="tree", spread=0, dtype=dtype, heads=4, kv_heads=2, dim=64)
    c.seen[150], c.seen[199] = [140, 150], [199]
    c.mask = c._packed()
    bits(c.k).zero_()
    bits(c.k)[..., 0] = 0x38  # 1
    c.ks.fill_(1.0)
    c.vs.fill_(1.0)  # (what fp32 holds beside such a score is no scale of v's)
    c.q.zero_()
    zero = c.reference()
    size = 2.0 ** 15 if dtype == torch.float16 else 2.0 ** 122  # of q: the rest is the scale's
    c.q[..., 0] = math.copysign(min(abs(score), size), score)
    c.scale = abs(score) / min(abs(score), size)
    z = c.scale * c.q[0, 0, 0].item()
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache, batch, c.heads)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    smcsd.smc_tree_attention8(cache, 0, batch, c.q, out, ws, mask=c.mask, lse=lse, scale=c.scale)
    assert smcsd.smc_device_status(ws) == 0
    ref, ref_lse, tol, tol_lse = zero  # (of scores 0: alike as well)
    assert ((out.double() - ref).abs() <= tol).all()
    assert ((lse.double() - (ref_lse + z)).abs() <= tol_lse + 8 * E32 * abs(z)).all()


# ---- norms, rotation, quantised cache write ------------------------------------

def _append(c, q, k, v, table, aligned=True, **kw):
    """The case's cache after a call, its rows' addresses a vector's multiples or one element past them."""
    def place(t):
        wide = torch.empty((*t.shape[:2], t.shape[2] + 16 // t.element_size()), dtype=t.dtype, device="cuda")
        at = wide[..., :t.shape[2]] if aligned else wide[..., 1:t.shape[2] + 1]
        return at.copy_(t)
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache)
    out = torch.empty_like(q)
    kept = [t.clone() for t in (bits(c.k), bits(c.v), c.ks, c.vs)]
    smcsd.smc_qk_norm_rope8(cache, 0, batch, place(q), place(k), place(v), table, out, ws, **kw)
    assert smcsd.smc_device_status(ws) == 0
    got = [t.clone() for t in (bits(c.k), bits(c.v), c.ks, c.vs)]
    for t, old in zip((bits(c.k), bits(c.v), c.ks, c.vs), kept):
        t.copy_(old)
    return got


@pytest.mark.parametrize("dtype,dim,rot,interleaved,norm", [
    (torch.bfloat16, 128, 128, False, True), (torch.bfloat16, 64, 64, True, True), (torch.float16, 96, 64, True, True),
    (torch.float16, 256, 128, False, True), (torch.float32, 128, 128, False, True), (torch.float32, 80, 40, False, False),
    (torch.bfloat16, 128, 128, False, False), (torch.float32, 64, 64, True, False)])
def test_append_stores_the_same_whatever_the_alignment(dtype, dim, rot, interleaved, norm):
    c = Cache8Case([37, 0, 90], [900, 700, 1100], heads=8, kv_heads=8, dim=dim, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(dim)
    q, k, v = (torch.randn((c.rows, 8, dim), generator=g, device="cuda").to(dtype) for _ in range(3))
    w = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(dtype) if norm else None
    kw = dict(q_weight=w, k_weight=w, interleaved=interleaved)
    table = rope_table(1300, rot)
    for a, b in zip(_append(c, q, k, v, table, **kw), _append(c, q, k, v, table, aligned=False, **kw)):
        assert torch.equal(a, b)


def _beside_a_scale(count):
    """(a, b, cos, sin) in fp32 with a cos - b sin within a step of 448, on the one side rounded product by product and
    on the other with the second product left whole."""
    rng = np.random.default_rng(3)
    found = []
    while len(found) < count:
        angle = rng.uniform(0.3, 1.2, 4000)
        c, s = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
        b = rng.uniform(-450, -150, 4000).astype(np.float32)
        a = ((448 + b.astype(np.float64) * s) / c).astype(np.float32)
        stepwise = a * c - b * s
        whole = ((a * c).astype(np.float64) - b.astype(np.float64) * s).astype(np.float32)
        other = a * s + b * c  # the other of the pair
        for i in np.nonzero(((stepwise <= 448) != (whole <= 448)) & (np.abs(other) < 440))[0]:
            found.append((a[i], b[i], c[i], s[i], stepwise[i]))
    return np.array(found[:count], dtype=np.float32)


@pytest.mark.parametrize("aligned", [True, False])
def test_append_of_a_largest_key_beside_a_scale(aligned):
    """Its products are rounded one by one, whatever the alignment: the scale is the rounded difference's."""
    found = _beside_a_scale(60)
    c = Cache8Case([0], [60], heads=1, kv_heads=1, dim=16, dtype=torch.float32, block=1)
    k = torch.zeros((60, 1, 16))
    k[:, 0, 0], k[:, 0, 8] = torch.from_numpy(found[:, 0].copy()), torch.from_numpy(found[:, 1].copy())
    table = torch.zeros((60, 16))
    table[:, :8] = 1
    table[:, 0], table[:, 8] = torch.from_numpy(found[:, 2].copy()), torch.from_numpy(found[:, 3].copy())
    k = k.cuda()
    _, _, ks, _ = _append(c, k, k, torch.zeros_like(k), table.cuda(), aligned)
    got = ks[0, c.tables[0, :60].long(), 0].cpu().numpy()
    assert (got == np.where(found[:, 4] <= 448, 1.0, 2.0)).all()


# ---- the calls together ---------------------------------------------------------

def _step(c, cache, batch, ws, q, k, v, table, out, path, n_path, pairs, counts):
    """Drafted tokens stored and attended to, the accepted path moved, a block copied."""
    turned = torch.empty_like(q)
    smcsd.smc_qk_norm_rope8(cache, 0, batch, q, k, v, table, turned, ws)
    smcsd.smc_tree_attention8(cache, 0, batch, turned, out, ws, mask=c.mask, scale=c.scale)
    smcsd.kv_compact_tokens8(cache, batch, path, n_path, ws)
    smcsd.kv_copy_blocks8(cache, pairs, counts, ws)


def test_a_step_captured_and_replayed_is_the_step():
    c = Cache8Case([70, 33, 900], [9, 5, 12], mask="tree", spread=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    table = rope_table(1000, 128)
    make = lambda: [torch.randn((c.rows, n, 128), generator=g, device="cuda").to(c.dtype) for n in (8, 2, 2)]  # noqa: E731
    rows = make()
    path = torch.tensor([[0, 3, 8], [1, 4, -1], [5, 6, 11]], dtype=torch.int32, device="cuda")
    n_path = torch.tensor([3, 2, 3], dtype=torch.int32, device="cuda")
    free = sorted(set(range(c.blocks)) - set(c.tables.flatten().tolist()))
    pairs = torch.tensor([[[int(c.tables[0, 4]), free[0]], [int(c.tables[2, 56]), free[1]]]], dtype=torch.int32, device="cuda")
    counts = torch.tensor([2], dtype=torch.int32, device="cuda")
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache, batch, c.heads)
    out = torch.empty_like(c.q)
    held = (bits(c.k), bits(c.v), c.ks, c.vs)
    start = [t.clone() for t in held]

    def put_back():
        for t, old in zip(held, start):
            t.copy_(old)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        _step(c, cache, batch, ws, *rows, table, out, path, n_path, pairs, counts)
    for turn in range(3):
        for t, new in zip(rows, make()):
            t.copy_(new)
        n_path.copy_(torch.tensor([3 - turn, 2, 3 - turn]))
        put_back()
        _step(c, cache, batch, ws, *rows, table, out, path, n_path, pairs, counts)
        want = [t.clone() for t in (*held, out)]
        put_back()
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (*held, out)))
        assert not torch.equal(want[0], start[0])
    assert smcsd.smc_device_status(ws) == 0


def test_two_streams_at_once_with_a_workspace_each():
    """Calls that run beside one another, on caches and workspaces of their own, do not meet."""
    cases = [Cache8Case([20000, 30], [8, 3], heads=16, kv_heads=4, seed=i, mask="tree") for i in range(2)]
    calls, streams = [], [torch.cuda.Stream() for _ in cases]
    for c in cases:
        cache, batch = c.cache(smcsd), c.batch(smcsd)
        ws = smcsd.alloc_cache8_workspace(cache, batch, c.heads)
        out = torch.empty_like(c.q)
        smcsd.smc_tree_attention8(cache, 0, batch, c.q, out, ws, mask=c.mask, scale=c.scale)
        calls.append((c, cache, batch, ws, out.clone(), torch.empty_like(out)))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (c, cache, batch, ws, want, out) in zip(streams, calls):
            out.record_stream(st)
            smcsd.smc_tree_attention8(cache, 0, batch, c.q, out, ws, mask=c.mask, scale=c.scale, stream=st)
        torch.cuda.synchronize()
        for c, _, _, ws, want, out in calls:
            assert torch.equal(out, want) and smcsd.smc_device_status(ws) == 0
            out.fill_(7)
        torch.cuda.synchronize()


@pytest.mark.parametrize("block", [16, 20])
def test_blocks_past_what_32_bits_count(block):
    """A pool of more than 2^32 bytes, of which a call's blocks are the last ones: every entry point finds them."""
    blocks, kv_heads, dim = (1 << 32) // (block * 8 * 128) + 3000, 8, 128
    small = Cache8Case([333, 60], [7, 9], heads=8, kv_heads=kv_heads, dim=dim, block=block, spread=2)
    # the same call in a small pool and in the large one, whose last blocks stand for the small one's
    shift = blocks - small.blocks
    big_k, big_v = (torch.zeros((1, blocks, block, kv_heads, dim), dtype=torch.uint8, device="cuda") for _ in range(2))
    big_k[:, shift:], big_v[:, shift:] = bits(small.k), bits(small.v)
    big_ks, big_vs = (torch.ones((1, blocks, kv_heads), device="cuda") for _ in range(2))
    big_ks[:, shift:], big_vs[:, shift:] = small.ks, small.vs
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((small.rows, 8, dim), generator=g, device="cuda").to(small.dtype) for _ in range(3))
    path = torch.tensor([[2, 5], [0, 7]], dtype=torch.int32, device="cuda")
    n_path = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    free = sorted(set(range(small.blocks)) - set(small.tables.flatten().tolist()))
    counts = torch.tensor([1], dtype=torch.int32, device="cuda")
    table, outs = rope_table(400, dim), []
    for cache, at in ((small.cache(smcsd), 0), (smcsd.make_cache8(big_k.view(E4M3), big_v.view(E4M3), big_ks, big_vs), shift)):
        tables = torch.where(small.tables < 0, -1, small.tables + at).to(torch.int32)
        batch = smcsd.make_batch(tables, small.seq_len, small.max_new, row_start=small.row_start, rows=small.rows)
        pairs = torch.tensor([[[int(tables[0, 3]), free[0] + at]]], dtype=torch.int32, device="cuda")
        ws = smcsd.alloc_cache8_workspace(cache, batch, 8)
        out = torch.empty_like(q)
        _step(small, cache, batch, ws, q, k, v, table, out, path, n_path, pairs, counts)
        assert smcsd.smc_device_status(ws) == 0
        outs.append(out)
    assert torch.equal(*outs)
    assert torch.equal(big_k[:, shift:], bits(small.k)) and torch.equal(big_v[:, shift:], bits(small.v))
    assert torch.equal(big_ks[:, shift:], small.ks) and torch.equal(big_vs[:, shift:], small.vs)
    assert not big_k[:, :shift].any() and torch.all(big_ks[:, :shift] == 1)
