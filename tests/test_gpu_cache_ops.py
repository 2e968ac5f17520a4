"""The paged cache's operators on the GPU against 64-bit references: tree
attention, norms with rotation and cache write, block copies, path compaction
and truncation."""
import math

import numpy as np
import pytest
import torch

import smc_speculative_decoding_gb300 as smcsd
from smc_speculative_decoding_gb300.workloads import make_kv_state

from cache_cases import CacheCase, qk_reference, rope_table
from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from smc_speculative_decoding_gb300 import build
    build.build()


def _attend(c, batch=None, lse=True, out=None, stream=None, workspace=None, **kw):
    cache = c.cache(smcsd)
    batch = c.batch(smcsd) if batch is None else batch
    ws = smcsd.alloc_cache_workspace(cache, batch, c.heads) if workspace is None else workspace
    out = torch.full((c.rows, c.heads, c.dim), 7.0, dtype=c.dtype, device="cuda") if out is None else out
    lses = torch.full((c.rows, c.heads), 7.0, device="cuda") if lse else None
    smcsd.smc_tree_attention(cache, c.layer, batch, c.q, out, ws, mask=c.mask, lse=lses,
                             scale=c.scale, stream=stream, **kw)
    return out, lses, ws


def _check_attention(c, out, lse, ws):
    assert smcsd.smc_device_status(ws) == 0
    ref, ref_lse, tol, tol_lse = c.reference()
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse), empty) and torch.all(lse[empty] == -math.inf)
    assert torch.all(out[empty] == 0)
    assert torch.isfinite(out).all()
    excess = ((out.double() - ref).abs() - tol).max().item() if ref.numel() else 0
    assert excess <= 0, f"out is {excess} past its bound"
    off = (lse.double() - ref_lse).abs()[~empty] - tol_lse[~empty]
    assert not off.numel() or off.max().item() <= 0


SHAPES = [
    # ctx, new, keywords
    ([5], [1], {}),
    ([0], [1], {}),
    ([127], [1], {}),
    ([128], [1], {}),
    ([129, 1, 640], [3, 1, 5], {}),
    ([300, 0, 17, 256], [5, 5, 0, 2], dict(mask="tree")),
    ([0, 3], [40, 33], dict(mask="tree")),
    ([0, 0, 200], [6, 1, 9], dict(mask="holes")),
    ([0, 70], [4, 4], dict(mask="none")),
    ([1000], [64], dict(mask="tree", heads=16, kv_heads=2)),       # 512 rows of a key head
    ([700, 100], [70, 65], dict(mask="tree", heads=8, kv_heads=4)),  # masks of three words
    ([513, 90], [200, 170], dict(heads=4, kv_heads=2)),            # rows past one tile, chain
    ([2000], [1], dict(heads=64, kv_heads=1)),
    ([260, 31], [7, 2], dict(heads=6, kv_heads=2, dim=64)),        # three heads of a key head
    ([260, 31], [7, 2], dict(heads=5, kv_heads=5, dim=80, mask="tree")),
    ([260, 31], [7, 2], dict(heads=4, kv_heads=1, dim=96)),
    ([260, 31], [7, 2], dict(heads=4, kv_heads=2, dim=8)),
    ([260, 31], [7, 2], dict(heads=4, kv_heads=2, dim=40)),
    ([400], [11], dict(block=1)),
    ([400, 9], [11, 3], dict(block=20)),
    ([400, 9], [11, 3], dict(block=24)),
    ([400, 9], [11, 3], dict(block=256)),
    ([400, 9], [11, 3], dict(block=136)),
    ([3000], [4], dict(block=64, heads=4, kv_heads=4)),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ctx,new,kw", SHAPES)
def test_attention(ctx, new, kw, dtype):
    c = CacheCase(ctx, new, dtype=dtype, poison=True, seed=len(ctx) + sum(ctx), **kw)
    _check_attention(c, *_attend(c))


@pytest.mark.parametrize("order,strided,block", [("hnd", False, 16), ("nhd", True, 16),
                                                 ("hnd", True, 20), ("hnd", False, 64)])
def test_attention_memory_orders(order, strided, block):
    c = CacheCase([200, 60], [6, 9], order=order, strided=strided, block=block, layers=3, layer=2,
                  mask="tree", poison=True)
    _check_attention(c, *_attend(c))


@pytest.mark.parametrize("group,shared,ctx,new", [
    (4, 512, [600, 512, 700, 530], [5, 5, 5, 5]),
    (2, 100, [100, 110, 300, 100], [3, 2, 1, 4]),   # less than one tile is shared
    (8, 640, [650] * 8 + [700] * 8, [17] * 16),     # more rows than one tile over the shared part
    (3, 0, [50, 60, 70], [2, 2, 2]),
    (2, 384, [384, 384], [1, 0]),
    (4, 256, [300, 290, 280, 310, 0, 5, 0, 1], [0, 3, 0, 2, 1, 1, 0, 2]),  # one prompt shares nothing
    (2, 1024, [1100, 1030], [30, 35]),
])
@pytest.mark.parametrize("mask", ["chain", "tree"])
@pytest.mark.parametrize("slots", [0, 3100])  # tables as large as those whose shared blocks are read once
def test_attention_shared_prefix(group, shared, ctx, new, mask, slots):
    shared = min([shared] + [c for c in ctx if shared and c >= shared]) if shared else 0
    ctx = [max(c, shared) if i // group == 0 else c for i, c in enumerate(ctx)]
    one = any(c < shared for c in ctx)
    c = CacheCase(ctx, new, group=group, shared=0 if one else shared, heads=8, kv_heads=2, mask=mask, poison=True,
                  slots=slots)
    if one:  # only the first prompt's sequences share their leading blocks
        n = shared // c.block
        c.tables[1:group, :n] = c.tables[:1, :n]
    out, lse, ws = _attend(c)
    _check_attention(c, out, lse, ws)
    again, lse2, _ = _attend(c, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("other", ["ended", "other_blocks"])
@pytest.mark.parametrize("group,shared,ctx,new", [
    (4, 512, [600, 512, 700, 530], [0, 5, 5, 5]),                        # the first has no rows
    (4, 256, [300, 300, 270, 290] * 2, [0, 0, 3, 2, 4, 0, 1, 2]),        # the first two of a prompt; one in the middle
    (3, 640, [650, 700, 690] * 2, [0, 1, 0, 0, 40, 40]),                 # a prompt with one sequence left
])
@pytest.mark.parametrize("slots", [0, 3100])
def test_attention_shared_prefix_beside_sequences_without_rows(group, shared, ctx, new, other, slots):
    """Sequences without new tokens have no say in what a prompt's others share: their tables may be given back
    (-1) or lead to other blocks."""
    c = CacheCase(ctx, new, group=group, shared=shared, mask="tree", slots=slots)
    want = CacheCase(ctx, new, group=group, shared=shared, mask="tree", slots=slots).reference()
    n = shared // c.block
    for s, m in enumerate(new):
        if m:
            continue
        if other == "ended":
            c.tables[s], c.seq_len[s] = -1, 0
        else:
            c.tables[s, :n] = c.tables[s, 0].clone()  # (an order of the same blocks would give the same result)
    out, lse, ws = _attend(c)
    assert smcsd.status_names(smcsd.smc_device_status(ws)) == []
    ref, ref_lse, tol, tol_lse = want
    assert ((out.double() - ref).abs() <= tol).all()
    assert ((lse.double() - ref_lse).abs() <= tol_lse).all()
    again, lse2, _ = _attend(c, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("sequences,group,new,low,high,kw", [
    (150, 1, 1, 0, 260, dict()),                     # units that end inside a multiprocessor's run, joined in it
    (150, 1, 5, 60, 200, dict(mask="tree", block=20)),  # element copies
    (270, 1, 3, 1, 130, dict(dim=64)),               # more sequences than are counted without a plan
    (160, 16, 5, 100, 400, dict(slots=700)),         # own parts after a shared one
    (96, 1, 40, 0, 300, dict(kv_heads=8, heads=24)),  # units of one row tile and of two, by turns
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_many_short(sequences, group, new, low, high, kw, dtype):
    """More units than multiprocessors: several to each, of like and of unlike lengths."""
    ctx = [low + 37 * i * i % (high - low + 1) for i in range(sequences)]
    news = [1 + (i * 7) % (2 * new) if new > 1 else 1 for i in range(sequences)]
    shared = min(ctx) // 16 * 16 if group > 1 else 0
    c = CacheCase(ctx, news, group=group, shared=shared, dtype=dtype, poison=True,
                  **{"heads": 8, "kv_heads": 4, **kw})
    out, lse, ws = _attend(c)
    _check_attention(c, out, lse, ws)
    again, lse2, _ = _attend(c, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("news,low,high,kw", [
    ([2, 2, 3, 40], 0, 60, {}),             # tiles that reach past the committed tokens from the first on
    ([1, 5, 5, 64, 33], 0, 400, {}),
    ([1, 2, 60], 0, 150, dict(dim=64)),
    ([2, 40, 1, 1], 30, 200, dict(block=20)),  # element copies
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_of_two_row_tiles_behind_units_side_by_side(news, low, high, kw, dtype):
    """Several units to a multiprocessor: short ones side by side, then one whose tiles both softmax groups use."""
    ctx = [low + 53 * i * i % (high - low + 1) for i in range(160)]
    c = CacheCase(ctx, [news[i % len(news)] for i in range(160)], mask="tree", dtype=dtype, poison=True, sigma=3.0,
                  heads=8, kv_heads=2, **kw)
    out, lse, ws = _attend(c)
    _check_attention(c, out, lse, ws)
    for _ in range(3):
        again, lse2, _ = _attend(c, workspace=ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def _check_like_double(c, out, lse):
    """Against torch in 64 bits on padded tensors: for shapes that the loops
    of the reference would take long over."""
    S, T, rep = len(c.ctx), c.tables.shape[1] * c.block, c.heads // c.kv_heads
    at = torch.arange(T, device="cuda")[None].expand(S, -1)
    slot = c.tables.long().clamp(min=0).gather(1, at // c.block)
    k, v = (x[c.layer][slot, at % c.block].double() for x in (c.k, c.v))
    held = at < c.seq_len[:, None]
    for b in range(S):
        r0, r1, n = int(c.starts[b]), int(c.starts[b + 1]), c.lengths[b]
        if r0 == r1:
            continue
        q = c.q[r0:r1].double().unflatten(1, (c.kv_heads, rep))
        z = torch.einsum("rhgd,thd->rhgt", q, k[b, :n]) * c.scale
        sees = torch.zeros((r1 - r0, n), dtype=torch.bool, device="cuda")
        sees[:, :c.ctx[b]] = True
        for r in range(r0, r1):
            cols = list(range(r - r0 + 1)) if c.seen is None else c.seen[r]
            sees[r - r0, [c.ctx[b] + j for j in cols]] = True
        z = z.masked_fill(~sees[:, None, None], -math.inf)
        p = torch.softmax(z, -1)
        want = torch.einsum("rhgt,thd->rhgd", p, v[b, :n])
        mag = torch.einsum("rhgt,thd->rhgd", p, v[b, :n].abs())
        u = torch.finfo(c.dtype).eps / 2
        got = out[r0:r1].double().unflatten(1, (c.kv_heads, rep))
        # weights and result rounded once each, fp32 scores and sums
        assert ((got - want).abs() <= 1.01 * u * (mag + want.abs()) + 1e-3 * u * mag + 2.0 ** -17 * mag).all()
        got = lse[r0:r1].double().unflatten(1, (c.kv_heads, rep))
        assert ((got - torch.logsumexp(z, -1)).abs() <= 1e-5).all()


@pytest.mark.parametrize("ctx,new,kw", [
    ([3000, 9000, 500, 0, 6400, 77], [5, 64, 1, 30, 128, 2], dict(mask="tree", heads=32, kv_heads=8)),
    ([20000, 100], [8, 8], dict(mask="tree", heads=64, kv_heads=8, block=64)),
    ([1500] * 40, [16] * 40, dict(heads=16, kv_heads=4, block=32)),
    ([900, 1100, 1300, 700] * 12, [5] * 48, dict(heads=16, kv_heads=4, group=4, shared=640)),
    ([900, 1100, 1300, 700] * 12, [5] * 48, dict(heads=16, kv_heads=4, group=4, shared=640, slots=400)),
    ([700] * 48, [70] * 48, dict(heads=16, kv_heads=4, group=16, shared=512, slots=400, mask="tree")),
    ([130] * 400, [1] * 400, dict(heads=8, kv_heads=2)),           # more sequences than one CTA counts
    ([3000] * 3, [40] * 3, dict(heads=12, kv_heads=4, dim=64, mask="tree")),
    ([2500, 40], [30, 30], dict(heads=24, kv_heads=1, dim=96, block=20, mask="tree")),  # odd blocks: element copies
    ([5000], [2], dict(heads=128, kv_heads=1)),                     # as many heads as a row tile holds
])
def test_attention_of_larger_batches(ctx, new, kw):
    c = CacheCase(ctx, new, poison=False, **kw)
    out, lse, ws = _attend(c)
    assert smcsd.smc_device_status(ws) == 0
    _check_like_double(c, out, lse)
    again, lse2, _ = _attend(c, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_attention_of_many_sequences():
    rng = np.random.default_rng(3)
    ctx, new = rng.integers(0, 300, 300).tolist(), rng.integers(0, 4, 300).tolist()
    c = CacheCase(ctx, new, heads=2, kv_heads=1, dim=64)
    _check_attention(c, *_attend(c))


def test_attention_of_a_long_cache():
    c = CacheCase([40000], [3], heads=4, kv_heads=2, block=64, mask="tree")
    _check_attention(c, *_attend(c))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_attention_ignores_what_a_row_does_not_see(value):
    """A new token that holds NaN or infinities reaches only the rows that see
    it."""
    c = CacheCase([150, 10], [9, 9], mask="tree", heads=8, kv_heads=2)
    bad, s = 4, 1
    at = c.ctx[s] + bad
    c.v[0, c.tables[s, at // c.block], at % c.block] = value
    out, lse, ws = _attend(c)
    clean = CacheCase([150, 10], [9, 9], mask="tree", heads=8, kv_heads=2)
    ref, ref_lse, tol, tol_lse = clean.reference()
    for r in range(c.rows):
        seen = r >= c.starts[s] and bad in c.seen[r]
        if seen:
            assert not torch.isfinite(out[r]).any()
            if not math.isnan(value):
                assert torch.all(out[r] == value)
        else:
            assert ((out[r].double() - ref[r]).abs() <= tol[r]).all()
    # a key likewise
    c = CacheCase([150, 10], [9, 9], mask="tree", heads=8, kv_heads=2)
    c.k[0, c.tables[s, at // c.block], at % c.block] = value
    out, lse, ws = _attend(c)
    for r in range(c.rows):
        if not (r >= c.starts[s] and bad in c.seen[r]):
            assert ((out[r].double() - ref[r]).abs() <= tol[r]).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx,new,bad,kw", [
    ([150, 10], [9, 40], 3, dict(heads=8)),            # 160 rows of a key head: two row tiles, one of them in part
    ([0, 30], [50, 64], 5, dict(heads=8)),            # 256 rows; the tile before the last one holds the token
    ([9000], [48], 1, dict(heads=8)),                 # cut between multiprocessors
    ([700, 90], [33, 60], 0, dict(heads=12, dim=64)),  # six heads of a key head: units of 252 rows and of the rest
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_of_two_row_tiles_ignores_what_a_row_does_not_see(ctx, new, bad, kw, value, dtype):
    """Both softmax groups read the tile of V that holds the token, and either may be the one that zeroes it."""
    s = len(ctx) - 1
    at = ctx[s] + bad
    c = CacheCase(ctx, new, mask="tree", kv_heads=2, dtype=dtype, **kw)
    ref, _, tol, _ = c.reference()
    c.v[0, c.tables[s, at // c.block], at % c.block] = value
    out, lse, ws = _attend(c)
    sees = torch.tensor([r >= c.starts[s] and bad in c.seen[r] for r in range(c.rows)], device="cuda")
    assert sees.any() and not sees.all()
    if math.isnan(value):
        assert torch.isnan(out[sees]).all()
    else:
        assert torch.all(out[sees] == value)
    assert ((out.double() - ref).abs() <= tol)[~sees].all()
    again, _, _ = _attend(c, workspace=ws)
    assert torch.equal(torch.nan_to_num(out, nan=7.0), torch.nan_to_num(again, nan=7.0))


def test_attention_of_large_scores():
    """Scores of several hundred: only differences from the maximum matter."""
    c = CacheCase([300, 40], [5, 5], sigma=20.0, mask="tree")
    _check_attention(c, *_attend(c))


def test_attention_rows_past_the_last_sequence_are_untouched():
    c = CacheCase([100, 50], [3, 2])
    rows = c.rows + 4
    q = torch.cat([c.q, torch.full((4, c.heads, c.dim), float("nan"), dtype=c.dtype, device="cuda")])
    cache = c.cache(smcsd)
    batch = smcsd.make_batch(c.tables, c.seq_len, c.max_new, row_start=c.row_start, rows=rows)
    ws = smcsd.alloc_cache_workspace(cache, batch, c.heads)
    out = torch.full((rows, c.heads, c.dim), 7.0, dtype=c.dtype, device="cuda")
    lse = torch.full((rows, c.heads), 7.0, device="cuda")
    smcsd.smc_tree_attention(cache, 0, batch, q, out, ws, lse=lse, scale=c.scale)
    _check_attention(c, out[:c.rows], lse[:c.rows], ws)
    assert torch.all(out[c.rows:] == 7) and torch.all(lse[c.rows:] == 7)


def test_attention_is_repeatable_and_leaves_its_workspace_reusable():
    c = CacheCase([5000, 900], [6, 40], mask="tree", heads=16, kv_heads=4)
    out, lse, ws = _attend(c)
    for _ in range(5):
        again, lse2, _ = _attend(c, workspace=ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert smcsd.smc_device_status(ws) == 0


def test_attention_uniform_batch_without_lse_on_another_stream():
    c = CacheCase([333, 20, 64], [4, 4, 4])
    want, _, _ = _attend(c)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, lse, ws = _attend(c, batch=c.batch(smcsd, uniform=True), lse=False, stream=st)
    st.synchronize()
    assert lse is None and torch.equal(got, want)


def test_attention_in_a_cuda_graph():
    """A captured call reads lengths, tables and masks at its replay."""
    c = CacheCase([700, 90], [5, 5], mask="tree")
    d = CacheCase([500, 100], [5, 5], mask="tree", seed=5)  # fits the pool of c
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache_workspace(cache, batch, c.heads)
    out, lse, _ = _attend(c, batch=batch, workspace=ws)
    out, lse = torch.empty_like(out), torch.empty_like(lse)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        smcsd.smc_tree_attention(cache, 0, batch, c.q, out, ws, mask=c.mask, lse=lse, scale=c.scale)
    g.replay()
    torch.cuda.synchronize()
    _check_attention(c, out, lse, ws)
    n = min(c.k.shape[1], d.k.shape[1])
    assert n >= int(d.tables.max()) + 1
    c.k[:, :n], c.v[:, :n], c.q[:] = d.k[:, :n], d.v[:, :n], d.q
    c.mask[:], c.seq_len[:] = d.mask, d.seq_len
    width = min(c.tables.shape[1], d.tables.shape[1])
    c.tables[:, :width] = d.tables[:, :width]
    g.replay()
    torch.cuda.synchronize()
    _check_attention(d, out, lse, ws)


def test_attention_reports_bad_state_and_touches_nothing_else():
    c = CacheCase([100, 50], [3, 2])
    cases = []
    t = c.tables.clone()
    t[0, 1] = c.blocks
    cases.append((dict(tables=t), "bad_block"))
    t = c.tables.clone()
    t[1, 0] = -1
    cases.append((dict(tables=t), "bad_block"))
    cases.append((dict(seq_len=torch.tensor([100000, 52], dtype=torch.int32, device="cuda")), "bad_block"))
    cases.append((dict(seq_len=torch.tensor([103, 1], dtype=torch.int32, device="cuda")), "bad_block"))
    cases.append((dict(seq_len=torch.tensor([-5, 52], dtype=torch.int32, device="cuda")), "bad_block"))
    cases.append((dict(row_start=torch.tensor([0, 3, 9], dtype=torch.int32, device="cuda")), "bad_rows"))
    cases.append((dict(row_start=torch.tensor([0, 4, 5], dtype=torch.int32, device="cuda")), "bad_rows"))
    cases.append((dict(row_start=torch.tensor([3, 0, 5], dtype=torch.int32, device="cuda")), "bad_rows"))
    cache = c.cache(smcsd)
    out = torch.empty((c.rows, c.heads, c.dim), dtype=c.dtype, device="cuda")
    for kw, bit in cases:
        kw = dict(tables=c.tables, seq_len=c.seq_len, row_start=c.row_start) | kw
        batch = smcsd.make_batch(kw["tables"], kw["seq_len"], 3, row_start=kw["row_start"], rows=c.rows)
        ws = smcsd.alloc_cache_workspace(cache, batch, c.heads)
        smcsd.smc_tree_attention(cache, 0, batch, c.q, out, ws, scale=c.scale)
        torch.cuda.synchronize()
        assert bit in smcsd.status_names(smcsd.smc_device_status(ws, clear=True)), (kw, bit)
        batch = c.batch(smcsd)  # the same workspace serves the next call
        smcsd.smc_tree_attention(cache, 0, batch, c.q, out, ws, scale=c.scale)
        ref, _, tol, _ = c.reference()
        assert ((out.double() - ref).abs() <= tol).all()
        assert smcsd.smc_device_status(ws) == 0


# ---- norms, rotation, cache write -------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim,rot,interleaved,norm,offset,kw", [
    (128, 128, False, True, 0.0, {}),
    (128, 64, True, True, 0.0, dict(order="hnd")),
    (64, 64, True, False, 0.0, dict(block=20)),
    (96, 96, False, True, 1.0, dict(strided=True)),
    (80, 40, False, True, 0.0, {}),
    (72, 24, False, True, 0.0, {}),
    (128, 0, False, True, 0.0, {}),
    (256, 256, False, True, 0.0, {}),
    (256, 32, True, True, 0.0, {}),
    (14, 6, True, True, 0.0, {}),
    (33, 10, False, True, 0.0, {}),
    (1, 0, False, True, 0.0, {}),
])
def test_qk_norm_rope(dim, rot, interleaved, norm, offset, kw, dtype):
    c = CacheCase([37, 0, 90], [5, 1, 7], heads=6, kv_heads=2, dim=dim, dtype=dtype, layers=2, layer=1, **kw)
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((c.rows, 10 * dim), generator=g, device="cuda").to(dtype)
    q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([6 * dim, 2 * dim, 2 * dim], dim=1))
    qw, kw_ = ((torch.randn(dim, generator=g, device="cuda") * 0.3 + 1 - offset).to(dtype) for _ in range(2))
    if not norm:
        qw = kw_ = None
    table = rope_table(200, rot)
    pos = torch.randint(0, 200, (c.rows,), generator=g, device="cuda").to(torch.int32)
    before = (c.k.clone(), c.v.clone())
    own = torch.cat([torch.arange(a, a + m) for a, m in zip(c.ctx, c.new)]).to(torch.int32).cuda()
    for positions in (pos, None):
        cache, batch = c.cache(smcsd), c.batch(smcsd)
        ws = smcsd.alloc_cache_workspace(cache)
        out = torch.empty((c.rows, 6, dim), dtype=dtype, device="cuda")
        smcsd.smc_qk_norm_rope(cache, 1, batch, q, k, v, table, out, ws, positions=positions,
                               q_weight=qw, k_weight=kw_, eps=1e-5, weight_offset=offset,
                               interleaved=interleaved)
        assert smcsd.smc_device_status(ws) == 0
        at = own if positions is None else positions
        for got, x, w in ((out, q, qw), (None, k, kw_)):
            ref, tol = qk_reference(x, w, table, at, rot, interleaved, 1e-5, offset)
            if got is None:
                got = torch.stack([c.k[1, c.tables[s, p // c.block], p % c.block]
                                   for s in range(3) for p in range(c.ctx[s], c.lengths[s])])
            assert ((got.double() - ref).abs() <= tol).all()
    stored = torch.stack([c.v[1, c.tables[s, p // c.block], p % c.block]
                          for s in range(3) for p in range(c.ctx[s], c.lengths[s])])
    assert torch.equal(stored, v)
    # nothing but the new tokens' slots of this layer changed
    for now, old in ((c.k, before[0]), (c.v, before[1])):
        for s in range(3):
            for p in range(c.ctx[s], c.lengths[s]):
                b = c.tables[s, p // c.block]
                now[1, b, p % c.block] = old[1, b, p % c.block]
        assert torch.equal(now, old)


def test_qk_in_place_far_positions_and_bad_rows():
    c = CacheCase([3, 8], [2, 3], heads=4, kv_heads=2, dim=128)
    x = torch.randn((c.rows, 4, 128), device="cuda").to(c.dtype)
    k, v = (torch.randn((c.rows, 2, 128), device="cuda").to(c.dtype) for _ in range(2))
    table = rope_table(70000, 128)
    pos = torch.tensor([69999, 65535, 0, 70000, -1], dtype=torch.int32, device="cuda")
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache_workspace(cache)
    ref, tol = qk_reference(x[:3], None, table, pos[:3], 128, False, 1e-6, 0.0)
    want = x.clone()
    smcsd.smc_qk_norm_rope(cache, 0, batch, x, k, v, table, x, ws, positions=pos)
    assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_rows"]
    assert ((x[:3].double() - ref).abs() <= tol).all() and torch.equal(x[3:], want[3:])
    c.tables[0, 0] = c.blocks + 5
    smcsd.smc_qk_norm_rope(cache, 0, batch, x, k, v, table, x, ws)
    assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_block"]


@pytest.mark.parametrize("heads,kv_heads,dim,norm_q,norm_k", [
    (32, 8, 128, True, False), (32, 8, 128, False, True), (71, 1, 64, True, True), (3, 3, 96, False, True),
    (64, 64, 128, True, True), (1, 1, 8, True, True), (100, 4, 256, True, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_qk_heads_and_one_norm(heads, kv_heads, dim, norm_q, norm_k, dtype):
    c = CacheCase([20, 3, 64, 0], [4, 4, 1, 3], heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(heads)
    q, k, v = (torch.randn((c.rows, n, dim), generator=g, device="cuda").to(dtype) for n in (heads, kv_heads, kv_heads))
    w = (torch.randn(dim, generator=g, device="cuda") * 0.2 + 1).to(dtype)
    table = rope_table(100, dim)
    own = torch.cat([torch.arange(a, a + m) for a, m in zip(c.ctx, c.new)]).to(torch.int32).cuda()
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache_workspace(cache)
    out = torch.empty_like(q)
    smcsd.smc_qk_norm_rope(cache, 0, batch, q, k, v, table, out, ws, q_weight=w if norm_q else None,
                           k_weight=w if norm_k else None)
    assert smcsd.smc_device_status(ws) == 0
    at = [(c.tables[s, p // c.block], p % c.block) for s in range(4) for p in range(c.ctx[s], c.lengths[s])]
    stored = torch.stack([c.k[0, b, o] for b, o in at])
    for got, x, normed in ((out, q, norm_q), (stored, k, norm_k)):
        ref, tol = qk_reference(x, w if normed else None, table, own, dim, False, 1e-6, 0.0)
        assert ((got.double() - ref).abs() <= tol).all()
    assert torch.equal(torch.stack([c.v[0, b, o] for b, o in at]), v)


def test_qk_rows_of_zeros_and_infinities():
    """A zero row has no direction: eps keeps it 0; a row with an infinity is
    NaN, as its formula is."""
    c = CacheCase([3], [3], heads=2, kv_heads=1, dim=64)
    q = torch.zeros((3, 2, 64), dtype=c.dtype, device="cuda")
    q[1, 0, 5] = float("inf")
    k = torch.zeros((3, 1, 64), dtype=c.dtype, device="cuda")
    w = torch.ones(64, dtype=c.dtype, device="cuda")
    out = torch.empty_like(q)
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache_workspace(cache)
    smcsd.smc_qk_norm_rope(cache, 0, batch, q, k, k, rope_table(10, 64), out, ws, q_weight=w, k_weight=w)
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0) and torch.all(out[1, 1] == 0)
    assert torch.isnan(out[1, 0, 5])


# ---- blocks -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,block,kw", [(128, 16, {}), (64, 24, dict(order="hnd")),
                                          (80, 5, dict(strided=True)), (3, 7, {}), (1, 1, {}),
                                          (128, 256, dict(layers=1))])
def test_copy_blocks(dim, block, kw, dtype):
    c = CacheCase([block * 9] * 3, [1] * 3, dim=dim, block=block, dtype=dtype, **({"layers": 3} | kw))
    before = c.k.clone(), c.v.clone()
    ids = torch.randperm(c.blocks)[:16].to(torch.int32)
    pairs = torch.stack([ids[:8], ids[8:]], 1).view(2, 4, 2).contiguous().cuda()
    counts = torch.tensor([4, 2], dtype=torch.int32, device="cuda")
    cache = c.cache(smcsd)
    ws = smcsd.alloc_cache_workspace(cache)
    smcsd.kv_copy_blocks(cache, pairs, counts, ws)
    assert smcsd.smc_device_status(ws) == 0
    for old in before:
        for lst, n in enumerate((4, 2)):
            for src, dst in pairs[lst, :n].tolist():
                old[:, dst] = old[:, src]
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])


def test_copy_blocks_reports_bad_pairs_and_counts():
    c = CacheCase([64], [1], layers=2)
    cache = c.cache(smcsd)
    ws = smcsd.alloc_cache_workspace(cache)
    before = c.k.clone()
    pairs = torch.tensor([[[0, c.blocks], [1, 2]], [[-1, 0], [0, 0]]], dtype=torch.int32, device="cuda")
    smcsd.kv_copy_blocks(cache, pairs, torch.tensor([2, 0], dtype=torch.int32, device="cuda"), ws)
    assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_block"]
    before[:, 2] = before[:, 1]
    assert torch.equal(c.k, before)
    for bad in (3, -1):
        smcsd.kv_copy_blocks(cache, pairs, torch.tensor([0, bad], dtype=torch.int32, device="cuda"), ws)
        assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_rows"]
    assert torch.equal(c.k, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,block,kw", [(128, 16, {}), (64, 24, dict(order="hnd")),
                                          (80, 5, dict(strided=True)), (3, 7, {}), (128, 1, {})])
def test_compact_tokens(dim, block, kw, dtype):
    rng = np.random.default_rng(dim)
    new = [40, 1, 9, 17, 33]
    c = CacheCase([33, 0, 7, 100, 16], new, dim=dim, block=block, dtype=dtype, layers=3, **kw)
    most = 33
    path = [sorted(rng.choice(m, rng.integers(0, m + 1), replace=False).tolist()) for m in new]
    path[4] = list(range(33))  # the whole chain: nothing moves
    path[0] = list(range(7, 40))
    n_path = torch.tensor([len(p) for p in path], dtype=torch.int32, device="cuda")
    padded = torch.tensor([p + [-1] * (most - len(p)) for p in path], dtype=torch.int32, device="cuda")
    before = c.k.clone(), c.v.clone()
    want = c.k.clone(), c.v.clone()
    for s, p in enumerate(path):
        for i, j in enumerate(p):
            a, b = c.ctx[s] + j, c.ctx[s] + i
            for w, old in zip(want, before):
                w[:, c.tables[s, b // block], b % block] = old[:, c.tables[s, a // block], a % block]
    cache = c.cache(smcsd)
    ws = smcsd.alloc_cache_workspace(cache)
    smcsd.kv_compact_tokens(cache, c.batch(smcsd), padded, n_path, ws)
    assert smcsd.smc_device_status(ws) == 0
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])


def test_compact_of_long_paths():
    """Paths longer than the moves that one pass places."""
    rng = np.random.default_rng(8)
    new = [300, 200]
    c = CacheCase([5, 31], new, dim=64, layers=2, block=16)
    path = [sorted(rng.choice(300, 190, replace=False).tolist()), sorted(rng.choice(200, 65, replace=False).tolist())]
    n_path = torch.tensor([len(p) for p in path], dtype=torch.int32, device="cuda")
    padded = torch.tensor([p + [0] * (200 - len(p)) for p in path], dtype=torch.int32, device="cuda")
    before = c.k.clone(), c.v.clone()
    want = c.k.clone(), c.v.clone()
    for s, p in enumerate(path):
        for i, j in enumerate(p):
            a, b = c.ctx[s] + j, c.ctx[s] + i
            for w, old in zip(want, before):
                w[:, c.tables[s, b // 16], b % 16] = old[:, c.tables[s, a // 16], a % 16]
    cache = c.cache(smcsd)
    ws = smcsd.alloc_cache_workspace(cache)
    smcsd.kv_compact_tokens(cache, c.batch(smcsd), padded, n_path, ws)
    assert smcsd.smc_device_status(ws) == 0
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])
    # a bad index deep in a path is reported, whichever pass it falls in
    for at in (3, 63, 64, 70, 189):
        bad = padded.clone()
        bad[0, at] = bad[0, at - 1]
        smcsd.kv_compact_tokens(cache, c.batch(smcsd), bad, n_path, ws)
        assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_rows"], at


def test_compact_reports_bad_paths():
    c = CacheCase([5, 6], [4, 4])
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache_workspace(cache)
    n = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    for path in ([[3, 4], [0, 0]], [[2, 1], [0, 0]], [[-1, 1], [0, 0]], [[2, 2], [0, 0]]):
        smcsd.kv_compact_tokens(cache, batch, torch.tensor(path, dtype=torch.int32, device="cuda"), n, ws)
        assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_rows"], path
    smcsd.kv_compact_tokens(cache, batch, torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device="cuda"),
                            torch.tensor([3, -1], dtype=torch.int32, device="cuda"), ws)
    assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_rows"]


@pytest.mark.parametrize("dim,block,kw", [(64, 16, {}), (3, 7, {}), (64, 4, dict(order="hnd")), (128, 1, {})])
def test_compact_skips_bad_entries_and_touches_nothing_else(dim, block, kw):
    """Entries that are out of range, do not ascend, or lie ahead of their place are skipped alone; paths may be
    longer than the new tokens, whose last sequence fills its table and the pool."""
    rng = np.random.default_rng(block)
    new = [2, 30, 0, 9, 2]
    ctx = [5, 31, 7, 0, 4 * block - 2]
    most = 100
    path = rng.integers(-3, 33, (5, most))
    path[0] = [0] * 99 + [1]
    path[1, :40] = np.sort(path[1, :40])
    path[3] = [-1] * 4 + list(range(96))
    path[4] = [9] * 98 + [0, 1]
    n_path = [100, 100, 3, 12, 100]
    c = CacheCase(ctx, new, dim=dim, block=block, layers=2, **kw)
    T = max(-(-n // block) for n in c.lengths)
    c.tables = c.tables[:, :T].contiguous()
    want = c.k.clone(), c.v.clone()
    for s, m in enumerate(new):
        last = -1
        for i, j in enumerate(path[s, :n_path[s]].tolist()):
            if not 0 <= j < m:
                continue
            if j > last and j >= i:
                a, b = ctx[s] + j, ctx[s] + i
                for w in want:  # (no place is a later source)
                    w[:, c.tables[s, b // block], b % block] = w[:, c.tables[s, a // block], a % block].clone()
            last = max(last, j)
    cache = c.cache(smcsd)
    ws = smcsd.alloc_cache_workspace(cache)
    smcsd.kv_compact_tokens(cache, c.batch(smcsd), torch.tensor(path, dtype=torch.int32, device="cuda"),
                            torch.tensor(n_path, dtype=torch.int32, device="cuda"), ws)
    assert smcsd.status_names(smcsd.smc_device_status(ws)) == ["bad_rows"]
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])


def _truncated(kv, new_len, block, pool):
    """The KV state after kv_truncate, by loops."""
    kv = {k: v.copy() for k, v in kv.items()}
    B, N, _ = kv["tables"].shape
    for b in range(B):
        freed = []
        for n in range(N):
            keep, held = okv.n_blocks(new_len[b, n], block), okv.n_blocks(kv["seq_len"][b, n], block)
            for t in range(keep, held):
                blk = kv["tables"][b, n, t]
                kv["tables"][b, n, t] = -1
                kv["refcount"][blk] -= 1
                if kv["refcount"][blk] == 0:
                    freed.append(blk)
            kv["seq_len"][b, n] = new_len[b, n]
        for blk in sorted(freed):
            kv["free_list"][b, kv["free_top"][b]] = blk
            kv["free_top"][b] += 1
    return kv


@pytest.mark.parametrize("B,N,prefix,block,drafted", [(3, 4, 40, 16, 30), (2, 1, 0, 4, 5), (2, 64, 100, 16, 9),
                                                      (1, 7, 33, 1, 20)])
def test_truncate_gives_blocks_back(B, N, prefix, block, drafted):
    T = (prefix + 4 * drafted) // block + 2
    P = N * T + 1
    kv = make_kv_state(B, N, prefix, block, T, P, device="cuda")
    params = smcsd.make_params(B, N, 1, 64, "f32")
    kvs = smcsd.make_kv(params, kv, block)
    ws = smcsd.alloc_workspace(params, kvs)
    rng = np.random.default_rng(N)
    anc = torch.arange(N, dtype=torch.int32, device="cuda").repeat(B)
    for round_ in range(3):
        res = torch.zeros(B, dtype=torch.int32, device="cuda")
        smcsd.kv_blocktable_remap(params, kvs, anc, res, drafted, ws)
        assert smcsd.smc_device_status(ws) == 0
        state = {k: v.cpu().numpy().astype(np.int64) for k, v in kv.items()}
        lens = state["seq_len"]
        new_len = lens - rng.integers(0, drafted + 1, lens.shape)
        if round_ == 2:
            new_len[:, ::2] = 0  # some particles end
        want = _truncated(state, new_len, block, P)
        smcsd.kv_truncate(params, kvs, torch.tensor(new_len, dtype=torch.int32, device="cuda"), ws)
        assert smcsd.smc_device_status(ws) == 0
        for key in ("tables", "seq_len", "refcount", "free_top"):
            assert np.array_equal(kv[key].cpu().numpy(), want[key]), key
        got = kv["free_list"].cpu().numpy()
        for b in range(B):
            top = int(want["free_top"][b])
            assert np.array_equal(got[b, :top], want["free_list"][b, :top])
        live = okv.live_references(want["tables"], want["seq_len"], block)
        for blk in range(B * P):
            assert want["refcount"][blk] == live.get(blk, 0)


def test_truncate_reports_bad_lengths():
    kv = make_kv_state(1, 2, 40, 16, 4, 12, device="cuda")
    params = smcsd.make_params(1, 2, 1, 64, "f32")
    kvs = smcsd.make_kv(params, kv, 16)
    ws = smcsd.alloc_workspace(params, kvs)
    before = {k: v.clone() for k, v in kv.items()}
    for bad in ([41, 40], [-1, 40]):
        smcsd.kv_truncate(params, kvs, torch.tensor(bad, dtype=torch.int32, device="cuda"), ws)
        assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_block"]
        assert all(torch.equal(kv[k], before[k]) for k in kv)
