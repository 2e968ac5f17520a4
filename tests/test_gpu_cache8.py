"""The 8-bit paged cache's operators on the GPU against 64-bit references:
tree attention, norms with rotation and quantised cache write, block copies and
path compaction."""
import math

import numpy as np
import pytest
import torch

import smc_speculative_decoding_gb300 as smcsd

from cache_cases import qk_reference, rope_table
from cache8_cases import E4M3, Cache8Case, bits, checked_scale, compacted, np_path, rounded

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
    ws = smcsd.alloc_cache8_workspace(cache, batch, c.heads) if workspace is None else workspace
    out = torch.full((c.rows, c.heads, c.dim), 7.0, dtype=c.dtype, device="cuda") if out is None else out
    lses = torch.full((c.rows, c.heads), 7.0, device="cuda") if lse else None
    smcsd.smc_tree_attention8(cache, c.layer, batch, c.q, out, ws, mask=c.mask, lse=lses,
                              scale=c.scale, stream=stream, **kw)
    return out, lses, ws


def _check_attention(c, out, lse, ws, want=None):
    assert smcsd.status_names(smcsd.smc_device_status(ws)) == []
    ref, ref_lse, tol, tol_lse = c.reference() if want is None else want
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse), empty) and torch.all(lse[empty] == -math.inf)
    assert torch.all(out[empty] == 0)
    assert torch.isfinite(out).all()
    excess = ((out.double() - ref).abs() - tol).max().item() if ref.numel() else 0
    assert excess <= 0, f"out is {excess} past its bound"
    off = (lse.double() - ref_lse).abs()[~empty] - tol_lse[~empty]
    assert not off.numel() or off.max().item() <= 0, f"lse is {off.max().item()} past its bound"


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
    ([300, 20], [3, 2], dict(heads=128, kv_heads=1)),               # as many heads as a key head may have
    ([300, 20], [3, 2], dict(heads=100, kv_heads=1)),
    ([260, 31], [7, 2], dict(heads=6, kv_heads=2, dim=64)),        # three heads of a key head
    ([260, 31], [7, 2], dict(heads=5, kv_heads=5, dim=80, mask="tree")),
    ([260, 31], [7, 2], dict(heads=4, kv_heads=1, dim=96)),
    ([260, 31], [7, 2], dict(heads=4, kv_heads=2, dim=16)),
    ([260, 31], [7, 2], dict(heads=4, kv_heads=2, dim=48)),
    ([400], [11], dict(block=1)),
    ([400, 9], [11, 3], dict(block=20)),
    ([400, 9], [11, 3], dict(block=24)),
    ([400, 9], [11, 3], dict(block=256)),
    ([400, 9], [11, 3], dict(block=136)),
    ([3000], [4], dict(block=64, heads=4, kv_heads=4)),
    ([260, 31], [7, 2], dict(spread=6, odd_scales=True)),
    ([900, 31], [20, 2], dict(spread=12)),                         # scales far apart
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ctx,new,kw", SHAPES)
def test_attention(ctx, new, kw, dtype):
    c = Cache8Case(ctx, new, dtype=dtype, poison=True, seed=len(ctx) + sum(ctx), **kw)
    _check_attention(c, *_attend(c))


@pytest.mark.parametrize("order,strided,block", [("hnd", False, 16), ("nhd", True, 16),
                                                 ("hnd", True, 20), ("hnd", False, 64)])
def test_attention_memory_orders(order, strided, block):
    c = Cache8Case([200, 60], [6, 9], order=order, strided=strided, block=block, layers=3, layer=2,
                   mask="tree", poison=True)
    _check_attention(c, *_attend(c))


@pytest.mark.parametrize("group,shared,ctx,new", [
    (4, 512, [600, 512, 700, 530], [5, 5, 5, 5]),
    (2, 100, [100, 110, 300, 100], [3, 2, 1, 4]),   # less than one tile is shared
    (8, 640, [650] * 8 + [700] * 8, [17] * 16),     # more rows than one tile over the shared part
    (3, 0, [50, 60, 70], [2, 2, 2]),
    (2, 384, [384, 384], [1, 0]),
    (4, 512, [600, 512, 700, 530], [0, 5, 5, 5]),   # the first has no rows
    (2, 1024, [1100, 1030], [30, 35]),
])
@pytest.mark.parametrize("mask", ["chain", "tree"])
@pytest.mark.parametrize("slots", [0, 12400])  # tables as large as those whose shared blocks are read once
def test_attention_shared_prefix(group, shared, ctx, new, mask, slots):
    c = Cache8Case(ctx, new, group=group, shared=shared, heads=8, kv_heads=2, mask=mask, poison=True, slots=slots)
    out, lse, ws = _attend(c)
    _check_attention(c, out, lse, ws)
    again, lse2, _ = _attend(c, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("sequences,group,new,low,high,kw", [
    (150, 1, 1, 0, 260, dict()),                     # several units to a CTA
    (150, 1, 5, 60, 200, dict(mask="tree", block=20)),  # element copies
    (270, 1, 3, 1, 130, dict(dim=64)),               # more sequences than are counted without a plan
    (160, 16, 5, 100, 400, dict(slots=1400)),        # own parts after a shared one
    (96, 1, 40, 0, 300, dict(kv_heads=8, heads=24)),  # units of one row tile and of two, by turns
    (160, 1, 20, 0, 150, dict(mask="tree")),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_many_short(sequences, group, new, low, high, kw, dtype):
    """More units than multiprocessors: several to each, of like and of unlike lengths."""
    ctx = [low + 37 * i * i % (high - low + 1) for i in range(sequences)]
    news = [1 + (i * 7) % (2 * new) if new > 1 else 1 for i in range(sequences)]
    shared = min(ctx) // 16 * 16 if group > 1 else 0
    c = Cache8Case(ctx, news, group=group, shared=shared, dtype=dtype, poison=True,
                   **{"heads": 8, "kv_heads": 4, **kw})
    out, lse, ws = _attend(c)
    _check_attention(c, out, lse, ws)
    again, lse2, _ = _attend(c, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("ctx,new,kw", [
    ([3000, 9000, 500, 0, 6400, 77], [5, 64, 1, 30, 128, 2], dict(mask="tree", heads=32, kv_heads=8)),
    ([20000, 100], [8, 8], dict(mask="tree", heads=64, kv_heads=8, block=64)),
    ([1500] * 40, [16] * 40, dict(heads=16, kv_heads=4, block=32)),
    ([900, 1100, 1300, 700] * 12, [5] * 48, dict(heads=16, kv_heads=4, group=4, shared=640)),
    ([900, 1100, 1300, 700] * 12, [5] * 48, dict(heads=16, kv_heads=4, group=4, shared=640, slots=900)),
    ([700] * 48, [70] * 48, dict(heads=16, kv_heads=4, group=16, shared=512, slots=900, mask="tree")),
    ([130] * 400, [1] * 400, dict(heads=8, kv_heads=2)),           # more sequences than one CTA counts
    ([3000] * 3, [40] * 3, dict(heads=12, kv_heads=4, dim=64, mask="tree")),
    ([2500, 40], [30, 30], dict(heads=24, kv_heads=1, dim=96, block=20, mask="tree")),  # odd blocks: element copies
    ([40000], [3], dict(heads=4, kv_heads=2, block=64, mask="tree")),
    ([70000], [1], dict(heads=8, kv_heads=1, block=16)),
])
def test_attention_of_larger_batches(ctx, new, kw):
    c = Cache8Case(ctx, new, **kw)
    out, lse, ws = _attend(c)
    _check_attention(c, out, lse, ws)
    again, lse2, _ = _attend(c, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("ctx,new,bad,kw", [
    ([150, 10], [9, 9], 4, dict(heads=8)),
    ([150, 10], [9, 40], 3, dict(heads=8)),            # 160 rows of a key head
    ([9000], [48], 1, dict(heads=8)),                  # cut between multiprocessors
    ([700, 90], [33, 60], 0, dict(heads=12, dim=64)),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_ignores_what_a_row_does_not_see(ctx, new, bad, kw, dtype):
    """A new token that holds NaN reaches only the rows that see it."""
    s = len(ctx) - 1
    at = ctx[s] + bad
    c = Cache8Case(ctx, new, mask="tree", kv_heads=2, dtype=dtype, **kw)
    ref, _, tol, _ = c.reference()
    sees = torch.tensor([r >= c.starts[s] and bad in c.seen[r] for r in range(c.rows)], device="cuda")
    assert sees.any() and not sees.all()
    block = c.tables[s, at // c.block]
    for which, some in (("v", 5), ("v", None), ("k", None)):
        x = bits(c.v if which == "v" else c.k)[0, block, at % c.block]
        kept = x.clone()
        x[..., some] = 0x7f  # one column, or all
        out, lse, ws = _attend(c)
        assert smcsd.status_names(smcsd.smc_device_status(ws)) == []
        hit = out[sees] if some is None else out[sees][..., some]
        assert torch.isnan(hit).all()
        if some is not None:
            rest = [d for d in range(c.dim) if d != some]
            assert ((out.double() - ref).abs() <= tol)[..., rest].all()
        assert ((out.double() - ref).abs() <= tol)[~sees].all()
        again, _, _ = _attend(c, workspace=ws)
        assert torch.equal(torch.nan_to_num(out, nan=7.0), torch.nan_to_num(again, nan=7.0))
        x.copy_(kept)


def test_attention_of_a_committed_nan_and_of_rows_with_infinities():
    c = Cache8Case([300, 40], [5, 5], mask="tree")
    bits(c.v)[0, c.tables[0, 3], 2, 0, 9] = 0x7f
    c.q[6, 1, 3] = float("inf")
    c.q[7, 2, 3] = float("nan")
    ref, _, tol, _ = c.reference()
    out, lse, ws = _attend(c)
    rep = c.heads // c.kv_heads
    assert torch.isnan(out[:5, :rep, 9]).all() and torch.isnan(out[6, 1]).all() and torch.isnan(out[7, 2]).all()
    good = torch.ones_like(out, dtype=torch.bool)
    good[:5, :rep, 9] = good[6, 1] = good[7, 2] = False
    assert ((out.double() - ref).abs() <= tol)[good].all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_of_large_scores_and_a_heavy_first_token(dtype):
    c = Cache8Case([300, 40], [5, 5], sigma=20.0, mask="tree", dtype=dtype)
    _check_attention(c, *_attend(c))
    # one token takes most of the weight, 20000 alike share the rest: each 2^-17 of it and less
    c = Cache8Case([20000], [2], heads=2, kv_heads=1, spread=0, dtype=dtype)
    b = c.tables[0, 0]
    bits(c.k).zero_()
    bits(c.k)[0, b, 0, 0, 0] = 0x7e  # 448
    c.q.zero_()
    c.q[..., 0] = 16.0
    for z in (11.0, 12.5, 14.0):
        c.scale = z / (16.0 * 448 * c.ks[0, b, 0].item())
        out, lse, ws = _attend(c)
        _check_attention(c, out, lse, ws)


def test_attention_of_scales_beyond_the_range():
    """Scales count as within [2^-100, 2^100]; a block of zeros may have the least one."""
    c = Cache8Case([100], [3], heads=4, kv_heads=1)
    b = c.tables[0, 2]
    bits(c.k)[0, b] = 0
    bits(c.v)[0, b] = 0
    want = c.reference()
    for s in (0.0, 2.0 ** -100, 2.0 ** -126, -1.0, float("nan")):
        c.ks[0, b] = s
        c.vs[0, b] = s
        _check_attention(c, *_attend(c), want=want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ctx,first,size", [(300, 8, 0), (300, 9, 8), (640, 24, 8), (3000, 8, 0), (3000, 160, 3)])
def test_attention_of_zeros_ahead_of_values(ctx, first, size, dtype):
    """Whole tiles of values that are zero, under the least scale, weigh as much as what follows them."""
    c = Cache8Case([ctx, 20], [5, 5], heads=8, kv_heads=2, mask="tree", dtype=dtype)
    size = min(size, 7) if dtype == torch.float16 else size  # (448 * 2^8 is out of fp16's range)
    c.vs *= 2.0 ** size / c.vs.max().item()
    for i in range(first):
        b = c.tables[0, i]
        bits(c.v)[0, b] = 0
        c.vs[0, b] = 2.0 ** -100
    _check_attention(c, *_attend(c))


def test_attention_rows_past_the_last_sequence_are_untouched():
    c = Cache8Case([100, 50], [3, 2])
    rows = c.rows + 4
    q = torch.cat([c.q, torch.full((4, c.heads, c.dim), float("nan"), dtype=c.dtype, device="cuda")])
    cache = c.cache(smcsd)
    batch = smcsd.make_batch(c.tables, c.seq_len, c.max_new, row_start=c.row_start, rows=rows)
    ws = smcsd.alloc_cache8_workspace(cache, batch, c.heads)
    out = torch.full((rows, c.heads, c.dim), 7.0, dtype=c.dtype, device="cuda")
    lse = torch.full((rows, c.heads), 7.0, device="cuda")
    smcsd.smc_tree_attention8(cache, 0, batch, q, out, ws, lse=lse, scale=c.scale)
    _check_attention(c, out[:c.rows], lse[:c.rows], ws)
    assert torch.all(out[c.rows:] == 7) and torch.all(lse[c.rows:] == 7)


def test_attention_of_strided_queries_uniform_batch_on_another_stream():
    c = Cache8Case([333, 20, 64], [4, 4, 4], strided=True)
    want, _, _ = _attend(c)
    wide = torch.full((c.rows, c.heads, c.dim + 8), 7.0, dtype=c.dtype, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, lse, ws = _attend(c, batch=c.batch(smcsd, uniform=True), lse=False, stream=st, out=wide[..., :c.dim])
    st.synchronize()
    assert lse is None and torch.equal(got, want) and torch.all(wide[..., c.dim:] == 7)


def test_attention_in_a_cuda_graph():
    """A captured call reads lengths, tables and masks at its replay."""
    c = Cache8Case([700, 90], [5, 5], mask="tree")
    d = Cache8Case([500, 100], [5, 5], mask="tree", seed=5)  # fits the pool of c
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache, batch, c.heads)
    out, lse, _ = _attend(c, batch=batch, workspace=ws)
    out, lse = torch.empty_like(out), torch.empty_like(lse)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        smcsd.smc_tree_attention8(cache, 0, batch, c.q, out, ws, mask=c.mask, lse=lse, scale=c.scale)
    g.replay()
    torch.cuda.synchronize()
    _check_attention(c, out, lse, ws)
    n = min(c.k.shape[1], d.k.shape[1])
    assert n >= int(d.tables.max()) + 1
    bits(c.k)[:, :n], bits(c.v)[:, :n], c.q[:] = bits(d.k)[:, :n], bits(d.v)[:, :n], d.q
    c.ks[:, :n], c.vs[:, :n] = d.ks[:, :n], d.vs[:, :n]
    c.mask[:], c.seq_len[:] = d.mask, d.seq_len
    width = min(c.tables.shape[1], d.tables.shape[1])
    c.tables[:, :width] = d.tables[:, :width]
    g.replay()
    torch.cuda.synchronize()
    _check_attention(d, out, lse, ws)


def test_attention_reports_bad_state_and_touches_nothing_else():
    c = Cache8Case([100, 50], [3, 2])
    cases = []
    t = c.tables.clone()
    t[0, 1] = c.blocks
    cases.append((dict(tables=t), "bad_block"))
    t = c.tables.clone()
    t[1, 0] = -1
    cases.append((dict(tables=t), "bad_block"))
    for lens in ([100000, 52], [103, 1], [-5, 52]):
        cases.append((dict(seq_len=torch.tensor(lens, dtype=torch.int32, device="cuda")), "bad_block"))
    for starts in ([0, 3, 9], [0, 4, 5], [3, 0, 5]):
        cases.append((dict(row_start=torch.tensor(starts, dtype=torch.int32, device="cuda")), "bad_rows"))
    cache = c.cache(smcsd)
    ref, _, tol, _ = c.reference()
    for kw, bit in cases:
        kw = dict(tables=c.tables, seq_len=c.seq_len, row_start=c.row_start) | kw
        batch = smcsd.make_batch(kw["tables"], kw["seq_len"], 3, row_start=kw["row_start"], rows=c.rows)
        ws = smcsd.alloc_cache8_workspace(cache, batch, c.heads)
        out = torch.empty((c.rows, c.heads, c.dim), dtype=c.dtype, device="cuda")
        smcsd.smc_tree_attention8(cache, 0, batch, c.q, out, ws, scale=c.scale)
        torch.cuda.synchronize()
        assert bit in smcsd.status_names(smcsd.smc_device_status(ws, clear=True)), (kw, bit)
        batch = c.batch(smcsd)  # the same workspace serves the next call
        smcsd.smc_tree_attention8(cache, 0, batch, c.q, out, ws, scale=c.scale)
        assert ((out.double() - ref).abs() <= tol).all()
        assert smcsd.smc_device_status(ws) == 0


# ---- norms, rotation, quantised cache write ----------------------------------

def _check_append(c, before, x, ref, tol, which):
    """The new tokens' elements and scales of one layer against rows ref [rows, kv_heads, dim] in 64 bits that the
    fp32 evaluation is at most tol off; `before`: that layer's (bits, scales)."""
    old_bits, old_scale = before
    now, scale = (c.k, c.ks) if which == "k" else (c.v, c.vs)
    now, scale = bits(now)[c.layer], scale[c.layer]
    want_rest, want_scale = old_bits.clone(), old_scale.clone()
    for s in range(len(c.ctx)):
        p = c.ctx[s]
        while p < c.lengths[s]:
            block, off = int(c.tables[s, p // c.block]), p % c.block
            n = min(c.block - off, c.lengths[s] - p)
            r = int(c.starts[s]) + p - c.ctx[s]
            y, t = ref[r:r + n], tol[r:r + n]
            finite = torch.where(torch.isfinite(y), y, 0.0)
            old = old_scale[block].double() if off else None
            amax, err = finite.abs().amax(dim=(0, 2)), t.amax(dim=(0, 2))
            got = scale[block].double()
            assert checked_scale(got, amax, err, old), (which, s, p)
            stored = now[block, off:off + n].view(E4M3).double() * got[None, :, None]
            half = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * got[None, :, None])
            nan = ~torch.isfinite(y)
            assert torch.equal(torch.isnan(stored), nan)
            assert ((stored - y).abs() <= half * 1.0001 + 1.2 * t)[~nan].all()
            if off:  # the tokens ahead, under the new scale
                f = (old_scale[block].double() / got)[None, :, None]
                x8 = old_bits[block, :off].view(E4M3).double()
                again = torch.where(f == 1, x8, rounded((x8 * f).float().double()))
                assert torch.equal(now[block, :off].view(E4M3).double(), again)
                want_rest[block, :off] = now[block, :off]
            want_rest[block, off:off + n] = now[block, off:off + n]
            want_scale[block] = scale[block]
            p += n
    assert torch.equal(now, want_rest) and torch.equal(scale, want_scale)  # nothing else changed


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("dim,rot,interleaved,norm,offset,kw", [
    (128, 128, False, True, 0.0, {}),
    (128, 64, True, True, 0.0, dict(order="hnd")),
    (64, 64, True, False, 0.0, dict(block=20)),
    (96, 96, False, True, 1.0, dict(strided=True)),
    (80, 40, False, True, 0.0, {}),
    (72, 24, False, True, 0.0, {}),
    (128, 0, False, True, 0.0, dict(block=64)),
    (256, 256, False, True, 0.0, {}),
    (256, 32, True, True, 0.0, {}),
    (14, 6, True, True, 0.0, {}),
    (33, 10, False, True, 0.0, {}),
    (1, 0, False, True, 0.0, dict(block=1)),
    (128, 128, False, False, 0.0, dict(block=128, spread=4)),
])
def test_append(dim, rot, interleaved, norm, offset, kw, dtype):
    c = Cache8Case([37, 0, 90, 250], [5, 1, 7, 40], heads=6, kv_heads=2, dim=dim, dtype=dtype, layers=2, layer=1, **kw)
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((c.rows, 10 * dim), generator=g, device="cuda").to(dtype)
    q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([6 * dim, 2 * dim, 2 * dim], dim=1))
    qw, kw_ = ((torch.randn(dim, generator=g, device="cuda") * 0.3 + 1 - offset).to(dtype) for _ in range(2))
    if not norm:
        qw = kw_ = None
    table = rope_table(300, rot)
    pos = torch.randint(0, 300, (c.rows,), generator=g, device="cuda").to(torch.int32)
    own = torch.cat([torch.arange(a, a + m) for a, m in zip(c.ctx, c.new)]).to(torch.int32).cuda()
    for positions in (pos, None):
        before = {n: (bits(x).clone(), s.clone()) for n, x, s in (("k", c.k, c.ks), ("v", c.v, c.vs))}
        cache, batch = c.cache(smcsd), c.batch(smcsd)
        ws = smcsd.alloc_cache8_workspace(cache)
        out = torch.empty((c.rows, 6, dim), dtype=dtype, device="cuda")
        smcsd.smc_qk_norm_rope8(cache, 1, batch, q, k, v, table, out, ws, positions=positions,
                                q_weight=qw, k_weight=kw_, eps=1e-5, weight_offset=offset, interleaved=interleaved)
        assert smcsd.status_names(smcsd.smc_device_status(ws)) == []
        at = own if positions is None else positions
        ref, tol = qk_reference(q, qw, table, at, rot, interleaved, 1e-5, offset)
        assert ((out.double() - ref).abs() <= tol).all()
        # (a key's fp32 evaluation: the bound of the reference for rows of fp32)
        ref, tol = qk_reference(k.float(), kw_, table, at, rot, interleaved, 1e-5, offset)
        _check_append(c, (before["k"][0][1], before["k"][1][1]), k, ref, tol, "k")
        _check_append(c, (before["v"][0][1], before["v"][1][1]), v, v.double(), torch.zeros_like(ref), "v")
        for n, x, s in (("k", c.k, c.ks), ("v", c.v, c.vs)):
            assert torch.equal(bits(x)[0], before[n][0][0]) and torch.equal(s[0], before[n][1][0])


@pytest.mark.parametrize("heads,kv_heads,dim,norm_q,norm_k,block", [
    (32, 8, 128, True, False, 16), (32, 8, 128, False, True, 64), (71, 1, 64, True, True, 16), (3, 3, 96, False, True, 8),
    (64, 64, 128, True, True, 16), (1, 1, 8, True, True, 16), (100, 4, 256, True, False, 16), (5, 8, 64, True, True, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_heads_and_one_norm(heads, kv_heads, dim, norm_q, norm_k, block, dtype):
    c = Cache8Case([20, 3, 64, 0, 9], [4, 4, 1, 3, 200], heads=kv_heads, kv_heads=kv_heads, dim=dim, dtype=dtype, block=block)
    g = torch.Generator(device="cuda").manual_seed(heads)
    q, k, v = (torch.randn((c.rows, n, dim), generator=g, device="cuda").to(dtype) for n in (heads, kv_heads, kv_heads))
    v = v * torch.logspace(-6, 6, c.rows, device="cuda")[:, None, None].to(dtype)  # scales from small to large
    w = (torch.randn(dim, generator=g, device="cuda") * 0.2 + 1).to(dtype)
    table = rope_table(300, dim)
    own = torch.cat([torch.arange(a, a + m) for a, m in zip(c.ctx, c.new)]).to(torch.int32).cuda()
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    before = {n: (bits(x)[0].clone(), s[0].clone()) for n, x, s in (("k", c.k, c.ks), ("v", c.v, c.vs))}
    ws = smcsd.alloc_cache8_workspace(cache)
    out = torch.empty_like(q)
    smcsd.smc_qk_norm_rope8(cache, 0, batch, q, k, v, table, out, ws, q_weight=w if norm_q else None,
                            k_weight=w if norm_k else None)
    assert smcsd.smc_device_status(ws) == 0
    ref, tol = qk_reference(q, w if norm_q else None, table, own, dim, False, 1e-6, 0.0)
    assert ((out.double() - ref).abs() <= tol).all()
    ref, tol = qk_reference(k.float(), w if norm_k else None, table, own, dim, False, 1e-6, 0.0)
    _check_append(c, before["k"], k, ref, tol, "k")
    _check_append(c, before["v"], v, v.double(), torch.zeros_like(ref), "v")
    # the same tokens again: nothing changes
    kept = [t.clone() for t in (bits(c.k), bits(c.v), c.ks, c.vs, out)]
    smcsd.smc_qk_norm_rope8(cache, 0, batch, q, k, v, table, out, ws, q_weight=w if norm_q else None,
                            k_weight=w if norm_k else None)
    assert all(torch.equal(a, b) for a, b in zip(kept, (bits(c.k), bits(c.v), c.ks, c.vs, out)))


def test_append_token_by_token_grows_a_blocks_scale():
    """Tokens of growing size, one call each: every call rounds the block's tokens under its new scale."""
    c = Cache8Case([0], [16], heads=1, kv_heads=1, dim=32, block=16)
    table = rope_table(20, 0)
    x = torch.randn((16, 1, 32), device="cuda").to(c.dtype) * torch.exp2(torch.arange(16, device="cuda"))[:, None, None].to(c.dtype)
    cache = c.cache(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache)
    out = torch.empty((1, 1, 32), dtype=c.dtype, device="cuda")
    want, scale = torch.zeros((16, 32), dtype=torch.float64, device="cuda"), 0.0
    block = int(c.tables[0, 0])
    for i in range(16):
        batch = smcsd.make_batch(c.tables, torch.tensor([i + 1], dtype=torch.int32, device="cuda"), 1)
        smcsd.smc_qk_norm_rope8(cache, 0, batch, x[i:i + 1], x[i:i + 1], x[i:i + 1], table, out, ws)
        need = 2.0 ** math.ceil(math.log2(x[i].abs().max().item() / 448))
        new = max(scale, need)
        if i and new != scale:
            want[:i] = rounded(want[:i] * (scale / new))
        scale = new
        want[i] = rounded(x[i, 0].double() / scale)
        for a, s in ((c.k, c.ks), (c.v, c.vs)):
            assert s[0, block, 0].item() == scale
            assert torch.equal(a[0, block, :i + 1, 0].double(), want[:i + 1])
    assert smcsd.smc_device_status(ws) == 0


def test_append_in_place_far_positions_and_bad_rows():
    c = Cache8Case([3, 8], [2, 3], heads=4, kv_heads=2, dim=128)
    x = torch.randn((c.rows, 4, 128), device="cuda").to(c.dtype)
    k, v = (torch.randn((c.rows, 2, 128), device="cuda").to(c.dtype) for _ in range(2))
    v[3] = 1e6  # skipped: has no say in the block's scale
    table = rope_table(70000, 128)
    pos = torch.tensor([69999, 65535, 0, 70000, -1], dtype=torch.int32, device="cuda")
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache)
    ref, tol = qk_reference(x[:3], None, table, pos[:3], 128, False, 1e-6, 0.0)
    want, kept = x.clone(), bits(c.v)[0, c.tables[1, 0], 9:11].clone()
    smcsd.smc_qk_norm_rope8(cache, 0, batch, x, k, v, table, x, ws, positions=pos)
    assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_rows"]
    assert ((x[:3].double() - ref).abs() <= tol).all() and torch.equal(x[3:], want[3:])
    assert torch.equal(bits(c.v)[0, c.tables[1, 0], 9:11], kept)
    assert c.vs[0, c.tables[1, 0]].max().item() < 1
    c.tables[0, 0] = c.blocks + 5
    smcsd.smc_qk_norm_rope8(cache, 0, batch, x, k, v, table, x, ws)
    assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_block"]


def test_append_rows_past_the_last_sequence_are_untouched():
    c = Cache8Case([5, 30], [3, 0], heads=2, kv_heads=2, dim=64)
    rows = c.rows + 5
    q, k, v = (torch.randn((rows, 2, 64), device="cuda").to(c.dtype) for _ in range(3))
    out = torch.full_like(q, 7.0)
    cache = c.cache(smcsd)
    batch = smcsd.make_batch(c.tables, c.seq_len, c.max_new, row_start=c.row_start, rows=rows)
    ws = smcsd.alloc_cache8_workspace(cache)
    smcsd.smc_qk_norm_rope8(cache, 0, batch, q, k, v, rope_table(100, 64), out, ws)
    assert smcsd.smc_device_status(ws) == 0
    assert torch.all(out[c.rows:] == 7) and not torch.any(out[:c.rows] == 7)


def test_append_of_zeros_infinities_and_nan():
    """A block of zeros gets the least scale; what is not finite is stored as NaN and has no say in a scale."""
    c = Cache8Case([16], [3], heads=2, kv_heads=1, dim=64)
    k = torch.zeros((3, 1, 64), dtype=c.dtype, device="cuda")
    v = torch.ones((3, 1, 64), dtype=c.dtype, device="cuda")
    v[1, 0, 5], v[2, 0, 7], v[0, 0, 9] = float("inf"), float("nan"), -float("inf")
    q = torch.zeros((3, 2, 64), dtype=c.dtype, device="cuda")
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache)
    smcsd.smc_qk_norm_rope8(cache, 0, batch, q, k, v, rope_table(20, 64), torch.empty_like(q), ws)
    b = int(c.tables[0, 1])
    assert c.ks[0, b, 0].item() == 2.0 ** -100 and torch.all(c.k[0, b, :3].float() == 0)
    assert c.vs[0, b, 0].item() == 2.0 ** -8
    got = c.v[0, b, :3, 0].float() * 2.0 ** -8
    assert torch.equal(torch.isnan(got), ~torch.isfinite(v[:, 0])) and torch.all(got[torch.isfinite(v[:, 0])] == 1)


def test_append_rounds_to_nearest_even():
    """Every e4m3 number, every midpoint between two and their neighbours, under a scale of 1."""
    grid = torch.arange(0, 0x7f, dtype=torch.uint8).view(E4M3).double()
    mid = (grid[1:] + grid[:-1]) / 2
    x = torch.cat([grid, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    x = torch.cat([x, -x])
    n = -(-x.numel() // 63)
    rows = torch.zeros((n, 64), dtype=torch.float64)
    rows[:, 0] = 448
    rows[:, 1:] = torch.nn.functional.pad(x, (0, n * 63 - x.numel())).view(n, 63)
    c = Cache8Case([0], [n], heads=1, kv_heads=1, dim=64, dtype=torch.float32, block=32)
    v = rows.float()[:, None].cuda()
    cache, batch = c.cache(smcsd), c.batch(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache)
    smcsd.smc_qk_norm_rope8(cache, 0, batch, v, v, v, rope_table(100, 0), torch.empty_like(v), ws)
    for a, s in ((c.k, c.ks), (c.v, c.vs)):
        got = torch.cat([a[0, c.tables[0, t], :min(32, n - 32 * t), 0] .double() for t in range(-(-n // 32))])
        assert all(s[0, c.tables[0, t], 0] == 1 for t in range(-(-n // 32)))
        assert torch.equal(got, rounded(v[:, 0].double()))


# ---- blocks -----------------------------------------------------------------

@pytest.mark.parametrize("dim,block,kw", [(128, 16, {}), (64, 24, dict(order="hnd")), (80, 5, dict(strided=True)),
                                          (3, 7, {}), (1, 1, {}), (128, 256, dict(layers=1)), (36, 3, {})])
def test_copy_blocks(dim, block, kw):
    c = Cache8Case([block * 9] * 3, [1] * 3, dim=dim, block=block, kv_heads=2, heads=2, **({"layers": 3} | kw))
    before = [t.clone() for t in (bits(c.k), bits(c.v), c.ks, c.vs)]
    ids = torch.randperm(c.blocks)[:16].to(torch.int32)
    pairs = torch.stack([ids[:8], ids[8:]], 1).view(2, 4, 2).contiguous().cuda()
    counts = torch.tensor([4, 2], dtype=torch.int32, device="cuda")
    cache = c.cache(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache)
    smcsd.kv_copy_blocks8(cache, pairs, counts, ws)
    assert smcsd.smc_device_status(ws) == 0
    for old in before:
        for lst, n in enumerate((4, 2)):
            for src, dst in pairs[lst, :n].tolist():
                old[:, dst] = old[:, src]
    assert all(torch.equal(a, b) for a, b in zip(before, (bits(c.k), bits(c.v), c.ks, c.vs)))
    smcsd.kv_copy_blocks8(cache, torch.full_like(pairs, c.blocks), counts, ws)
    assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_block"]
    smcsd.kv_copy_blocks8(cache, pairs, counts + 2, ws)
    assert smcsd.status_names(smcsd.smc_device_status(ws, clear=True)) == ["bad_rows"]


def _compact(c, path, most=None):
    most = max([1] + [len(p) for p in path]) if most is None else most
    n_path = torch.tensor([len(p) for p in path], dtype=torch.int32, device="cuda")
    padded = torch.tensor([p + [-1] * (most - len(p)) for p in path], dtype=torch.int32, device="cuda")
    cache = c.cache(smcsd)
    ws = smcsd.alloc_cache8_workspace(cache)
    smcsd.kv_compact_tokens8(cache, c.batch(smcsd), padded, n_path, ws)
    return smcsd.status_names(smcsd.smc_device_status(ws))


def _check_compact(c, want):
    for name, x, s in (("k", c.k, c.ks), ("v", c.v, c.vs)):
        data, scale = want[name]
        assert torch.equal(s.double(), scale)
        assert torch.equal(x.double(), data)


@pytest.mark.parametrize("dim,block,kw", [
    (128, 16, {}), (64, 24, dict(order="hnd")), (80, 5, dict(strided=True)), (3, 7, {}), (128, 1, {}),
    (128, 16, dict(spread=3)), (64, 64, dict(spread=3)), (32, 1000, dict(spread=3)), (36, 8, dict(odd_scales=True)),
    (256, 16, dict(kv_heads=24, heads=24, layers=1)), (128, 16, dict(spread=0))])
def test_compact_tokens(dim, block, kw):
    rng = np.random.default_rng(dim)
    new = [40, 1, 9, 17, 33]
    c = Cache8Case([33, 0, 7, 100, 16], new, dim=dim, block=block, **({"layers": 3} | kw))
    path = [np_path(rng, m, m) for m in new]
    path[4] = list(range(33))  # the whole chain: nothing moves
    path[0] = list(range(7, 40))
    want = compacted(c, path)
    assert _compact(c, path) == []
    _check_compact(c, want)


@pytest.mark.parametrize("block", [16, 130, 1024])
def test_compact_of_long_paths(block):
    """Paths longer than the moves whose places are found at a time."""
    rng = np.random.default_rng(8)
    new = [2600, 1500]
    c = Cache8Case([5, 31], new, dim=16, heads=2, kv_heads=2, layers=2, block=block, spread=2)
    path = [sorted(rng.choice(2600, 2290, replace=False).tolist()), sorted(rng.choice(1500, 65, replace=False).tolist())]
    want = compacted(c, path)
    assert _compact(c, path) == []
    _check_compact(c, want)
    for at in (3, 255, 256, 1030, 2289):  # a bad index deep in a path is reported, whichever pass it falls in
        bad = [list(path[0]), path[1]]
        bad[0][at] = bad[0][at - 1]
        assert _compact(c, bad) == ["bad_rows"], at


@pytest.mark.parametrize("dim,block,kw", [(64, 16, {}), (3, 7, {}), (64, 4, dict(order="hnd")), (128, 1, {})])
def test_compact_skips_bad_entries_and_touches_nothing_else(dim, block, kw):
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
    c = Cache8Case(ctx, new, dim=dim, block=block, layers=2, spread=2, **kw)
    T = max(-(-n // block) for n in c.lengths)
    c.tables = c.tables[:, :T].contiguous()
    path = [path[s, :n].tolist() for s, n in enumerate(n_path)]
    want = compacted(c, path)
    assert _compact(c, path, most) == ["bad_rows"]
    _check_compact(c, want)
    c.tables[1, (31 + 25) // block] = c.blocks  # where the second token comes from
    assert "bad_block" in _compact(c, [[], [1, 25], [], [], []], most)
