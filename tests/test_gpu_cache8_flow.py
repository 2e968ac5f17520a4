"""The 8-bit cache's entry points used together, as in examples/draft_scoring.py
with --bits 8: what each particle's table leads to stays its own history, up to
the rounding of blocks whose scale has grown, and the attention over it is that
history's."""
import os
import sys

import pytest
import torch

from cache8_cases import Q_LEFT, WEIGHT, WEIGHT_FLOOR
from cache_cases import E32, half_step

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from smc_speculative_decoding_gb300 import build
    build.build()


def _held(st, table, n):
    """Keys and values [layers, n, kv_heads, dim] behind a table in 64 bits, and their scales [layers, n, kv_heads]."""
    at = torch.arange(n, device="cuda")
    block = table.long()[at // st["block_size"]]
    out = []
    for x, s in ((st["k"], st["cache"].k_scale), (st["v"], st["cache"].v_scale)):
        scale = s[:, block].double()
        out += [x[:, block, at % st["block_size"]].double() * scale[..., None], scale]
    return out


def _same_up_to_scales(now, scale, before, old_scale):
    """Values under scales that may have grown: a power of two's growth rounds only below e4m3's smallest normal
    number, each time by half of 2^-9 of the scale then: less than 2^-9 of the last one in all."""
    assert (scale >= old_scale).all()
    same = (scale == old_scale)[..., None].expand_as(now)
    assert torch.equal(now[same], before[same])
    assert ((now - before).abs() <= 2.0 ** -9 * scale[..., None]).all()


@pytest.mark.parametrize("prompts,n,K,prefix,block", [(3, 8, 4, 200, 16), (2, 5, 2, 7, 4), (1, 16, 4, 64, 32)])
def test_particles_keep_their_histories(prompts, n, K, prefix, block):
    import draft_scoring as ds
    shadow = {}
    seen_resampling = []

    def observe(step, st):
        if "ancestors" in st:
            for b in range(prompts):
                if st["resampled"][b]:
                    seen_resampling.append(step)
                    old = [shadow[b, i] for i in range(n)]
                    for i in range(n):
                        shadow[b, i] = old[int(st["ancestors"][b, i])]
            return
        kv, T = st["kv"], K + 1
        for b in range(prompts):
            for i in range(n):
                length = int(kv["seq_len"][b, i])
                k, ks, v, vs = _held(st, kv["tables"][b, i], length)
                if (b, i) in shadow:
                    wk, wks, wv, wvs = shadow[b, i]
                    m = length - T
                    assert wk.shape[1] == m
                    _same_up_to_scales(k[:, :m], ks[:, :m], wk, wks)
                    _same_up_to_scales(v[:, :m], vs[:, :m], wv, wvs)
                shadow[b, i] = (k, ks, v, vs)
        b, i = step % prompts, step % n
        k, ks, v, vs = shadow[b, i]
        length = k.shape[1]
        for layer, (q, o) in enumerate(st["seen"]):
            rep = q.shape[1] // k.shape[2]
            rows = slice((b * n + i) * T, (b * n + i + 1) * T)
            x = q[rows].double().unflatten(1, (-1, rep))
            scale = q.shape[2] ** -0.5
            z = torch.einsum("rhgd,thd->rhgt", x, k[layer]) * scale
            late = torch.arange(length, device="cuda")[None] > length - T + torch.arange(T, device="cuda")[:, None]
            p = torch.softmax(z.masked_fill(late[:, None, None], -torch.inf), -1)
            want = torch.einsum("rhgt,thd->rhgd", p, v[layer])
            mag = torch.einsum("rhgt,thd->rhgd", p, v[layer].abs())
            a = scale * ((q.shape[2] + 2) * E32 * torch.einsum("rhgd,thd->rhgt", x.abs(), k[layer].abs()) +
                         Q_LEFT * x.abs().amax(-1, keepdim=True) * k[layer].abs().sum(-1).T[None, :, None]).amax()
            floor = WEIGHT_FLOOR * (p * vs[layer].T[None, :, None]).amax(-1, keepdim=True) * \
                (v[layer].abs() / vs[layer][..., None]).sum(0)[None, :, None]
            tol = (2 * a + 2.0 ** -19 + 2 * length * E32 + WEIGHT) * 1.01 * mag + half_step(q.dtype) * 1.01 * want.abs() + floor
            got = o[rows].double().unflatten(1, (-1, rep))
            assert ((got - want).abs() <= tol).all()

    tokens, saved = ds.particles(prompts, n, K=K, steps=7, prefix=prefix, block_size=block, observe=observe, bits=8)
    assert tokens.shape == (prompts, n, 7 * (K + 1)) and 0 <= saved < 1
    assert seen_resampling, "no step resampled: the flow was not exercised"


@pytest.mark.parametrize("M,prefix,block", [(12, 37, 16), (33, 16, 4), (5, 0 + 1, 8)])
def test_trees_leave_the_accepted_path(M, prefix, block):
    import draft_scoring as ds
    want = {}
    rounds = []

    def observe(round_, st):
        kv = st["kv"]
        for s in range(kv["seq_len"].numel()):
            c, n = int(st["committed"][s]), int(st["n_path"][s])
            if st.get("after"):
                length = int(kv["seq_len"].view(-1)[s])
                assert length == c + n
                k, ks, v, vs = _held(st, kv["tables"][s, 0], length)
                for now, scale, (before, old) in ((k, ks, want[s][0]), (v, vs, want[s][1])):
                    # (a moved token's scale is its new block's, the larger one)
                    assert ((now - before).abs() <= 2.0 ** -10 * scale[..., None]).all() and (scale >= old).all()
                used = -(-length // st["block_size"])
                assert torch.all(kv["tables"][s, 0, used:] == -1)
            else:
                k, ks, v, vs = _held(st, kv["tables"][s, 0], c + M)
                keep = torch.cat([torch.arange(c, device="cuda"), c + st["path"][s, :n].long()])
                want[s] = ((k[:, keep], ks[:, keep]), (v[:, keep], vs[:, keep]))
        rounds.append(round_)

    lengths = ds.tree(3, M=M, prefix=prefix, block_size=block, observe=observe, bits=8)
    assert torch.all(lengths > prefix) and len(rounds) == 8


def test_two_bits_widths_agree_on_the_logits():
    """The same tokens through both caches: attention outputs differ by the cache's rounding alone."""
    import draft_scoring as ds
    seen = {}

    def observe(bits):
        def see(step, st):
            if step == 0 and "seen" in st:
                seen[bits] = st["seen"][0]
        return see

    for bits in (8, 16):
        ds.particles(2, 4, steps=1, prefix=50, observe=observe(bits), bits=bits)
    (q8, o8), (q16, o16) = seen[8], seen[16]
    assert torch.equal(q8, q16)
    # an element of the cache is off by 2^-4 of it at most, in the mean by less than half of that; the output is a mean
    # over many: a relative error of the whole below 2^-4
    assert (o8.double() - o16.double()).norm() <= 2.0 ** -4 * o16.double().norm()
