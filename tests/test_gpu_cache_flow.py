"""The cache's entry points used together, as in examples/draft_scoring.py:
what each particle's table leads to stays its own history through resampling,
copy-on-write, tree compaction and truncation, and the attention over it is
that history's."""
import os
import sys

import pytest
import torch

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
    """Keys and values [layers, n, kv_heads, dim] behind a table."""
    at = torch.arange(n, device="cuda")
    block = table.long()[at // st["block_size"]]
    return st["k"][:, block, at % st["block_size"]], st["v"][:, block, at % st["block_size"]]


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
        kv = st["kv"]
        T = K + 1
        for b in range(prompts):
            for i in range(n):
                length = int(kv["seq_len"][b, i])
                k, v = _held(st, kv["tables"][b, i], length)
                if (b, i) in shadow:
                    wk, wv = shadow[b, i]
                    assert wk.shape[1] == length - T
                    assert torch.equal(k[:, :length - T], wk) and torch.equal(v[:, :length - T], wv), (step, b, i)
                shadow[b, i] = (k.clone(), v.clone())
        # one particle's attention, in 64 bits, over what its table leads to
        b, i = step % prompts, step % n
        k, v = shadow[b, i]
        length = k.shape[1]
        for layer, (q, o) in enumerate(st["seen"]):
            rep = q.shape[1] // k.shape[2]
            rows = slice((b * n + i) * T, (b * n + i + 1) * T)
            x = q[rows].double().unflatten(1, (-1, rep))
            scale = q.shape[2] ** -0.5
            z = torch.einsum("rhgd,thd->rhgt", x, k[layer].double()) * scale
            late = torch.arange(length, device="cuda")[None] > length - T + torch.arange(T, device="cuda")[:, None]
            p = torch.softmax(z.masked_fill(late[:, None, None], -torch.inf), -1)
            want = torch.einsum("rhgt,thd->rhgd", p, v[layer].double())
            mag = torch.einsum("rhgt,thd->rhgd", p, v[layer].double().abs())
            a = (q.shape[2] + 2) * E32 * scale * torch.einsum("rhgd,thd->rhgt", x.abs(), k[layer].double().abs()).amax()
            u = half_step(q.dtype)
            tol = (2 * a + 2.0 ** -20 + 2 * length * E32 + u) * 1.01 * mag + u * 1.01 * want.abs()
            got = o[rows].double().unflatten(1, (-1, rep))
            assert ((got - want).abs() <= tol).all()

    tokens, saved = ds.particles(prompts, n, K=K, steps=7, prefix=prefix, block_size=block, observe=observe)
    assert tokens.shape == (prompts, n, 7 * (K + 1)) and 0 <= saved < 1
    assert seen_resampling, "no step resampled: the flow was not exercised"


@pytest.mark.parametrize("M,prefix,block", [(12, 37, 16), (33, 16, 4), (5, 0 + 1, 8)])
def test_trees_leave_the_accepted_path(M, prefix, block):
    import draft_scoring as ds
    want = {}
    free0 = []

    def observe(round_, st):
        kv = st["kv"]
        S = kv["seq_len"].numel()
        for s in range(S):
            c, n = int(st["committed"][s]), int(st["n_path"][s])
            if st.get("after"):
                length = int(kv["seq_len"].view(-1)[s])
                assert length == c + n
                k, v = _held(st, kv["tables"][s, 0], length)
                assert torch.equal(k, want[s][0]) and torch.equal(v, want[s][1])
                used = -(-length // st["block_size"])
                assert torch.all(kv["tables"][s, 0, used:] == -1)
                assert int(kv["free_top"][s]) + used == kv["free_list"].shape[1]
            else:
                k, v = _held(st, kv["tables"][s, 0], c + M)
                keep = torch.cat([torch.arange(c, device="cuda"), c + st["path"][s, :n].long()])
                want[s] = (k[:, keep].clone(), v[:, keep].clone())
        free0.append(round_)

    lengths = ds.tree(3, M=M, prefix=prefix, block_size=block, observe=observe)
    assert torch.all(lengths > prefix) and len(free0) == 8
