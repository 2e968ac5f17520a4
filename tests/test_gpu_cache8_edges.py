"""The 8-bit paged cache's operators at the edges of what their calls may say,
against 64-bit references."""
import pytest
import torch

import smc_speculative_decoding_gb300 as smcsd

from cache8_cases import Cache8Case, compacted

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
