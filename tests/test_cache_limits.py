"""The largest calls on the paged cache's entry points, without a GPU: what 32
bits would not count is refused before anything is launched."""
import ctypes

import pytest

from smc_speculative_decoding_gb300 import binding as bd
from test_cache8_refusals import _cache8, _qk
from test_cache_refusals import ARG, PTR, WS, _batch, _cache, lib  # noqa: F401


@pytest.mark.parametrize("most,code", [(1 << 30, WS), ((1 << 30) + 1, ARG), ((1 << 31) - 1, ARG)])
def test_paths(lib, most, code):  # noqa: F811
    b = ctypes.byref(_batch())  # (no workspace: what passes the other checks is refused for that)
    assert lib.kv_compact_tokens(ctypes.byref(_cache()), b, PTR, PTR, most, None, 0, None) == code
    assert lib.kv_compact_tokens8(ctypes.byref(_cache8()), b, PTR, PTR, most, None, 0, None) == code


@pytest.mark.parametrize("rows,code", [(1 << 30, WS), ((1 << 30) + 1, ARG), ((1 << 31) - 1, ARG)])
def test_rows_of_a_quantised_write(lib, rows, code):  # noqa: F811
    assert _qk(lib, batch=_batch(rows=rows), ws=None, ws_bytes=0) == code
