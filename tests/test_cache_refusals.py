"""Refusals of the paged cache's entry points, without a GPU: every bad
argument gets its code before anything is launched."""
import ctypes
import os
import shutil
import subprocess

import pytest

from smc_speculative_decoding_gb300 import binding as bd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x10000  # never dereferenced: validation fails first
ARG, DTYPE, WS = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from smc_speculative_decoding_gb300 import build
    build.build()
    return bd.lib()


def _cache(**kw):
    f = dict(k=PTR, v=PTR, layer_stride=8 * 4096, block_stride=4096, token_stride=256, head_stride=128,
             layers=2, blocks=8, block_size=16, kv_heads=2, head_dim=128, dtype=bd.SMC_BF16) | kw
    return bd.smc_cache(*(f[n] for n, _ in bd.smc_cache._fields_))


def _batch(**kw):
    f = dict(tables=PTR, seq_len=PTR, row_start=PTR, S=4, T=8, rows=12, max_new=3, group=2) | kw
    return bd.smc_batch(*(f[n] for n, _ in bd.smc_batch._fields_))


def _attn(lib, p=None, cache=None, batch=None, layer=0, q=PTR, mask=None, out=PTR, ws=PTR, ws_bytes=1 << 40, **kw):
    f = dict(q_heads=8, mask_words=0, scale=0.1, reserved=0, q_row_stride=1024, q_head_stride=128,
             out_row_stride=1024, out_head_stride=128) | kw
    params = bd.smc_attn_params(*(f[n] for n, _ in bd.smc_attn_params._fields_))
    return lib.smc_tree_attention(ctypes.byref(params), ctypes.byref(cache or _cache()), layer,
                                  ctypes.byref(batch or _batch()), q, mask, out, None, ws, ws_bytes, None)


def _qk(lib, cache=None, batch=None, layer=0, q=PTR, k=PTR, v=PTR, rope=PTR, out=PTR, ws=PTR, ws_bytes=256, **kw):
    f = dict(q_heads=8, rot_dim=128, max_pos=10, interleaved=0, eps=1e-6, weight_offset=0.0,
             q_row_stride=1, q_head_stride=1, k_row_stride=1, k_head_stride=1, v_row_stride=1,
             v_head_stride=1, out_row_stride=1, out_head_stride=1) | kw
    params = bd.smc_qk_params(*(f[n] for n, _ in bd.smc_qk_params._fields_))
    return lib.smc_qk_norm_rope(ctypes.byref(params), ctypes.byref(cache or _cache()), layer,
                                ctypes.byref(batch or _batch()), q, k, v, None, None, None, rope, out,
                                ws, ws_bytes, None)


BAD_CACHES = [dict(k=None), dict(v=None), dict(layers=0), dict(blocks=0), dict(block_size=0), dict(kv_heads=0),
              dict(head_dim=0), dict(block_stride=-4096), dict(token_stride=-256), dict(layer_stride=-1),
              dict(head_stride=-128), dict(k=PTR + 1)]
BAD_BATCHES = [dict(tables=None), dict(seq_len=None), dict(S=0), dict(T=0), dict(rows=-1), dict(max_new=0),
               dict(max_new=(1 << 16) + 1), dict(group=0), dict(group=3), dict(row_start=None, rows=11)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches(lib, kw):
    c, b = _cache(**kw), _batch()
    assert lib.smc_cache_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 8) == 0
    assert lib.smc_cache_workspace_bytes(ctypes.byref(c), None, 0) == 0
    assert _attn(lib, cache=c) == ARG and _qk(lib, cache=c) == ARG
    assert lib.kv_copy_blocks(ctypes.byref(c), PTR, PTR, 1, 1, PTR, 256, None) == ARG
    assert lib.kv_compact_tokens(ctypes.byref(c), ctypes.byref(b), PTR, PTR, 1, PTR, 256, None) == ARG


@pytest.mark.parametrize("kw", BAD_BATCHES)
def test_bad_batches(lib, kw):
    c, b = _cache(), _batch(**kw)
    assert lib.smc_cache_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 8) == 0
    assert _attn(lib, batch=b) == ARG and _qk(lib, batch=b) == ARG
    assert lib.kv_compact_tokens(ctypes.byref(c), ctypes.byref(b), PTR, PTR, 1, PTR, 256, None) == ARG


@pytest.mark.parametrize("kw", [
    dict(q_heads=0), dict(q_heads=7), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(reserved=1), dict(mask_words=-1), dict(mask=PTR, mask_words=0), dict(q=None),
    dict(out=None), dict(layer=-1), dict(layer=2), dict(q=PTR + 2), dict(out=PTR + 8), dict(q_row_stride=1001),
    dict(q_head_stride=4), dict(out_row_stride=-8), dict(out_head_stride=129), dict(cache=_cache(head_dim=136)),
    dict(cache=_cache(head_dim=20)), dict(cache=_cache(token_stride=260)), dict(cache=_cache(k=PTR + 2)),
    dict(cache=_cache(layer_stride=4), layer=1), dict(q_row_stride=0), dict(q_head_stride=0),
    dict(q_heads=258)])
def test_bad_attention_arguments(lib, kw):
    assert _attn(lib, **kw) == ARG


@pytest.mark.parametrize("kw", [
    dict(q_heads=0), dict(rot_dim=-2), dict(rot_dim=130), dict(rot_dim=3), dict(max_pos=0), dict(interleaved=2),
    dict(eps=-1e-6), dict(eps=float("nan")), dict(weight_offset=float("inf")), dict(q=None), dict(k=None),
    dict(v=None), dict(out=None), dict(rope=None), dict(layer=2), dict(layer=-1), dict(q_row_stride=-1),
    dict(out_head_stride=-1), dict(q=PTR + 1), dict(cache=_cache(head_dim=264))])
def test_bad_qk_arguments(lib, kw):
    assert _qk(lib, **kw) == ARG


def test_dtypes_and_workspaces(lib):
    for dtype in (3, -1):
        c = _cache(dtype=dtype)
        assert _attn(lib, cache=c) == DTYPE and _qk(lib, cache=c) == DTYPE
        assert lib.kv_copy_blocks(ctypes.byref(c), PTR, PTR, 1, 1, PTR, 256, None) == DTYPE
        assert lib.smc_cache_workspace_bytes(ctypes.byref(c), None, 0) == 0
    assert _attn(lib, cache=_cache(dtype=bd.SMC_F32)) == DTYPE  # attention takes 16-bit caches
    need = lib.smc_cache_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(_batch()), 8)
    assert need >= 256 and need % 256 == 0
    for ws, size in ((None, need), (PTR + 16, need), (PTR, need - 1)):
        assert _attn(lib, ws=ws, ws_bytes=size) == WS
    for ws, size in ((None, 256), (PTR + 16, 256), (PTR, 255)):
        assert _qk(lib, ws=ws, ws_bytes=size) == WS
        assert lib.kv_copy_blocks(ctypes.byref(_cache()), PTR, PTR, 1, 1, ws, size, None) == WS
        assert lib.kv_compact_tokens(ctypes.byref(_cache()), ctypes.byref(_batch()), PTR, PTR, 1, ws, size, None) == WS


def test_bad_block_calls(lib):
    c, b = _cache(), _batch()
    for pairs, counts, lists, most in ((None, PTR, 1, 1), (PTR, None, 1, 1), (PTR, PTR, 0, 1), (PTR, PTR, 1, 0),
                                       (PTR, PTR, 1 << 20, 1 << 20)):
        assert lib.kv_copy_blocks(ctypes.byref(c), pairs, counts, lists, most, PTR, 256, None) == ARG
    for path, n, most in ((None, PTR, 1), (PTR, None, 1), (PTR, PTR, 0)):
        assert lib.kv_compact_tokens(ctypes.byref(c), ctypes.byref(b), path, n, most, PTR, 256, None) == ARG
    p = bd.smc_params(2, 4, 3, 64, 0, 1.0, 0.5, 0, 0)
    kv = bd.smc_kv(*[PTR] * 7, 8, 16, 64)
    need = lib.smc_workspace_bytes(ctypes.byref(p), ctypes.byref(kv))
    assert lib.kv_truncate(None, ctypes.byref(kv), PTR, PTR, need, None) == ARG
    assert lib.kv_truncate(ctypes.byref(p), None, PTR, PTR, need, None) == ARG
    assert lib.kv_truncate(ctypes.byref(p), ctypes.byref(kv), None, PTR, need, None) == ARG
    assert lib.kv_truncate(ctypes.byref(p), ctypes.byref(kv), PTR, PTR, need - 1, None) == WS
    bad = bd.smc_params(2, 4, 3, 64, 7, 1.0, 0.5, 0, 0)
    assert lib.kv_truncate(ctypes.byref(bad), ctypes.byref(kv), PTR, PTR, need, None) == DTYPE


def test_tables_with_room_for_more_tokens_than_32_bits_count(lib):
    c = _cache(kv_heads=1, head_dim=8, token_stride=8, head_stride=8, block_stride=128, layer_stride=1024)
    kw = dict(S=1, rows=1, max_new=1, group=1)
    for T, fits in (((1 << 31) // 16, False), ((1 << 31) // 16 - 255, False), ((1 << 31) // 16 - 256, True)):
        b = _batch(T=T, **kw)
        assert (lib.smc_cache_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 1) > 0) == fits
        if not fits:
            assert _attn(lib, cache=c, batch=b, q_heads=1) == ARG


def test_a_call_without_rows_is_accepted(lib):
    b = _batch(rows=0)
    need = lib.smc_cache_workspace_bytes(ctypes.byref(_cache()), ctypes.byref(b), 8)
    assert need >= 256
    assert _attn(lib, batch=b, q=None, out=None) == 0
    assert _qk(lib, batch=b, q=None, k=None, v=None, out=None) == 0


def test_struct_layouts_match_the_c_compiler(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    structs = [bd.smc_cache, bd.smc_batch, bd.smc_attn_params, bd.smc_qk_params]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "smcsd.h"', 'int main(void){']
    for st in structs:
        n = st.__name__
        lines.append(f'printf("{n} - %zu\\n", sizeof({n}));')
        lines += [f'printf("{n} {f} %zu\\n", offsetof({n}, {f}));' for f, _ in st._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join([*lines, "return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", f"-I{ROOT}/include", str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    by = {st.__name__: st for st in structs}
    for line in out.splitlines():
        name, field, size = line.split()
        want = ctypes.sizeof(by[name]) if field == "-" else getattr(by[name], field).offset
        assert want == int(size), line


def test_the_binding_refuses_tensors_it_cannot_pass():
    import torch
    t = torch.zeros((1, 4, 16, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bd.make_cache(t, t)
    with pytest.raises(TypeError):
        bd.make_cache(None, t)


def test_the_binding_refuses_a_mask_without_words(monkeypatch):
    """It has no address, and no mask means a chain."""
    import torch
    monkeypatch.setattr(bd, "_rows", lambda *a: (PTR, 1024, 128))
    q = torch.zeros((12, 8, 128), dtype=torch.bfloat16)
    for shape in ((12, 0), (11, 1), (12,)):
        with pytest.raises(ValueError, match="at least one word"):
            bd.smc_tree_attention(_cache(), 0, _batch(), q, q, None, mask=torch.zeros(shape, dtype=torch.int32))
