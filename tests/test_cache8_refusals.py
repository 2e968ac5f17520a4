"""Refusals of the 8-bit paged cache's entry points, without a GPU: every bad
argument gets its code before anything is launched."""
import ctypes
import os
import shutil
import subprocess

import pytest

from smc_speculative_decoding_gb300 import binding as bd
from test_cache_refusals import ARG, BAD_BATCHES, BAD_CACHES, DTYPE, PTR, ROOT, WS, _batch, lib  # noqa: F401


def _cache8(k_scale=PTR, v_scale=PTR, scales=(16, 2, 1), **kw):
    f = dict(k=PTR, v=PTR, layer_stride=8 * 4096, block_stride=4096, token_stride=256, head_stride=128,
             layers=2, blocks=8, block_size=16, kv_heads=2, head_dim=128, dtype=bd.SMC_E4M3) | kw
    return bd.smc_cache8(bd.smc_cache(*(f[n] for n, _ in bd.smc_cache._fields_)), k_scale, v_scale, *scales)


def _attn(lib, cache=None, batch=None, layer=0, dtype=bd.SMC_BF16, q=PTR, mask=None, out=PTR, ws=PTR,
          ws_bytes=1 << 40, **kw):
    f = dict(q_heads=8, mask_words=0, scale=0.1, reserved=0, q_row_stride=1024, q_head_stride=128,
             out_row_stride=1024, out_head_stride=128) | kw
    params = bd.smc_attn_params(*(f[n] for n, _ in bd.smc_attn_params._fields_))
    return lib.smc_tree_attention8(ctypes.byref(params), ctypes.byref(cache or _cache8()), layer,
                                   ctypes.byref(batch or _batch()), dtype, q, mask, out, None, ws, ws_bytes, None)


def _qk(lib, cache=None, batch=None, layer=0, dtype=bd.SMC_BF16, q=PTR, k=PTR, v=PTR, rope=PTR, out=PTR, ws=PTR,
        ws_bytes=256, **kw):
    f = dict(q_heads=8, rot_dim=128, max_pos=10, interleaved=0, eps=1e-6, weight_offset=0.0,
             q_row_stride=1, q_head_stride=1, k_row_stride=1, k_head_stride=1, v_row_stride=1,
             v_head_stride=1, out_row_stride=1, out_head_stride=1) | kw
    params = bd.smc_qk_params(*(f[n] for n, _ in bd.smc_qk_params._fields_))
    return lib.smc_qk_norm_rope8(ctypes.byref(params), ctypes.byref(cache or _cache8()), layer,
                                 ctypes.byref(batch or _batch()), dtype, q, k, v, None, None, None, rope, out,
                                 ws, ws_bytes, None)


def _copy(lib, cache=None, pairs=PTR, counts=PTR, lists=1, most=1, ws=PTR, ws_bytes=256):
    return lib.kv_copy_blocks8(ctypes.byref(cache or _cache8()), pairs, counts, lists, most, ws, ws_bytes, None)


def _compact(lib, cache=None, batch=None, path=PTR, n=PTR, most=1, ws=PTR, ws_bytes=256):
    return lib.kv_compact_tokens8(ctypes.byref(cache or _cache8()), ctypes.byref(batch or _batch()), path, n, most,
                                  ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [kw for kw in BAD_CACHES if kw != dict(k=PTR + 1)] + [
    dict(k_scale=None), dict(v_scale=None), dict(k_scale=PTR + 2), dict(v_scale=PTR + 1), dict(scales=(-1, 2, 1)),
    dict(scales=(16, -2, 1)), dict(scales=(16, 2, -1))])
def test_bad_caches(lib, kw):  # noqa: F811
    c, b = _cache8(**kw), _batch()
    assert lib.smc_cache8_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 8) == 0
    assert lib.smc_cache8_workspace_bytes(ctypes.byref(c), None, 0) == 0
    assert _attn(lib, cache=c) == ARG and _qk(lib, cache=c) == ARG
    assert _copy(lib, cache=c) == ARG and _compact(lib, cache=c) == ARG


@pytest.mark.parametrize("kw", BAD_BATCHES)
def test_bad_batches(lib, kw):  # noqa: F811
    c, b = _cache8(), _batch(**kw)
    assert lib.smc_cache8_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 8) == 0
    assert _attn(lib, batch=b) == ARG and _qk(lib, batch=b) == ARG and _compact(lib, batch=b) == ARG


@pytest.mark.parametrize("kw", [
    dict(q_heads=0), dict(q_heads=7), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(reserved=1), dict(mask_words=-1), dict(mask=PTR, mask_words=0), dict(q=None),
    dict(out=None), dict(layer=-1), dict(layer=2), dict(q=PTR + 2), dict(out=PTR + 8), dict(q_row_stride=1001),
    dict(q_head_stride=4), dict(out_row_stride=-8), dict(out_head_stride=129), dict(cache=_cache8(head_dim=144)),
    dict(cache=_cache8(head_dim=120)), dict(cache=_cache8(token_stride=264)), dict(cache=_cache8(k=PTR + 8)),
    dict(cache=_cache8(layer_stride=8), layer=1), dict(q_row_stride=0), dict(q_head_stride=0), dict(q_heads=258)])
def test_bad_attention_arguments(lib, kw):  # noqa: F811
    assert _attn(lib, **kw) == ARG


@pytest.mark.parametrize("kw", [
    dict(q_heads=0), dict(rot_dim=-2), dict(rot_dim=130), dict(rot_dim=3), dict(max_pos=0), dict(interleaved=2),
    dict(eps=-1e-6), dict(eps=float("nan")), dict(weight_offset=float("inf")), dict(q=None), dict(k=None),
    dict(v=None), dict(out=None), dict(rope=None), dict(layer=2), dict(layer=-1), dict(q_row_stride=-1),
    dict(out_head_stride=-1), dict(q=PTR + 1), dict(q=PTR + 2, dtype=bd.SMC_F32),
    dict(cache=_cache8(head_dim=264)), dict(cache=_cache8(kv_heads=65536))])
def test_bad_qk_arguments(lib, kw):  # noqa: F811
    assert _qk(lib, **kw) == ARG


def test_dtypes_and_workspaces(lib):  # noqa: F811
    for dtype in (bd.SMC_BF16, bd.SMC_F32, 4, -1):  # an 8-bit cache is one of e4m3
        c = _cache8(dtype=dtype)
        assert _attn(lib, cache=c) == DTYPE and _qk(lib, cache=c) == DTYPE
        assert _copy(lib, cache=c) == DTYPE and _compact(lib, cache=c) == DTYPE
        assert lib.smc_cache8_workspace_bytes(ctypes.byref(c), None, 0) == 0
    for dtype in (bd.SMC_F32, bd.SMC_E4M3, 4, -1):
        assert _attn(lib, dtype=dtype) == DTYPE
    for dtype in (bd.SMC_E4M3, 4, -1):
        assert _qk(lib, dtype=dtype) == DTYPE
    need = lib.smc_cache8_workspace_bytes(ctypes.byref(_cache8()), ctypes.byref(_batch()), 8)
    assert need >= 256 and need % 256 == 0
    for ws, size in ((None, need), (PTR + 16, need), (PTR, need - 1)):
        assert _attn(lib, ws=ws, ws_bytes=size) == WS
    for ws, size in ((None, 256), (PTR + 16, 256), (PTR, 255)):
        assert _qk(lib, ws=ws, ws_bytes=size) == WS
        assert _copy(lib, ws=ws, ws_bytes=size) == WS and _compact(lib, ws=ws, ws_bytes=size) == WS


def test_bad_block_calls(lib):  # noqa: F811
    for kw in (dict(pairs=None), dict(counts=None), dict(lists=0), dict(most=0), dict(lists=1 << 20, most=1 << 20)):
        assert _copy(lib, **kw) == ARG
    for kw in (dict(path=None), dict(n=None), dict(most=0), dict(cache=_cache8(block_size=1025)),
               dict(cache=_cache8(kv_heads=65536))):
        assert _compact(lib, **kw) == ARG


def test_the_other_entry_points_refuse_8_bits(lib):  # noqa: F811
    c, b = _cache8().data, _batch()
    assert lib.smc_cache_workspace_bytes(ctypes.byref(c), None, 0) == 0
    assert lib.kv_copy_blocks(ctypes.byref(c), PTR, PTR, 1, 1, PTR, 256, None) == DTYPE
    assert lib.kv_compact_tokens(ctypes.byref(c), ctypes.byref(b), PTR, PTR, 1, PTR, 256, None) == DTYPE


def test_null_structs(lib):  # noqa: F811
    b = ctypes.byref(_batch())
    assert lib.smc_cache8_workspace_bytes(None, b, 8) == 0
    assert lib.smc_tree_attention8(None, ctypes.byref(_cache8()), 0, b, 1, PTR, None, PTR, None, PTR, 1 << 30, None) == ARG
    assert lib.kv_copy_blocks8(None, PTR, PTR, 1, 1, PTR, 256, None) == ARG
    assert lib.kv_compact_tokens8(None, b, PTR, PTR, 1, PTR, 256, None) == ARG


def test_tables_with_room_for_more_tokens_than_32_bits_count(lib):  # noqa: F811
    c = _cache8(kv_heads=1, head_dim=16, token_stride=16, head_stride=16, block_stride=256, layer_stride=2048)
    kw = dict(S=1, rows=1, max_new=1, group=1)
    for T, fits in (((1 << 31) // 16, False), ((1 << 31) // 16 - 255, False), ((1 << 31) // 16 - 256, True)):
        b = _batch(T=T, **kw)
        assert (lib.smc_cache8_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 1) > 0) == fits
        if not fits:
            assert _attn(lib, cache=c, batch=b, q_heads=1) == ARG


def test_a_call_without_rows_is_accepted(lib):  # noqa: F811
    b = _batch(rows=0)
    assert _attn(lib, batch=b, q=None, out=None) == 0
    assert _qk(lib, batch=b, q=None, k=None, v=None, out=None) == 0


def test_struct_layout_matches_the_c_compiler(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "smcsd.h"', 'int main(void){',
             'printf("- %zu\\n", sizeof(smc_cache8));']
    lines += [f'printf("{f} %zu\\n", offsetof(smc_cache8, {f}));' for f, _ in bd.smc_cache8._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join([*lines, "return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        field, size = line.split()
        want = ctypes.sizeof(bd.smc_cache8) if field == "-" else getattr(bd.smc_cache8, field).offset
        assert want == int(size), line


def test_the_binding_refuses_tensors_it_cannot_pass():
    import torch
    x = torch.zeros((1, 4, 16, 2, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones((1, 4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        bd.make_cache8(x, x, s, s)
    with pytest.raises(TypeError):
        bd.make_cache8(x, x, None, s)
    for q in (torch.zeros((12, 8, 128)), torch.zeros((12, 8, 128), dtype=torch.float64)):
        with pytest.raises(ValueError, match="must be one of"):
            bd.smc_tree_attention8(_cache8(), 0, _batch(), q, q, None)
    with pytest.raises(TypeError):
        bd.smc_qk_norm_rope8(_cache8(), 0, _batch(), None, None, None, None, None, None)
