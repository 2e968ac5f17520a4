"""Thin Python binding of libsmcsd.so (include/smcsd.h), by ctypes.

Argument marshalling only: every function checks that the tensors it is given
are CUDA, contiguous and of the expected dtype and size, passes their device
pointers and the caller's stream to the C entry point of the same name, and
raises ``SmcError`` on a non-zero return.  All arithmetic runs in the
library's kernels; there is no CPU path.  PyTorch supplies device memory and
streams only.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsmcsd.so")

SMC_F32, SMC_BF16, SMC_F16 = 0, 1, 2

# device status bits (smcsd.h)
DEV_BITS = {
    0x01: "bad_token", 0x02: "nonfinite", 0x04: "empty_row", 0x08: "all_zero_weight",
    0x10: "pool_exhausted", 0x20: "table_overflow", 0x40: "bad_block", 0x80: "timeout",
    0x100: "bad_rows",
}


class SmcError(RuntimeError):
    """A non-zero return code of a libsmcsd entry point."""

    def __init__(self, fn, code, text):
        super().__init__(f"{fn} returned {code}: {text}")
        self.code = code


class smc_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("V", ctypes.c_int32), ("dtype", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("ess_frac", ctypes.c_float), ("seed", ctypes.c_uint64), ("step", ctypes.c_uint32)]


class smc_kv(ctypes.Structure):
    _fields_ = [("tables", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("refcount", ctypes.c_void_p), ("free_list", ctypes.c_void_p),
                ("free_top", ctypes.c_void_p), ("cow_pairs", ctypes.c_void_p),
                ("n_cow", ctypes.c_void_p), ("T", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("P", ctypes.c_int32)]


class smc_step_opts(ctypes.Structure):
    _fields_ = [("log_potential", ctypes.c_void_p), ("temperature", ctypes.c_float),
                ("top_p", ctypes.c_float), ("reserved", ctypes.c_int32 * 2)]


class smc_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("block_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("layers", ctypes.c_int32),
                ("blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class smc_batch(ctypes.Structure):
    _fields_ = [("tables", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("row_start", ctypes.c_void_p), ("S", ctypes.c_int32), ("T", ctypes.c_int32),
                ("rows", ctypes.c_int32), ("max_new", ctypes.c_int32), ("group", ctypes.c_int32)]


class smc_attn_params(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("mask_words", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64)]


class smc_qk_params(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("max_pos", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("k_row_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_row_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64)]


_lib = None

_SIGS = {
    "smc_abi_version": (ctypes.c_int32, []),
    "smc_strerror": (ctypes.c_char_p, [ctypes.c_int32]),
    "smc_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(smc_params), ctypes.POINTER(smc_kv)]),
    "smc_workspace_init": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "smc_device_status": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int32,
                                           ctypes.POINTER(ctypes.c_int32), ctypes.c_void_p]),
    "smc_step": (ctypes.c_int32, [ctypes.POINTER(smc_params)] + [ctypes.c_void_p] * 8 +
                 [ctypes.POINTER(smc_kv), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "smc_resample": (ctypes.c_int32, [ctypes.POINTER(smc_params)] + [ctypes.c_void_p] * 4 +
                     [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "kv_blocktable_remap": (ctypes.c_int32, [ctypes.POINTER(smc_params), ctypes.POINTER(smc_kv),
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "sps_verify": (ctypes.c_int32, [ctypes.POINTER(smc_params)] + [ctypes.c_void_p] * 5 +
                   [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "sps_verify_ex": (ctypes.c_int32, [ctypes.POINTER(smc_params)] + [ctypes.c_void_p] * 5 +
                      [ctypes.POINTER(smc_step_opts), ctypes.c_void_p, ctypes.c_size_t,
                       ctypes.c_void_p]),
    "smc_set_row_timing_events": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p]),
    "smc_set_step_clock": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32]),
    "smc_selftest_bounded_wait": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32,
                                                   ctypes.c_int32, ctypes.c_void_p]),
    "smc_step_ex": (ctypes.c_int32, [ctypes.POINTER(smc_params), ctypes.POINTER(smc_step_opts)] +
                    [ctypes.c_void_p] * 8 +
                    [ctypes.POINTER(smc_kv), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "smc_draft_sample": (ctypes.c_int32, [ctypes.POINTER(smc_params), ctypes.c_void_p,
                                          ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_size_t, ctypes.c_void_p]),
    "smc_kv_usage": (ctypes.c_int32, [ctypes.POINTER(smc_params), ctypes.POINTER(smc_kv),
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "smc_cache_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(smc_cache),
                                                    ctypes.POINTER(smc_batch), ctypes.c_int32]),
    "smc_tree_attention": (ctypes.c_int32, [ctypes.POINTER(smc_attn_params),
                                            ctypes.POINTER(smc_cache), ctypes.c_int32,
                                            ctypes.POINTER(smc_batch)] + [ctypes.c_void_p] * 4 +
                           [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "smc_qk_norm_rope": (ctypes.c_int32, [ctypes.POINTER(smc_qk_params),
                                          ctypes.POINTER(smc_cache), ctypes.c_int32,
                                          ctypes.POINTER(smc_batch)] + [ctypes.c_void_p] * 8 +
                         [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "kv_copy_blocks": (ctypes.c_int32, [ctypes.POINTER(smc_cache), ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "kv_compact_tokens": (ctypes.c_int32, [ctypes.POINTER(smc_cache), ctypes.POINTER(smc_batch),
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                           ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "kv_truncate": (ctypes.c_int32, [ctypes.POINTER(smc_params), ctypes.POINTER(smc_kv),
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                     ctypes.c_void_p]),
}


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m smc_speculative_decoding_gb300.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(fn, rc):
    if rc != 0:
        raise SmcError(fn, rc, lib().smc_strerror(rc).decode())


def _ptr(t, name, dtype=None, numel=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, got {t.numel()}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_params(B, N, K, V, dtype="bf16", alpha=1.0, ess_frac=0.5, seed=0, step=0):
    """smc_params for a shape; dtype is "bf16"/"f32" or a torch dtype."""
    if dtype in ("bf16", torch.bfloat16):
        code = SMC_BF16
    elif dtype in ("f32", torch.float32):
        code = SMC_F32
    else:
        raise ValueError(f"unsupported dtype {dtype!r}")
    return smc_params(int(B), int(N), int(K), int(V), code, float(alpha), float(ess_frac),
                      int(seed), int(step) & 0xFFFFFFFF)


_KV_KEYS = ("tables", "seq_len", "refcount", "free_list", "free_top", "cow_pairs", "n_cow")


def make_kv(params, kv, block_size):
    """smc_kv over a dict of int32 CUDA tensors (see workloads.make_kv_state)."""
    B, N = params.B, params.N
    T = kv["tables"].shape[-1]
    P = kv["free_list"].shape[-1]
    sizes = dict(tables=B * N * T, seq_len=B * N, refcount=B * P, free_list=B * P,
                 free_top=B, cow_pairs=B * N * 2, n_cow=B)
    ptrs = {k: _ptr(kv[k], f"kv[{k!r}]", torch.int32, sizes[k]) for k in _KV_KEYS}
    return smc_kv(*(ptrs[k] for k in _KV_KEYS), int(T), int(block_size), int(P))


def smc_abi_version():
    return lib().smc_abi_version()


def smc_strerror(code):
    return lib().smc_strerror(int(code)).decode()


def smc_workspace_bytes(params, kv=None):
    n = lib().smc_workspace_bytes(ctypes.byref(params), ctypes.byref(kv) if kv is not None else None)
    if n == 0:
        raise SmcError("smc_workspace_bytes", -1, "invalid shape")
    return n


def alloc_workspace(params, kv=None, device="cuda"):
    """A zero-filled workspace tensor of smc_workspace_bytes() bytes."""
    return torch.zeros(smc_workspace_bytes(params, kv), dtype=torch.uint8, device=device)


def smc_workspace_init(workspace, stream=None):
    _check("smc_workspace_init", lib().smc_workspace_init(
        _ptr(workspace, "workspace"), workspace.numel(), _stream(stream)))


def smc_device_status(workspace, clear=False, stream=None):
    """Device status bits of a workspace (synchronises the stream)."""
    out = ctypes.c_int32(0)
    _check("smc_device_status", lib().smc_device_status(
        _ptr(workspace, "workspace"), int(bool(clear)), ctypes.byref(out), _stream(stream)))
    return out.value


def smc_set_row_timing_events(rows_begin=None, rows_end=None):
    """Record two torch.cuda.Event objects (created with enable_timing=True)
    around the row pass of every later step; None, None turns it off.

    The events are recorded once here, on the current stream, so that torch
    creates them and treats them as recorded; the library records them
    again, around the row pass, at every later step."""
    def handle(ev):
        if ev is None:
            return None
        if not isinstance(ev, torch.cuda.Event):
            raise TypeError("expected a torch.cuda.Event")
        ev.record()
        return ctypes.c_void_p(ev.cuda_event)
    _check("smc_set_row_timing_events",
           lib().smc_set_row_timing_events(handle(rows_begin), handle(rows_end)))


def smc_set_step_clock(stamps=None, counter=None):
    """Device-side step clock: `stamps` (int64 CUDA tensor) receives the GPU
    timer (ns) as each later step's row pass starts, at index counter[0]++
    (`counter`: int32 CUDA tensor of one element, zeroed by the caller).
    None turns it off."""
    if stamps is None:
        _check("smc_set_step_clock", lib().smc_set_step_clock(None, None, 0))
        return
    if not (stamps.is_cuda and stamps.dtype == torch.int64 and counter is not None
            and counter.is_cuda and counter.dtype == torch.int32 and counter.numel() >= 1):
        raise TypeError("stamps: int64 CUDA tensor; counter: int32 CUDA tensor")
    _check("smc_set_step_clock",
           lib().smc_set_step_clock(ctypes.c_void_p(stamps.data_ptr()),
                                    ctypes.c_void_p(counter.data_ptr()), stamps.numel()))


def smc_selftest_bounded_wait(workspace, kind, poll_limit=1000, stream=None):
    """Run one of the library's bounded waits (kind 0: counter, 1: mbarrier)
    against a condition nothing satisfies; it raises the timeout status bit
    in `workspace` (a zeroed uint8 CUDA tensor of at least 8 bytes)."""
    _check("smc_selftest_bounded_wait",
           lib().smc_selftest_bounded_wait(ctypes.c_void_p(workspace.data_ptr()),
                                           workspace.numel() * workspace.element_size(),
                                           kind, poll_limit, _stream(stream)))


def status_names(bits):
    return [name for bit, name in DEV_BITS.items() if bits & bit]


def _logit_dtype(params):
    return torch.bfloat16 if params.dtype == SMC_BF16 else torch.float32


def smc_step(params, target_logits, draft_logits, draft_tokens, log_weights, tokens_out,
             ancestors, ess, resampled, kv=None, workspace=None, stream=None):
    B, N, K, V = params.B, params.N, params.K, params.V
    ld = _logit_dtype(params)
    args = [
        _ptr(target_logits, "target_logits", ld, B * N * (K + 1) * V),
        _ptr(draft_logits, "draft_logits", ld, B * N * K * V),
        _ptr(draft_tokens, "draft_tokens", torch.int32, B * N * K),
        _ptr(log_weights, "log_weights", torch.float32, B * N),
        _ptr(tokens_out, "tokens_out", torch.int32, B * N * (K + 1)),
        _ptr(ancestors, "ancestors", torch.int32, B * N),
        _ptr(ess, "ess", torch.float32, B),
        _ptr(resampled, "resampled", torch.int32, B),
    ]
    _check("smc_step", lib().smc_step(
        ctypes.byref(params), *args, ctypes.byref(kv) if kv is not None else None,
        _ptr(workspace, "workspace"), workspace.numel(), _stream(stream)))


def smc_step_ex(params, target_logits, draft_logits, draft_tokens, log_weights, tokens_out,
                ancestors, ess, resampled, kv=None, workspace=None, stream=None,
                temperature=1.0, log_potential=None, top_p=1.0):
    """smc_step with a temperature, a top-p nucleus and an optional [B, N]
    fp32 CUDA tensor of per-particle log-potential increments (smc_step_ex in
    smcsd.h)."""
    B, N, K, V = params.B, params.N, params.K, params.V
    ld = _logit_dtype(params)
    opts = smc_step_opts(
        _ptr(log_potential, "log_potential", torch.float32, B * N) if log_potential is not None
        else None, float(temperature), float(top_p))
    args = [
        _ptr(target_logits, "target_logits", ld, B * N * (K + 1) * V),
        _ptr(draft_logits, "draft_logits", ld, B * N * K * V),
        _ptr(draft_tokens, "draft_tokens", torch.int32, B * N * K),
        _ptr(log_weights, "log_weights", torch.float32, B * N),
        _ptr(tokens_out, "tokens_out", torch.int32, B * N * (K + 1)),
        _ptr(ancestors, "ancestors", torch.int32, B * N),
        _ptr(ess, "ess", torch.float32, B),
        _ptr(resampled, "resampled", torch.int32, B),
    ]
    _check("smc_step_ex", lib().smc_step_ex(
        ctypes.byref(params), ctypes.byref(opts), *args,
        ctypes.byref(kv) if kv is not None else None,
        _ptr(workspace, "workspace"), workspace.numel(), _stream(stream)))


def smc_draft_sample(params, draft_logits, position, tokens_out, workspace, stream=None):
    """One token per particle from softmax(alpha * l) of draft_logits [B, N, V]."""
    B, N, V = params.B, params.N, params.V
    _check("smc_draft_sample", lib().smc_draft_sample(
        ctypes.byref(params), _ptr(draft_logits, "draft_logits", _logit_dtype(params), B * N * V),
        int(position), _ptr(tokens_out, "tokens_out", torch.int32, B * N),
        _ptr(workspace, "workspace"), workspace.numel(), _stream(stream)))


def smc_kv_usage(params, kv, used_blocks, unshared_blocks, stream=None):
    """Per prompt: blocks in use with sharing, and blocks unshared copies would hold."""
    B = params.B
    _check("smc_kv_usage", lib().smc_kv_usage(
        ctypes.byref(params), ctypes.byref(kv), _ptr(used_blocks, "used_blocks", torch.int32, B),
        _ptr(unshared_blocks, "unshared_blocks", torch.int32, B), _stream(stream)))


def smc_resample(params, log_weights, ancestors, ess, resampled, workspace, stream=None):
    B, N = params.B, params.N
    _check("smc_resample", lib().smc_resample(
        ctypes.byref(params), _ptr(log_weights, "log_weights", torch.float32, B * N),
        _ptr(ancestors, "ancestors", torch.int32, B * N), _ptr(ess, "ess", torch.float32, B),
        _ptr(resampled, "resampled", torch.int32, B), _ptr(workspace, "workspace"),
        workspace.numel(), _stream(stream)))


def kv_blocktable_remap(params, kv, ancestors, resampled, n_append, workspace, stream=None):
    B, N = params.B, params.N
    _check("kv_blocktable_remap", lib().kv_blocktable_remap(
        ctypes.byref(params), ctypes.byref(kv), _ptr(ancestors, "ancestors", torch.int32, B * N),
        _ptr(resampled, "resampled", torch.int32, B), int(n_append),
        _ptr(workspace, "workspace"), workspace.numel(), _stream(stream)))


def sps_verify(params, target_logits, draft_logits, draft_tokens, tokens_out, n_emitted,
               workspace, stream=None):
    B, K, V = params.B, params.K, params.V
    ld = _logit_dtype(params)
    _check("sps_verify", lib().sps_verify(
        ctypes.byref(params), _ptr(target_logits, "target_logits", ld, B * (K + 1) * V),
        _ptr(draft_logits, "draft_logits", ld, B * K * V),
        _ptr(draft_tokens, "draft_tokens", torch.int32, B * K),
        _ptr(tokens_out, "tokens_out", torch.int32, B * (K + 1)),
        _ptr(n_emitted, "n_emitted", torch.int32, B),
        _ptr(workspace, "workspace"), workspace.numel(), _stream(stream)))


def sps_verify_ex(params, target_logits, draft_logits, draft_tokens, tokens_out, n_emitted,
                  workspace, stream=None, temperature=1.0, top_p=1.0):
    """sps_verify under a temperature and a top-p nucleus (sps_verify_ex in
    smcsd.h)."""
    B, K, V = params.B, params.K, params.V
    ld = _logit_dtype(params)
    opts = smc_step_opts(None, float(temperature), float(top_p))
    _check("sps_verify_ex", lib().sps_verify_ex(
        ctypes.byref(params), _ptr(target_logits, "target_logits", ld, B * (K + 1) * V),
        _ptr(draft_logits, "draft_logits", ld, B * K * V),
        _ptr(draft_tokens, "draft_tokens", torch.int32, B * K),
        _ptr(tokens_out, "tokens_out", torch.int32, B * (K + 1)),
        _ptr(n_emitted, "n_emitted", torch.int32, B), ctypes.byref(opts),
        _ptr(workspace, "workspace"), workspace.numel(), _stream(stream)))


def smc_step_noalloc(params, target_logits, draft_logits, draft_tokens, log_weights, tokens_out,
                     ancestors, ess, resampled, status_bits, kv=None, stream=None):
    """smc_step without a caller workspace: the library's own fixed scratch
    array is used (see smc_step_noalloc in smcsd.h).  status_bits is a CUDA
    int32 tensor of one element that receives this call's device status."""
    fn = lib().smc_step_noalloc
    fn.restype = ctypes.c_int32
    fn.argtypes = [ctypes.POINTER(smc_params)] + [ctypes.c_void_p] * 8 + \
        [ctypes.POINTER(smc_kv), ctypes.c_void_p, ctypes.c_void_p]
    B, N, K, V = params.B, params.N, params.K, params.V
    ld = _logit_dtype(params)
    args = [
        _ptr(target_logits, "target_logits", ld, B * N * (K + 1) * V),
        _ptr(draft_logits, "draft_logits", ld, B * N * K * V),
        _ptr(draft_tokens, "draft_tokens", torch.int32, B * N * K),
        _ptr(log_weights, "log_weights", torch.float32, B * N),
        _ptr(tokens_out, "tokens_out", torch.int32, B * N * (K + 1)),
        _ptr(ancestors, "ancestors", torch.int32, B * N),
        _ptr(ess, "ess", torch.float32, B),
        _ptr(resampled, "resampled", torch.int32, B),
    ]
    _check("smc_step_noalloc", fn(ctypes.byref(params), *args,
                                  ctypes.byref(kv) if kv is not None else None,
                                  _ptr(status_bits, "status_bits", torch.int32, 1),
                                  _stream(stream)))


# ---- the paged cache's data ------------------------------------------------

_CACHE_DTYPES = {torch.float32: SMC_F32, torch.bfloat16: SMC_BF16, torch.float16: SMC_F16}
_CACHE_TORCH = {code: dtype for dtype, code in _CACHE_DTYPES.items()}


def _addr(t, name, dtype, numel=None):
    """The address of a contiguous CUDA tensor, for the calls of a decoding
    loop: the checks of _ptr, the common case in one expression."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (numel is None or t.numel() == numel)):
        return t.data_ptr()
    return _ptr(t, name, dtype, numel).value


def _raw_stream(stream, tensor):
    """The stream's handle; without one, the current stream of the tensor's
    device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(tensor.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def make_cache(k, v):
    """smc_cache over keys and values [layers, blocks, block_size, kv_heads,
    head_dim]: CUDA tensors of one dtype (fp32, bf16 or fp16), one shape and
    one set of strides, the last of them 1 (a head-major cache, or a slice of
    a larger one, is passed as a view).  The struct keeps the tensors alive."""
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
        if t.dim() != 5 or t.dtype not in _CACHE_DTYPES:
            raise ValueError(f"{name} must be [layers, blocks, block_size, kv_heads, head_dim] "
                             f"in fp32, bf16 or fp16, got {tuple(t.shape)} {t.dtype}")
    if k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
        raise ValueError("k and v must have one shape, dtype and set of strides")
    if k.numel() == 0 or (k.stride(4) != 1 and k.shape[4] > 1):
        raise ValueError("k and v must not be empty and their last axis must be contiguous")
    cache = smc_cache(k.data_ptr(), v.data_ptr(), *k.stride()[:4], *k.shape, _CACHE_DTYPES[k.dtype])
    cache.tensors = (k, v)
    return cache


def make_batch(tables, seq_len, max_new, row_start=None, rows=None, group=1):
    """smc_batch over a call's sequences: tables [S, T] (or [B, N, T], as in
    the KV state) and seq_len [S] int32, at most max_new new tokens each;
    row_start [S + 1] int32 when their numbers differ, with `rows` rows in the
    arrays (default S * max_new).  group: consecutive sequences of one prompt.
    The struct keeps the tensors alive."""
    S = seq_len.numel()
    T = tables.shape[-1]
    if rows is None:
        rows = S * max_new
    batch = smc_batch(_ptr(tables, "tables", torch.int32, S * T),
                      _ptr(seq_len, "seq_len", torch.int32),
                      None if row_start is None else _ptr(row_start, "row_start", torch.int32, S + 1),
                      S, T, int(rows), int(max_new), int(group))
    batch.tensors = (tables, seq_len, row_start)
    return batch


def smc_cache_workspace_bytes(cache, batch=None, q_heads=0):
    n = lib().smc_cache_workspace_bytes(
        ctypes.byref(cache), None if batch is None else ctypes.byref(batch), int(q_heads))
    if n == 0:
        raise SmcError("smc_cache_workspace_bytes", -1, "invalid shape")
    return n


def alloc_cache_workspace(cache, batch=None, q_heads=0, device="cuda"):
    """A zero-filled workspace for the cache entry points: with a batch and
    q_heads for all of them, without for those that take no batch."""
    return torch.zeros(smc_cache_workspace_bytes(cache, batch, q_heads), dtype=torch.uint8,
                       device=device)


def _rows(t, name, dtype, shape):
    """A [rows, heads, head_dim] CUDA tensor of the cache's dtype, its last
    axis contiguous: its address and its row and head strides."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape:
        row, head, dim = t.stride()
        if dim == 1 or shape[2] == 1:
            return t.data_ptr(), row, head
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {shape} in {dtype}, got {tuple(t.shape)} {t.dtype}")
    raise ValueError(f"{name}'s last axis must be contiguous")


def smc_tree_attention(cache, layer, batch, q, out, workspace, mask=None, lse=None, scale=None,
                       stream=None):
    """Attention of the new tokens q [rows, q_heads, head_dim] over their
    sequences' caches into out; mask [rows, words] int32 of packed bits (None:
    a chain), lse [rows, q_heads] fp32 (None: not wanted), scale (None:
    head_dim ** -0.5).  See smc_tree_attention in smcsd.h."""
    rows, dim, dtype = batch.rows, cache.head_dim, _CACHE_TORCH[cache.dtype]
    if q.dim() != 3:
        raise ValueError("q must be [rows, q_heads, head_dim]")
    heads = q.shape[1]
    shape = (rows, heads, dim)
    qp, q_row, q_head = _rows(q, "q", dtype, shape)
    op, o_row, o_head = _rows(out, "out", dtype, shape)
    words = 0
    if mask is not None:
        # (a tensor of no words has no address: it would count as no mask, which is a chain)
        if mask.dim() != 2 or mask.shape[0] != rows or mask.shape[1] < 1:
            raise ValueError(f"mask must be [{rows}, words] with at least one word, got {tuple(mask.shape)}")
        words = mask.shape[1]
    params = smc_attn_params(heads, words, dim ** -0.5 if scale is None else scale, 0,
                             q_row, q_head, o_row, o_head)
    _check("smc_tree_attention", (_lib or lib()).smc_tree_attention(
        ctypes.byref(params), ctypes.byref(cache), layer, ctypes.byref(batch), qp,
        None if mask is None else _addr(mask, "mask", torch.int32), op,
        None if lse is None else _addr(lse, "lse", torch.float32, rows * heads),
        _addr(workspace, "workspace", torch.uint8), workspace.numel(), _raw_stream(stream, workspace)))


def smc_qk_norm_rope(cache, layer, batch, q, k, v, rope, q_out, workspace, positions=None,
                     q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, interleaved=False,
                     stream=None):
    """Norms and rotation of the new tokens' q [rows, q_heads, head_dim] (into
    q_out) and k [rows, kv_heads, head_dim] (into the cache, with v).  rope
    [max_pos, rot_dim] fp32: cosines, then sines; positions [rows] int32
    (None: the tokens' own); weights [head_dim] (None: no norm).  See
    smc_qk_norm_rope in smcsd.h."""
    rows, dim, dtype = batch.rows, cache.head_dim, _CACHE_TORCH[cache.dtype]
    if q.dim() != 3 or rope.dim() != 2:
        raise ValueError("q must be [rows, q_heads, head_dim] and rope [max_pos, rot_dim]")
    heads = q.shape[1]
    shape, kv_shape = (rows, heads, dim), (rows, cache.kv_heads, dim)
    qp, q_row, q_head = _rows(q, "q", dtype, shape)
    kp, k_row, k_head = _rows(k, "k", dtype, kv_shape)
    vp, v_row, v_head = _rows(v, "v", dtype, kv_shape)
    op, o_row, o_head = _rows(q_out, "q_out", dtype, shape)
    max_pos, rot = rope.shape
    params = smc_qk_params(heads, rot, max_pos, 1 if interleaved else 0, eps, weight_offset, q_row,
                           q_head, k_row, k_head, v_row, v_head, o_row, o_head)
    _check("smc_qk_norm_rope", (_lib or lib()).smc_qk_norm_rope(
        ctypes.byref(params), ctypes.byref(cache), layer, ctypes.byref(batch), qp, kp, vp,
        None if q_weight is None else _addr(q_weight, "q_weight", dtype, dim),
        None if k_weight is None else _addr(k_weight, "k_weight", dtype, dim),
        None if positions is None else _addr(positions, "positions", torch.int32, rows),
        _addr(rope, "rope", torch.float32), op, _addr(workspace, "workspace", torch.uint8), workspace.numel(),
        _raw_stream(stream, workspace)))


def kv_copy_blocks(cache, pairs, counts, workspace, stream=None):
    """Copies blocks pairs[l, i, 0] to pairs[l, i, 1], i < counts[l], in every
    layer: a step's cow_pairs [B, N, 2] and n_cow [B]."""
    if pairs.dim() != 3 or pairs.shape[2] != 2:
        raise ValueError(f"pairs must be [lists, max_pairs, 2], got {tuple(pairs.shape)}")
    lists, most = pairs.shape[:2]
    _check("kv_copy_blocks", (_lib or lib()).kv_copy_blocks(
        ctypes.byref(cache), _addr(pairs, "pairs", torch.int32),
        _addr(counts, "counts", torch.int32, lists), lists, most, _addr(workspace, "workspace", torch.uint8),
        workspace.numel(), _raw_stream(stream, workspace)))


def kv_compact_tokens(cache, batch, path, n_path, workspace, stream=None):
    """Moves new tokens path[s, i] (ascending), i < n_path[s], to new token i
    of their sequence, in every layer; path [S, max_path], n_path [S] int32."""
    if path.dim() != 2:
        raise ValueError(f"path must be [S, max_path], got {tuple(path.shape)}")
    _check("kv_compact_tokens", (_lib or lib()).kv_compact_tokens(
        ctypes.byref(cache), ctypes.byref(batch),
        _addr(path, "path", torch.int32, batch.S * path.shape[1]),
        _addr(n_path, "n_path", torch.int32, batch.S), path.shape[1],
        _addr(workspace, "workspace", torch.uint8), workspace.numel(), _raw_stream(stream, workspace)))


def kv_truncate(params, kv, new_len, workspace, stream=None):
    """Shortens every particle to new_len [B, N] int32 tokens and gives the
    blocks past them back."""
    _check("kv_truncate", (_lib or lib()).kv_truncate(
        ctypes.byref(params), ctypes.byref(kv),
        _addr(new_len, "new_len", torch.int32, params.B * params.N), _addr(workspace, "workspace", torch.uint8),
        workspace.numel(), _raw_stream(stream, workspace)))
