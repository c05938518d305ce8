"""weight_only_bit_gb300 -- fused 4-bit weight-only dequant-GEMV (W4A16) for GB300.

Python binding of libw4 (include/w4.h).  Each function has the C name and argument order,
accepts device buffers as torch tensors (or raw integer addresses), and returns the C status
code; `check(status)` turns a non-zero status into W4Error.  All arithmetic runs in libw4's CUDA
kernels; this module only marshals arguments.  `stream=None` means torch's current CUDA stream.
"""
from __future__ import annotations

import ctypes
import struct

from ._lib import (GemvDesc, GemvPlan, KvCache, W4Error, lib, SYMBOLS, W4_OK, W4_ERR_NULL, W4_ERR_SHAPE, W4_ERR_ALIGN,
                   W4_ERR_BLOCKSIZE, W4_ERR_CUDA, W4_ERR_TIMEOUT, W4_ERR_UNSUPPORTED, W4_FMT_NF4,
                   W4_FMT_INT4, W4_FMT_FP4, W4_MAX_BATCH, W4_MAX_K, W4_KERNEL_SMALL_BATCH, W4_KERNEL_TCGEN05,
                   W4_ERR_LIMIT, W4_ERR_RANGE, W4_MAX_SEQS, W4_MAX_GROUP, W4_MAX_DRAFTS)

__all__ = [
    "w4_nf4_codebook", "w4_quantize_nf4", "w4_quantize_int4", "w4_dequantize_nf4", "w4_dequantize_int4",
    "w4_gemv_nf4", "w4_gemv_int4", "w4_gemv_sequence", "w4_step_workspace_bytes", "w4_step_create",
    "w4_step_launch",
    "w4_step_destroy", "w4_status_str", "w4_last_cuda_error", "w4_device_check", "w4_launch_count",
    "w4_inject_timeout_once", "w4_gemv_levels_noalloc", "w4_gemv_plan",
    "w4_quantize_fp4", "w4_dequantize_fp4", "w4_gemv_fp4", "w4_step_run_host",
    "w4_kv_cache", "w4_kv_append", "w4_attn_workspace_bytes", "w4_attn_kv8", "w4_spec_verify_workspace_bytes",
    "w4_spec_verify", "KvCache", "W4_ERR_RANGE", "W4_MAX_SEQS", "W4_MAX_GROUP", "W4_MAX_DRAFTS",
    "check", "W4Error", "GemvDesc", "GemvPlan", "W4_FMT_NF4", "W4_FMT_INT4", "W4_FMT_FP4", "W4_MAX_BATCH",
    "W4_MAX_K",
    "W4_KERNEL_SMALL_BATCH", "W4_KERNEL_TCGEN05",
]


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw = None          # (device index, device -> stream handle), once torch has set CUDA up


def _current_stream():
    """Handle of torch's current stream; 0 without a GPU.  torch.cuda.current_stream() builds an object and
    asks the driver whether a GPU is there: 3.7 us a call, as long as a launch; the handle itself is
    0.2 us."""
    global _raw
    if _raw is not None:
        return _raw[1](_raw[0]())
    import torch
    if not torch.cuda.is_available():
        return 0
    s = torch.cuda.current_stream().cuda_stream
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if get is not None:
        _raw = (torch.cuda.current_device, get)
    return s


def _stream(s):
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def check(status: int, what: str = "") -> int:
    if status != W4_OK:
        raise W4Error(status, what)
    return status


def w4_nf4_codebook():
    """Host function: returns (status, list of 16 floats)."""
    out = (ctypes.c_float * 16)()
    st = lib().w4_nf4_codebook(out)
    return st, list(out)


def w4_quantize_nf4(W, packed, absmax, codebook, N, K, blocksize=64, stream=None):
    return lib().w4_quantize_nf4(_ptr(W), _ptr(packed), _ptr(absmax), _ptr(codebook), N, K, blocksize,
                                 _stream(stream))


def w4_quantize_int4(W, packed, scale, N, K, group=128, stream=None):
    return lib().w4_quantize_int4(_ptr(W), _ptr(packed), _ptr(scale), N, K, group, _stream(stream))


def w4_quantize_fp4(W, packed, scale, N, K, group=32, stream=None):
    return lib().w4_quantize_fp4(_ptr(W), _ptr(packed), _ptr(scale), N, K, group, _stream(stream))


def w4_dequantize_nf4(packed, absmax, codebook, W_out, N, K, blocksize=64, stream=None):
    return lib().w4_dequantize_nf4(_ptr(packed), _ptr(absmax), _ptr(codebook), _ptr(W_out), N, K, blocksize,
                                   _stream(stream))


def w4_dequantize_int4(packed, scale, W_out, N, K, group=128, stream=None):
    return lib().w4_dequantize_int4(_ptr(packed), _ptr(scale), _ptr(W_out), N, K, group, _stream(stream))


def w4_dequantize_fp4(packed, scale, W_out, N, K, group=32, stream=None):
    return lib().w4_dequantize_fp4(_ptr(packed), _ptr(scale), _ptr(W_out), N, K, group, _stream(stream))


def w4_gemv_nf4(packed, absmax, codebook, x, y, M, N, K, blocksize=64, stream=None):
    return lib().w4_gemv_nf4(_ptr(packed), _ptr(absmax), _ptr(codebook), _ptr(x), _ptr(y), M, N, K, blocksize,
                             _stream(stream))


def w4_gemv_int4(packed, scale, x, y, M, N, K, group=128, stream=None):
    return lib().w4_gemv_int4(_ptr(packed), _ptr(scale), _ptr(x), _ptr(y), M, N, K, group, _stream(stream))


def w4_gemv_fp4(packed, scale, x, y, M, N, K, group=32, stream=None):
    return lib().w4_gemv_fp4(_ptr(packed), _ptr(scale), _ptr(x), _ptr(y), M, N, K, group, _stream(stream))


def _descs(descs):
    arr = (GemvDesc * len(descs))()
    for i, d in enumerate(descs):
        arr[i] = GemvDesc(d["format"], _ptr(d["packed"]), _ptr(d["scales"]), _ptr(d.get("codebook")),
                          _ptr(d["x"]), _ptr(d["y"]), d["M"], d["N"], d["K"], d["blocksize"], d.get("level", i))
    return arr


def w4_gemv_sequence(descs, stream=None):
    """descs: sequence of dicts with keys format, packed, scales, codebook, x, y, M, N, K, blocksize and
    optionally level (default: the descriptor's index, i.e. every GEMV waits for the one before)."""
    arr = _descs(descs)
    return lib().w4_gemv_sequence(arr, len(descs), _stream(stream))


def w4_step_workspace_bytes(count: int) -> int:
    return lib().w4_step_workspace_bytes(count)


def w4_step_create(descs, workspace):
    """Returns (status, handle).  workspace: device buffer of w4_step_workspace_bytes(len(descs))."""
    arr = _descs(descs)
    h = ctypes.c_void_p()
    st = lib().w4_step_create(arr, len(descs), _ptr(workspace), ctypes.byref(h))
    return st, h.value


def w4_step_launch(step, stream=None):
    return lib().w4_step_launch(step, _stream(stream))


def w4_step_run_host(step, x_host, x_dev, x_bytes, y_host, y_dev, y_bytes, stream=None):
    """x_host / y_host: pinned host tensors (or raw addresses); x_dev / y_dev: the step's device
    input and output buffers."""
    return lib().w4_step_run_host(step, _ptr(x_host), _ptr(x_dev), x_bytes, _ptr(y_host), _ptr(y_dev), y_bytes,
                                  _stream(stream))


def w4_step_destroy(step):
    return lib().w4_step_destroy(step)


def w4_status_str(status: int) -> str:
    return lib().w4_status_str(status).decode()


def w4_last_cuda_error() -> int:
    return lib().w4_last_cuda_error()


def w4_device_check(stream=None) -> int:
    return lib().w4_device_check(_stream(stream))


def w4_gemv_plan(format: int, M: int, N: int, K: int, blocksize: int, sm_count: int = 152):
    """Host function: returns (status, dict of w4_gemv_plan_t's fields); no device call."""
    out = GemvPlan()
    st = lib().w4_gemv_plan(format, M, N, K, blocksize, sm_count, ctypes.byref(out))
    return st, {name: getattr(out, name) for name, _ in GemvPlan._fields_}


def w4_launch_count() -> int:
    return lib().w4_launch_count()


def w4_inject_timeout_once() -> int:
    return lib().w4_inject_timeout_once()


def w4_gemv_levels_noalloc(descs, stream=None) -> int:
    """One persistent launch of the descriptors with the level counters inside libw4, for callers
    that cannot allocate device memory; see include/w4.h for its limits and its one-time set-up."""
    arr = _descs(descs)
    return lib().w4_gemv_levels_noalloc(arr, len(descs), _stream(stream))


# ---------------------------------------------------------------- paged 8-bit cache, attention, drafts


def _nbytes(workspace, given):
    if given is not None:
        return given
    if workspace is None:
        return 0
    if isinstance(workspace, int):
        raise W4Error(W4_ERR_SHAPE, "a workspace given as an address needs workspace_bytes")
    return workspace.numel() * workspace.element_size()


def w4_kv_cache(k, v, k_scale, v_scale, page_table, *, num_pages, kv_heads, page_tokens, head_dim, table_stride,
                page_stride=0, scale_stride=0):
    """The cache descriptor that w4_kv_append and w4_attn_kv8 take (w4_kv_cache of include/w4.h); it
    keeps the tensors it was made of."""
    c = KvCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), page_stride, scale_stride, num_pages,
                kv_heads, page_tokens, head_dim, table_stride)
    c.tensors = (k, v, k_scale, v_scale, page_table)
    return c


_append_args = struct.Struct("11P4q8i").pack        # w4_kv_append_args


def w4_kv_append(cache, q, k, v, q_out, rope_cos, rope_sin, q_start, kv_len, tokens, batch, q_heads, max_q,
                 max_position, rotary_dim, interleaved=0, positions=None, q_stride=0, k_stride=0, v_stride=0,
                 q_out_stride=0, stream=None):
    """Rotates q and k, appends k and v to the cache; strides are elements from row to row (0: dense)."""
    # one packed block: with 22 arguments for ctypes to convert, the call took 6.9 us and not 5.3
    return lib().w4_kv_append_block(_append_args(
        0 if cache is None else ctypes.addressof(cache), _ptr(q) or 0, _ptr(k) or 0, _ptr(v) or 0, _ptr(q_out) or 0,
        _ptr(rope_cos) or 0, _ptr(rope_sin) or 0, _ptr(positions) or 0, _ptr(q_start) or 0, _ptr(kv_len) or 0,
        _stream(stream) or 0, q_stride, k_stride, v_stride, q_out_stride, tokens, batch, q_heads, max_q, max_position,
        rotary_dim, 1 if interleaved else 0, 0))


def w4_attn_workspace_bytes(tokens: int, batch: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return lib().w4_attn_workspace_bytes(tokens, batch, q_heads, kv_heads, head_dim)


_attn_args = struct.Struct("8P3q6ifi").pack          # w4_attn_kv8_args


def w4_attn_kv8(cache, q, out, lse, q_start, kv_len, tokens, batch, q_heads, max_q, softmax_scale, workspace, causal=1,
                window=0, q_stride=0, out_stride=0, workspace_bytes=None, stream=None):
    """Attention of the new rows over the cache.  workspace: w4_attn_workspace_bytes(...) bytes, zeroed once."""
    return lib().w4_attn_kv8_block(_attn_args(
        0 if cache is None else ctypes.addressof(cache), _ptr(q) or 0, _ptr(out) or 0, _ptr(lse) or 0, _ptr(q_start) or 0,
        _ptr(kv_len) or 0, _ptr(workspace) or 0, _stream(stream) or 0, q_stride, out_stride,
        _nbytes(workspace, workspace_bytes), tokens, batch, q_heads, max_q, 1 if causal else 0, window, softmax_scale, 0))


def w4_spec_verify_workspace_bytes(batch: int, drafts: int, vocab: int) -> int:
    return lib().w4_spec_verify_workspace_bytes(batch, drafts, vocab)


def w4_spec_verify(target, draft, draft_tokens, u, e, tokens, accepted, logprob, batch, drafts, vocab, temperature,
                   workspace, n_drafts=None, target_stride=0, draft_stride=0, workspace_bytes=None, stream=None):
    """Verification of drafted tokens from logits.  workspace: w4_spec_verify_workspace_bytes(...) bytes,
    zeroed once."""
    return lib().w4_spec_verify(_ptr(target), _ptr(draft), _ptr(draft_tokens), _ptr(u), _ptr(e), _ptr(tokens),
                                _ptr(accepted), _ptr(logprob), batch, drafts, vocab, temperature, _ptr(n_drafts),
                                target_stride, draft_stride, _ptr(workspace), _nbytes(workspace, workspace_bytes),
                                _stream(stream))
