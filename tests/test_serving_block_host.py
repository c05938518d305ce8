"""The calls that take their arguments in one block: every field lands where the separate call has it."""
import ctypes

import pytest

import weight_only_bit_gb300 as w4
from weight_only_bit_gb300 import _lib

A = 1 << 20        # fake, never dereferenced device addresses


def _cache(**kw):
    d = dict(num_pages=8, kv_heads=2, page_tokens=64, head_dim=128, table_stride=4)
    d.update(kw)
    return w4.w4_kv_cache(A, A, A, A, A, **d)


APPEND = dict(q=A, k=A, v=A, q_out=A, rope_cos=A, rope_sin=A, positions=None, q_start=A, kv_len=A, tokens=0, batch=2,
              q_heads=12, max_q=2, max_position=100, rotary_dim=128, interleaved=0, q_stride=0, k_stride=0, v_stride=0,
              q_out_stride=0, stream=0)
ATTN = dict(q=A, out=A, lse=A, q_start=A, kv_len=A, tokens=0, batch=2, q_heads=12, max_q=2, softmax_scale=0.1, causal=1,
            window=0, q_stride=0, out_stride=0, workspace=A, workspace_bytes=1 << 40, stream=0)

# one bad value at a time; what the separate call answers is what the block's must
APPEND_BAD = [("q", None), ("k", None), ("v", None), ("q_out", None), ("rope_cos", None), ("rope_sin", None),
              ("q_start", None), ("kv_len", None), ("q", A + 8), ("k", A + 8), ("v", A + 8), ("q_out", A + 8),
              ("rope_cos", A + 8), ("rope_sin", A + 8), ("positions", A + 2), ("q_start", A + 2), ("kv_len", A + 2),
              ("tokens", -1), ("batch", 0), ("batch", w4.W4_MAX_SEQS + 1), ("q_heads", 3), ("max_q", -1),
              ("max_position", 0), ("rotary_dim", 8), ("rotary_dim", 144), ("q_stride", 12 * 128 + 4),
              ("k_stride", 100), ("v_stride", 2 * 128 + 4), ("q_out_stride", -8)]
ATTN_BAD = [("q", None), ("out", None), ("workspace", None), ("q_start", None), ("kv_len", None), ("q", A + 8),
            ("out", A + 8), ("lse", A + 2), ("q_start", A + 2), ("kv_len", A + 2), ("workspace", A + 8), ("tokens", -1),
            ("batch", 0), ("q_heads", 3), ("max_q", -1), ("softmax_scale", 0.0), ("softmax_scale", -1.0),
            ("softmax_scale", float("inf")), ("softmax_scale", float("nan")), ("window", -1), ("q_stride", 12 * 128 + 4),
            ("out_stride", 100), ("workspace_bytes", 100)]


def _raw_append(cache, d):
    return _lib.lib().w4_kv_append(cache, d["q"], d["k"], d["v"], d["q_out"], d["rope_cos"], d["rope_sin"], d["positions"],
                                   d["q_start"], d["kv_len"], d["tokens"], d["batch"], d["q_heads"], d["max_q"],
                                   d["max_position"], d["rotary_dim"], d["interleaved"], d["q_stride"], d["k_stride"],
                                   d["v_stride"], d["q_out_stride"], d["stream"])


def _raw_attn(cache, d):
    return _lib.lib().w4_attn_kv8(cache, d["q"], d["out"], d["lse"], d["q_start"], d["kv_len"], d["tokens"], d["batch"],
                                  d["q_heads"], d["max_q"], d["softmax_scale"], d["causal"], d["window"], d["q_stride"],
                                  d["out_stride"], d["workspace"], d["workspace_bytes"], d["stream"])


@pytest.mark.parametrize("name,value", [(None, None)] + APPEND_BAD)
def test_append_block(libw4, name, value):
    d = dict(APPEND)
    if name:
        d[name] = value
    want = _raw_append(_cache(), d)
    assert (want == w4.W4_OK) == (name is None)
    assert w4.w4_kv_append(_cache(), **d) == want


@pytest.mark.parametrize("name,value", [(None, None)] + ATTN_BAD)
def test_attention_block(libw4, name, value):
    d = dict(ATTN)
    if name:
        d[name] = value
    want = _raw_attn(_cache(), d)
    assert (want == w4.W4_OK) == (name is None)
    assert w4.w4_attn_kv8(_cache(), **d) == want


def test_no_block(libw4):
    assert _lib.lib().w4_kv_append_block(None) == w4.W4_ERR_NULL
    assert _lib.lib().w4_attn_kv8_block(None) == w4.W4_ERR_NULL
    assert w4.w4_kv_append(None, **APPEND) == w4.W4_ERR_NULL
    assert w4.w4_attn_kv8(None, **ATTN) == w4.W4_ERR_NULL


def test_block_sizes():
    P, L, I = ctypes.sizeof(ctypes.c_void_p), 8, 4
    assert len(w4._append_args(*[0] * 23)) == 11 * P + 4 * L + 8 * I
    assert len(w4._attn_args(*[0] * 17, 0.0, 0)) == 8 * P + 3 * L + 8 * I
