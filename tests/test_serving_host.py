"""The cache, attention and verification entry points on the host: argument checks before any CUDA call,
workspace sizes, and pins of the 64-bit definitions that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest

import weight_only_bit_gb300 as w4
from oracle import serving as sv
from weight_only_bit_gb300 import _lib

A = 1 << 20        # fake, never dereferenced device addresses


def _cache(**kw):
    d = dict(num_pages=8, kv_heads=2, page_tokens=64, head_dim=128, table_stride=4)
    ptrs = {n: kw.pop(n, A) for n in ("k", "v", "k_scale", "v_scale", "page_table")}
    d.update(kw)
    return w4.w4_kv_cache(ptrs["k"], ptrs["v"], ptrs["k_scale"], ptrs["v_scale"], ptrs["page_table"], **d)


def _append(cache=None, **kw):
    d = dict(q=A, k=A, v=A, q_out=A, rope_cos=A, rope_sin=A, q_start=A, kv_len=A, tokens=3, batch=2, q_heads=12, max_q=2,
             max_position=100, rotary_dim=128, stream=0)
    d.update(kw)
    return w4.w4_kv_append(cache or _cache(), **d)


def _attn(cache=None, **kw):
    d = dict(q=A, out=A, lse=A, q_start=A, kv_len=A, tokens=3, batch=2, q_heads=12, max_q=2, softmax_scale=0.1, workspace=A,
             workspace_bytes=1 << 40, stream=0)
    d.update(kw)
    return w4.w4_attn_kv8(cache or _cache(), **d)


def _verify(**kw):
    d = dict(target=A, draft=A, draft_tokens=A, u=A, e=A, tokens=A, accepted=A, logprob=A, batch=2, drafts=3, vocab=100,
             temperature=1.0, workspace=A, workspace_bytes=1 << 40, stream=0)
    d.update(kw)
    return w4.w4_spec_verify(**d)


@pytest.mark.parametrize("call", [_append, _attn])
def test_cache_refusals(libw4, call):
    for name in ("k", "v", "k_scale", "v_scale", "page_table"):
        assert call(_cache(**{name: None})) == w4.W4_ERR_NULL
    assert call(_cache(num_pages=0)) == w4.W4_ERR_SHAPE
    assert call(_cache(kv_heads=0)) == w4.W4_ERR_SHAPE
    assert call(_cache(table_stride=0)) == w4.W4_ERR_SHAPE
    for page in (0, 8, 24, 48, 256):
        assert call(_cache(page_tokens=page)) == w4.W4_ERR_UNSUPPORTED
    for dim in (0, 32, 96, 256):
        assert call(_cache(head_dim=dim)) == w4.W4_ERR_UNSUPPORTED
    assert call(_cache(page_stride=2 * 64 * 128 - 16)) == w4.W4_ERR_SHAPE          # pages would overlap
    assert call(_cache(page_stride=2 * 64 * 128 + 8)) == w4.W4_ERR_ALIGN
    assert call(_cache(scale_stride=1)) == w4.W4_ERR_SHAPE
    assert call(_cache(k=A + 8)) == w4.W4_ERR_ALIGN
    assert call(_cache(k_scale=A + 2)) == w4.W4_ERR_ALIGN
    assert call(_cache(page_table=A + 2)) == w4.W4_ERR_ALIGN
    assert _lib.lib().w4_kv_append(None, *[None] * 9, *[0] * 11, None) == w4.W4_ERR_NULL


@pytest.mark.parametrize("call", [_append, _attn])
def test_batch_refusals(libw4, call):
    assert call(q_start=None) == w4.W4_ERR_NULL
    assert call(kv_len=None) == w4.W4_ERR_NULL
    assert call(tokens=-1) == w4.W4_ERR_SHAPE
    assert call(batch=0) == w4.W4_ERR_SHAPE
    assert call(max_q=-1) == w4.W4_ERR_SHAPE
    assert call(q_heads=13) == w4.W4_ERR_SHAPE                                     # not a multiple of kv_heads
    assert call(q_heads=2 * (w4.W4_MAX_GROUP + 1)) == w4.W4_ERR_UNSUPPORTED
    assert call(batch=w4.W4_MAX_SEQS + 1) == w4.W4_ERR_UNSUPPORTED
    assert call(tokens=1 << 28) == w4.W4_ERR_UNSUPPORTED
    assert call(q_stride=12 * 128 - 8) == w4.W4_ERR_SHAPE
    assert call(q_stride=12 * 128 + 4) == w4.W4_ERR_ALIGN
    assert call(q=A + 2) == w4.W4_ERR_ALIGN
    assert call(q_start=A + 1) == w4.W4_ERR_ALIGN
    assert call(tokens=0) == w4.W4_OK                                               # nothing to do, nothing launched
    assert call(max_q=0) == w4.W4_OK


def test_append_refusals(libw4):
    assert _append(k=None) == w4.W4_ERR_NULL
    assert _append(q=None) == w4.W4_ERR_NULL                                        # q_out without q
    assert _append(q=None, q_out=None, tokens=0) == w4.W4_OK
    assert _append(rope_cos=None) == w4.W4_ERR_NULL
    assert _append(rope_cos=None, rope_sin=None, rotary_dim=0, max_position=0, tokens=0) == w4.W4_OK
    for r in (-16, 8, 24, 144):
        assert _append(rotary_dim=r) == w4.W4_ERR_SHAPE
    assert _append(max_position=0) == w4.W4_ERR_SHAPE
    assert _append(k_stride=128) == w4.W4_ERR_SHAPE
    assert _append(rope_sin=A + 4) == w4.W4_ERR_ALIGN
    assert _append(q_out_stride=12 * 128 + 1) == w4.W4_ERR_ALIGN


def test_attention_refusals(libw4):
    assert _attn(q=None) == w4.W4_ERR_NULL
    assert _attn(out=None) == w4.W4_ERR_NULL
    assert _attn(workspace=None) == w4.W4_ERR_NULL
    assert _attn(workspace=A + 4) == w4.W4_ERR_ALIGN
    assert _attn(workspace_bytes=16) == w4.W4_ERR_SHAPE
    assert _attn(window=-1) == w4.W4_ERR_SHAPE
    assert _attn(softmax_scale=math.inf) == w4.W4_ERR_SHAPE
    assert _attn(softmax_scale=math.nan) == w4.W4_ERR_SHAPE
    assert _attn(out_stride=100) == w4.W4_ERR_SHAPE
    with pytest.raises(w4.W4Error):
        w4.w4_attn_kv8(_cache(), A, A, A, A, A, 3, 2, 12, 2, 0.1, A, stream=0)      # an address needs its size
    assert w4.w4_attn_workspace_bytes(1, 1, 12, 2, 128) > 0
    assert w4.w4_attn_workspace_bytes(1, 1, 12, 2, 80) == 0
    assert w4.w4_attn_workspace_bytes(1, 0, 12, 2, 64) == 0


def test_verify_refusals(libw4):
    for name in ("target", "draft_tokens", "u", "e", "tokens", "accepted", "workspace"):
        assert _verify(**{name: None}) == w4.W4_ERR_NULL
    for t in (-1.0, math.nan, math.inf):
        assert _verify(temperature=t) == w4.W4_ERR_SHAPE
    assert _verify(temperature=1e-5) == w4.W4_ERR_UNSUPPORTED
    assert _verify(batch=0) == w4.W4_ERR_SHAPE
    assert _verify(drafts=0) == w4.W4_ERR_SHAPE
    assert _verify(vocab=0) == w4.W4_ERR_SHAPE
    assert _verify(drafts=w4.W4_MAX_DRAFTS + 1) == w4.W4_ERR_UNSUPPORTED
    assert _verify(vocab=(1 << 24) + 1) == w4.W4_ERR_UNSUPPORTED
    assert _verify(target_stride=99) == w4.W4_ERR_SHAPE
    assert _verify(draft_stride=99) == w4.W4_ERR_SHAPE
    assert _verify(target=A + 1) == w4.W4_ERR_ALIGN
    assert _verify(e=A + 2) == w4.W4_ERR_ALIGN
    assert _verify(workspace_bytes=64) == w4.W4_ERR_SHAPE
    assert w4.w4_spec_verify_workspace_bytes(2, 3, 100) > 0
    assert w4.w4_spec_verify_workspace_bytes(2, 0, 100) == 0
    assert w4.w4_status_str(w4.W4_ERR_RANGE) != w4.w4_status_str(-100)


def test_cache_struct_matches_the_header(libw4):
    assert ctypes.sizeof(w4.KvCache) == 5 * 8 + 2 * 8 + 5 * 4 + 4


# ------------------------------------------------------------------ the definitions themselves
def test_e4m3_values():
    v = sv.E4M3
    assert v[0x00] == 0 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1 and v[0x7e] == 448
    assert v[0xb8] == -1 and np.isnan(v[0x7f]) and np.isnan(v[0xff])
    assert np.all(np.diff(v[:0x7f]) > 0)


def test_e4m3_round_is_the_nearest_value_with_ties_to_even():
    grid = sv.E4M3[:0x7f]
    mids = (grid[1:] + grid[:-1]) / 2                    # exact ties
    got = sv.e4m3_round(mids)
    for i, m in enumerate(mids):
        assert got[i] == grid[i + (i & 1)], m            # the even code of i, i + 1
    x = np.random.default_rng(1).uniform(-500, 500, 2000) * 10.0 ** np.random.default_rng(2).uniform(-5, 0, 2000)
    near = np.concatenate([-grid[::-1], grid])
    d = np.abs(near[None] - np.clip(x, -448, 448)[:, None]).min(axis=1)
    assert np.array_equal(np.abs(sv.e4m3_round(x) - np.clip(x, -448, 448)), d)


def test_power_scale():
    assert sv.power_scale(448.0) == 1 and sv.power_scale(np.nextafter(448.0, 500)) == 2
    assert sv.power_scale(0.0) == 2.0 ** -60 and sv.power_scale(1.75) == 2.0 ** -8


def test_rotation_is_one_of_the_plane():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 64))
    ang = rng.uniform(0, 6, 16)
    for inter in (False, True):
        y = sv.rotate(x, np.cos(ang), np.sin(ang), 32, inter)
        assert np.allclose((y ** 2).sum(), (x ** 2).sum()) and np.array_equal(y[:, 32:], x[:, 32:])
        back = sv.rotate(y, np.cos(-ang), np.sin(-ang), 32, inter)
        assert np.allclose(back, x)
    quarter = sv.rotate(np.eye(1, 64), np.zeros(16), np.ones(16), 32, False)
    assert quarter[0, 16] == 1 and np.count_nonzero(np.abs(quarter) > 1e-12) == 1


def test_attention_rows_by_hand():
    k = np.array([[1.0, 0], [0, 1], [1, 1]])
    v = np.array([[1.0, 0], [0, 2], [3, 3]])
    q = np.array([[[0.0, 0]]])
    out, lse, mag = sv.attention_rows(q, k, v, [1], 3, 1.0, True, 0)
    assert np.allclose(out, [[[0.5, 1]]]) and np.allclose(lse, math.log(2)) and np.allclose(mag, out)
    out, lse, _ = sv.attention_rows(q, k, v, [2], 3, 1.0, True, 1)
    assert np.allclose(out, [[[3, 3]]]) and np.allclose(lse, 0)
    out, lse, _ = sv.attention_rows(q, k, v, [-1], 3, 1.0, False, 0)
    assert not out.any() and lse[0, 0] == -np.inf


def test_verification_draws_from_the_target():
    """Accept-or-redraw gives the target's distribution whatever the draft's (the property the operator
    exists for); 4000 draws over 4 tokens, compared within 5 standard deviations."""
    rng = np.random.default_rng(7)
    target = np.log(np.array([[0.5, 0.2, 0.2, 0.1], [0.25] * 4]))
    draft = np.log(np.array([[0.1, 0.6, 0.1, 0.2]]))
    counts = np.zeros(4)
    n = 4000
    for _ in range(n):
        x = rng.choice(4, p=np.exp(draft[0]))
        out, *_ = sv.verify(target, draft, [x], rng.random(1), rng.exponential(size=4), 1.0)
        counts[out[0]] += 1
    p = np.exp(target[0])
    assert np.all(np.abs(counts / n - p) < 5 * np.sqrt(p * (1 - p) / n))


def test_verification_greedy_and_edges():
    target = np.array([[0.0, 3, 3], [1, 0, 0], [0, 0, 1]])
    assert sv.verify(target, None, [1, 0], None, None, 0)[:2] == ([1, 0, 2], 2)     # a tie goes to the lower token
    assert sv.verify(target, None, [2, 0], None, None, 0)[:2] == ([1], 0)
    out, acc, lp, _ = sv.verify(np.full((2, 3), -np.inf), None, [1], [0.5], np.ones(3), 1.0)
    assert out == [-1] and acc == 0 and lp == [-np.inf]
