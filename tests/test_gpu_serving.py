"""Cache append, attention and draft verification on the GPU against the 64-bit definitions of
oracle/serving.py."""
import math

import numpy as np
import pytest

import weight_only_bit_gb300 as w4
from oracle import serving as sv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
DEV = "cuda"
NAN_CODE = 0x7F


class Case:
    """A ragged batch over a paged cache whose unused places hold NaN codes and table entries of -1."""

    def __init__(self, new, total, q_heads=12, kv_heads=2, dim=128, page=16, seed=0, extra_pages=3, page_stride=0,
                 scale_stride=0, power=False, pad_q=0):
        rng = np.random.default_rng(seed)
        self.new, self.total = list(new), list(total)
        self.hq, self.hkv, self.d, self.page = q_heads, kv_heads, dim, page
        self.batch, self.tokens, self.max_q = len(new), sum(new), max(new + [1])
        pages = [-(-t // page) for t in total]
        self.num_pages = sum(pages) + extra_pages
        self.width = max(pages + [1]) + 1
        order = rng.permutation(self.num_pages)
        self.table = np.full((self.batch, self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        block = kv_heads * page * dim
        self.page_bytes = page_stride or block
        self.sstride = scale_stride or kv_heads
        self.rng = rng

        def pool():
            p = np.full((self.num_pages, kv_heads, page, dim), NAN_CODE, np.uint8)
            codes = torch.from_numpy(rng.standard_normal(p.shape).astype(np.float32) * 56).clamp(-448, 448).to(FP8)
            codes = codes.view(torch.uint8).numpy()
            for b, t in enumerate(total):
                for k, pg in enumerate(self.table[b, :pages[b]]):
                    r = min(page, t - k * page)
                    p[pg, :, :r] = codes[pg, :, :r]
            return p

        self.k, self.v = pool(), pool()
        e = rng.uniform(-1, 1, (2, self.num_pages, kv_heads))
        e = np.exp2(np.rint(e) if power else e)
        self.ks, self.vs = (e[0] * 2.0 ** -6).astype(np.float32), (e[1] * 2.0 ** -7).astype(np.float32)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.q_stride = q_heads * dim + pad_q
        self.q = np.full((max(self.tokens, 1), self.q_stride), np.nan, np.float16)
        self.q[:, :q_heads * dim] = rng.standard_normal((max(self.tokens, 1), q_heads * dim))
        self.page_stride, self.scale_stride = page_stride, scale_stride

    def upload(self):
        def strided(x, bytes_):
            flat = torch.full((self.num_pages, bytes_), NAN_CODE, dtype=torch.uint8, device=DEV)
            flat[:, :x[0].size] = torch.from_numpy(x.reshape(self.num_pages, -1)).to(DEV)
            return flat

        def scales(x):
            flat = torch.full((self.num_pages, self.sstride), math.nan, device=DEV)
            flat[:, :self.hkv] = torch.from_numpy(x).to(DEV)
            return flat

        self.gk, self.gv = strided(self.k, self.page_bytes), strided(self.v, self.page_bytes)
        self.gks, self.gvs = scales(self.ks), scales(self.vs)
        self.gtable = torch.from_numpy(self.table).to(DEV)
        self.gstart = torch.from_numpy(self.start).to(DEV)
        self.glen = torch.tensor(self.total, dtype=torch.int32, device=DEV)
        self.cache = w4.w4_kv_cache(self.gk, self.gv, self.gks, self.gvs, self.gtable, num_pages=self.num_pages,
                                    kv_heads=self.hkv, page_tokens=self.page, head_dim=self.d, table_stride=self.width,
                                    page_stride=self.page_stride, scale_stride=self.scale_stride)
        return self

    def workspace(self):
        n = w4.w4_attn_workspace_bytes(self.tokens, self.batch, self.hq, self.hkv, self.d)
        return torch.zeros(n, dtype=torch.uint8, device=DEV)

    def attend(self, causal=True, window=0, out_pad=0, ws=None, stream=None, lse=True, max_q=None):
        stride = self.hq * self.d + out_pad
        out = torch.full((max(self.tokens, 1), stride), math.nan, dtype=torch.float16, device=DEV)
        gl = torch.full((max(self.tokens, 1), self.hq), math.nan, device=DEV) if lse else None
        q = torch.from_numpy(self.q).to(DEV)
        ws = self.workspace() if ws is None else ws
        torch.cuda.current_stream().synchronize()
        w4.check(w4.w4_attn_kv8(self.cache, q, out, gl, self.gstart, self.glen, self.tokens, self.batch, self.hq,
                                max_q or self.max_q, self.d ** -0.5, ws, causal=causal, window=window,
                                q_stride=self.q_stride, out_stride=stride, stream=stream))
        w4.check(w4.w4_device_check(stream))
        return out, gl

    def values(self, b, h):
        """Keys and values of a sequence's head in 64 bits."""
        t = self.total[b]
        pg = self.table[b, :-(-t // self.page)] if t else self.table[b, :0]
        k = sv.E4M3[self.k[pg, h]].reshape(-1, self.d) * np.repeat(self.ks[pg, h].astype(np.float64), self.page)[:, None]
        v = sv.E4M3[self.v[pg, h]].reshape(-1, self.d) * np.repeat(self.vs[pg, h].astype(np.float64), self.page)[:, None]
        return k[:t], v[:t]

    def compare(self, out, lse, causal=True, window=0):
        """Every output against the definition.  Bound: each weight is rounded to FP16 (2^-11, or 2^-25 of the
        largest weight times the largest |v| below FP16's normal range), its exponent carries the FP32
        error of the logit (2^-18 allows for the sum's order over D terms), the output is rounded to FP16."""
        out = out.cpu().numpy()[:, :self.hq * self.d].reshape(-1, self.hq, self.d).astype(np.float64)
        lse = lse.cpu().numpy().astype(np.float64) if lse is not None else None
        g = self.hq // self.hkv
        for b in range(self.batch):
            lo, hi = self.start[b], self.start[b + 1]
            if lo == hi:
                continue
            pos = np.arange(self.total[b] - (hi - lo), self.total[b])
            for h in range(self.hkv):
                k, v = self.values(b, h)
                q = self.q[lo:hi, h * g * self.d:(h + 1) * g * self.d].reshape(-1, g, self.d)
                want, wlse, mag = sv.attention_rows(q, k, v, pos, self.total[b], self.d ** -0.5, causal, window)
                got = out[lo:hi, h * g:(h + 1) * g]
                big = np.abs(v).max() if v.size else 0.0
                tol = (2.0 ** -11 + 2.0 ** -18) * mag + 2.0 ** -11 * np.abs(want) + (len(v) * 2.0 ** -25 + 2.0 ** -24) * big
                bad = np.abs(got - want) > tol
                assert not bad.any() and np.isfinite(got).all(), (b, h, np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])
                if lse is not None:
                    gl = lse[lo:hi, h * g:(h + 1) * g]
                    none = np.isinf(wlse)
                    assert np.array_equal(np.isneginf(gl), none) and not got[none].any()
                    assert np.all(np.abs(gl - wlse)[~none] <= 1e-5 * (1 + np.abs(wlse[~none])))


def check(case, causal=True, window=0, **kw):
    case.upload()
    out, lse = case.attend(causal=causal, window=window, **kw)
    case.compare(out, lse, causal, window)
    return out, lse


EDGE = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, 700]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [(12, 2, 128), (8, 8, 64), (28, 4, 128), (8, 1, 64), (64, 2, 128)])
def test_single_tokens_at_every_edge(libw4, heads, page):
    check(Case([1] * len(EDGE), EDGE, *heads, page=page, seed=page))


@pytest.mark.parametrize("q_len", [2, 3, 5, 9, 16, 33, 70, 130])
@pytest.mark.parametrize("heads,page", [((12, 2, 128), 32), ((16, 4, 64), 16), ((5, 5, 128), 64), ((12, 4, 128), 128)])
def test_several_rows(libw4, q_len, heads, page):
    total = [q_len, q_len + 1, q_len + 63, 400 + q_len]
    check(Case([q_len] * 4, total, *heads, page=page, seed=q_len))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 7, 64, 100, 1000])
@pytest.mark.parametrize("dim", [64, 128])
def test_masks(libw4, causal, window, dim):
    check(Case([1, 5, 40, 3, 200], [300, 301, 40, 129, 500], 8, 2, dim, page=16, seed=window), causal, window)


def test_rows_that_see_nothing(libw4):
    """Empty sequences, sequences without new rows, and padding rows before position 0: zeros and -infinity."""
    for new, total in (([1, 1, 1], [0, 0, 0]), ([4, 0, 3], [2, 100, 0]), ([3, 1, 7], [1, 1, 0]), ([40, 2], [9, 0])):
        for causal in (True, False):
            check(Case(new, total, 12, 2, 128, page=16, seed=1), causal)
            check(Case(new, total, 8, 4, 64, page=64, seed=2), causal, 5)


def test_ragged_mix_of_chunks_and_single_tokens(libw4):
    rng = np.random.default_rng(5)
    new = [1, 300, 1, 1, 77, 0, 513, 2]
    total = [n + int(rng.integers(0, 900)) if n else 40 for n in new]
    check(Case(new, total, 12, 2, 128, page=64, seed=5))
    check(Case(new, total, 16, 4, 64, page=16, seed=6), window=200)


def test_long_cache_is_split_and_joined_deterministically(libw4):
    c = Case([1], [40001], 12, 2, 128, page=64, seed=8)
    out, lse = check(c)
    ws = c.workspace()
    for _ in range(3):
        o2, l2 = c.attend(ws=ws)                       # the workspace is ready again after each call
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert int(ws[:4096].max()) == 0
    check(Case([3, 1], [20011, 9003], 32, 8, 128, page=128, seed=9))
    check(Case([50], [9001], 12, 2, 128, page=16, seed=10))


def test_many_short_sequences(libw4):
    rng = np.random.default_rng(11)
    total = [int(x) for x in rng.integers(0, 90, 1000)]
    check(Case([1] * 1000, total, 4, 2, 64, page=16, seed=11))


def test_strides_and_missing_lse(libw4):
    c = Case([5, 1, 17], [70, 1, 400], 12, 2, 128, page=16, seed=12, page_stride=2 * 16 * 128 + 4096, scale_stride=5, pad_q=264)
    check(c, out_pad=72)
    out, _ = c.attend(lse=False)
    c.compare(out, None)
    out, lse = c.attend(max_q=200)                      # a loose bound on the rows per sequence
    c.compare(out, lse)


def test_pages_beyond_four_gigabytes(libw4):
    c = Case([1, 4], [130, 65], 4, 1, 128, page=64, seed=13, page_stride=1 << 30, extra_pages=2).upload()
    out, lse = c.attend()
    c.compare(out, lse)


def test_nan_in_a_masked_key_stays_out(libw4):
    """A key that holds NaN reaches the rows that see it and no others (same tile, same row block)."""
    c = Case([6], [70], 12, 2, 128, page=16, seed=14)
    c.k[c.table[0, 66 // 16], :, 66 % 16, 5] = NAN_CODE
    c.upload()
    out, lse = c.attend()
    o = out.view(6, 12, 128)
    assert torch.isfinite(o[:2]).all() and torch.isfinite(lse[:2]).all()           # rows at 64, 65
    assert torch.isnan(o[2:]).all() and torch.isnan(lse[2:]).all()                 # rows at 66 ... 69
    c = Case([100], [300], 12, 2, 128, page=16, seed=15)
    c.k[c.table[0, 250 // 16], :, 250 % 16, 5] = NAN_CODE
    c.upload()
    out, lse = c.attend()
    assert torch.isfinite(out[:50]).all() and torch.isnan(out[50:]).all()


def test_large_logits_and_tiny_scales(libw4):
    c = Case([1, 3], [500, 333], 12, 2, 128, page=32, seed=16)
    c.ks *= 64                                          # softmax close to one key
    c.vs *= np.exp2(np.random.default_rng(1).integers(-30, 12, c.vs.shape)).astype(np.float32)
    c.upload()
    out, lse = c.attend()
    # values down to 2^-37: the bound's absolute part is that of the largest value, FP16's own range ends at 2^-24
    c.compare(out, lse)


def test_another_stream_and_a_graph(libw4):
    c = Case([1, 2], [900, 64], 12, 2, 128, page=64, seed=17).upload()
    want, wl = c.attend()
    s = torch.cuda.Stream()
    got, gl = c.attend(stream=s)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    out, q, ws = torch.zeros_like(want), torch.from_numpy(c.q).to(DEV), c.workspace()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.check(w4.w4_attn_kv8(c.cache, q, out, None, c.gstart, c.glen, c.tokens, c.batch, c.hq, c.max_q, c.d ** -0.5, ws))
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    c.glen.copy_(torch.tensor([700, 64], dtype=torch.int32))      # the same graph at another length
    c.total = [700, 64]
    graph.replay()
    torch.cuda.synchronize()
    c.compare(out, None)


def test_bad_page_ids_and_lengths_are_reported(libw4):
    c = Case([1], [100], 12, 2, 128, page=16, seed=18)
    c.table[0, 2] = c.num_pages
    c.upload()
    with pytest.raises(w4.W4Error) as e:
        c.attend()
    assert e.value.status == w4.W4_ERR_RANGE
    assert w4.w4_device_check() == w4.W4_OK             # reported once
    c = Case([1], [100], 12, 2, 128, page=16, seed=18).upload()
    c.glen.fill_(10 ** 6)                                # more tokens than the page table holds
    with pytest.raises(w4.W4Error):
        c.attend()
    c.glen.fill_(100)
    c.compare(*c.attend())


# ---------------------------------------------------------------------------------------------- append
def run_append(c, rotary_dim, interleaved, positions=None, poison=None, inplace=False, seed=3, with_q=True):
    """Appends the case's new tokens; returns what was given and what came out."""
    rng = np.random.default_rng(seed)
    d, w = c.d, (c.hq + 2 * c.hkv) * c.d
    qkv = rng.standard_normal((max(c.tokens, 1), w)).astype(np.float16)
    qkv[:, c.hq * d:(c.hq + c.hkv) * d:29] *= 8
    if poison:
        poison(qkv)
    qkv[:, (c.hq + c.hkv) * d:] *= np.float16(0.5)
    top = max(c.total + [1]) + 7
    ang = rng.uniform(0, 6, (top, max(rotary_dim, 2) // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    g = torch.from_numpy(qkv).to(DEV)
    q_out = g if inplace else torch.full((max(c.tokens, 1), c.hq * d), math.nan, dtype=torch.float16, device=DEV)
    es = 2
    gc, gs = torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV)
    gp = torch.from_numpy(positions).to(DEV) if positions is not None else None
    w4.check(w4.w4_kv_append(c.cache, g if with_q else None, g.data_ptr() + es * c.hq * d, g.data_ptr() + es * (c.hq + c.hkv) * d,
                             q_out if with_q else None, gc, gs, c.gstart, c.glen, c.tokens, c.batch, c.hq, c.max_q, top,
                             rotary_dim, interleaved=interleaved, positions=gp, q_stride=w, k_stride=w, v_stride=w,
                             q_out_stride=w if inplace else 0))
    w4.check(w4.w4_device_check())
    return qkv, cos.astype(np.float64), sin.astype(np.float64), q_out.cpu().numpy()[:, :c.hq * d]


def pool_of(c, flat):
    n = c.hkv * c.page * c.d
    return flat[:, :n].cpu().numpy().reshape(c.num_pages, c.hkv, c.page, c.d)


def check_append(c, rotary_dim, interleaved, positions=None, **kw):
    """Codes within half an E4M3 step of the 64-bit value (plus the FP32 rounding of the rotation, 3 roundings
    of the two products), scales equal, q within FP16's half step (plus the same), all else untouched."""
    qkv, cos, sin, q_out = run_append(c, rotary_dim, interleaved, positions, **kw)
    gk, gv = pool_of(c, c.gk), pool_of(c, c.gv)
    gks, gvs = c.gks.cpu().numpy()[:, :c.hkv], c.gvs.cpu().numpy()[:, :c.hkv]
    d, p = c.d, c.page
    want = {"k": c.k.copy(), "v": c.v.copy()}
    scales = {"k": c.ks.copy(), "v": c.vs.copy()}
    got, gsc = {"k": gk, "v": gv}, {"k": gks, "v": gvs}
    written = {n: np.zeros(c.k.shape[:3], bool) for n in want}
    for b in range(c.batch):
        lo, n, t = int(c.start[b]), c.new[b], c.total[b]
        rows = [(lo + i, t - n + i) for i in range(n)]
        x = {"k": {}, "v": {}}
        for r, pos in rows:
            if pos < 0:
                if kw.get("with_q", True):
                    assert not q_out[r].any()
                continue
            rp = pos if positions is None else int(positions[r])
            row = qkv[r].astype(np.float64).reshape(-1, d)
            ca, sa = cos[rp][:rotary_dim // 2], sin[rp][:rotary_dim // 2]
            q, k, v = row[:c.hq], row[c.hq:c.hq + c.hkv], row[c.hq + c.hkv:]
            eps = 2.0 ** -22 * 2 * np.abs(row).max()
            if kw.get("with_q", True):
                wq = sv.rotate(q, ca, sa, rotary_dim, interleaved)
                assert np.all(np.abs(q_out[r].reshape(-1, d) - wq) <= 2.0 ** -11 * np.abs(wq) + 2.0 ** -25 + eps)
            x["k"][pos], x["v"][pos] = (sv.rotate(k, ca, sa, rotary_dim, interleaved), eps), (v, 0.0)
        for name in ("k", "v"):
            for pg in sorted({pos // p for pos in x[name]}):
                here = [pos for pos in x[name] if pos // p == pg]
                pid, first = int(c.table[b, pg]), min(here) % p
                for h in range(c.hkv):
                    s = sv.power_scale(max(np.abs(x[name][q_][0][h]).max() for q_ in here))
                    old = float(scales[name][pid, h])
                    if first > 0:
                        s = max(s, old)
                    assert gsc[name][pid, h] == np.float32(s), (name, b, pg, h)
                    scales[name][pid, h] = s
                    if first > 0:
                        held = sv.E4M3[want[name][pid, h, :first]]
                        assert np.array_equal(sv.E4M3[got[name][pid, h, :first]], sv.e4m3_round(held * (old / s)))
                    for q_ in here:
                        val, eps = x[name][q_][0][h], x[name][q_][1]
                        g = sv.E4M3[got[name][pid, h, q_ % p]]
                        y = val / s
                        assert np.all(np.abs(g - y) <= sv.e4m3_ulp(np.abs(y) + eps / s) / 2 + eps / s), (name, b, q_, h)
                written[name][pid, :, :max(here) % p + 1] = True
    for name in want:
        keep = ~written[name]
        assert np.array_equal(got[name][keep], want[name][keep])
        assert np.array_equal(gsc[name], scales[name])


APPEND = [([1] * 9, [1, 2, 15, 16, 17, 64, 65, 128, 129]), ([5, 1, 7, 3], [5, 1, 70, 131]), ([200, 33], [200, 250]),
          ([0, 4, 0, 1], [9, 4, 0, 33]), ([130], [1000])]


@pytest.mark.parametrize("new,total", APPEND)
@pytest.mark.parametrize("heads,page,rot", [((12, 2, 128), 16, 128), ((12, 2, 128), 64, 64), ((8, 8, 64), 32, 64),
                                             ((7, 1, 64), 128, 16), ((4, 4, 128), 128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(libw4, new, total, heads, page, rot, interleaved):
    check_append(Case(new, total, *heads, page=page, seed=21, power=True).upload(), rot, interleaved)


def test_append_padding_positions_strides(libw4):
    c = Case([6, 3, 2], [4, 3, 0], 12, 2, 128, page=16, seed=22, power=True, page_stride=2 * 16 * 128 + 16,
             scale_stride=3).upload()
    check_append(c, 128, False)
    c = Case([6, 3], [40, 3], 12, 2, 128, page=16, seed=23, power=True).upload()
    check_append(c, 64, False, positions=np.array([0, 0, 3, 9, 1, 2, 40, 7, 7], np.int32))
    c = Case([6, 3], [40, 3], 12, 2, 128, page=16, seed=24).upload()               # scales that are no powers of two
    c2 = Case([6, 3], [40, 3], 12, 2, 128, page=16, seed=24, power=True)
    assert not np.array_equal(c.ks, c2.ks)
    run_append(c, 128, False)
    check_append(Case([5], [69], 8, 2, 64, page=64, seed=25, power=True).upload(), 64, True, inplace=True)
    check_append(Case([5], [69], 8, 2, 64, page=64, seed=25, power=True).upload(), 64, True, with_q=False)


def test_append_grows_a_scale_and_keeps_the_page(libw4):
    """A token far larger than the page's others: the others move to the new scale, rounded again."""
    c = Case([1], [40], 12, 2, 128, page=64, seed=26, power=True)
    c.ks[:], c.vs[:] = 2.0 ** -12, 2.0 ** -13
    check_append(c.upload(), 0, False)
    again = [t.clone() for t in (c.gk, c.gv, c.gks, c.gvs)]
    run_append(c, 0, False)                              # the same token again changes nothing
    assert all(torch.equal(a, b) for a, b in zip(again, (c.gk, c.gv, c.gks, c.gvs)))


def test_append_infinities_and_nan(libw4):
    c = Case([3], [35], 12, 2, 128, page=16, seed=27, power=True).upload()
    k0, v0 = 12 * 128, 14 * 128

    def poison(x):
        x[0, k0 + 3] = np.inf
        x[1, v0 + 128 + 7] = np.nan                      # token 1, kv head 1
        x[2, v0 + 5] = -np.inf

    run_append(c, 0, False, poison=poison)
    gk, gv = sv.E4M3[pool_of(c, c.gk)], sv.E4M3[pool_of(c, c.gv)]
    at = [(int(c.table[0, p // 16]), p % 16) for p in (32, 33, 34)]
    assert gk[at[0][0], 0, at[0][1], 3] == 448 and np.isfinite(gk[at[0][0], 0, at[0][1]]).all()
    assert gv[at[2][0], 0, at[2][1], 5] == -448
    assert np.isnan(gk[at[1][0], 1, at[1][1]]).all() and gv[at[1][0], 1, at[1][1], 7] == 0
    assert np.isfinite(gk[at[1][0], 0, at[1][1]]).all() and np.isfinite(gv[at[1][0]][:, 0:3]).all()
    assert np.isfinite(c.gks.cpu().numpy()[at[0][0]]).all()
    out, lse = c.attend()                                # rows at 32, 33, 34 of 12 heads; head 6 ... 11 read kv head 1
    o = out.view(3, 12, 128)
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[1:, :6]).all() and torch.isnan(o[1:, 6:]).all()


def test_append_out_of_range_is_reported_and_skipped(libw4):
    c = Case([2], [40], 12, 2, 128, page=16, seed=28, power=True)
    c.table[0, 2] = c.num_pages + 5
    c.upload()
    before = c.gk.clone()
    with pytest.raises(w4.W4Error) as e:
        run_append(c, 0, False)
    assert e.value.status == w4.W4_ERR_RANGE and torch.equal(before, c.gk)
    c = Case([2], [40], 12, 2, 128, page=16, seed=28, power=True).upload()
    with pytest.raises(w4.W4Error):
        run_append(c, 128, False, positions=np.array([3, 10 ** 6], np.int32))
    assert w4.w4_device_check() == w4.W4_OK


def test_append_then_attend_across_page_growth(libw4):
    """Tokens appended one by one into an empty cache, then read: against the definition on the codes."""
    steps = 70
    c = Case([1, 1], [steps, steps], 12, 2, 128, page=32, seed=29, power=True)
    c.k[:], c.v[:] = NAN_CODE, NAN_CODE
    c.ks[:], c.vs[:] = np.nan, np.nan
    c.upload()
    for t in range(1, steps + 1):
        c.total = [t, t]
        c.glen.fill_(t)
        run_append(c, 128, False, seed=t)
    c.k, c.v = pool_of(c, c.gk), pool_of(c, c.gv)
    c.ks, c.vs = c.gks.cpu().numpy(), c.gvs.cpu().numpy()
    c.compare(*c.attend())


# ---------------------------------------------------------------------------------------------- verify
def run_verify(target, draft, drafted, u, e, temperature, n_drafts=None, tstride=0, dstride=0, ws=None):
    b, n1, v = target.shape
    n = n1 - 1

    def put(x, stride):
        if x is None:
            return None
        flat = torch.full((x.shape[0] * x.shape[1], stride or v), math.nan, dtype=torch.float16, device=DEV)
        flat[:, :v] = torch.from_numpy(x.reshape(-1, v)).to(DEV)
        return flat

    up = lambda x: None if x is None else torch.from_numpy(x).to(DEV)  # noqa: E731
    tokens = torch.full((b, n1), -7, dtype=torch.int32, device=DEV)
    accepted = torch.full((b,), -7, dtype=torch.int32, device=DEV)
    logprob = torch.full((b, n1), math.nan, device=DEV)
    if ws is None:
        ws = torch.zeros(w4.w4_spec_verify_workspace_bytes(b, n, v), dtype=torch.uint8, device=DEV)
    args = [put(target, tstride), put(draft, dstride), up(drafted), up(u), up(e)]
    for _ in range(2):                                   # the workspace is ready again after each call
        w4.check(w4.w4_spec_verify(*args, tokens, accepted, logprob, b, n, v, temperature, ws, n_drafts=up(n_drafts),
                                   target_stride=tstride, draft_stride=dstride))
        w4.check(w4.w4_device_check())
        res = tokens.cpu().numpy(), accepted.cpu().numpy(), logprob.cpu().numpy()
    return res


def check_verify(target, draft, drafted, u, e, temperature, n_drafts=None, **kw):
    tokens, accepted, logprob = run_verify(target, draft, drafted, u, e, temperature, n_drafts, **kw)
    b, n1, _ = target.shape
    sure = 0
    for i in range(b):
        n = n1 - 1 if n_drafts is None else int(np.clip(n_drafts[i], 0, n1 - 1))
        want, acc, lp, margin = sv.verify(target[i, :n + 1], None if draft is None else draft[i], drafted[i, :n],
                                          None if u is None else u[i], None if e is None else e[i], temperature)
        if margin < 1e-4:                                # FP32 may decide the other way
            continue
        sure += 1
        assert list(tokens[i]) == want + [-1] * (n1 - len(want)) and accepted[i] == acc, (i, tokens[i], want)
        got = logprob[i, :len(want)].astype(np.float64)
        lp = np.array(lp)
        fin = np.isfinite(lp)
        assert np.array_equal(np.isneginf(got), np.isneginf(lp))
        # FP32 of (x - m) c and of the logarithm of the sum
        assert np.all(np.abs(got - lp)[fin] <= 4e-6 * (1 + np.abs(lp[fin])))
        assert not logprob[i, len(want):].any()
    assert sure >= 0.8 * b                               # margins are small for few of the seeded inputs
    return accepted


def inputs(b, n, v, seed, t=1.0):
    rng = np.random.default_rng(seed)
    target = rng.standard_normal((b, n + 1, v)) * 1.5
    target[..., rng.integers(0, v, 6)] += 6
    noisy = target[:, :n] + 0.7 * rng.standard_normal((b, n, v))
    drafted = (noisy / (t or 0.3) - np.log(rng.exponential(size=noisy.shape))).argmax(-1).astype(np.int32)
    return (target.astype(np.float16), noisy.astype(np.float16), drafted, rng.random((b, n)).astype(np.float32),
            np.maximum(rng.exponential(size=(b, v)), 1e-9).astype(np.float32))


@pytest.mark.parametrize("b,n,v", [(1, 1, 1), (3, 1, 2), (5, 4, 7), (40, 3, 300), (2, 31, 1000), (6, 5, 32003), (1, 4, 151936)])
@pytest.mark.parametrize("t", [0.0, 0.6, 1.0])
@pytest.mark.parametrize("with_draft", [True, False])
def test_verify(libw4, b, n, v, t, with_draft):
    target, draft, drafted, u, e = inputs(b, n, v, 31 + v, t)
    check_verify(target, draft if with_draft else None, drafted, u, e, t)


def test_verify_ragged_counts_and_strides(libw4):
    target, draft, drafted, u, e = inputs(8, 4, 501, 41)
    nd = np.array([0, 1, 2, 3, 4, 9, -1, 2], np.int32)
    for t in (0.0, 0.8):
        acc = check_verify(target, draft, drafted, u, e, t, nd, tstride=513, dstride=700)
        assert np.all(acc <= np.clip(nd, 0, 4))


def test_verify_accepts_all_and_none(libw4):
    target, draft, drafted, u, e = inputs(6, 4, 2000, 42)
    acc = check_verify(target, target[:, :4].copy(), drafted, u * 0.99, e, 1.0)     # p = q: u q < p always
    assert np.all(acc == 4)
    hidden = target.copy()
    for b in range(6):
        hidden[b, 0, drafted[b, 0]] = -np.inf
    assert np.all(check_verify(hidden, draft, drafted, u, e, 1.0) == 0)


def test_verify_masked_and_odd_logits(libw4):
    target, draft, drafted, u, e = inputs(4, 3, 999, 43)
    target[0, :, 100:] = -np.inf                         # a top-k mask
    draft[0, :, 50:] = -65504
    drafted[0] = [3, 150, 5]
    target[1] = -np.inf                                  # no token at all
    target[2, 0, 7], target[2, 0, 9] = np.nan, np.inf     # NaN never, infinity as the largest value
    drafted[2, 0] = 9
    drafted[3] = [-1, 5000, 2]                           # outside the vocabulary: refused
    for t in (0.0, 1.0):
        acc = check_verify(target, draft, drafted, u, e, t)
        assert acc[1] == 0 and acc[3] == 0 and acc[2] >= 1
    tokens, _, logprob = run_verify(target, draft, drafted, u, e, 1.0)
    assert tokens[1, 0] == -1 and np.isneginf(logprob[1, 0])


def test_verify_ties_go_to_the_lowest_token(libw4):
    target = np.zeros((2, 2, 40000), np.float16)
    drafted = np.array([[39999], [0]], np.int32)
    e = np.ones((2, 40000), np.float32)
    u = np.full((2, 1), 0.99999, np.float32)
    tokens, acc, _ = run_verify(target, None, drafted, u, e, 0.0)
    assert list(tokens[0]) == [0, -1] and list(tokens[1]) == [0, 0] and list(acc) == [0, 1]
    tokens, acc, _ = run_verify(target, None, drafted, u, e, 1.0)
    assert list(tokens[0]) == [0, -1] and list(tokens[1]) == [1, -1] and list(acc) == [0, 0]
