"""Measured cases of the serving operators around the 4-bit projections: appending keys and values to a
paged 8-bit cache (with the position rotation), attention over that cache, and the verification of
drafted tokens.

Each operator has a plain form (elementary torch operations in 32 bits) and the library's own call; `own`
says which of the two `run` makes.  `exact` computes the same outputs in 64 bits from the definitions.
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one user, early in a conversation: one new token, a few hundred cached ones (latency)
        attention("attn_one_short", batch=1, q_len=1, kv_max=257, page=16),
        # one user, one new token at the end of a very long document
        attention("attn_one_long", batch=1, q_len=1, kv_max=131071, page=64),
        # a serving batch, every sequence at its own length, one of them empty
        attention("attn_batch_ragged", batch=64, q_len=1, kv_max=8192, page=64, ragged=True),
        # a serving batch that verifies four drafted tokens a sequence (five query rows each)
        attention("attn_draft_batch", batch=16, q_len=5, kv_max=6001, page=32, ragged=True, q_heads=32, kv_heads=8),
        # chunked prompts and single tokens in one batch, sliding window, small heads, small pages
        attention("attn_chunk_window", batch=8, q_len=517, kv_max=16384, page=16, ragged=True, q_ragged=True,
                  q_heads=16, kv_heads=4, head_dim=64, window=4096),
        # a whole prompt, causal
        attention("attn_prompt", batch=1, q_len=8191, kv_max=8191, page=64),
        # one user, one new token
        append("append_one", batch=1, q_len=1, kv_max=257, page=16),
        # a serving batch, one new token each, every page at another fill
        append("append_batch", batch=256, q_len=1, kv_max=2048, page=64, ragged=True),
        # two long prompts
        append("append_prompt", batch=2, q_len=8191, kv_max=8191, page=64, q_heads=32, kv_heads=8),
        # one user's four drafted tokens, with the draft model's logits
        verify("verify_one", batch=1, drafts=4, vocab=151936, temperature=0.8),
        # a serving batch with the draft model's logits
        verify("verify_batch", batch=48, drafts=5, vocab=151936, temperature=1.0),
        # drafts copied out of the context (no draft model), odd vocabulary
        verify("verify_lookup", batch=16, drafts=7, vocab=32003, temperature=0.6, with_draft=False),
    ]


def attention(name, *, batch, q_len, kv_max, page, ragged=False, q_ragged=False, q_heads=12, kv_heads=2, head_dim=128,
              window=0, causal=True):
    return _named(name, {"op": "attention", "batch": batch, "q_len": q_len, "kv_max": kv_max, "page": page,
                         "ragged": ragged, "q_ragged": q_ragged, "q_heads": q_heads, "kv_heads": kv_heads,
                         "head_dim": head_dim, "window": window, "causal": causal})


def append(name, *, batch, q_len, kv_max, page, ragged=False, q_heads=12, kv_heads=2, head_dim=128, rotary_dim=None,
           interleaved=False):
    return _named(name, {"op": "append", "batch": batch, "q_len": q_len, "kv_max": kv_max, "page": page,
                         "ragged": ragged, "q_ragged": False, "q_heads": q_heads, "kv_heads": kv_heads,
                         "head_dim": head_dim, "rotary_dim": rotary_dim or head_dim, "interleaved": interleaved})


def verify(name, *, batch, drafts, vocab, temperature, with_draft=True):
    return _named(name, {"op": "verify", "batch": batch, "drafts": drafts, "vocab": vocab, "temperature": temperature,
                         "with_draft": with_draft})


def _named(name, case):
    return dict(case, name=name) if name else case


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


#: query heads and key/value heads: the repository's own decode step (12 over 2), and generic ones
HEADS = [(12, 2, 128), (12, 2, 128), (32, 8, 128), (16, 16, 128), (16, 4, 64), (28, 4, 128), (8, 1, 64)]


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "append", "verify"])
    if op == "verify":
        vocab = rng.choice([151936, _log_int(rng, 1000, 160000)])
        drafts = rng.randint(1, 8)
        return verify(None, batch=_log_int(rng, 1, max(1, min(128, 40_000_000 // (vocab * drafts)))), drafts=drafts,
                      vocab=vocab, temperature=rng.choice([0.0, 0.5, 0.8, 1.0, round(rng.uniform(0.3, 1.5), 2)]),
                      with_draft=rng.random() < 0.7)
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        q_len = rng.choice([1, rng.randint(2, 9), _log_int(rng, 16, 8191)])
        batch = _log_int(rng, 1, max(1, min(256, 16000 // q_len)))
        kv_max = q_len + _log_int(rng, 1, 2048)
        return append(None, batch=batch, q_len=q_len, kv_max=kv_max, page=page, ragged=rng.random() < 0.7, q_heads=hq,
                      kv_heads=hkv, head_dim=d, rotary_dim=rng.choice([d, d // 2]), interleaved=rng.random() < 0.3)
    kind = rng.choice(["one", "one", "draft", "chunk", "prompt"])
    window = rng.choice([0, 0, 0, _log_int(rng, 100, 8192)])
    if kind == "prompt":
        q_len = _log_int(rng, 64, 6000)
        batch = _log_int(rng, 1, max(1, min(8, 6000 // q_len)))
        return attention(None, batch=batch, q_len=q_len, kv_max=q_len, page=page, ragged=False, q_ragged=rng.random() < 0.5,
                         q_heads=min(hq, 16) if hq != 28 else 12, kv_heads=min(hkv, 4), head_dim=d, window=window,
                         causal=rng.random() < 0.8)
    q_len = 1 if kind == "one" else rng.randint(2, 9) if kind == "draft" else _log_int(rng, 16, 600)
    kv_max = q_len + _log_int(rng, 32, 60000 if kind != "chunk" else 16000)
    most = 500_000_000 // (kv_max * hkv * d * 2)
    if kind == "chunk":
        most = min(most, 250_000_000 // (q_len * kv_max * hq // 8))
    batch = _log_int(rng, 1, max(1, min(128, most)))
    return attention(None, batch=batch, q_len=q_len, kv_max=kv_max, page=page, ragged=rng.random() < 0.7,
                     q_ragged=kind != "one" and rng.random() < 0.5, q_heads=hq, kv_heads=hkv, head_dim=d, window=window)


def _lengths(case):
    """(new tokens, tokens in the cache with the new ones) of each sequence; by the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new, total = [], []
    for b in range(case["batch"]):
        n = rng.randint(1, case["q_len"]) if case["q_ragged"] and b else case["q_len"]
        if case["ragged"]:
            t = n + rng.randint(0, case["kv_max"] - case["q_len"])
        else:
            t = n + case["kv_max"] - case["q_len"]
        new.append(n)
        total.append(t)
    if case["ragged"] and case["batch"] > 2 and case["op"] == "attention":
        total[1] = 0  # a slot whose sequence has no tokens: all of its rows are empty
    return new, total


def _visible(case, n, t):
    """Sum over a sequence's new tokens of the keys that each of them sees, and the keys that any of them sees."""
    w = case["window"] or t + 1
    seen, first = 0, t
    for i in range(n):
        hi = (t - n + i + 1) if case["causal"] else t
        lo = max(0, t - n + i + 1 - w)
        if hi > lo:
            seen += hi - lo
            first = min(first, lo)
    return seen, t - first


def work(case):
    if case["op"] == "verify":
        rows = case["drafts"] + 1 + (case["drafts"] if case["with_draft"] else 0)
        per = rows * case["vocab"] * 2 + (case["vocab"] * 4 if case["temperature"] > 0 else 0) + case["drafts"] * 8
        return {"bytes": case["batch"] * (per + (case["drafts"] + 1) * 8 + 4), "flops": case["batch"] * rows * case["vocab"] * 4}
    new, total = _lengths(case)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        t = sum(new)
        return {"bytes": t * d * (4 * hq + 6 * hkv) + t * case["rotary_dim"] * 4 + t // case["page"] * hkv * 8,
                "flops": t * (hq + 2 * hkv) * d * 4}
    seen = [_visible(case, n, t) for n, t in zip(new, total)]
    return {"bytes": sum(k for _, k in seen) * hkv * 2 * d + sum(new) * hq * (4 * d + 4),
            "flops": sum(s for s, _ in seen) * hq * 4 * d}


# ---------------------------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    s = _prepare_verify(case, seed) if case["op"] == "verify" else _prepare_cache(case, seed)
    if own:
        import weight_only_bit_gb300 as w4
        s["w4"] = w4
        if case["op"] == "verify":
            s["workspace"] = torch.zeros(w4.w4_spec_verify_workspace_bytes(case["batch"], case["drafts"], case["vocab"]),
                                         dtype=torch.uint8, device=DEV)
        else:
            s["cache"] = w4.w4_kv_cache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"],
                                        num_pages=s["k_pool"].shape[0], kv_heads=case["kv_heads"],
                                        page_tokens=case["page"], head_dim=case["head_dim"],
                                        table_stride=s["table"].shape[1])
        if case["op"] == "attention":
            n = w4.w4_attn_workspace_bytes(s["tokens"], case["batch"], case["q_heads"], case["kv_heads"], case["head_dim"])
            s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=DEV)
    return s


def _prepare_cache(case, seed):
    g = _generator(seed)
    new, total = _lengths(case)
    b, p, d, hkv, hq = case["batch"], case["page"], case["head_dim"], case["kv_heads"], case["q_heads"]
    pages = [-(-t // p) for t in total]
    width = max(1, max(pages))
    used = sum(pages)
    pool = used + 3
    # pages in an arbitrary order, as an allocator hands them out; unused table entries are -1
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32, device=DEV)
    counts = torch.tensor(pages, device=DEV)
    table[torch.arange(width, device=DEV)[None, :] < counts[:, None]] = order[:used]
    s = {"case": dict(case), "table": table, "tokens": sum(new), "max_q": max(new)}
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device=DEV)

    def codes():
        x = torch.empty((pool, hkv, p, d), dtype=FP8, device=DEV)
        step = max(1, (1 << 27) // (hkv * p * d))
        for i in range(0, pool, step):
            x[i:i + step] = (torch.randn(x[i:i + step].shape, generator=g, device=DEV) * 56).clamp_(-448, 448).to(FP8)
        return x

    def scales(mid, power):
        e = torch.rand((pool, hkv), generator=g, device=DEV) * 2 - 1
        return (torch.exp2(e.round()) if power else torch.exp2(e)) * mid

    s["k_pool"], s["v_pool"] = codes(), codes()
    t = s["tokens"]
    if case["op"] == "attention":
        # scales of any value, as a calibrated cache has them
        s["k_scale"], s["v_scale"] = scales(2.0 ** -5.5, False), scales(2.0 ** -6.5, False)
        s["q"] = torch.randn((t, hq, d), generator=g, device=DEV).half()
        s["out"] = torch.empty((t, hq, d), dtype=torch.float16, device=DEV)
        s["lse"] = torch.empty((t, hq), dtype=torch.float32, device=DEV)
    else:
        s["k_scale"], s["v_scale"] = scales(2.0 ** -6, True), scales(2.0 ** -7, True)
        # one fused projection's output: q, k and v are column ranges of it; some key channels are large
        qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device=DEV)
        qkv[:, hq * d:(hq + hkv) * d:37] *= 6
        s["qkv"] = qkv.half()
        s["q"], s["k"], s["v"] = s["qkv"].split([hq * d, hkv * d, hkv * d], dim=1)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.float16, device=DEV)
        r = case["rotary_dim"]
        inv = 1e6 ** (-torch.arange(r // 2, dtype=torch.float64, device=DEV) * 2 / r)
        ang = torch.arange(case["kv_max"] + 1, dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    return s


def _prepare_verify(case, seed):
    g = _generator(seed)
    b, n, v = case["batch"], case["drafts"], case["vocab"]
    # a few likely tokens over a broad floor; the draft model's logits are the target's with noise
    target = torch.randn((b, n + 1, v), generator=g, device=DEV) * 1.5
    top = torch.randint(0, v, (b, n + 1, 12), generator=g, device=DEV)
    target.scatter_(2, top, 10 + 2.5 * torch.randn(top.shape, generator=g, device=DEV))
    noisy = target[:, :n] + 0.7 * torch.randn((b, n, v), generator=g, device=DEV)
    t = case["temperature"] or 0.25
    race = noisy / t - torch.empty_like(noisy).exponential_(generator=g).log_()
    s = {"case": dict(case), "target": target.half(), "draft_tokens": race.argmax(2).to(torch.int32),
         "draft": noisy.half() if case["with_draft"] else None,
         "u": torch.rand((b, n), generator=g, device=DEV),
         "e": torch.empty((b, v), device=DEV).exponential_(generator=g).clamp_min_(1e-12)}
    s["tokens"] = torch.empty((b, n + 1), dtype=torch.int32, device=DEV)
    s["accepted"] = torch.empty((b,), dtype=torch.int32, device=DEV)
    s["logprob"] = torch.empty((b, n + 1), dtype=torch.float32, device=DEV)
    return s


# -------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attention": _attention_plain, "append": _append_plain, "verify": _verify_plain}[op](s)
    w4, c = s["w4"], s["case"]
    if op == "attention":
        w4.check(w4.w4_attn_kv8(s["cache"], s["q"], s["out"], s["lse"], s["q_start"], s["kv_len"], s["tokens"], c["batch"],
                                c["q_heads"], s["max_q"], c["head_dim"] ** -0.5, s["workspace"], causal=c["causal"],
                                window=c["window"]))
        return {"out": s["out"], "lse": s["lse"]}
    if op == "append":
        w4.check(w4.w4_kv_append(s["cache"], s["q"], s["k"], s["v"], s["q_out"], s["cos"], s["sin"], s["q_start"],
                                 s["kv_len"], s["tokens"], c["batch"], c["q_heads"], s["max_q"], s["cos"].shape[0],
                                 c["rotary_dim"], interleaved=c["interleaved"], q_stride=s["qkv"].shape[1],
                                 k_stride=s["qkv"].shape[1], v_stride=s["qkv"].shape[1]))
        return _cache_out(s)
    w4.check(w4.w4_spec_verify(s["target"], s["draft"], s["draft_tokens"], s["u"], s["e"], s["tokens"], s["accepted"],
                               s["logprob"], c["batch"], c["drafts"], c["vocab"], c["temperature"], s["workspace"]))
    return {"tokens": s["tokens"], "accepted": s["accepted"], "logprob": s["logprob"]}


def _cache_out(s):
    return {"q": s["q_out"], "k_codes": s["k_pool"], "v_codes": s["v_pool"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------------------------------------ plain forms
def _places(s):
    """Sequence and position of each new token."""
    t = torch.arange(s["tokens"], device=DEV)
    start, kv = s["q_start"].long(), s["kv_len"].long()
    b = (t[:, None] >= start[None, 1:]).sum(1)
    return b, kv[b] - start[b + 1] + t


def _attention_plain(s):
    c = s["case"]
    hq, hkv, d, p = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    nb, nq = c["batch"], s["max_q"]
    b, pos = _places(s)
    start = s["q_start"].long()
    slot = torch.arange(s["tokens"], device=DEV) - start[b]
    q = torch.zeros((nb, nq, hq, d), device=DEV)
    q[b, slot] = s["q"].float()
    q = q.view(nb, nq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(nb, hkv, -1, d)
    table = s["table"].long().clamp_min(0)

    def gather(pool, scale):
        x = pool.view(torch.uint8)[table].view(FP8).float() * scale[table][..., None, None]  # [nb, pages, hkv, p, d]
        return x.permute(0, 2, 1, 3, 4).reshape(nb, hkv, -1, d)

    k, v = gather(s["k_pool"], s["k_scale"]), gather(s["v_pool"], s["v_scale"])
    at = torch.full((nb, nq), -1, device=DEV, dtype=torch.long)
    at[b, slot] = pos
    j = torch.arange(k.shape[2], device=DEV)
    kv = s["kv_len"].long()
    seen = (j < kv[:, None, None]) & (at[:, :, None] >= 0)
    if c["causal"]:
        seen = seen & (j <= at[:, :, None])
    if c["window"]:
        seen = seen & (j > at[:, :, None] - c["window"])
    x = torch.matmul(q, k.transpose(2, 3)).view(nb, hkv, hq // hkv, nq, -1) * d ** -0.5
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-3e38)
    x = torch.exp(x - m)
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(nb, hkv, -1, x.shape[-1]), v).view(nb, hkv, hq // hkv, nq, d) / l.clamp_min(1e-30)
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(nb, nq, hq, d)
    return {"out": o[b, slot].half(), "lse": lse.permute(0, 3, 1, 2).reshape(nb, nq, hq)[b, slot].contiguous()}


def _rotate(x, cos, sin, rotary_dim, interleaved):
    """x [T, heads, D] in 32 bits; cos, sin [T, rotary_dim / 2]."""
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rotary_dim:2], x[..., 1:rotary_dim:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rotary_dim // 2], x[..., rotary_dim // 2:rotary_dim]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., rotary_dim:]], -1)


def _power_scale(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^-60."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -60)).clamp_min(-60)
    return torch.ldexp(torch.ones_like(amax), e)


def _append_plain(s):
    c = s["case"]
    hq, hkv, d, p = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    t = s["tokens"]
    b, pos = _places(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _rotate(s["q"].float().view(t, hq, d), cos, sin, c["rotary_dim"], c["interleaved"])
    s["q_out"].copy_(q)
    k = _rotate(s["k"].float().view(t, hkv, d), cos, sin, c["rotary_dim"], c["interleaved"])
    page = s["table"].long()[b, pos // p]
    old = s["kv_len"].long() - (s["q_start"][1:] - s["q_start"][:-1]).long()  # tokens that were there
    part = (old % p > 0).nonzero()[:, 0] if c["batch"] > 1 else torch.arange(1, device=DEV)
    first = s["table"].long()[part, (old[part] // p).clamp_max(s["table"].shape[1] - 1)]
    fill = (old % p)[part]
    for pool, scale, x in ((s["k_pool"], s["k_scale"], k), (s["v_pool"], s["v_scale"], s["v"].float().view(t, hkv, d))):
        amax = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
        most = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, hkv), amax, "amax")
        was = torch.zeros_like(scale)
        was[first] = scale[first] * (fill > 0)[:, None]
        new = torch.maximum(was, _power_scale(most))
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEV)
        touched[page] = True
        # tokens that share a page with new ones go over to its new scale
        rows = torch.arange(p, device=DEV)
        bits = pool.view(torch.uint8)
        held = bits[first]
        ratio = torch.where(was[first] > 0, was[first] / new[first], torch.ones_like(new[first]))
        again = (held.view(FP8).float() * ratio[..., None, None]).to(FP8).view(torch.uint8)
        keep = (rows[None, :] < fill[:, None])[:, None, :, None]
        bits[first] = torch.where(keep, again, held)
        scale.copy_(torch.where(touched[:, None], new, scale))
        bits[page, :, pos % p] = (x / scale[page][..., None]).clamp(-448, 448).to(FP8).view(torch.uint8)
    return _cache_out(s)


def _log_softmax(x, t):
    x = x.float() / t
    x = x - x.amax(-1, keepdim=True)
    return x - torch.log(torch.exp(x).sum(-1, keepdim=True))


def _verify_plain(s):
    c = s["case"]
    b, n, v = c["batch"], c["drafts"], c["vocab"]
    target, x = s["target"], s["draft_tokens"].long()
    greedy = c["temperature"] == 0
    logp = _log_softmax(target, c["temperature"] or 1.0)
    rows = torch.arange(b, device=DEV)
    if greedy:
        best = logp.argmax(-1)
        ok = best[:, :n] == x
    else:
        p = torch.exp(logp)
        px = p[:, :n].gather(2, x[..., None])[..., 0]
        if s["draft"] is not None:
            q = torch.exp(_log_softmax(s["draft"], c["temperature"]))
            ok = s["u"] * q.gather(2, x[..., None])[..., 0] < px
        else:
            ok = s["u"] < px
    accepted = ok.long().cumprod(1).sum(1)
    if greedy:
        token = best[rows, accepted]
    else:
        pr = p[rows, accepted]
        at = accepted.clamp_max(n - 1)
        if s["draft"] is not None:
            res = (pr - q[rows, at]).clamp_min(0)
        else:
            res = pr.scatter(1, x[rows, at][:, None], 0.0)
        res = torch.where((accepted == n)[:, None] | (res.amax(1, keepdim=True) <= 0), pr, res)
        token = (res / s["e"]).argmax(1)
    i = torch.arange(n + 1, device=DEV)
    tokens = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(i < accepted[:, None], tokens, torch.where(i == accepted[:, None], token[:, None], -1))
    lp = logp.gather(2, tokens.clamp_min(0)[..., None])[..., 0]
    return {"tokens": tokens.to(torch.int32), "accepted": accepted.to(torch.int32),
            "logprob": torch.where(tokens >= 0, lp, torch.zeros_like(lp))}


# ------------------------------------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _attention_exact, "append": _append_exact, "verify": _verify_exact}[case["op"]](s)


def _attention_exact(s):
    c = s["case"]
    p, d = c["page"], c["head_dim"]
    per = c["q_heads"] // c["kv_heads"]
    out = torch.zeros((s["tokens"], c["q_heads"], d), dtype=torch.float64, device=DEV)
    lse = torch.full((s["tokens"], c["q_heads"]), -math.inf, dtype=torch.float64, device=DEV)
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    pools = [s[name].view(torch.uint8) for name in ("k_pool", "v_pool")]
    for b, t in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if t == 0 or hi == lo:
            continue
        pages = s["table"][b, :-(-t // p)].long()
        pos = torch.arange(t - (hi - lo), t, device=DEV)
        j = torch.arange(t, device=DEV)
        hide = torch.zeros((hi - lo, t), dtype=torch.bool, device=DEV)
        if c["causal"]:
            hide |= j[None] > pos[:, None]
        if c["window"]:
            hide |= j[None] <= pos[:, None] - c["window"]
        hide |= pos[:, None] < 0
        for h in range(c["kv_heads"]):
            k = (pools[0][pages, h].view(FP8).double() * s["k_scale"][pages, h].double()[:, None, None]).reshape(-1, d)[:t]
            v = (pools[1][pages, h].view(FP8).double() * s["v_scale"][pages, h].double()[:, None, None]).reshape(-1, d)[:t]
            for g in range(h * per, (h + 1) * per):
                x = (s["q"][lo:hi, g].double() @ k.T) * (1 / math.sqrt(d))
                x[hide] = -math.inf
                l = torch.logsumexp(x, 1)
                lse[lo:hi, g] = l
                w = torch.exp(x - l[:, None])
                w[torch.isinf(l)] = 0
                out[lo:hi, g] = w @ v
    return {"out": out, "lse": lse}


def _nearest_e4m3(x):
    """The values of the 8-bit format nearest to x (64 bits, ties to even), at most 448 in size."""
    _, e = torch.frexp(x.abs())
    ulp = torch.ldexp(torch.ones_like(x), (e - 1).clamp_min(-6) - 3)
    return (torch.round(x / ulp) * ulp).clamp(-448, 448)


def _append_exact(s):
    c = s["case"]
    p, d, r, hkv, hq = c["page"], c["head_dim"], c["rotary_dim"], c["kv_heads"], c["q_heads"]
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    big = {"k_codes": s["k_pool"].float(), "v_codes": s["v_pool"].float()}
    scale = {"k_codes": s["k_scale"].double(), "v_codes": s["v_scale"].double()}
    at = torch.cat([torch.arange(t - (hi - lo), t, device=DEV) for lo, hi, t in zip(starts, starts[1:], lens)])
    cos, sin = s["cos"][at].double(), s["sin"][at].double()

    def turned(x):
        x = x.double().view(s["tokens"], -1, d).clone()
        i = torch.arange(r // 2, device=DEV)
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(cos, sin)[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    new = {"k_codes": turned(s["k"]), "v_codes": s["v"].double().view(s["tokens"], hkv, d)}
    table = s["table"].tolist()
    for name, pool in big.items():
        for b, t in enumerate(lens):
            lo, pos = starts[b], lens[b] - (starts[b + 1] - starts[b])
            while pos < t:
                page, row = table[b][pos // p], pos % p
                n = min(p - row, t - pos)
                x = new[name][lo:lo + n]
                sc = torch.exp2(torch.ceil(torch.log2(x.abs().amax((0, 2)) / 448))).clamp_min(2.0 ** -60)
                if row:
                    sc = torch.maximum(sc, scale[name][page])
                    pool[page, :, :row] = _nearest_e4m3(pool[page, :, :row].double() * (scale[name][page] / sc)[:, None, None]).float()
                scale[name][page] = sc
                pool[page, :, row:row + n] = _nearest_e4m3(x / sc[None, :, None]).transpose(0, 1).float()
                lo, pos = lo + n, pos + n
    return {"q": turned(s["q"]), "k_scale": scale["k_codes"], "v_scale": scale["v_codes"], **big}


def _verify_exact(s):
    """The log-probabilities of the tokens that the definition gives in 64 bits."""
    c = s["case"]
    n, t = c["drafts"], c["temperature"]
    tokens, counts, logprob = [], [], []
    for b in range(c["batch"]):
        logp = [torch.log_softmax(s["target"][b, i].double() / (t or 1.0), 0) for i in range(n + 1)]
        q = None if s["draft"] is None or not t else [torch.softmax(s["draft"][b, i].double() / t, 0) for i in range(n)]
        got = []
        for i, x in enumerate(s["draft_tokens"][b].tolist()):
            if not t:
                ok = int((s["target"][b, i] == s["target"][b, i].max()).nonzero()[0]) == x
            else:
                ok = bool(s["u"][b, i].double() * (1.0 if q is None else q[i][x]) < logp[i][x].exp())
            if not ok:
                break
            got.append(x)
        i = len(got)
        if not t:
            got.append(int((s["target"][b, i] == s["target"][b, i].max()).nonzero()[0]))
        else:
            rest = logp[i].exp()
            if i < n:
                if q is None:
                    rest[int(s["draft_tokens"][b, i])] = 0
                else:
                    rest = (rest - q[i]).clamp_min(0)
            got.append(int((rest / s["e"][b].double()).argmax()))
        tokens.append(got + [-1] * (n - i))
        counts.append(i)
        logprob.append([float(logp[k][x]) for k, x in enumerate(got)] + [0.0] * (n - i))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "accepted": torch.tensor(counts, dtype=torch.int32),
            "logprob": torch.tensor(logprob, dtype=torch.float64)}
