"""FP64 CPU definitions of the serving operators (append to a paged 8-bit cache, attention over it, draft
verification), in numpy, sharing no code with the CUDA path.  Used only by the tests."""
from __future__ import annotations

import math

import numpy as np


def e4m3_values() -> np.ndarray:
    """The 256 values of the E4M3 code (sign, 4 exponent bits with bias 7, 3 mantissa bits; no infinities,
    0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = math.nan
        elif e == 0:
            out[c] = sign * m * 2.0 ** -9
        else:
            out[c] = sign * (8 + m) * 2.0 ** (e - 10)
    return out


E4M3 = e4m3_values()


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Value nearest to x in E4M3, ties to the even code, saturating at +-448; NaN stays."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    ulp = 2.0 ** (np.maximum(e, -6) - 3)
    return np.clip(np.rint(x / ulp) * ulp, -448, 448)


def e4m3_ulp(x: np.ndarray) -> np.ndarray:
    """Spacing of E4M3 around |x| (x in the code's own range)."""
    a = np.abs(np.asarray(x, np.float64))
    e = np.floor(np.log2(np.where(a > 0, a, 1e-30)))
    return 2.0 ** (np.maximum(e, -6) - 3)


def power_scale(amax: float) -> float:
    """The smallest power of two s with amax <= 448 s, at least 2^-60."""
    s = 2.0 ** -60
    while amax > 448 * s:
        s *= 2
    return s


def rotate(x, cos, sin, rotary_dim, interleaved):
    """x [heads, D]; cos, sin [rotary_dim / 2]."""
    y = np.array(x, np.float64)
    i = np.arange(rotary_dim // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)
    y[:, a] = x[:, a] * cos - x[:, b] * sin
    y[:, b] = x[:, b] * cos + x[:, a] * sin
    return y


def attention_rows(q, keys, values, positions, kv_len, scale, causal, window):
    """q [n, G, D] of one kv head, keys / values [kv_len, D] in float64.  Returns out, lse, and per output
    the sum of w |v| / sum w (for error bounds)."""
    n, g, d = q.shape
    out, mag = np.zeros((n, g, d)), np.zeros((n, g, d))
    lse = np.full((n, g), -np.inf)
    j = np.arange(kv_len)
    for i in range(n):
        p = positions[i]
        see = (j >= 0) & (p >= 0)
        if causal:
            see &= j <= p
        if window:
            see &= j > p - window
        if not see.any():
            continue
        x = (q[i].astype(np.float64) @ keys[see].T) * scale
        m = x.max(axis=1, keepdims=True)
        w = np.exp(x - m)
        s = w.sum(axis=1, keepdims=True)
        out[i] = w @ values[see] / s
        mag[i] = w @ np.abs(values[see]) / s
        lse[i] = (m + np.log(s))[:, 0]
    return out, lse, mag


def softmax(x, t):
    x = np.where(np.isnan(x), -np.inf, np.minimum(np.asarray(x, np.float64), 65504.0))
    m = x.max()
    if m == -np.inf:
        return np.zeros_like(x), np.full_like(x, -np.inf)
    y = (x - m) / t
    lp = y - np.log(np.exp(y).sum())
    return np.exp(lp), lp


def verify(target, draft, drafted, u, e, temperature):
    """One sequence: target [n + 1, V], draft [n, V] or None, drafted [n], u [n], e [V].  Returns tokens
    (accepted ones and the new one), accepted, log-probabilities, and the smallest relative margin of
    the decisions taken."""
    n, vocab = len(drafted), target.shape[1]
    t = temperature or 1.0
    out, lps, margin = [], [], np.inf

    def first_max(x):
        """Index of the first largest, and how far the next value is below it."""
        k = int(np.argmax(x))
        rest = np.delete(x, k)
        gap = (x[k] - rest.max()) / abs(x[k]) if rest.size and x[k] else np.inf
        return k, gap

    for i in range(n):
        p, lp = softmax(target[i], t)
        x = int(drafted[i])
        inside = 0 <= x < vocab
        if temperature == 0:
            clean = np.where(np.isnan(target[i]), -np.inf, np.minimum(target[i].astype(np.float64), 65504.0))
            ok = inside and clean.max() > -np.inf and int(np.argmax(clean)) == x
        else:
            q = softmax(draft[i], t)[0] if draft is not None else None
            ok = False
            if inside:
                a, b = u[i] * (q[x] if q is not None else 1.0), p[x]
                ok = a < b
                margin = min(margin, abs(a - b) / max(a, b, 1e-300))
        if not ok:
            break
        out.append(x)
        lps.append(lp[x])
    acc = len(out)
    p, lp = softmax(target[acc], t)
    if temperature == 0:
        clean = np.where(np.isnan(target[acc]), -np.inf, np.minimum(target[acc].astype(np.float64), 65504.0))
        token = int(np.argmax(clean)) if clean.max() > -np.inf else -1
    else:
        res = p.copy()
        if acc < n:
            if draft is not None:
                res = np.maximum(p - softmax(draft[acc], t)[0], 0)
            elif 0 <= int(drafted[acc]) < vocab:
                res[int(drafted[acc])] = 0
        if res.max() <= 0:
            res = p
        token = -1
        if res.max() > 0:
            token, gap = first_max(res / e)
            margin = min(margin, gap)
    out.append(token)
    lps.append(lp[token] if token >= 0 else -np.inf)
    return out, acc, lps, margin
