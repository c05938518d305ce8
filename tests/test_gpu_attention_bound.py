"""Attention where the logits climb along the keys, so that the running bound has to move: by less and by more than
the weights may grow before it does, inside a block of keys and between blocks, in few rows and in many."""
import numpy as np
import pytest

from oracle import serving as sv
from test_gpu_serving import Case, check

pytestmark = pytest.mark.gpu

# A key whose channels are all `a` has, with q of ones and a scale of 2^-6, the base-2 logit a * sqrt(D) * 2^-6 * log2(e):
# at D = 64 these are 0, 5.4, 11.5, 18.8, 31.7, 51.9, 80.8, at D = 128 sqrt(2) times that.
LEVELS = np.array([0.0, 30.0, 64.0, 104.0, 176.0, 288.0, 448.0])


def _code(value):
    return int(np.nonzero(sv.E4M3 == value)[0][0])


def _climbing(new, total, heads, page, rises, seed):
    """Level i of LEVELS is reached at key rises[i - 1]; between, keys take any level reached so far."""
    c = Case(new, total, *heads, page=page, seed=seed)
    rng = np.random.default_rng(seed)
    c.q[:] = 1.0
    c.ks[:] = 2.0 ** -6
    codes = np.array([_code(x) for x in LEVELS], np.uint8)
    for b, t in enumerate(total):
        level = np.searchsorted(np.array(rises), np.arange(t), side="right")
        for h in range(c.hkv):
            pick = (rng.random(t) * (level + 1)).astype(int)
            for i, r in enumerate(rises):
                if r < t:
                    pick[r] = i + 1
            for j in range(t):
                c.k[c.table[b, j // page], h, j % page] = codes[pick[j]]
    return c


@pytest.mark.parametrize("heads", [(12, 2, 128), (16, 4, 64), (4, 4, 64)])
@pytest.mark.parametrize("new", [1, 7, 40, 150])
@pytest.mark.parametrize("rises", [(3, 20, 40, 70, 135, 300), (0, 63, 64, 127, 128, 191), (100, 101, 102, 103, 104, 105),
                                   (640, 641, 660, 670, 690, 699)])
def test_climbing_logits(libw4, heads, new, rises):
    c = _climbing([new, min(new, 3)], [700, 699], heads, 32, rises, seed=new)
    check(c, causal=True)
    check(c, causal=False)


@pytest.mark.parametrize("heads", [(12, 2, 128), (16, 4, 64)])
def test_climbing_logits_in_a_window(libw4, heads):
    c = _climbing([130, 260], [1500, 400], heads, 16, (3, 350, 700, 1050, 1390, 1400), seed=5)
    check(c, causal=True, window=300)
