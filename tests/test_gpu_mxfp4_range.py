"""GPU parity: paged attention over the 4-bit cache at the ends of its numbers' range, against the float64 oracle on the values
that the cache holds. Tolerances are the oracle's (oracle.attention.attention_tolerance), those of test_gpu_mxfp4_cache.py where
scores are of ordinary size."""
import numpy as np
import pytest
import torch

from oracle import attention as A
from tests.test_gpu_mxfp4_cache import SHAPES, Paged4

pytestmark = pytest.mark.gpu

# One key's value: its weight's rounding to bf16, where the sum takes the weight as it was, and the result's own, 2^-8 each.
ONE_KEY = 2.0 ** -7


def one_key_takes_all(p, scale):
    """Where fp32 can tell a row's best key from its second: (rows, that key's value). Scores are sums of up to 128 products,
    off by no more than 128 * 2^-24 of the products' magnitudes, so a lead of 2^-16 of those is one; and a lead of 256 leaves
    the others no weight."""
    q = p.q.double().cpu().numpy()
    sure, want = np.zeros(q.shape[:3], dtype=bool), np.zeros(q.shape)
    for b, n in enumerate(p.lens):
        mine = p.table[b, :p.used[b]].cpu().numpy()
        k, v = (t[mine].transpose(0, 2, 1, 3).reshape(-1, *t.shape[1::2])[:n] for t in p.values)
        for r in range(p.rows):
            see = A.visible(n - p.rows + r, n, 0, 0)
            for h in range(q.shape[2]):
                hk = h // (q.shape[2] // k.shape[1])
                s = k[see, hk] @ q[b, r, h] * scale
                size = (np.abs(k[see, hk]) @ np.abs(q[b, r, h])).max() * abs(scale)
                best = int(np.argmax(s))
                second = np.max(np.delete(s, best), initial=-np.inf)
                sure[b, r, h] = s[best] - second > max(256.0, 2.0 ** -16 * size)
                want[b, r, h] = v[see[best], hk]
    return sure, want


@pytest.mark.parametrize("rows,Hq", SHAPES[:2])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [20, 25, 28, 29, 30, 31, 34, 60, 95])
def test_large_scores(power, D, rows, Hq):
    """Scores of 2^power and their negatives: every row has one key's value."""
    p = Paged4([rows + 15, 700], rows, Hq, 1, D, 16, seed=power)
    p.q *= 2.0 ** (power // 2)
    p.cache.k_s += power - power // 2
    p.reread()
    for scale in (D ** -0.5, -D ** -0.5):
        got = p.run(scale=scale).double().cpu().numpy()
        sure, want = one_key_takes_all(p, scale)
        assert sure.mean() > 0.9 and np.isfinite(got).all()
        assert (np.abs(got - want) <= ONE_KEY * np.abs(want))[sure].all()


@pytest.mark.parametrize("rows,Hq", SHAPES[:2])
@pytest.mark.parametrize("power", [0, 20, 21, 22, 24, 26, 30, 40])
def test_equal_keys_share_at_any_score(power, rows, Hq):
    """All keys are the same, and all scores, of 2^power and more; their values' mean comes out."""
    p = Paged4([700, 90], rows, Hq, 1, 64, 16, seed=3)
    p.cache.k[:], p.cache.k_s[:] = 0x22, 127                    # ones
    p.q[:] = 2.0 ** power * 1.25
    p.reread()
    p.check()
    p.check(scale=-0.3)
