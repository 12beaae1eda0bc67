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


@pytest.mark.parametrize("rows,Hq", SHAPES)
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


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("power", [0, 20, 21, 22, 24, 26, 30, 40])
def test_equal_keys_share_at_any_score(power, rows, Hq):
    """All keys are the same, and all scores, of 2^power and more; their values' mean comes out."""
    p = Paged4([700, 90], rows, Hq, 1, 64, 16, seed=3)
    p.cache.k[:], p.cache.k_s[:] = 0x22, 127                    # ones
    p.q[:] = 2.0 ** power * 1.25
    p.reread()
    p.check()
    p.check(scale=-0.3)


def _spread(p, r, block):
    """Every other row's largest query elements 2^r times the others, where they meet keys of nothing: one element and codes of
    zero, or a block of queries and keys whose scale makes up for it."""
    if block:
        p.q[:, ::2, :, 32:64] *= 2.0 ** r
        p.cache.k_s[..., 1] -= r
    else:
        p.q[:, ::2, :, 3] = 2.0 ** r
        p.cache.k[..., 1] &= 0x0F                               # element 3 is the high half of byte 1
    p.reread()


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("r", [10, 17, 20, 24, 26, 31, 34, 60, 100])
def test_queries_with_elements_far_apart(r, block, D, rows, Hq):
    p = Paged4([700, 90], rows, Hq, 1, D, 16, seed=r)
    _spread(p, r, block)
    p.check()
    p.check(200, 3)


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("r", [20, 26, 60, 100])
def test_small_query_blocks_that_large_keys_make_up_for(r, rows, Hq):
    """A row's first block is of ordinary size and meets codes of zero, its second is 2^-r of that and meets scales of 2^r."""
    p = Paged4([700, 90], rows, Hq, 1, 64, 16, seed=r)
    p.q[..., 32:] *= 2.0 ** -r
    p.cache.k[..., :16] = 0
    p.cache.k_s[..., 1] += r
    p.reread()
    p.check()


@pytest.mark.parametrize("rows,Hq", SHAPES)
def test_scales_at_their_ends(rows, Hq):
    """Keys of scale byte 0 and of the largest, some among ordinary ones, with queries that make up for them; factors of the scores
    far from one."""
    for q, k, scale in ((2.0 ** 124, -126, None), (2.0 ** -120, 120, None), (2.0 ** 30, 30, 2.0 ** -63),
                        (2.0 ** -25, -25, 2.0 ** 47), (2.0 ** 60, 40, 2.0 ** -103), (2.0 ** -70, -40, 2.0 ** 107)):
        p = Paged4([300, 90], rows, Hq, 1, 64, 16, seed=4)
        p.cache.k_s.copy_(torch.clamp(p.cache.k_s.int() + k, 0, 255).byte())
        p.q *= q
        p.reread()
        p.check(scale=scale)
    p = Paged4([300, 90], rows, Hq, 1, 64, 16, seed=5, q_scale=2.0 ** -63)
    for j in (3, 40, 250):                       # keys of 2^66 among others whose scores are next to nothing
        p.cache.k_s[p.at(0, j)] += 66
    p.cache.k_s[p.at(0, 77)] = 0
    p.reread()
    p.check()
    p.check(100, 4)


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
def test_values_beside_ones_of_2_to_the_127(D, rows, Hq):
    """Values of 2^-40, and a token whose values are the largest of the format: in the last row's own place, which the others do not
    see; and where every row's weight of it is zero."""
    def small(seed):
        p = Paged4([200, 1300], rows, Hq, 1, D, 16, seed=seed)
        p.cache.v_s -= 40
        return p
    p = small(6)
    for b, n in enumerate(p.lens):
        p.cache.v[p.at(b, n - 1)], p.cache.v_s[p.at(b, n - 1)] = 0x22, 254          # 2^127
    p.reread()
    got = p.run().double().cpu().numpy()
    p.B.attention_status()
    want, mag = p.oracle()
    near = np.abs(got - want) <= p.tolerance(want, mag)
    # what the rest of the values' sum may be off is not what the largest one may
    for b in range(2):
        rest = np.abs(got - want)[b, :-1]
        assert (rest <= A.attention_tolerance(want, mag)[b, :-1] + 2.0 ** -30 * 2.0 ** -38 * p.lens[b]).all()
    assert near.all()
    p = small(7)
    p.q[..., 0] = 100.0
    p.cache.k[..., 0] = (p.cache.k[..., 0] & 0xF0) | 7
    large = [(0, 100), (1, 3), (1, 777)]
    for b, j in large:
        p.cache.k[p.at(b, j) + (0,)] = (p.cache.k[p.at(b, j) + (0,)] & 0xF0) | 15     # -6 instead of 6
        p.cache.v[p.at(b, j)], p.cache.v_s[p.at(b, j)] = 0x22, 254
        p.cache.k_s[p.at(b, j)] += 3
    p.reread()
    got = p.run().double().cpu().numpy()
    p.B.attention_status()
    # Such a key's score is so far below the row's best that its weight, below e^-88 < 2^-126, is none that fp32 has.
    q = p.q.double().cpu().numpy()
    for b, j in large:
        mine = p.table[b, :p.used[b]].cpu().numpy()
        k = p.values[0][mine].transpose(0, 2, 1, 3).reshape(-1, D)[:p.lens[b] - rows + 1]       # what all rows see
        s = np.einsum("rhd,nd->rhn", q[b], k) * D ** -0.5
        assert (s.max(-1) - s[..., j] > 88).all()
        p.values[1][p.at(b, j)] = 0
    want, mag = p.oracle()
    assert (np.abs(got - want) <= A.attention_tolerance(want, mag) + 2.0 ** -30 * 2.0 ** -38 * 1300).all()


@pytest.mark.parametrize("rows,Hq", SHAPES[:2])
@pytest.mark.parametrize("power", [0, 120, 124])
def test_sums_of_large_values(power, rows, Hq):
    """The mean of thousands of values of 2^power and more, with weights that refer to one far below them (5.5, of equal keys)."""
    p = Paged4([1300, 9001, 90], rows, Hq, 1, 64, 16, seed=11)
    p.cache.k[:], p.cache.k_s[:] = 0x22, 127
    p.q[:] = 0.6875
    p.cache.v &= 0x33                            # 0 to 1.5
    p.cache.v_s += power
    p.reread()
    p.check()
    p.check(700, 50)


@pytest.mark.parametrize("rows,Hq", SHAPES[:2])
def test_keys_past_the_largest_number_of_fp32(rows, Hq):
    """Scales of 2^126 and 2^127 and codes up to 6, which an append of the largest bf16 values stores (4 * 2^126), with queries that
    are zero or make up for them."""
    p = Paged4([300, 90], rows, Hq, 1, 64, 16, seed=8)
    p.q *= 2.0 ** -100
    p.q[..., 32:] *= 2.0 ** -26
    p.q[..., 40:50] = 0
    p.cache.k_s[..., 0] += 100
    p.cache.k_s[..., 1] = 253 + (torch.arange(16, device="cuda") & 1)
    p.reread()
    p.check()
