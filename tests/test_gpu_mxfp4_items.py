"""GPU parity: paged attention over the 4-bit cache where a block takes item after item, so that what its warps hand on from one to the
next (queries, sums, the join's buffer, the ring's phases) is used again and again; and how finely weights are rounded."""
import numpy as np
import pytest
import torch

from tests.test_gpu_mxfp4_cache import SHAPES, Paged4

pytestmark = pytest.mark.gpu


# 608 or 456 blocks for 8 rows to a key head, 304 for 15, 152 for 18: at least 3 times as many items each
@pytest.mark.parametrize("rows,Hq,Hkv", [(1, 96, 12), (3, 30, 6), (6, 9, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_more_pieces_than_the_gpu_has_room_for(D, rows, Hq, Hkv):
    rng = np.random.default_rng(D)
    lens = [int(n) for n in np.concatenate((rng.integers(1, 60, 130), rng.integers(100, 900, 30)))] + [0, 3, 1500, 2049]
    rng.shuffle(lens)
    p = Paged4(lens, rows, Hq, Hkv, D, 16, seed=rows)
    p.check()
    want = [p.run(), p.run(200, 5)]
    for _ in range(5):                  # one behind the other, without a wait between them
        got = [p.run(), p.run(200, 5)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a sequence by itself, in which no block has a second item
    for b in (0, 7, lens.index(1500), lens.index(2049)):
        one = p.B.moe_paged_attention(p.q[b:b + 1].contiguous(), p.cache, p.table[b:b + 1].contiguous(), p.seq_lens()[b:b + 1],
                                      max(lens))
        assert torch.equal(one[0], want[0][b])
    p.B.attention_status()


@pytest.mark.parametrize("rows,Hq", SHAPES[:2])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_are_rounded_to_f16(D, rows, Hq):
    """Two visible keys whose values are v and -v, and weights a and b, a + b = 1. With weights off by relative d and e, the result
    is off by 2ab(d - e) v, so by at most 2^-11 |v| for f16's 2^-11 (half a step). The result's rounding to bf16 adds 2^-8 of it.
    fp32 scores, sums of 128 products of together less than 8, are off by less than 128 * 2^-24 * 8 = 2^-14, the result by half of
    their difference at most, 2^-14 |v|. Weights of bf16, eight times as coarse, do not stay within that."""
    p = Paged4([300, 91], rows, Hq, 1, D, 16, seed=D, q_scale=0.1)
    for b, n in enumerate(p.lens):      # neighbours differ in sign
        for j in range(n):
            p.cache.v[p.at(b, j)], p.cache.v_s[p.at(b, j)] = p.cache.v[p.at(b, 0)] ^ (0x88 * (j % 2)), p.cache.v_s[p.at(b, 0)]
    p.reread()
    got = p.run(window=2).double().cpu().numpy()
    p.B.attention_status()
    want, mag = p.oracle(window=2)
    tol = (2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -8 * np.abs(want) + 1e-30
    assert (np.abs(got - want) <= tol).all()
    # the same with weights of bf16, by the definition
    q = p.q.double().cpu().numpy()
    outside = 0
    for b, n in enumerate(p.lens):
        mine = p.table[b, :p.used[b]].cpu().numpy()
        k, v = (t[mine].transpose(0, 2, 1, 3).reshape(-1, D)[:n] for t in p.values)
        for r in range(rows):
            at = n - rows + r
            s = q[b, r] @ k[at - 1:at + 1].T * D ** -0.5
            w = torch.from_numpy(np.exp(s - s.max(-1, keepdims=True))).bfloat16().double().numpy()
            out = w @ v[at - 1:at + 1] / w.sum(-1, keepdims=True)
            outside += int((np.abs(out - want[b, r]) > tol[b, r]).sum())
    assert outside > 0
