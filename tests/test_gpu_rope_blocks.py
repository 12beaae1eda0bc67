"""Rotary calls of many tokens, whose blocks take 2, 4 or 8 tokens and end inside one: bit for bit what the same rows give in calls of
so few tokens that a block has one, with nothing else written; and near the definition."""
import numpy as np
import pytest
import torch

from tests.test_gpu_rope import _cache, _equal, _freq, _near, _oracle, _pos, _rows, _twin

pytestmark = pytest.mark.gpu

CHUNK = 500                             # tokens of a call whose blocks have one each
# 152 multiprocessors: 2 tokens a block from 1216 on, 4 from 2432 on, 8 from 4864 on where heads are few; all of these end inside one
LENGTHS = [1217, 2433, 2435, 4865, 4870, 10007]


def _guarded(T, heads, D):
    """Rows with 9 more behind them, and a look at whether these are as they were."""
    wide = torch.full((T + 9, heads, D), 7, dtype=torch.bfloat16, device="cuda")
    return wide[:T], lambda: bool((wide[T:] == 7).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,dim,Hq,Hkv", [(128, 128, 3, 1), (128, 64, 40, 8), (80, 80, 4, 4), (64, 24, 20, 3)])
@pytest.mark.parametrize("T", LENGTHS)
def test_rows(T, D, dim, Hq, Hkv, interleaved):
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(T + D)
    freq, axis = _freq(dim // 2), [i % 2 for i in range(dim // 2)]
    r = B.Rotary(freq, axis=axis, axes=2, interleaved=interleaved)
    pos = rng.integers(0, 100000, (2, T))
    q, k = _rows(rng, T, Hq, D), _rows(rng, T, Hkv, D)
    (qo, q_kept), (ko, k_kept) = _guarded(T, Hq, D), _guarded(T, Hkv, D)
    B.moe_rope(r, q, k, _pos(pos), q_out=qo, k_out=ko)
    assert q_kept() and k_kept()
    for at in range(0, T, CHUNK):
        one = B.moe_rope(r, q[at:at + CHUNK], k[at:at + CHUNK], _pos(pos[:, at:at + CHUNK]))
        assert torch.equal(qo[at:at + CHUNK], one[0]) and torch.equal(ko[at:at + CHUNK], one[1])
    _near(ko[-50:], *_oracle(k[-50:], pos[:, -50:], freq, axis=axis, interleaved=interleaved))


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("D,dim,Hq,Hkv", [(128, 128, 3, 1), (128, 64, 20, 4), (64, 64, 5, 2), (64, 24, 20, 3), (128, 32, 12, 2)])
@pytest.mark.parametrize("T", LENGTHS)
def test_append(T, D, dim, Hq, Hkv, fmt):
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(T + dim)
    r = B.Rotary(_freq(dim // 2))
    pos = rng.integers(0, 100000, T)
    qkv = _rows(rng, T, Hq + 2 * Hkv, D)
    q, k, v = qkv.split((Hq, Hkv, Hkv), dim=1)
    one = _cache(T // 16 + 3, 16, Hkv, D, fmt)
    two = _twin(one)
    slots = rng.permutation(one.pages * 16)[:T].astype(np.int32)
    slots[5::11] = -1
    slots = torch.from_numpy(slots).cuda()
    (qo, q_kept), (ko, k_kept) = _guarded(T, Hq, D), _guarded(T, Hkv, D)
    B.moe_rope_kv_append(r, one, q, k, v, _pos(pos), slots, q_out=qo, k_out=ko)
    assert q_kept() and k_kept()
    for at in range(0, T, CHUNK):
        rows = slice(at, at + CHUNK)
        k_one = torch.empty((len(k[rows]), Hkv, D), dtype=torch.bfloat16, device="cuda")
        q_one = B.moe_rope_kv_append(r, two, q[rows], k[rows], v[rows], _pos(pos[rows]), slots[rows].contiguous(), k_out=k_one)
        assert torch.equal(qo[rows], q_one) and torch.equal(ko[rows], k_one)
    assert _equal(one, two)             # what nobody stored to among it
    if fmt == "bf16":                   # and the keys are those that a call without a cache turns
        three = _twin(one)
        B.moe_kv_append(three, B.moe_rope(r, q, k, _pos(pos))[1], v, slots)
        assert _equal(one, three)
    B.attention_status()
