"""GPU parity: scores so large that fp32 cannot tell them from a neighbour 2^8 away: one key's value, or the mean of equal keys,
comes out of every kernel of the attention, over every format."""
import numpy as np
import pytest
import torch

from tests.test_gpu_mxfp4_range import ONE_KEY, one_key_takes_all
from tests.test_gpu_paged_attention import Paged

pytestmark = pytest.mark.gpu

POWERS = [24, 27, 28, 29, 31, 32, 33, 36, 50, 95]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,Hq", [(1, 8), (3, 5), (6, 8), (60, 3)])
@pytest.mark.parametrize("power", POWERS)
def test_paged_attention(power, rows, Hq, mx):
    p = Paged([rows + 15, 1400], rows, Hq, 1, 64, 16, mx, seed=power)
    p.q *= 2.0 ** power
    for scale in (0.125, -0.125):
        got = p.run(scale=scale).double().cpu().numpy()
        sure, want = one_key_takes_all(p, scale)
        assert sure.mean() > 0.9 and np.isfinite(got).all()
        assert (np.abs(got - want) <= ONE_KEY * np.abs(want))[sure].all()
    if mx:
        p.cache.k[:], p.cache.k_s[:] = 0x38, 127                # ones
    else:
        p.cache.k[:] = 1.0
    p.values[0][:] = 1.0
    p.q[:] = 2.0 ** power * 1.25
    p.check()
    p.check(scale=-0.3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", POWERS)
def test_prompt_attention(power, D):
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(power)
    lens, Hq, Hkv = [300, 1, 17, 130], 4, 2
    cu = np.concatenate(([0], np.cumsum(lens)))
    q, k, v = (torch.from_numpy(rng.standard_normal((cu[-1], h, D)).astype(np.float32)).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    q *= 2.0 ** power
    bounds = torch.from_numpy(cu.astype(np.int32)).cuda()
    q64, k64, v64 = (t.double().cpu().numpy() for t in (q, k, v))
    for scale in (0.125, -0.125):
        got = B.moe_prefill_attention(q, k, v, bounds, scale=scale).double().cpu().numpy()
        assert np.isfinite(got).all()
        told = 0
        for b, n in enumerate(lens):
            for t in range(n):
                for h in range(Hq):
                    keys, vals = (a[cu[b]:cu[b] + t + 1, h // 2] for a in (k64, v64))
                    s = keys @ q64[cu[b] + t, h] * scale
                    size = (np.abs(keys) @ np.abs(q64[cu[b] + t, h])).max() * abs(scale)
                    best = int(np.argmax(s))
                    if s[best] - np.max(np.delete(s, best), initial=-np.inf) > max(256.0, 2.0 ** -16 * size):
                        want = vals[best]
                        assert (np.abs(got[cu[b] + t, h] - want) <= ONE_KEY * np.abs(want)).all()
                        told += 1
        assert told > 0.9 * cu[-1] * Hq
    B.attention_status()
