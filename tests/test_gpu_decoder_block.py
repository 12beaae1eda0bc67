"""The example's decoder block at a small size: each stage against the oracle on the inputs that it really had, and the
experts' rows against the layer's own call, bit for bit."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import formats as F

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("mxfp8", [False, True])
@pytest.mark.parametrize("window,sinks,rows", [(0, 0, 6), (40, 3, 2)])
def test_prompt_and_decode_steps(mxfp8, window, sinks, rows, monkeypatch):
    import decoder_block as E
    B = E.B
    hidden, heads, heads_kv, dim, page = 256, 8, 2, 64, 16
    block = E.DecoderBlock(hidden, heads, heads_kv, dim, 8, 2, 128, window, sinks)
    cache = B.KvCache.empty(64, page, heads_kv, dim, mxfp8=mxfp8)
    calls = []

    def spy(name):
        inner = getattr(B, name)

        def call(*a, **kw):
            r = inner(*a, **kw)
            torch.cuda.synchronize()
            keep = [t.clone() if torch.is_tensor(t) else t for t in a]
            calls.append((name, keep, kw, r))
            return r
        monkeypatch.setattr(B, name, call)
    for name in ("moe_add_rmsnorm_mxfp8", "moe_prefill_attention", "moe_paged_attention", "moe_combine"):
        spy(name)
    lens, steps = [70, 5, 1], 3
    outs = E.run(lens, rows, steps, block, cache, hidden)
    monkeypatch.undo()
    assert [o.shape[0] for o in outs] == [sum(lens)] + [len(lens) * rows] * steps
    want = {"moe_add_rmsnorm_mxfp8": 2 * (1 + steps), "moe_prefill_attention": 1, "moe_paged_attention": steps,
            "moe_combine": 1 + steps}
    assert {n: sum(c[0] == n for c in calls) for n in want} == want

    norm = None
    for name, a, kw, r in calls:
        if name == "moe_add_rmsnorm_mxfp8":
            norm = r
            h, y = A.add_rmsnorm(_np(a[0]), None if a[2] is None else _np(a[2]), _np(a[1]), 1e-6)
            assert np.all(np.abs(_np(r[0]) - y) <= 2.0 ** -8 * np.abs(y) + 1e-38)
            assert np.all(np.abs(_np(r[1]) - h) <= 2.0 ** -8 * np.abs(h))
        elif name == "moe_prefill_attention":
            q, k, v, cu = (_np(t) for t in a[:4])
            got, cu = _np(r), cu.astype(int)
            for b, n in enumerate(lens):
                s = slice(cu[b], cu[b + 1])
                out, mag = A.attend_heads(q[s], k[s], v[s], 0, dim ** -0.5, window, sinks)
                assert np.all(np.abs(got[s] - out) <= A.attention_tolerance(out, mag))
        elif name == "moe_combine":             # the layer's own call on the norm's bf16 rows
            assert torch.equal(r, block.moe.forward(norm[0]))
    # the last step's attention over what the cache holds now
    name, a, kw, r = [c for c in calls if c[0] == "moe_paged_attention"][-1]
    vals = [cache.k, cache.v]
    if mxfp8:
        vals = [F.dequant_blocks(F.decode_e4m3(t.cpu().numpy()), s.cpu().numpy())
                for t, s in ((cache.k, cache.k_s), (cache.v, cache.v_s))]
    else:
        vals = [_np(t) for t in vals]
    q, got, table = _np(a[0]), _np(r), a[2].cpu().numpy()
    for b, n in enumerate(a[3].tolist()):
        assert n == lens[b] + 2 * (steps - 1) + rows
        k, v = (t[table[b]].transpose(0, 2, 1, 3).reshape(-1, heads_kv, dim)[:n] for t in vals)
        out, mag = A.attend_heads(q[b], k, v, n - rows, dim ** -0.5, window, sinks)
        assert np.all(np.abs(got[b] - out) <= A.attention_tolerance(out, mag))
