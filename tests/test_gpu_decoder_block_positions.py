"""The example's decoder block with positions, over every kind of cache: the turn and the append against the oracle on the inputs
that they really had, the attention over what the cache then holds, and a prompt read back from the cache."""
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


def _values(cache):
    if cache.k_s is None:
        return [_np(t) for t in (cache.k, cache.v)]
    out = []
    for t, s in ((cache.k, cache.k_s), (cache.v, cache.v_s)):
        t = t.cpu().numpy()
        codes = F.decode_e2m1(F.unpack_e2m1(t)) if cache.desc.format == 4 else F.decode_e4m3(t)
        out.append(F.dequant_blocks(codes, s.cpu().numpy()))
    return out


@pytest.mark.parametrize("fmt", [{}, {"mxfp8": True}, {"mxfp4": True}])
@pytest.mark.parametrize("dim,rot,axes,window,sinks,rows", [(64, 64, 1, 0, 0, 6), (128, 64, 2, 40, 3, 2), (64, 32, 1, 0, 0, 1)])
def test_prompt_and_decode_steps(dim, rot, axes, window, sinks, rows, fmt, monkeypatch):
    import decoder_block as E
    B = E.B
    hidden, heads, heads_kv, page = 256, 8, 2, 16
    freq = [10000.0 ** (-i / (rot // 2)) for i in range(rot // 2)]
    axis = [i % axes for i in range(rot // 2)]
    rotary = B.Rotary(freq, axis=axis, axes=axes)
    block = E.DecoderBlock(hidden, heads, heads_kv, dim, 8, 2, 128, window, sinks, rotary=rotary)
    cache = B.KvCache.empty(64, page, heads_kv, dim, **fmt)
    calls, inner = [], {n: getattr(B, n) for n in ("moe_rope_kv_append", "moe_prefill_attention", "moe_paged_attention")}

    def append(rot_, c, q, k, v, pos, slots, q_out=None, k_out=None):
        if axes > 1:                            # the same place along every axis but the last
            pos = torch.stack([pos] * (axes - 1) + [pos // 3]).contiguous()
        keep = [t.clone() for t in (q, k, v, pos, slots)]
        r = inner["moe_rope_kv_append"](rot_, c, q, k, v, pos, slots, q_out=q_out, k_out=k_out)
        calls.append(("append", keep, r.clone(), None if k_out is None else k_out.clone()))
        return r

    def spy(name):
        def call(*a, **kw):
            r = inner[name](*a, **kw)
            calls.append((name, [t.clone() if torch.is_tensor(t) else t for t in a], r.clone(), None))
            return r
        monkeypatch.setattr(B, name, call)
    monkeypatch.setattr(B, "moe_rope_kv_append", append)
    spy("moe_prefill_attention")
    spy("moe_paged_attention")
    lens, steps = [70, 5, 1], 3
    outs = E.run(lens, rows, steps, block, cache, hidden)
    monkeypatch.undo()
    assert all(o.isfinite().all() for o in outs) and len(calls) == 2 * (1 + steps)
    for name, a, r, turned in calls:
        if name == "append":
            for got, x in ((r, a[0]), (turned, a[1])):
                if got is not None:
                    want, mag = A.rope(_np(x), _np(a[3]).reshape(axes, -1), freq, axis=axis)
                    assert np.all(np.abs(_np(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag)
        elif name == "moe_prefill_attention":
            q, k, v, cu = (_np(t) for t in a[:4])
            for b in range(len(lens)):
                s = slice(int(cu[b]), int(cu[b + 1]))
                out, mag = A.attend_heads(q[s], k[s], v[s], 0, dim ** -0.5, window, sinks)
                assert np.all(np.abs(_np(r)[s] - out) <= A.attention_tolerance(out, mag))
            # the append's keys, turned, are what the prompt's attention read
            assert torch.equal(a[1], calls[0][3]) and torch.equal(a[0], calls[0][2])
    vals = _values(cache)
    # the prompt's tokens that are still in the cache hold its turned keys, to the format's half step of their block
    table = [c for c in calls if c[0] == "moe_paged_attention"][-1][1][2].cpu().numpy()
    k = vals[0][table[0]].transpose(0, 2, 1, 3).reshape(-1, heads_kv, dim)[:lens[0]]
    want = _np(calls[0][3])[:lens[0]]
    # of a block's largest value (2 of 6, 32 of 448, an 8-bit fraction), and the bf16 rounding of what it is compared with
    part = 2 / 6 / 2 if "mxfp4" in fmt else 2.0 ** -4 if fmt else 0.0
    most = np.abs(want).reshape(*want.shape[:2], -1, 32).max(-1).repeat(32, axis=-1)
    assert np.all(np.abs(k - want) <= 2 * part * most + 2.0 ** -8 * np.abs(want))
    # the last step's attention over what the cache holds now
    name, a, r, _ = [c for c in calls if c[0] == "moe_paged_attention"][-1]
    for b, n in enumerate(a[3].tolist()):
        assert n == lens[b] + 2 * (steps - 1) + rows
        k, v = (t[table[b]].transpose(0, 2, 1, 3).reshape(-1, heads_kv, dim)[:n] for t in vals)
        out, mag = A.attend_heads(_np(a[0])[b], k, v, n - rows, dim ** -0.5, window, sinks)
        tol = A.attention_tolerance(out, mag) + 2.0 ** -30 * np.repeat(np.abs(v).sum(0), heads // heads_kv, 0)   # f16 weights
        assert np.all(np.abs(_np(r)[b] - out) <= tol)


def test_a_step_in_a_graph_on_another_stream():
    """Append with the turn and attention captured together: the next step's positions, slots and lengths are the replay's."""
    from block_scaled_fp8_moe_gb300 import binding as B
    g = torch.Generator(device="cuda").manual_seed(1)
    n, heads, heads_kv, dim = 3, 8, 2, 128
    rotary = B.Rotary([10000.0 ** (-i / 64) for i in range(64)])
    caches = [B.KvCache.empty(30, 16, heads_kv, dim, mxfp4=True) for _ in range(2)]
    table = torch.randperm(30, generator=g, device="cuda").int().view(n, 10)
    pos, lens = torch.tensor([5, 0, 61], dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    slots = torch.empty(n, dtype=torch.int32, device="cuda")
    qkv = torch.randn(n, heads + 2 * heads_kv, dim, generator=g, device="cuda").bfloat16()
    q, k, v = qkv.split((heads, heads_kv, heads_kv), dim=1)

    def place():
        slots.copy_(table[torch.arange(n, device="cuda"), (pos // 16).long()] * 16 + pos % 16)
        lens.copy_(pos + 1)
    ws = [torch.zeros(m, dtype=torch.uint8, device="cuda")
          for m in (256, B.moe_paged_attention_workspace_bytes(n, 1, heads, heads_kv, dim, 160))]
    turned, out = torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 1, heads, dim, dtype=torch.bfloat16, device="cuda")
    place()

    def step(cache, ws_):
        B.moe_rope_kv_append(rotary, cache, q, k, v, pos, slots, q_out=turned, ws=ws_[0])
        return B.moe_paged_attention(turned.view(n, 1, heads, dim), cache, table, lens, 160, out=out, ws=ws_[1])
    step(caches[0], ws)                          # once outside, as a user warms up; the same cells are written again
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step(caches[0], ws)
    for i in range(20):
        place()
        qkv.normal_(generator=g)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        got = out.clone()
        want = step(caches[1], ws)
        assert torch.equal(got, want) and torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v_s, caches[1].v_s)
        pos += 1
    for w in ws:
        B.moe_check_device_status(w)
