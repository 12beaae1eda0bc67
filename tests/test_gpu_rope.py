"""GPU parity: rotary positions, alone and on the way into the cache, against the definition in 64 bits.

Tolerance of a turned value a c - b s: its rounding to bf16, 2^-8 of it; cosine and sine off by at most 4e-7 (two units in the
last place, and the angle's rounding to 24 bits of half a turn, 2^-25 * pi) and two roundings of fp32, 2^-23, of |a| + |b|: below
2^-20 of those."""
import math

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import formats as F

pytestmark = pytest.mark.gpu


def _near(got, want, mag):
    got = got.float().cpu().numpy()
    bad = np.abs(got - want) > 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag + 1e-38
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want).max()))


def _rows(rng, T, heads, D, spread=2.0):
    a = rng.standard_normal((T, heads, D)) * np.exp(spread * rng.standard_normal((T, heads, 1)))
    return torch.from_numpy(a.astype(np.float32)).bfloat16().cuda()


def _freq(half, base=10000.0):
    return [base ** (-i / half) for i in range(half)]


def _pos(p):
    return torch.from_numpy(np.ascontiguousarray(p, dtype=np.int32)).cuda()


def _oracle(x, pos, freq, **kw):
    return A.rope(x.float().cpu().numpy(), np.atleast_2d(np.asarray(pos)), freq, **kw)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,dim", [(1, 1, 1, 64, 64), (6, 32, 8, 128, 128), (131, 5, 1, 80, 80), (33, 3, 2, 96, 32),
                                            (7, 2, 0, 256, 256), (9, 16, 16, 72, 72), (65, 7, 1, 8, 8), (700, 9, 3, 128, 48),
                                            (3, 1, 1, 128, 24), (2, 0, 3, 64, 16), (5, 70, 1, 40, 40)])
def test_rows_heads_and_dimensions(T, Hq, Hkv, D, dim, inverse, interleaved):
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(T + D)
    freq = _freq(dim // 2)
    pos = rng.integers(0, 5000, T)
    q, k = _rows(rng, T, Hq, D), _rows(rng, T, Hkv, D)
    r = B.Rotary(freq, interleaved=interleaved, factor=1.25)
    qo, ko = B.moe_rope(r, q, k, _pos(pos), inverse=inverse)
    for got, x in ((qo, q), (ko, k)):
        want, mag = _oracle(x, pos, freq, interleaved=interleaved, factor=1.25, inverse=inverse)
        _near(got, want, mag)
        assert torch.equal(got[..., dim:], x[..., dim:])
    alone, none = B.moe_rope(r, q, None, _pos(pos), inverse=inverse)
    assert none is None and torch.equal(alone, qo)


@pytest.mark.parametrize("axes,axis", [(2, [0] * 16 + [1] * 16), (3, [i % 3 for i in range(32)]),
                                       (3, [0] * 8 + [1] * 12 + [2] * 12), (4, [3] * 5 + [i % 4 for i in range(27)])])
def test_several_axes(axes, axis):
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(axes)
    freq = _freq(32, 500000.0)
    pos = rng.integers(-300, 100000, (axes, 90))
    q, k = _rows(rng, 90, 6, 64), _rows(rng, 90, 2, 64)
    got = B.moe_rope(B.Rotary(freq, axis=axis, axes=axes), q, k, _pos(pos))
    for g, x in zip(got, (q, k)):
        _near(g, *_oracle(x, pos, freq, axis=axis))


def test_far_positions_and_odd_frequencies():
    """Every int32 position, frequencies of many turns a token, below zero, tiny and zero. The angle in 64 bits as a fraction of a
    turn, by whole numbers."""
    from block_scaled_fp8_moe_gb300 import binding as B
    from fractions import Fraction
    freq = [1.0, 0.1, -0.37, 100.0, 1e6, 1e-9, 0.0, math.pi]
    pos = [0, 1, -1, 131071, 10 ** 6 + 3, 2 ** 31 - 1, -2 ** 31, 77777777]
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257")
    x = torch.zeros(len(pos), 1, 16, dtype=torch.bfloat16, device="cuda")
    x[..., ::2] = 1
    got, _ = B.moe_rope(B.Rotary(freq, interleaved=True), x, None, _pos(pos))
    got = got.float().cpu().numpy()
    for t, p in enumerate(pos):
        for i, w in enumerate(freq):
            turn = float((p * Fraction(w) / two_pi) % 1) * 2 * math.pi
            for at, want in ((2 * i, math.cos(turn)), (2 * i + 1, math.sin(turn))):
                assert abs(got[t, 0, at] - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -20, (p, w)


def test_in_place_strided_and_other_rows():
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(0)
    for D, dim, T in ((128, 128, 77), (64, 24, 1), (96, 96, 300)):
        r = B.Rotary(_freq(dim // 2))
        wide = _rows(rng, T, 11, D)
        q, k = wide[:, :6], wide[:, 6:9]
        pos = _pos(rng.integers(0, 9999, T))
        want = B.moe_rope(r, q.contiguous(), k.contiguous(), pos)
        got = B.moe_rope(r, q, k, pos)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        before = wide[:, 9:].clone()
        out = torch.full((T, 9, D), 7, dtype=torch.bfloat16, device="cuda")
        B.moe_rope(r, q, k, pos, q_out=out[:, 2:8], k_out=k)
        assert torch.equal(out[:, 2:8], want[0]) and torch.equal(k, want[1]) and (out[:, [0, 1, 8]] == 7).all()
        B.moe_rope(r, q, None, pos, q_out=q)
        assert torch.equal(q, want[0]) and torch.equal(wide[:, 9:], before)


def test_the_gradient_is_the_inverse():
    """Against the formula's own gradient by torch in 64 bits, and against differences."""
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(3)
    T, H, D, freq, factor = 5, 3, 64, _freq(24), 1.1
    pos = rng.integers(0, 3000, T)
    x, dy = _rows(rng, T, H, D, 0.3), _rows(rng, T, H, D, 0.3)
    angle = torch.tensor(pos, dtype=torch.float64)[:, None, None] * torch.tensor(freq, dtype=torch.float64)

    def f(t):
        a, b = t[..., :24], t[..., 24:48]
        c, s = angle.cos() * factor, angle.sin() * factor
        return torch.cat((a * c - b * s, a * s + b * c, t[..., 48:]), -1)
    leaf = x.double().cpu().requires_grad_()
    (f(leaf) * dy.double().cpu()).sum().backward()
    r = B.Rotary(freq, factor=factor)
    got, _ = B.moe_rope(r, dy, None, _pos(pos), inverse=True)
    _, mag = _oracle(dy, pos, freq, factor=factor)
    _near(got, leaf.grad.numpy(), mag)
    # the result's change along dx, from the call itself; it is linear, and every one of its values is rounded by 2^-8
    dx = _rows(rng, T, H, D, 0.3)
    up, down = (B.moe_rope(r, (x + s * dx), None, _pos(pos))[0].double() for s in (1, -1))
    step = (x + dx).double() - (x - dx).double()
    left, right = ((up - down) * dy.double()).sum(), (step * got.double()).sum()
    bound = 2.0 ** -8 * (((up.abs() + down.abs()) * dy.double().abs()).sum() + (step * got.double()).abs().sum())
    assert (left - right).abs() <= bound


def test_values_that_are_not_finite_stay_in_their_pair():
    from block_scaled_fp8_moe_gb300 import binding as B
    x = _rows(np.random.default_rng(1), 3, 2, 64)
    r = B.Rotary(_freq(16))
    pos = _pos([5, 6, 7])
    want, _ = B.moe_rope(r, x, None, pos)
    x[1, 1, 3], x[2, 0, 40] = float("nan"), float("inf")
    got, _ = B.moe_rope(r, x, None, pos)
    assert got[1, 1, [3, 19]].isnan().all() and got[2, 0, 40] == float("inf")
    same = torch.ones_like(x, dtype=torch.bool)
    same[1, 1, [3, 19]] = same[2, 0, 40] = False
    assert torch.equal(got[same], want[same])


def _cache(pages, page, Hkv, D, fmt, seed=0):
    from block_scaled_fp8_moe_gb300 import binding as B
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = B.KvCache.empty(pages, page, Hkv, D, **({} if fmt == "bf16" else {fmt: True}))
    for t in (c.k, c.v, c.k_s, c.v_s):
        if t is not None:
            b = t.view(torch.uint8)
            b.copy_(torch.randint(0, 255, b.shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def _tensors(c):
    return [t for t in (c.k, c.v, c.k_s, c.v_s) if t is not None]


def _twin(c):
    from block_scaled_fp8_moe_gb300 import binding as B
    return B.KvCache(*(t.clone() for t in (c.k, c.v)), *(t.clone() for t in (c.k_s, c.v_s) if t is not None))


def _equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(_tensors(a), _tensors(b)))


def _slots(rng, T, cache):
    slots = rng.permutation(cache.pages * cache.page_size)[:T].astype(np.int32)
    slots[2::7] = -1
    return torch.from_numpy(slots).cuda()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("T,Hq,Hkv,D,dim,page", [(1, 1, 1, 64, 64, 8), (48, 64, 8, 128, 128, 16), (131, 5, 5, 64, 24, 64),
                                                 (700, 3, 1, 128, 48, 256), (5, 0, 2, 128, 128, 32), (2200, 8, 2, 64, 32, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_without_a_turn_and_with_quarters_of_one(T, Hq, Hkv, D, dim, page, fmt, interleaved):
    """A turn by nothing, or by quarters, is exact: the cache holds, bit for bit, what the append stores of the turned keys."""
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(T)
    qkv = _rows(rng, T, Hq + 2 * Hkv + 1, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:Hq + 2 * Hkv]
    r = B.Rotary([math.pi / 2] * (dim // 2), interleaved=interleaved)
    first = _cache(T // page + 3, page, Hkv, D, fmt)
    slots = _slots(rng, T, first)
    for pos in (np.zeros(T), rng.integers(0, 4, T)):
        one, two = _twin(first), _twin(first)
        k_out = torch.empty_like(k.contiguous())
        qo = B.moe_rope_kv_append(r, one, q, k, v, _pos(pos), slots, k_out=k_out)
        want_q, want_k = B.moe_rope(r, q, k, _pos(pos))
        assert torch.equal(qo, want_q) and torch.equal(k_out, want_k)
        if not pos.any():
            assert torch.equal(qo, q) and torch.equal(k_out, k)
        B.moe_kv_append(two, want_k, v, slots)
        assert _equal(one, two)
    B.attention_status()


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("D,dim,axes", [(128, 128, 1), (64, 64, 3), (128, 64, 2), (64, 24, 1)])
def test_append_turned_keys(D, dim, axes, fmt):
    """Every stored value is within half a step of the exact one, of the block's scale; a scale is the smallest that holds the
    block, or the next one where its largest value is at a border of two."""
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(D + dim)
    T, Hq, Hkv, page = 150, 4, 2, 16
    freq, axis = _freq(dim // 2), [i % axes for i in range(dim // 2)]
    pos = rng.integers(0, 100000, (axes, T))
    q, k, v = (_rows(rng, T, h, D) for h in (Hq, Hkv, Hkv))
    cache = _cache(T // page + 2, page, Hkv, D, fmt)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    two = _twin(cache)
    q_in = q.clone()
    assert B.moe_rope_kv_append(B.Rotary(freq, axis=axis, axes=axes), cache, q, k, v, _pos(pos), slots, q_out=q) is q
    _near(q, *_oracle(q_in, pos, freq, axis=axis))
    B.moe_kv_append(two, k, v, slots)
    assert torch.equal(cache.v.view(torch.uint8), two.v.view(torch.uint8))
    assert fmt == "bf16" or torch.equal(cache.v_s, two.v_s)
    want, mag = _oracle(k, pos, freq, axis=axis)
    got, scales = (None if t is None else t.transpose(1, 2).flatten(0, 1)[:T] for t in (cache.k, cache.k_s))
    if fmt == "bf16":
        return _near(got, want, mag)
    noise = 2.0 ** -20 * mag
    amax = np.abs(want).reshape(T, Hkv, -1, 32).max(-1)
    qmax, top_step = (448.0, 32.0) if fmt == "mxfp8" else (6.0, 2.0)
    s = scales.cpu().numpy().astype(int) - 127
    slack = noise.reshape(T, Hkv, -1, 32).max(-1)
    assert np.all(amax - slack <= qmax * 2.0 ** s) and np.all(amax + slack >= qmax * 2.0 ** (s - 1))
    codes = got.cpu().numpy()
    vals = F.decode_e4m3(codes) if fmt == "mxfp8" else F.decode_e2m1(F.unpack_e2m1(codes))
    unit = np.repeat(2.0 ** s, 32, axis=-1)
    # half a step at the value's own size: 3 (1) digits behind the first one, from the smallest normal value on
    digits, low = (3, 2.0 ** -6) if fmt == "mxfp8" else (1, 1.0)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want / unit), low))) - digits)
    assert np.all(np.abs(vals * unit - want) <= np.minimum(step, top_step) / 2 * unit * (1 + 2.0 ** -20) + noise)


def test_slots_out_of_range_are_left_out_and_reported():
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(0)
    r = B.Rotary(_freq(32))
    for fmt in ("bf16", "mxfp8", "mxfp4"):
        for bad in (64, -2, 2 ** 31 - 1, -2 ** 31):
            cache = _cache(4, 16, 2, 64, fmt)
            two = _twin(cache)
            q, k, v = (_rows(rng, 4, h, 64) for h in (3, 2, 2))
            slots = torch.tensor([3, bad, -1, 63], dtype=torch.int32, device="cuda")
            pos = _pos([1, 2, 3, 4])
            got = B.moe_rope_kv_append(r, cache, q, k, v, pos, slots)
            with pytest.raises(B.MoeError) as e:
                B.attention_status()
            assert e.value.code == B.MOE_ERR_DEVICE_INPUT
            slots[1] = -1
            assert torch.equal(B.moe_rope_kv_append(r, two, q, k, v, pos, slots), got) and _equal(cache, two)
            B.attention_status()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_keys_that_are_not_finite(fmt):
    from block_scaled_fp8_moe_gb300 import binding as B
    k = _rows(np.random.default_rng(1), 4, 1, 64)
    cache = _cache(1, 8, 1, 64, fmt)
    k[0, 0, 3], k[1, 0, 33], k[2, 0, 0], k[2, 0, 32] = float("nan"), float("inf"), 3e38, 3e38
    B.moe_rope_kv_append(B.Rotary(_freq(32)), cache, k[:, :0], k, k, _pos([1, 2, 1, 3]), torch.arange(4, dtype=torch.int32, device="cuda"))
    s = cache.k_s[0, 0].cpu().numpy()
    assert (s[:2] == 255).all() and s[3].max() < 255 and not cache.k[0, 0, :2].any()
    assert s[2].max() == 255                      # 3e38 (sin 1 + cos 1) is past fp32


def test_streams_graphs_and_workspaces():
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(5)
    q, k, v = (_rows(rng, 20, h, 128) for h in (4, 2, 2))
    r, pos, slots = B.Rotary(_freq(64)), _pos(np.arange(20)), torch.arange(20, dtype=torch.int32, device="cuda")
    ref = _cache(3, 16, 2, 128, "mxfp4")
    other, graphed = _twin(ref), _twin(ref)
    want = B.moe_rope_kv_append(r, ref, q, k, v, pos, slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = B.moe_rope_kv_append(r, other, q, k, v, pos, slots, stream=side)
    both = B.moe_rope(r, q, k, pos, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and _equal(other, ref) and torch.equal(both[0], want)
    ws, out = torch.zeros(256, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    x, graph = torch.zeros(4, device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x += 1
        with pytest.raises(ValueError, match="workspace"):
            B.moe_rope_kv_append(r, graphed, q, k, v, pos, slots, q_out=out)
        B.moe_rope_kv_append(r, graphed, q, k, v, pos, slots, q_out=out, ws=ws)
        B.moe_rope(r, out, None, pos, inverse=True, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert _equal(graphed, ref) and torch.equal(out, B.moe_rope(r, want, None, pos, inverse=True)[0])
    pos += 7                                      # the next replay's positions
    graph.replay()
    want = B.moe_rope_kv_append(r, ref, q, k, v, pos, slots)
    torch.cuda.synchronize()
    assert _equal(graphed, ref) and torch.equal(out, B.moe_rope(r, want, None, pos, inverse=True)[0])
    B.moe_check_device_status(ws)


def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes in, and a cache's page as far."""
    from block_scaled_fp8_moe_gb300 import binding as B
    T, Hq, D = 70001, 320, 128
    r = B.Rotary(_freq(64))
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[-3:] = _rows(np.random.default_rng(0), 3, Hq, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    want, _ = B.moe_rope(r, q[-3:], None, pos[-3:].contiguous())
    got, _ = B.moe_rope(r, q, None, pos, q_out=q)
    assert torch.equal(got[-3:], want) and not got[:-3].any()
    del q, got
    page, Hkv = 64, 8
    pages = 2 ** 31 // (Hkv * page * D) + 40
    c = B.KvCache.empty(pages, page, Hkv, D)
    k = _rows(np.random.default_rng(1), 100, Hkv, D)
    slots = torch.arange(100, dtype=torch.int32, device="cuda") + (pages - 2) * page
    B.moe_rope_kv_append(r, c, k, k, k, pos[:100], slots)
    stored = c.k[-2:].transpose(1, 2).flatten(0, 1)[:100]
    assert torch.equal(stored, B.moe_rope(r, k, None, pos[:100])[0])
    assert torch.equal(c.v[-2:].transpose(1, 2).flatten(0, 1)[:100], k) and not c.k[:-2].any()
    del c
    torch.cuda.empty_cache()


def test_refusals():
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(0)
    q, k = _rows(rng, 4, 3, 64), _rows(rng, 4, 2, 64)
    r, r2, pos = B.Rotary(_freq(32)), B.Rotary(_freq(32), axis=[0, 1] * 16), _pos([1, 2, 3, 4])
    cache, slots = _cache(2, 16, 2, 64, "bf16"), torch.arange(4, dtype=torch.int32, device="cuda")
    f, g = B.moe_rope, B.moe_rope_kv_append
    for call in (lambda: f(r, q.float(), k, pos), lambda: f(r, q, k[:3], pos), lambda: f(r, q, k, pos.long()),
                 lambda: f(r, q, k, pos[:3]), lambda: f(r2, q, k, pos), lambda: f(r, q, k[..., :32], pos),
                 lambda: f(r, q, k, pos, q_out=torch.empty_like(q[:3])), lambda: f(r, q, None, pos, k_out=k),
                 lambda: f(r, q.cpu(), k, pos), lambda: f(r, q.transpose(1, 2).contiguous().transpose(1, 2), k, pos),
                 lambda: f(r, q, k, pos, q_out=q.flatten(0, 1)[:4, None].expand(4, 3, 64)),
                 lambda: g(r, cache, q, k, k[:3], pos, slots), lambda: g(r, cache, q, q, k, pos, slots),
                 lambda: g(r, cache, q, k, k, pos, slots.long()), lambda: g(r, cache, q, k, k, pos, slots[:3]),
                 lambda: g(r, _cache(2, 16, 2, 128, "bf16"), q, k, k, pos, slots),
                 lambda: B.Rotary([]), lambda: B.Rotary([[1.0]]), lambda: B.Rotary([1.0] * 4, axis=[0] * 3),
                 lambda: B.Rotary([1.0] * 4, axis=[0, 1, 2, -1]), lambda: B.Rotary([1.0] * 4, axis=[0, 1, 2, 2], axes=2)):
        with pytest.raises(ValueError):
            call()
    for code, call in ((B.MOE_ERR_INVALID_ARG, lambda: B.Rotary([float("nan")])), (B.MOE_ERR_INVALID_ARG, lambda: B.Rotary([2e6])),
                       (B.MOE_ERR_UNSUPPORTED_SHAPE, lambda: f(B.Rotary(_freq(36)), q, k, pos)),
                       (B.MOE_ERR_UNSUPPORTED_SHAPE, lambda: f(B.Rotary(_freq(3)), q, k, pos)),
                       (B.MOE_ERR_UNSUPPORTED_SHAPE, lambda: f(B.Rotary(_freq(32), axes=5), q, k, _pos(np.zeros((5, 4))))),
                       (B.MOE_ERR_UNSUPPORTED_SHAPE, lambda: f(B.Rotary(_freq(32), factor=float("inf")), q, k, pos)),
                       (B.MOE_ERR_WORKSPACE, lambda: g(r, cache, q, k, k, pos, slots, ws=torch.zeros(128, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.code == code
    assert f(r, q[:0], k[:0], pos[:0])[0].shape == (0, 3, 64)
    r.dev += 1                                    # as if it had been made there
    with pytest.raises(ValueError, match="device"):
        f(r, q, k, pos)
