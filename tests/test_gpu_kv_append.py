"""GPU parity: new tokens into the paged cache. Copies and the MXFP8 rule are exact, so everything is compared bit for
bit, the places that nothing was stored to included."""
import numpy as np
import pytest
import torch

from oracle import attention as A

pytestmark = pytest.mark.gpu


def _cache(pages, page, Hkv, D, mx, seed=0):
    from block_scaled_fp8_moe_gb300 import binding as B
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = B.KvCache.empty(pages, page, Hkv, D, mxfp8=mx)
    for t in (c.k, c.v, c.k_s, c.v_s):
        if t is not None:
            b = t.view(torch.uint8)
            b.copy_(torch.randint(0, 255, b.shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def _rows(n, Hkv, D, seed, apart=0):
    rng = np.random.default_rng(seed)
    a = rng.standard_normal((n, 2 * Hkv + apart, D)) * 10.0 ** rng.uniform(-3, 3, (n, 1, 1))
    t = torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16).cuda()
    return t[:, :Hkv], t[:, Hkv:2 * Hkv]


def _want(cache, k, v, slots):
    """The cache's bytes afterwards, by the oracle."""
    out = []
    for rows, data, scales in ((k, cache.k, cache.k_s), (v, cache.v, cache.v_s)):
        a = rows.float().cpu().numpy()
        if scales is None:
            new, parts = rows.cpu().contiguous().view(torch.int16).numpy(), [data.cpu().view(torch.int16).numpy().copy()]
            news = [new]
        else:
            parts, news = [data.cpu().numpy().copy(), scales.cpu().numpy().copy()], A.quant_block_mxfp8(a)
        for t, slot in enumerate(slots):
            if 0 <= slot < cache.pages * cache.page_size:
                for part, new in zip(parts, news):
                    part[slot // cache.page_size, :, slot % cache.page_size] = new[t]
        out += parts
    return out


def _got(cache):
    ts = [cache.k, cache.k_s, cache.v, cache.v_s]
    return [t.cpu().view(torch.int16).numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
            for t in ts if t is not None]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,Hkv,D,page,apart", [(1, 1, 64, 8, 0), (5, 2, 128, 16, 0), (48, 8, 128, 16, 3),
                                                (131, 3, 64, 64, 1), (700, 5, 128, 256, 0)])
def test_append_matches_the_oracle(T, Hkv, D, page, apart, mx):
    from block_scaled_fp8_moe_gb300 import binding as B
    pages = T // page + 3
    rng = np.random.default_rng(T)
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[::7] = -1
    cache = _cache(pages, page, Hkv, D, mx)
    k, v = _rows(T, Hkv, D, T, apart)
    want = _want(cache, k, v, slots)
    B.moe_kv_append(cache, k, v, torch.from_numpy(slots).cuda())
    for a, b in zip(_got(cache), want):
        assert np.array_equal(a, b)
    B.attention_status()


def test_mxfp8_edges():
    from block_scaled_fp8_moe_gb300 import binding as B
    k, v = (t.contiguous() for t in _rows(10, 1, 64, 3))
    k[0] = 0
    k[1] = -0.0
    k[2] *= 1e-35
    k[3, 0, :32] = 448
    k[3, 0, 32:] = 450
    k[4, 0, 3] = float("nan")
    k[5, 0, 40] = float("inf")
    k[6, 0, 63] = float("-inf")
    k[7] = 3.3e38
    v[8, 0, 31] = float("nan")
    cache = _cache(2, 8, 1, 64, True)
    slots = np.arange(10, dtype=np.int32)
    want = _want(cache, k, v, slots)
    B.moe_kv_append(cache, k, v, torch.from_numpy(slots).cuda())
    for a, b in zip(_got(cache), want):
        assert np.array_equal(a, b)
    assert want[1][0, 0, 4, 0] == 255 and want[3][1, 0, 0, 0] == 255


def test_slots_out_of_range_are_left_out_and_reported():
    from block_scaled_fp8_moe_gb300 import binding as B
    for mx in (False, True):
        for bad in (64, -2, 2 ** 31 - 1, -2 ** 31):
            cache = _cache(4, 16, 2, 64, mx)
            k, v = _rows(4, 2, 64, 1)
            slots = np.array([3, bad, -1, 63], dtype=np.int32)
            want = _want(cache, k, v, slots)
            B.moe_kv_append(cache, k, v, torch.from_numpy(slots).cuda())
            for a, b in zip(_got(cache), want):
                assert np.array_equal(a, b)
            with pytest.raises(B.MoeError) as e:
                B.attention_status()
            assert e.value.code == B.MOE_ERR_DEVICE_INPUT
            B.attention_status()


def test_another_stream_and_a_captured_graph():
    from block_scaled_fp8_moe_gb300 import binding as B
    k, v = _rows(20, 2, 128, 5)
    slots = torch.arange(20, dtype=torch.int32, device="cuda")
    ref = _cache(3, 16, 2, 128, True)
    B.moe_kv_append(ref, k, v, slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _cache(3, 16, 2, 128, True)
    torch.cuda.synchronize()
    B.moe_kv_append(other, k, v, slots, stream=side)
    side.synchronize()
    assert torch.equal(other.k, ref.k) and torch.equal(other.v_s, ref.v_s)
    graphed = _cache(3, 16, 2, 128, True)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.moe_kv_append(graphed, k, v, slots, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_kv_append(graphed, k, v, slots, ws=ws)
    graphed.k.zero_()
    graph.replay()
    torch.cuda.synchronize()
    stored = lambda c: c.k.transpose(1, 2).flatten(0, 1)[:20]  # noqa: E731
    assert torch.equal(stored(graphed), stored(ref))


def test_refusals():
    from block_scaled_fp8_moe_gb300 import binding as B
    cache = _cache(3, 16, 2, 128, False)
    k, v = _rows(4, 2, 128, 5)
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    for call in (lambda: B.moe_kv_append(cache, k, v, slots.long()), lambda: B.moe_kv_append(cache, k[:3], v, slots),
                 lambda: B.moe_kv_append(cache, k[:, :1], v, slots), lambda: B.moe_kv_append(cache, k.float(), v, slots),
                 lambda: B.moe_kv_append(cache, k, v.transpose(1, 2).contiguous().transpose(1, 2), slots),
                 lambda: B.KvCache(cache.k, cache.v[:2]), lambda: B.KvCache(cache.k.float(), cache.v.float()),
                 lambda: B.KvCache(cache.k, cache.v, torch.zeros(3, 2, 16, 4, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for page, D in ((24, 128), (4, 128), (512, 128), (16, 96)):
        odd = B.KvCache.empty(2, page, 2, D)
        kk = torch.zeros(4, 2, D, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(B.MoeError) as e:
            B.moe_kv_append(odd, kk, kk, slots)
        assert e.value.code == B.MOE_ERR_UNSUPPORTED_SHAPE
    B.moe_kv_append(cache, k[:0], v[:0], slots[:0])


@pytest.mark.parametrize("stride", [131, 1, 2 ** 40])
def test_the_stride_of_a_single_row_does_not_matter(stride):
    from block_scaled_fp8_moe_gb300 import binding as B
    cache = _cache(3, 16, 2, 64, False)
    k, v = _rows(1, 2, 64, 5)
    odd = lambda t: t.contiguous().as_strided((1, 2, 64), (stride, 64, 1))  # noqa: E731
    slots = np.array([17], dtype=np.int32)
    want = _want(cache, k, v, slots)
    B.moe_kv_append(cache, odd(k), odd(v), torch.from_numpy(slots).cuda())
    for a, b in zip(_got(cache), want):
        assert np.array_equal(a, b)
    for t in (cache.k, cache.v):
        t.zero_()
    B.moe_kv_append(cache, odd(k), odd(v), torch.from_numpy(slots).cuda())
    lens, table = torch.tensor([18], dtype=torch.int32, device="cuda"), torch.tensor([[2, 1]], dtype=torch.int32, device="cuda")
    q = torch.cat([k, k], 1).view(1, 1, 4, 64)
    one = q.contiguous().as_strided((1, 1, 4, 64), (stride, stride, 64, 1))
    assert torch.equal(B.moe_paged_attention(one, cache, table, lens, 18), B.moe_paged_attention(q, cache, table, lens, 18))
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    assert torch.equal(B.moe_prefill_attention(odd(k), odd(k), odd(v), cu), B.moe_prefill_attention(k, k, v, cu))


def test_a_cache_on_another_device_is_refused():
    from block_scaled_fp8_moe_gb300 import binding as B
    cache = _cache(3, 16, 2, 64, False)
    k, v = _rows(2, 2, 64, 5)
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    cache.dev += 1                                # as if it had been made there
    with pytest.raises(ValueError, match="device"):
        B.moe_kv_append(cache, k, v, ids)
    with pytest.raises(ValueError, match="device"):
        B.moe_paged_attention(k.contiguous().view(2, 1, 2, 64), cache, ids.view(2, 1), ids, 16)
