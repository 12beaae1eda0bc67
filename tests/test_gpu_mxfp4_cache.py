"""GPU parity: the 4-bit cache. Appends are exact and compared bit for bit; attention is compared with the float64 oracle on
the values that the cache holds.

Tolerance: the oracle's own, which allows for weights rounded to bf16 (more than 16 rows a block) by 2^-8; f16's 2^-11 (up to 16
rows) are within it down to f16's smallest normal number. Below, f16's steps are 2^-24, so that a rounding is off by 2^-25
whatever the weight; weights are held 2^7 times themselves, so they are off by 2^-32 each, and the sum that they are divided by is
at least 2^-2, the least that the largest of them may be before their reference moves: at most 2^-30 of the values' magnitudes,
summed without weights, come on top. That shows where the keys that count have the code 0 in a column.
"""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import formats as F
from tests.test_gpu_paged_attention import Paged

pytestmark = pytest.mark.gpu

# rows and heads to a kv head of 1: up to 8 rows a block, up to 16, more than 16, more than a block
SHAPES = [(1, 8), (3, 5), (6, 8), (60, 3)]


def _values(codes, scales):
    return F.dequant_blocks(F.decode_e2m1(F.unpack_e2m1(codes.cpu().numpy())), scales.cpu().numpy())


class Paged4(Paged):
    """The same sequences, pages and poison, with the keys and values held in MXFP4."""

    def __init__(self, lens, rows, Hq, Hkv, D, page, seed=0, **kw):
        super().__init__(lens, rows, Hq, Hkv, D, page, False, seed, **kw)
        parts = [A.quant_block_mxfp4(t.float().cpu().numpy()) for t in (self.cache.k, self.cache.v)]
        self.cache = self.B.KvCache(*(torch.from_numpy(p[0]).cuda() for p in parts),
                                    *(torch.from_numpy(p[1]).cuda() for p in parts))
        assert self.cache.format == self.B.MOE_KV_MXFP4 and self.cache.D == D
        self.reread()

    def reread(self):
        self.values = [_values(*t) for t in ((self.cache.k, self.cache.k_s), (self.cache.v, self.cache.v_s))]

    def tolerance(self, want, mag):
        tol = A.attention_tolerance(want, mag)
        for b in range(len(self.lens)):
            mine = self.table[b, :self.used[b]].cpu().numpy()
            whole = np.nansum(np.abs(self.values[1][mine]), axis=(0, 2))            # [Hkv, D]; more than any row sees
            tol[b] += 2.0 ** -30 * np.repeat(whole, tol.shape[2] // whole.shape[0], 0)
        return tol

    def check(self, window=0, sinks=0, **kw):
        got = self.run(window, sinks, **kw).float().cpu().numpy()
        want, mag = self.oracle(window, sinks, kw.get("scale"))
        bad = np.abs(got - want) > self.tolerance(want, mag)
        assert not bad.any() and np.isfinite(got).all(), (int(bad.sum()), float(np.nanmax(np.abs(got - want))))
        self.B.attention_status()

    def at(self, b, j):
        return int(self.table[b, j // self.page]), slice(None), j % self.page


def _random_cache(pages, page, Hkv, D, seed=0):
    from block_scaled_fp8_moe_gb300 import binding as B
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = B.KvCache.empty(pages, page, Hkv, D, mxfp4=True)
    for t in (c.k, c.v, c.k_s, c.v_s):
        t.copy_(torch.randint(0, 255, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def _appended(cache, k, v, slots):
    """The cache's bytes afterwards, by the oracle."""
    out = []
    for rows, data, scales in ((k, cache.k, cache.k_s), (v, cache.v, cache.v_s)):
        parts = [data.cpu().numpy().copy(), scales.cpu().numpy().copy()]
        for t, slot in enumerate(slots):
            if 0 <= slot < cache.pages * cache.page_size:
                for part, new in zip(parts, A.quant_block_mxfp4(rows.float().cpu().numpy())):
                    part[slot // cache.page_size, :, slot % cache.page_size] = new[t]
        out += parts
    return out


def _same(cache, want):
    return all(np.array_equal(t.cpu().numpy(), w) for t, w in zip((cache.k, cache.k_s, cache.v, cache.v_s), want))


@pytest.mark.parametrize("T,Hkv,D,page,apart", [(1, 1, 64, 8, 0), (5, 2, 128, 16, 0), (48, 8, 128, 16, 3), (131, 3, 64, 64, 1)])
def test_append_matches_the_oracle(T, Hkv, D, page, apart):
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(T)
    pages = T // page + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[1::7] = -1
    rows = rng.standard_normal((T, 2 * Hkv + apart, D)) * 10.0 ** rng.uniform(-3, 3, (T, 1, 1))
    rows = torch.from_numpy(rows.astype(np.float32)).bfloat16().cuda()
    k, v = rows[:, :Hkv], rows[:, Hkv:2 * Hkv]
    cache = _random_cache(pages, page, Hkv, D)
    want = _appended(cache, k, v, slots)
    B.moe_kv_append(cache, k, v, torch.from_numpy(slots).cuda())
    assert _same(cache, want)
    B.attention_status()


def test_append_ties_borders_and_what_is_not_finite():
    from block_scaled_fp8_moe_gb300 import binding as B
    k = torch.zeros(9, 1, 64, dtype=torch.bfloat16, device="cuda")
    grid = torch.arange(32, device="cuda") / 4 * 0.75           # 0 to 5.8 in quarters of 0.75: ties of the scale 1 among them
    k[0, 0, :32], k[0, 0, 32:] = grid, -grid
    k[0, 0, 31] = k[0, 0, 63] = 6
    k[1, 0, :8] = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6], device="cuda")
    k[1, 0, 32:40] = -k[1, 0, :8]
    k[2] = -0.0
    k[3, 0, :32], k[3, 0, 32:] = 6, 6.03125                     # the border between two scales
    k[4, 0, 3], k[5, 0, 40], k[6, 0, 63] = float("nan"), float("inf"), float("-inf")
    k[7], k[8] = 3.3e38, 1e-39
    v = k.flip(0).contiguous()
    cache = _random_cache(2, 8, 1, 64)
    slots = np.arange(9, dtype=np.int32)
    want = _appended(cache, k, v, slots)
    B.moe_kv_append(cache, k, v, torch.from_numpy(slots).cuda())
    assert _same(cache, want) and want[1][0, 0, 4, 0] == 255


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,Hq,Hkv,page", [(1, 8, 1, 16), (1, 4, 4, 8), (6, 16, 2, 16), (2, 5, 1, 64), (7, 14, 2, 32),
                                              (3, 24, 3, 128), (1, 70, 1, 256), (16, 8, 1, 64), (17, 1, 1, 8), (64, 4, 1, 64)])
def test_lengths_heads_and_pages(rows, Hq, Hkv, page, D):
    Paged4([1, rows, 17, 0, 63, 64, 65, 129, 300, 2, 1400], rows, Hq, Hkv, D, page, seed=rows * 100 + Hq).check()


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (64, 4), (100, 70), (128, 300), (1000, 3), (257, 129)])
def test_windows_and_first_tokens(window, sinks, D, page, rows, Hq):
    Paged4([700, 5, 64, 129, 1, 333, 1100], rows, Hq, 1, D, page, seed=window).check(window, sinks)


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
def test_long_sequences_in_many_pieces(D, rows, Hq):
    Paged4([5000, 4097, 1, 2049, 9001], rows, Hq, 1, D, 32, seed=4).check()
    Paged4([9001, 4097], rows, Hq, 1, D, 64, seed=5).check(4100, 33)


@pytest.mark.parametrize("rows,Hq", SHAPES)
def test_scores_far_apart_and_growing(rows, Hq):
    p = Paged4([900, 33], rows, Hq, 1, 128, 16, seed=8, q_scale=6.0, spread=0.7)
    p.check()
    p.check(scale=-0.5)
    p.check(scale=0.0)


@pytest.mark.parametrize("rows,Hq", SHAPES)
def test_a_row_does_not_depend_on_its_batch(rows, Hq):
    p = Paged4([3000, 40, 777, 1025], rows, Hq, 1, 64, 16, seed=3, spread=1.5)
    whole = p.run()
    for b, n in enumerate(p.lens):
        for max_len in (n, 3000):
            one = p.B.moe_paged_attention(p.q[b:b + 1].contiguous(), p.cache, p.table[b:b + 1].contiguous(),
                                          p.seq_lens()[b:b + 1], max_len)
            assert torch.equal(one[0], whole[b])
    for _ in range(10):
        assert torch.equal(p.run(), whole)


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("span", [(100, 112), (60, 200), (7, 230)])
def test_value_scales_over_their_range(span, D, rows, Hq):
    """Scales of neighbouring values further apart than the codes' arithmetic holds, growing and falling along the sequence."""
    p = Paged4([300, 90, 1500], rows, Hq, 1, D, 16, seed=12, q_scale=2.0 ** -5)
    rng = np.random.default_rng(rows)
    p.cache.v_s.copy_(torch.from_numpy(rng.integers(*span, tuple(p.cache.v_s.shape), dtype=np.uint8)).cuda())
    p.cache.k_s.copy_(torch.from_numpy(rng.integers(0, 124, tuple(p.cache.k_s.shape), dtype=np.uint8)).cuda())
    p.reread()
    p.check()
    p.check(70, 5)
    for b, j in ((0, 7), (0, 250), (2, 1200), (2, 1499)):       # a few keys' scores far above the others'
        p.cache.k[p.at(b, j)], p.cache.k_s[p.at(b, j)] = 0x22, 137
    p.reread()
    p.check()


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
def test_one_block_far_above_and_zeros_below(D, rows, Hq):
    """One block of columns a thousand times the others, tokens of zeros with a scale of 2^-127, tokens 2^-20 of the others."""
    p = Paged4([400, 1300], rows, Hq, 1, D, 16, seed=6)
    p.cache.v_s[..., 1] += 10
    for j in range(0, 400, 3):
        p.cache.v[p.at(0, j)], p.cache.v_s[p.at(0, j)] = (0x80, 0) if j % 2 else (0x08, 3)
    for j in range(0, 1300, 5):
        p.cache.v_s[p.at(1, j)] -= 20
    p.cache.v[p.at(0, 0)], p.cache.v_s[p.at(0, 0)] = 0, 0       # the first token of all
    p.reread()
    p.check()
    p.check(200, 1)


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shift", [-60, -25, 20, 100])
def test_all_values_far_from_one(shift, D, rows, Hq):
    """Caches whose values are all small or all large, some sequences beginning with tokens of zeros, or with a window behind
    which the first steps' tokens are nobody's; and scores that are all far below or above zero."""
    p = Paged4([400, 1300, 90], rows, Hq, 1, D, 16, seed=6)
    p.cache.v_s += shift if shift > 0 else 256 + shift
    for j in range(150):
        p.cache.v[p.at(1, j)], p.cache.v_s[p.at(1, j)] = 0, 0
    p.reread()
    p.check()
    p.check(333, 0)
    p.check(70, 3)
    p.q[..., 1:] = 0
    for x in (-300.0, 30.0, -20.0):              # every score near x * (6 to 8) / sqrt(D), whose spread it keeps small
        p.q[..., 0] = x
        p.cache.k[..., 0] = (p.cache.k[..., 0] & 0xF0) | 7
        p.cache.k_s[..., 0] = 127
        p.reread()
        p.check()
        p.check(70, 3)


@pytest.mark.parametrize("rows,Hq", SHAPES)
def test_small_and_large_queries(rows, Hq):
    """Rows whose queries are 2^-100 and 2^100 times the others', and scales of keys that make up for it."""
    for power in (-100, 100, -120):
        p = Paged4([200], rows, Hq, 1, 64, 16, seed=2)
        p.q[0, ::2] *= 2.0 ** power
        if power == 100:
            p.cache.k_s[:] = 20
        if power == -100:
            p.cache.k_s[:] = 230
            p.q[0, 1::2] *= 0
        p.reread()
        p.check()


def _put(p, b, j, col):
    """NaN at key j of sequence b, in the column's block of 32."""
    p.cache.v_s[p.at(b, j) + (col // 32,)] = 255
    p.values[1][p.at(b, j) + (slice(col // 32 * 32, col // 32 * 32 + 32),)] = np.nan


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20), (700, 200)])
def test_nan_that_some_rows_see(window, sinks, D, rows, Hq):
    lens = [700, 300, 5000]
    p = Paged4(lens, rows, Hq, 1, D, 16, seed=rows + window)
    for b, n in enumerate(lens):
        _put(p, b, n - 1, 1)
        _put(p, b, max(n - rows + 2 - 150, 0), 41)
        _put(p, b, max(n - rows + 2 - 700, 0), 42)
    for j in range(200, 240):
        _put(p, 1, j, 50)
    got = p.run(window, sinks).float().cpu().numpy()
    p.B.attention_status()
    with np.errstate(all="ignore"):
        want, mag = p.oracle(window, sinks)
        near = np.abs(got - want) <= p.tolerance(want, mag)
    fine = np.isfinite(want)
    assert near[fine].all() and not fine.all() and np.isnan(got[~fine]).all()


@pytest.mark.parametrize("rows,Hq", SHAPES)
def test_nan_scales_of_keys_and_values(rows, Hq):
    p = Paged4([40 + rows], rows, Hq, 1, 64, 16, seed=2)
    p.cache.v_s[p.at(0, 21) + (1,)] = 255
    got = p.run()
    assert got[..., 32:].isnan().all() and got[..., :32].isfinite().all()
    p.cache.k_s[p.at(0, 21) + (0,)] = 255
    assert p.run().isnan().all()
    clean = p.run(8, 2)                           # no row sees it
    assert clean[:, -1].isfinite().all()


@pytest.mark.parametrize("rows,Hq", SHAPES)
def test_queries_that_are_not_finite(rows, Hq):
    p = Paged4([90, 70], rows, Hq, 1, 64, 16, seed=2)
    want = p.run()
    p.q[0, 0, 0, 5], p.q[1, 0, 0, 7] = float("nan"), float("inf")
    got = p.run()
    assert got[:, 0, 0].isnan().all()
    got[:, 0, 0] = want[:, 0, 0]
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows,Hq,D", [(2, 4, 64), (8, 1, 128), (4, 4, 128), (3, 4, 64), (6, 8, 64), (60, 3, 128)])
def test_rows_that_see_nothing_are_plus_zero(rows, Hq, D):
    for longest in (70, 9000):
        p = Paged4([1, rows - 1, 0, longest], rows, Hq, 1, D, 16, seed=2)
        p.cache.v |= 0x88
        got = p.run().view(torch.int16)
        assert not got[0, :rows - 1].any() and not got[1, :1].any() and not got[2].any() and got[3].any()
        p.B.attention_status()
        none = p.B.moe_paged_attention(p.q, p.cache, torch.full_like(p.table, -1), p.seq_lens(), longest).view(torch.int16)
        assert not none.any()
        with pytest.raises(p.B.MoeError):
            p.B.attention_status()


@pytest.mark.parametrize("rows,Hq", SHAPES)
def test_pages_and_lengths_out_of_range(rows, Hq):
    p = Paged4([500, 41], rows, Hq, 1, 64, 16, seed=9)
    want = p.run()
    for bad in (-1, p.cache.pages, 2 ** 31 - 1):
        table = p.table.clone()
        table[0, 2] = bad
        got = p.B.moe_paged_attention(p.q, p.cache, table, p.seq_lens(), 500)
        with pytest.raises(p.B.MoeError):
            p.B.attention_status()
        assert torch.equal(got[1], want[1]) and got[0].isfinite().all() and not torch.equal(got[0], want[0])
        lens = torch.tensor([501, 41], dtype=torch.int32, device="cuda")
        got = p.B.moe_paged_attention(p.q, p.cache, p.table, lens, 500)
        with pytest.raises(p.B.MoeError):
            p.B.attention_status()
        assert not got[0].any() and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows,Hq", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
def test_whatever_a_kernel_has_left(D, rows, Hq):
    """Shared and Tensor Memory hold what ran before, NaN and large numbers here."""
    p = Paged4([5, 17, 40, 700, 100, 3000], rows, Hq, 1, D, 16, seed=D + rows)
    want = [p.run(), p.run(30, 3)]
    p.check()
    for fill in (float("nan"), 1e30, 0.0):
        x = torch.full((20000, 8, D), fill, device="cuda", dtype=torch.bfloat16)
        cu = torch.tensor([0, 20000], dtype=torch.int32, device="cuda")
        p.B.moe_prefill_attention(x, x, x, cu, window=64)
        assert torch.equal(p.run(), want[0]) and torch.equal(p.run(30, 3), want[1])


@pytest.mark.parametrize("rows,Hq", SHAPES)
def test_strided_queries_streams_and_graphs(rows, Hq):
    p = Paged4([90, 410], rows, Hq, 1, 128, 16, seed=9)
    want = p.run()
    wide = torch.zeros(2, rows, Hq + 4, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, :, :Hq] = p.q
    plain, p.q = p.q, wide[:, :, :Hq]
    assert torch.equal(p.run(), want)
    p.q = plain
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    out = torch.empty_like(want)
    assert p.run(stream=side, out=out) is out
    side.synchronize()
    assert torch.equal(out, want)
    ws = torch.zeros(p.B.moe_paged_attention_workspace_bytes(2, rows, Hq, 1, 128, 410), dtype=torch.uint8, device="cuda")
    lens, graph = p.seq_lens(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.B.moe_paged_attention(p.q, p.cache, p.table, lens, 410, out=out, ws=ws)
    for n in ([90, 410], [3, 17], [0, 300]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(7)
        graph.replay()
        fresh = p.B.moe_paged_attention(p.q, p.cache, p.table, lens, 410)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), fresh.view(torch.int16))


def test_offsets_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes into the cache."""
    from block_scaled_fp8_moe_gb300 import binding as B
    Hkv, page, D = 4, 256, 128
    pages = 2 ** 32 // (Hkv * page * D // 2) + 40
    c = B.KvCache.empty(pages, page, Hkv, D, mxfp4=True)
    rng = np.random.default_rng(0)
    k, v = (torch.from_numpy(rng.standard_normal((300, Hkv, D)).astype(np.float32)).bfloat16().cuda() for _ in range(2))
    B.moe_kv_append(c, k, v, torch.arange(300, dtype=torch.int32, device="cuda") + (pages - 2) * page)
    vals = [_values(*(torch.from_numpy(p) for p in A.quant_block_mxfp4(t.float().cpu().numpy()))) for t in (k, v)]
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
    for heads in (8, 64, 128):
        q = torch.from_numpy(rng.standard_normal((1, 1, heads, D)).astype(np.float32)).bfloat16().cuda()
        got = B.moe_paged_attention(q, c, table, torch.tensor([300], dtype=torch.int32, device="cuda"), 300)
        want, mag = A.attend_heads(q[0].float().cpu().numpy(), *vals, 299, D ** -0.5)
        assert np.all(np.abs(got[0].float().cpu().numpy() - want) <= A.attention_tolerance(want, mag))
    B.attention_status()
    del c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,Hq", SHAPES[:3])
@pytest.mark.parametrize("load", [0, 3, 6])
def test_a_wait_that_runs_out_is_reported(load, rows, Hq):
    p = Paged4([12000] * 4, rows, Hq, 1, 64, 64, seed=load)         # pieces of 7 or 8 steps; each step one load, or two
    want = p.run()
    p.B.attention_status()
    p.B.moe_selftest_attention_hold(load)
    try:
        p.run()
        with pytest.raises(p.B.MoeError) as e:
            p.B.attention_status()
        assert e.value.code == p.B.MOE_ERR_TIMEOUT
    finally:
        p.B.moe_selftest_attention_hold()
    assert torch.equal(p.run(), want)
    p.B.attention_status()


def test_refusals():
    from block_scaled_fp8_moe_gb300 import binding as B
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    for call in (lambda: B.KvCache(u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 16, 3), u8(3, 2, 16, 3)),
                 lambda: B.KvCache(u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 16, 4), u8(3, 2, 16, 2)),
                 lambda: B.KvCache(u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 8, 4), u8(3, 2, 8, 4)),
                 lambda: B.KvCache(u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 16, 4).float(), u8(3, 2, 16, 4)),
                 lambda: B.KvCache.empty(3, 16, 2, 64, mxfp8=True, mxfp4=True)):
        with pytest.raises(ValueError):
            call()
    for page, D in ((24, 128), (4, 128), (512, 128), (16, 96)):
        odd = B.KvCache.empty(2, page, 2, D, mxfp4=True)
        kk = torch.zeros(4, 2, D, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(B.MoeError) as e:
            B.moe_kv_append(odd, kk, kk, torch.arange(4, dtype=torch.int32, device="cuda"))
        assert e.value.code == B.MOE_ERR_UNSUPPORTED_SHAPE
