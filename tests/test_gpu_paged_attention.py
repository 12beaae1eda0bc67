"""GPU parity: attention of a few new rows per sequence over the paged cache, against the float64 oracle on the values
that the cache holds. The tolerance is the oracle's own (oracle.attention.attention_tolerance)."""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import formats as F

pytestmark = pytest.mark.gpu


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


class Paged:
    """A cache that holds sequences of the given lengths in pages of a random order. What lies behind a sequence's end
    and in the pages that nobody has is poison: NaN, infinities, NaN scales."""

    def __init__(self, lens, rows, Hq, Hkv, D, page, mx, seed=0, q_scale=1.0, width=None, spread=0.0):
        from block_scaled_fp8_moe_gb300 import binding as B
        rng = np.random.default_rng(seed)
        self.B, self.lens, self.rows = B, lens, rows
        used = [-(-n // page) for n in lens]
        pages = sum(used) + 2
        width = max(max(used, default=0), 1) if width is None else width
        order = rng.permutation(pages)
        table = np.full((len(lens), width), -7, dtype=np.int32)
        k = np.full((pages, Hkv, page, D), np.nan, dtype=np.float32)
        k[:, :, ::2] = np.inf
        v = -k
        self.kv = []
        at = 0
        for b, n in enumerate(lens):
            mine = order[at:at + used[b]]
            at += used[b]
            table[b, :used[b]] = mine
            kb = rng.standard_normal((n, Hkv, D)) * np.exp(spread * rng.standard_normal((n, 1, 1)))
            vb = rng.standard_normal((n, Hkv, D)) * np.exp(spread * rng.standard_normal((n, Hkv, 1)))
            for j in range(n):
                k[mine[j // page], :, j % page] = kb[j]
                v[mine[j // page], :, j % page] = vb[j]
        k, v = _bf16(k), _bf16(v)
        if mx:
            parts = []
            for t in (k, v):
                q, s = A.quant_block_mxfp8(t.float().cpu().numpy())
                parts.append((q, s, F.dequant_blocks(F.decode_e4m3(q), s)))
            self.cache = B.KvCache(*(torch.from_numpy(p[0]).cuda() for p in parts),
                                   *(torch.from_numpy(p[1]).cuda() for p in parts))
            self.values = [p[2] for p in parts]
        else:
            self.cache = B.KvCache(k, v)
            self.values = [t.float().cpu().numpy().astype(np.float64) for t in (k, v)]
        self.table = torch.from_numpy(table).cuda()
        self.q = _bf16(rng.standard_normal((len(lens), rows, Hq, D)) * q_scale)
        self.page, self.used = page, used

    def seq_lens(self):
        return torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def oracle(self, window=0, sinks=0, scale=None, only=None):
        q = self.q.float().cpu().numpy()
        out, mag = np.zeros(q.shape), np.zeros(q.shape)
        for b, n in enumerate(self.lens):
            if only is not None and b not in only:
                continue
            mine = self.table[b, :self.used[b]].cpu().numpy()
            k, v = (t[mine].transpose(0, 2, 1, 3).reshape(-1, *t.shape[1::2])[:n] for t in self.values)
            out[b], mag[b] = A.attend_heads(q[b], k, v, n - self.rows, q.shape[-1] ** -0.5 if scale is None else scale,
                                            window, sinks)
        return out, mag

    def run(self, window=0, sinks=0, max_len=None, **kw):
        max_len = max(self.lens) if max_len is None else max_len
        return self.B.moe_paged_attention(self.q, self.cache, self.table, self.seq_lens(), max_len, window=window,
                                          sinks=sinks, **kw)

    def check(self, window=0, sinks=0, **kw):
        got = self.run(window, sinks, **kw).float().cpu().numpy()
        want, mag = self.oracle(window, sinks, kw.get("scale"))
        bad = np.abs(got - want) > A.attention_tolerance(want, mag)
        assert not bad.any() and np.isfinite(got).all(), (int(bad.sum()), float(np.nanmax(np.abs(got - want))))
        self.B.attention_status()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,Hq,Hkv,page", [(1, 8, 1, 16), (1, 4, 4, 8), (6, 16, 2, 16), (2, 5, 1, 64),
                                              (7, 14, 2, 32), (3, 24, 3, 128), (1, 70, 1, 256), (16, 8, 1, 64)])
def test_lengths_heads_and_pages(rows, Hq, Hkv, page, D, mx):
    lens = [1, rows, 17, 0, 63, 64, 65, 129, 300, 2]
    Paged(lens, rows, Hq, Hkv, D, page, mx, seed=rows * 100 + Hq).check()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 0), (64, 4), (100, 70), (128, 300), (1000, 3),
                                          (257, 129)])
def test_windows_and_first_tokens(window, sinks, mx):
    Paged([700, 5, 64, 129, 1, 333, 1100], 3, 8, 2, 64, 16, mx, seed=window).check(window, sinks)


@pytest.mark.parametrize("mx,D", [(False, 128), (True, 128), (False, 64), (True, 64)])
def test_long_sequences_in_many_pieces(mx, D):
    Paged([5000, 4097, 1, 2049, 9001], 2, 4, 1, D, 32, mx, seed=4).check()
    Paged([9001, 4097], 1, 4, 2, D, 64, mx, seed=5).check(4100, 33)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,Hq,Hkv", [(3, 8, 1), (9, 16, 1)])
def test_many_rows_where_the_pieces_of_a_sequence_change(rows, Hq, Hkv, mx):
    """8192 tokens and around: pieces of twice as many steps; 144 rows are two blocks of rows."""
    Paged([8064, 8065, 8192, 8193, 8320, 700], rows, Hq, Hkv, 64, 64, mx, seed=rows).check()
    Paged([8192, 8193, 9000], rows, Hq, Hkv, 64, 64, mx, seed=rows + 1).check(8100, 130)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,Hq,Hkv", [(1, 8, 1), (2, 8, 1), (4, 8, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_short_sequences_where_a_kernel_has_left_nan(D, rows, Hq, Hkv, mx):
    """Pages that a short sequence does not have leave their places in a block's shared memory as they were."""
    p = Paged([5, 17, 40, 70, 100, 129], rows, Hq, Hkv, D, 16, mx, seed=D + rows)
    nan = torch.full((20000, Hkv, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    q, cu = torch.zeros((20000, Hq, D), device="cuda", dtype=torch.bfloat16), torch.tensor([0, 20000], dtype=torch.int32, device="cuda")
    for _ in range(3):
        p.B.moe_prefill_attention(q, nan, nan, cu, window=300)
        p.check()
        p.check(30, 3)


def test_one_large_score_takes_all():
    """Scores far apart, and growing along the sequence, so that the running maximum moves again and again."""
    for mx in (False, True):
        p = Paged([900, 33], 2, 4, 2, 128, 16, mx, seed=8, q_scale=6.0, spread=0.7)
        p.check()
        p.check(scale=-0.5)
        p.check(scale=0.0)


def test_a_row_does_not_depend_on_its_batch():
    for mx in (False, True):
        p = Paged([3000, 40, 777, 1025], 4, 8, 2, 64, 16, mx, seed=3)
        whole = p.run()
        for b, n in enumerate(p.lens):
            for max_len in (n, n + 1, 3000):
                one = p.B.moe_paged_attention(p.q[b:b + 1].contiguous(), p.cache, p.table[b:b + 1].contiguous(),
                                              p.seq_lens()[b:b + 1], max_len)
                assert torch.equal(one[0], whole[b])


def test_later_rows_values_do_not_reach_earlier_rows():
    """Verification rows: what a draft token's key and value hold does not matter to the rows before it."""
    for bad in (float("nan"), float("inf"), 3e38):
        p = Paged([130, 64, 70], 6, 8, 2, 64, 16, False, seed=6)
        for b, n in enumerate(p.lens):
            for j in (n - 1, n - 2):
                page = int(p.table[b, j // p.page])
                p.cache.k[page, :, j % p.page] = bad
                p.cache.v[page, :, j % p.page, ::3] = bad
        p.values = [t.float().cpu().numpy().astype(np.float64) for t in (p.cache.k, p.cache.v)]
        got = p.run().float().cpu().numpy()
        with np.errstate(all="ignore"):
            want, mag = p.oracle()
        assert np.all(np.abs(got - want)[:, :4] <= A.attention_tolerance(want, mag)[:, :4])
        if bad != 3e38:
            assert not np.isfinite(got[:, 4:]).any(axis=(0, 1, 2)).all()


def test_values_that_are_not_finite_and_unseen_are_left_out():
    """Outside the window, between the first tokens and the window, inside the same pages."""
    p = Paged([400], 2, 4, 2, 128, 64, False, seed=7)
    for j in (3, 30, 250, 298):
        page = int(p.table[0, j // p.page])
        p.cache.k[page, :, j % p.page] = float("nan")
        p.cache.v[page, :, j % p.page] = float("-inf")
    p.values = [t.float().cpu().numpy().astype(np.float64) for t in (p.cache.k, p.cache.v)]
    p.check(100, 3)
    got = p.run(100, 4)                       # the fourth first token is one of them
    assert got.isnan().all()


def test_a_nan_scale_reads_as_nan():
    p = Paged([40], 1, 2, 1, 64, 16, True, seed=2)
    page = int(p.table[0, 1])
    p.cache.v_s[page, 0, 5, 1] = 255
    got = p.run()
    assert got[..., 32:].isnan().all() and got[..., :32].isfinite().all()
    p.cache.k_s[page, 0, 5, 0] = 255
    assert p.run().isnan().all()


def test_mxfp8_scales_over_their_range():
    """Blocks from 2^-120 to 2^100 in one cache; the largest decide the scores."""
    p = Paged([90], 1, 2, 1, 64, 16, True, seed=12)
    rng = np.random.default_rng(0)
    for t, x, span in ((p.cache.k, p.cache.k_s, (0, 120)), (p.cache.v, p.cache.v_s, (7, 227))):
        x.copy_(torch.from_numpy(rng.integers(*span, tuple(x.shape), dtype=np.uint8)).cuda())
        t &= 0xBF                             # finite codes, of at most 15/8
    p.values = [F.dequant_blocks(F.decode_e4m3(t.cpu().numpy()), s.cpu().numpy())
                for t, s in ((p.cache.k, p.cache.k_s), (p.cache.v, p.cache.v_s))]
    p.check()


def test_strided_queries_other_outputs_and_streams():
    p = Paged([90, 41], 3, 8, 2, 128, 16, False, seed=9)
    want = p.run()
    wide = torch.zeros(2, 3, 12, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, :, :8] = p.q
    plain, p.q = p.q, wide[:, :, :8]
    assert torch.equal(p.run(), want)
    p.q = plain
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    out = torch.empty_like(want)
    assert p.run(stream=side, out=out) is out
    side.synchronize()
    assert torch.equal(out, want)
    need = p.B.moe_paged_attention_workspace_bytes(2, 3, 8, 2, 128, 90)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    p.run(ws=ws)
    lens, graph = p.seq_lens(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.B.moe_paged_attention(p.q, p.cache, p.table, lens, 90, out=out, ws=ws)
    for n in ([90, 41], [3, 17], [0, 90]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        p.table[1, 3:] = p.table[0, 3:]       # the second sequence may be longer than it was made
        out.fill_(7)
        graph.replay()
        fresh = p.B.moe_paged_attention(p.q, p.cache, p.table, lens, 90)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), fresh.view(torch.int16))


def test_many_calls_in_turn_give_the_same_bits():
    p, small = Paged([4000, 30, 2500], 2, 8, 2, 128, 16, False, seed=1), Paged([50], 1, 8, 2, 128, 16, False, seed=2)
    want, want_small = p.run(), small.run()
    for _ in range(50):
        a, b = p.run(), small.run()
        assert torch.equal(a, want) and torch.equal(b, want_small)


def test_lengths_and_pages_out_of_range_are_reported():
    p = Paged([90, 41, 60], 1, 4, 2, 64, 16, False, seed=9)
    want = p.run()
    for bad in (-1, 91, 2 ** 31 - 1):
        got = p.B.moe_paged_attention(p.q, p.cache, p.table, torch.tensor([90, bad, 60], dtype=torch.int32,
                                                                          device="cuda"), 90)
        assert not got[1].any() and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
        with pytest.raises(p.B.MoeError) as e:
            p.B.attention_status()
        assert e.value.code == p.B.MOE_ERR_DEVICE_INPUT
    for mx in (False, True):
        p = Paged([90, 41, 60], 1, 4, 2, 64, 16, mx, seed=9)
        want = p.run()
        for bad in (-1, p.cache.pages, 2 ** 31 - 1):
            table = p.table.clone()
            table[0, 2] = bad                 # the keys 32 to 47 are left out
            got = p.B.moe_paged_attention(p.q, p.cache, table, p.seq_lens(), 90)
            with pytest.raises(p.B.MoeError):
                p.B.attention_status()
            assert torch.equal(got[1:], want[1:]) and got[0].isfinite().all() and not torch.equal(got[0], want[0])
            # a table without that page
            mine = [int(i) for i in p.table[0, :6] if int(i) != int(p.table[0, 2])]
            cut = torch.tensor([mine], dtype=torch.int32, device="cuda")
            short = p.B.moe_paged_attention(p.q[:1], p.cache, cut, torch.tensor([74], dtype=torch.int32, device="cuda"),
                                            74)
            tol = 2.0 ** -6                   # both are within the oracle's bound, of values below 4
            assert (got[0].float() - short[0].float()).abs().max() < tol
    p.B.attention_status()


# Blocks of many rows go another way than blocks of up to 16: the same checks there.
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,Hq,Hkv,page", [(17, 1, 1, 8), (6, 64, 2, 16), (64, 4, 1, 64), (5, 40, 1, 128),
                                              (3, 12, 2, 256)])
def test_many_rows(rows, Hq, Hkv, page, D, mx):
    lens = [1, rows, 17, 0, 127, 128, 129, 257, 700, 1400, 2]
    Paged(lens, rows, Hq, Hkv, D, page, mx, seed=rows * 100 + Hq).check()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 0), (64, 4), (100, 70), (128, 300), (1000, 3),
                                          (257, 129)])
def test_many_rows_windows_and_first_tokens(window, sinks, mx):
    Paged([700, 5, 64, 129, 1, 333, 1100], 5, 16, 2, 64, 16, mx, seed=window).check(window, sinks)
    Paged([1100, 2300], 4, 16, 2, 128, 64, mx, seed=window).check(window, sinks)


@pytest.mark.parametrize("mx", [False, True])
def test_many_rows_long_and_growing(mx):
    Paged([9001, 4097, 1, 2049, 12000], 6, 16, 2, 64, 32, mx, seed=4).check()
    p = Paged([900, 33, 5000], 6, 8, 1, 128, 16, mx, seed=8, q_scale=6.0, spread=0.7)
    p.check()
    p.check(scale=-0.5)
    p.check(scale=0.0)


@pytest.mark.parametrize("mx", [False, True])
def test_many_rows_do_not_depend_on_their_batch(mx):
    p = Paged([3000, 40, 777, 1025, 9000], 6, 16, 2, 64, 16, mx, seed=3)
    whole = p.run()
    for b, n in enumerate(p.lens):
        for max_len in (n, n + 1, 9000):
            one = p.B.moe_paged_attention(p.q[b:b + 1].contiguous(), p.cache, p.table[b:b + 1].contiguous(),
                                          p.seq_lens()[b:b + 1], min(max_len, 16 * p.table.shape[1]))
            assert torch.equal(one[0], whole[b])
    for _ in range(30):
        assert torch.equal(p.run(), whole)


@pytest.mark.parametrize("mx", [False, True])
def test_many_rows_values_that_are_not_finite(mx):
    """Unseen ones are left out; one that later rows see reaches those and their columns alone."""
    p = Paged([700, 300], 6, 8, 1, 128, 64, mx, seed=7)
    clean = p.run(100, 3)

    def put(b, j, key, value):
        page, at = int(p.table[b, j // 64]), j % 64
        if mx:
            if key:
                p.cache.k_s[page, :, at] = 255
            p.cache.v_s[page, :, at, value] = 255
        else:
            if key:
                p.cache.k[page, :, at] = float("nan")
            p.cache.v[page, :, at, 32 * value] = float("-inf")
    for j in (3, 30, 250, 593):                # the window of the first row begins at 595
        put(0, j, True, 0)
    assert torch.equal(p.run(100, 3), clean)
    put(1, 297, False, 2)                       # seen by the last three of six rows, at 297 to 299
    got = p.run(100, 3)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1, :3], clean[1, :3])
    hit = got[1, 3:].float()
    assert not hit[..., 64].isfinite().any()
    keep = [d for d in range(128) if not 64 <= d < 96]
    assert (hit[..., keep] - clean[1, 3:].float()[..., keep]).abs().max() < 2.0 ** -6   # both within the oracle's bound
    put(1, 296, True, 0)                        # and a key: the rows from the third on are lost
    got = p.run(100, 3)
    assert torch.equal(got[1, :2], clean[1, :2]) and got[1, 2:].isnan().all()


@pytest.mark.parametrize("mx", [False, True])
def test_many_rows_pages_out_of_range(mx):
    p = Paged([500, 41], 6, 8, 2, 64, 16, mx, seed=9)
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


@pytest.mark.parametrize("mx", [False, True])
def test_more_pieces_than_the_gpu_has_room_for(mx):
    lens = [int(n) for n in np.random.default_rng(1).integers(1, 1500, 60)] + [0, 3, 1500]
    Paged(lens, 3, 24, 4, 64, 16, mx, seed=5).check()


def test_offsets_past_32_bits():
    """Pages whose values lie more than 2^31 elements, and 2^32 bytes, into the cache."""
    from block_scaled_fp8_moe_gb300 import binding as B
    Hkv, page, D = 8, 64, 128
    for mx in (False, True):
        pages = 2 ** 31 // (Hkv * page * D) + 40
        c = B.KvCache.empty(pages, page, Hkv, D, mxfp8=mx)
        k, v = (_bf16(np.random.default_rng(i).standard_normal((100, Hkv, D))) for i in (0, 1))
        slots = torch.arange(100, dtype=torch.int32, device="cuda") + (pages - 2) * page
        B.moe_kv_append(c, k, v, slots)
        q = _bf16(np.random.default_rng(2).standard_normal((1, 1, 16, D)))
        table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda")
        got = B.moe_paged_attention(q, c, table, torch.tensor([100], dtype=torch.int32, device="cuda"), 100)
        vals = []
        for t in (k, v):
            a = t.float().cpu().numpy()
            if mx:
                cq, cs = A.quant_block_mxfp8(a)
                a = F.dequant_blocks(F.decode_e4m3(cq), cs)
            vals.append(a)
        want, mag = A.attend_heads(q[0].float().cpu().numpy(), *vals, 99, D ** -0.5)
        assert np.all(np.abs(got[0].float().cpu().numpy() - want) <= A.attention_tolerance(want, mag))
        B.attention_status()
        del c
    torch.cuda.empty_cache()


def test_refusals():
    p = Paged([90, 41], 2, 4, 2, 64, 16, False, seed=9)
    B, t, n = p.B, p.table, p.seq_lens()
    f = B.moe_paged_attention
    for call in (lambda: f(p.q.float(), p.cache, t, n, 90), lambda: f(p.q, p.cache, t.long(), n, 90),
                 lambda: f(p.q, p.cache, t[:1], n, 90), lambda: f(p.q, p.cache, t, n[:1], 90),
                 lambda: f(p.q, p.cache, t, n, 90, out=torch.empty_like(p.q[:1])),
                 lambda: f(p.q.cpu(), p.cache, t, n, 90), lambda: f(p.q.transpose(2, 3), p.cache, t, n, 90)):
        with pytest.raises(ValueError):
            call()
    small = torch.zeros(128, dtype=torch.uint8, device="cuda")
    for code, call in ((B.MOE_ERR_INVALID_ARG, lambda: f(p.q, p.cache, t, n, 16 * t.shape[1] + 1)),
                       (B.MOE_ERR_INVALID_ARG, lambda: f(p.q, p.cache, t, n, -1)),
                       (B.MOE_ERR_UNSUPPORTED_SHAPE, lambda: f(p.q[:, :, :3].contiguous(), p.cache, t, n, 90)),
                       (B.MOE_ERR_UNSUPPORTED_SHAPE, lambda: f(p.q, p.cache, t, n, 90, window=-1)),
                       (B.MOE_ERR_UNSUPPORTED_SHAPE, lambda: f(p.q, p.cache, t, n, 90, sinks=-1)),
                       (B.MOE_ERR_UNSUPPORTED_SHAPE, lambda: f(p.q, p.cache, t, n, 90, scale=float("nan"))),
                       (B.MOE_ERR_WORKSPACE, lambda: f(p.q, p.cache, t, n, 90, ws=small)),
                       (B.MOE_ERR_UNSUPPORTED_SHAPE,
                        lambda: f(torch.zeros(2, 65, 4, 64, dtype=torch.bfloat16, device="cuda"), p.cache, t, n, 90))):
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.code == code
    assert f(p.q[:0], p.cache, t[:0], n[:0], 0).shape == (0, 2, 4, 64)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,Hq", [(17, 1), (6, 4), (5, 8), (6, 8)])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_whatever_a_kernel_has_left(D, rows, Hq, mx):
    """A block's tile of 128 queries has rows that nobody owns: what an earlier kernel left there, large queries of a
    prompt here, must not reach the others, nor how their weights are rounded."""
    p = Paged([3000, 777, 1025], rows, Hq, 1, D, 16, mx, seed=rows)
    g = torch.Generator(device="cuda").manual_seed(5)
    cu = torch.tensor([0, 20000], dtype=torch.int32, device="cuda")
    kv = torch.randn((20000, 8, D), generator=g, device="cuda").bfloat16()
    want = []
    for size in (0.0, 1.0, 30.0, 1000.0):
        q = (size * torch.randn((20000, 8, D), generator=g, device="cuda")).bfloat16()
        p.B.moe_prefill_attention(q, kv, kv, cu, window=64)
        want.append([p.run(), p.run(300, 5)])
    for got in want[1:]:
        assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])


def _gives_up(p, load):
    """A call whose blocks wait for a load that does not complete: it ends, says so, and the next one is as ever."""
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


@pytest.mark.parametrize("mx,D,rows", [(False, 128, 2), (False, 64, 4), (True, 64, 2), (True, 128, 4)])
@pytest.mark.parametrize("load", [0, 3, 7])
def test_a_wait_that_runs_out_is_reported(load, mx, D, rows):
    """Pieces of 8 steps, one a block: the eighth is the last that a loading warp issues."""
    _gives_up(Paged([4096] * 4, rows, 8, 2, D, 64, mx, seed=load), load)


@pytest.mark.parametrize("mx,D", [(False, 128), (False, 64), (True, 64), (True, 128)])
@pytest.mark.parametrize("load", [0, 3, 7])
def test_many_rows_a_wait_that_runs_out_is_reported(load, mx, D):
    """Pieces of 4 steps, one a block: 8 tiles of keys and values, of which the loading warp has issued all but the held
    one's successors when the others give up."""
    _gives_up(Paged([4096] * 4, 6, 16, 2, D, 64, mx, seed=load), load)


def _put(p, b, j, col, x):
    """Value `x` (MXFP8: NaN in the column's block of 32) at key j of sequence b."""
    page, at = int(p.table[b, j // p.page]), j % p.page
    if p.cache.v_s is not None:
        p.cache.v_s[page, :, at, col // 32] = 255
    else:
        p.cache.v[page, :, at, col] = x
    p.values[1][page, :, at, slice(col // 32 * 32, col // 32 * 32 + 32) if p.cache.v_s is not None else col] = (
        np.nan if p.cache.v_s is not None else x)


def _check_not_finite(p, window=0, sinks=0):
    """Where the oracle's result is not finite, the same infinity or NaN; elsewhere as ever."""
    got = p.run(window, sinks).float().cpu().numpy()
    p.B.attention_status()
    with np.errstate(all="ignore"):
        want, mag = p.oracle(window, sinks)
        near = np.abs(got - want) <= A.attention_tolerance(want, mag)
    fine = np.isfinite(want)
    assert near[fine].all() and not fine.all()
    assert np.array_equal(np.where(fine, 0, got), np.where(fine, 0, want), equal_nan=True)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,Hq,lens", [(6, 16, [700, 300, 5000]), (60, 3, [700, 300, 5000])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20), (700, 200)])
def test_many_rows_infinities_and_nan_that_some_rows_see(window, sinks, rows, Hq, lens, D, mx):
    """In the last keys, at the windows' beginnings, among the first tokens, a whole step of them; infinities of either sign
    in one column, in steps at the mask's edge and in others."""
    inf = float("inf")
    p = Paged(lens, rows, Hq, 1, D, 16, mx, seed=rows + window)
    for b, n in enumerate(lens):
        _put(p, b, n - 1, 1, inf)
        _put(p, b, n - rows // 2, 40, -inf)
        _put(p, b, 10, 40, inf)
        _put(p, b, 19, 2, float("nan"))
        _put(p, b, max(n - rows + 3 - 150, 0), 41, inf)
        _put(p, b, max(n - rows + 3 - 700, 0), 42, inf)
    for j in range(200, 290):
        _put(p, 1, j, 50, inf)
    _check_not_finite(p, window, sinks)


@pytest.mark.parametrize("mx", [False, True])
def test_many_rows_infinities_beside_pages_out_of_range(mx):
    """A page that is not there makes its step no edge: what every row sees stays in the product."""
    p = Paged([500], 6, 8, 1, 64, 16, mx, seed=3)
    clean = p.run()
    _put(p, 0, 40, 3, float("inf"))
    table = p.table.clone()
    table[0, 3] = -1                               # keys 48 to 63
    got = p.B.moe_paged_attention(p.q, p.cache, table, p.seq_lens(), 500)
    with pytest.raises(p.B.MoeError):
        p.B.attention_status()
    cols = list(range(32)) if mx else [3]
    keep = [d for d in range(64) if d not in cols]
    assert not got[..., cols].isfinite().any() and got[..., keep].isfinite().all()
    assert not torch.equal(got[..., keep], clean[..., keep])


def test_a_captured_call_needs_its_own_workspace():
    """All captures share one stream, and with it they would share one buffer of partial results. Each with its own, two
    graphs can be replayed side by side."""
    a, b = Paged([9000, 700], 6, 8, 2, 64, 16, False, seed=1), Paged([4000, 30, 2500], 2, 8, 2, 64, 16, False, seed=2)
    B = a.B
    kv = torch.randn(3, 2, 64, device="cuda").bfloat16()
    slots, cu = torch.full((3,), -1, dtype=torch.int32, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    lens = [p.seq_lens() for p in (a, b)]
    outs = [torch.empty_like(p.q) for p in (a, b)]
    for stream in (None, torch.cuda.Stream()):
        graph, x = torch.cuda.CUDAGraph(), torch.zeros(4, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.graph(graph) if stream is None else torch.cuda.graph(graph, stream=stream):
            x += 1
            for call in (lambda s: B.moe_paged_attention(a.q, a.cache, a.table, lens[0], 9000, out=outs[0], stream=s),
                         lambda s: B.moe_kv_append(a.cache, kv, kv, slots, stream=s),
                         lambda s: B.moe_prefill_attention(kv, kv, kv, cu, out=kv, stream=s)):
                with pytest.raises(ValueError, match="workspace"):
                    call(stream)
        graph.replay()
        torch.cuda.synchronize()
        assert (x == 1).all()
    want, graphs = [a.run(), b.run()], []
    for p, n, out in zip((a, b), lens, outs):
        ws = torch.zeros(B.moe_paged_attention_workspace_bytes(*p.q.shape[:3], 2, 64, max(p.lens)), dtype=torch.uint8,
                         device="cuda")
        graphs.append((torch.cuda.CUDAGraph(), torch.cuda.Stream(), ws))
        with torch.cuda.graph(graphs[-1][0]):
            for _ in range(20):
                B.moe_paged_attention(p.q, p.cache, p.table, n, max(p.lens), out=out, ws=ws)
    for _ in range(5):
        for out in outs:
            out.fill_(7)
        torch.cuda.synchronize()
        for graph, stream, _ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    for _, _, ws in graphs:
        B.moe_check_device_status(ws)


def test_errors_found_before_a_workspace_grew_are_reported_once():
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        p = Paged([90, 41], 1, 4, 2, 64, 16, False, seed=9)
        p.B.moe_paged_attention(p.q, p.cache, p.table, torch.tensor([90, 91], dtype=torch.int32, device="cuda"), 90)
        big = Paged([9000] * 40, 4, 8, 2, 64, 64, False, seed=1)
        big.run()
        with pytest.raises(p.B.MoeError) as e:
            p.B.attention_status()
        assert e.value.code == p.B.MOE_ERR_DEVICE_INPUT
        p.B.attention_status()


@pytest.mark.parametrize("rows,Hq,Hkv", [(2, 4, 2), (3, 4, 1), (6, 16, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_of_minus_infinity(D, rows, Hq, Hkv):
    """A row whose scores are all minus infinity is 0 / 0; one finite score takes all; rows that see nothing stay zero, those
    whose pages are all out of range among them."""
    p = Paged([40, 1, 3000, 3000], rows, Hq, Hkv, D, 16, False, seed=2)
    p.q[..., 0] = 1
    p.cache.k[..., 0] = float("-inf")
    p.cache.k[int(p.table[3, 60]), :, 5, 0] = 1
    p.values[0] = p.cache.k.float().cpu().numpy().astype(np.float64)
    got = p.run().float().cpu().numpy()
    with np.errstate(all="ignore"):
        want, mag = p.oracle()
        near = np.abs(got - want) <= A.attention_tolerance(want, mag)
    assert np.isnan(want[0]).all() and np.isnan(want[2]).all() and np.isfinite(want[3]).all()
    assert (want[1, :rows - 1] == 0).all()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and near[~np.isnan(want)].all()
    none = p.B.moe_paged_attention(p.q, p.cache, torch.full_like(p.table, -1), p.seq_lens(), 3000)
    assert not none.any()
    with pytest.raises(p.B.MoeError):
        p.B.attention_status()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,Hq,Hkv,D,page", [(3, 4, 2, 64, 16), (1, 8, 1, 128, 64), (8, 1, 1, 64, 8), (5, 3, 1, 128, 32)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 0), (64, 4), (100, 70), (128, 300), (1000, 3),
                                          (257, 129)])
def test_few_rows_windows_and_first_tokens(window, sinks, rows, Hq, Hkv, D, page, mx):
    """Up to 8 rows, and up to 16."""
    Paged([700, 5, 64, 129, 1, 333, 1100], rows, Hq, Hkv, D, page, mx, seed=window).check(window, sinks)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,Hq", [(4, 2), (6, 1), (5, 3), (16, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20), (700, 200)])
def test_few_rows_infinities_and_nan_that_some_rows_see(window, sinks, rows, Hq, D, mx):
    """Keys that some rows see and others do not, with values that are not finite: added one by one."""
    inf = float("inf")
    lens = [700, 300, 5000]
    p = Paged(lens, rows, Hq, 1, D, 16, mx, seed=rows + window)
    for b, n in enumerate(lens):
        _put(p, b, n - 1, 1, inf)
        _put(p, b, n - 2, 40, -inf)
        _put(p, b, 10, 40, inf)
        _put(p, b, 19, 2, float("nan"))
        _put(p, b, max(n - rows + 2 - 150, 0), 41, inf)
        _put(p, b, max(n - rows + 2 - 700, 0), 42, inf)
    for j in range(200, 290):
        _put(p, 1, j, 50, inf)
    _check_not_finite(p, window, sinks)


@pytest.mark.parametrize("rows,Hq", [(1, 2), (2, 4), (3, 5), (6, 4), (6, 8)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_mxfp8_scales_over_their_range_for_every_kernel(window, sinks, D, rows, Hq):
    """Values of up to 2^110 in some blocks, whose scales one factor of the conversion does not hold, beside small ones."""
    p = Paged([300, 90, 1500], rows, Hq, 1, D, 16, True, seed=12, q_scale=2.0 ** -5)
    rng = np.random.default_rng(rows)
    for t, x, low, high in ((p.cache.k, p.cache.k_s, 0, 124), (p.cache.v, p.cache.v_s, 7, 237)):
        s = rng.integers(low, high, tuple(x.shape), dtype=np.uint8)
        x.copy_(torch.from_numpy(s).cuda())
        t &= 0xBF                             # finite codes, of at most 15/8
    p.values = [F.dequant_blocks(F.decode_e4m3(t.cpu().numpy()), s.cpu().numpy())
                for t, s in ((p.cache.k, p.cache.k_s), (p.cache.v, p.cache.v_s))]
    p.check(window, sinks)
    # a few keys' scores far above the others', by a scale of more than 134
    for b, j in ((0, 7), (0, 250), (2, 1200), (2, 1499)):
        page, at = int(p.table[b, j // 16]), j % 16
        p.cache.k[page, :, at] = 0x38         # ones
        p.cache.k_s[page, :, at] = 137
        p.cache.v_s[page, :, at] = 230
    p.values = [F.dequant_blocks(F.decode_e4m3(t.cpu().numpy()), s.cpu().numpy())
                for t, s in ((p.cache.k, p.cache.k_s), (p.cache.v, p.cache.v_s))]
    p.check(window, sinks)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,Hq,Hkv,D", [(2, 4, 2, 64), (8, 1, 1, 128), (4, 4, 1, 128), (3, 4, 1, 64), (6, 16, 2, 64), (60, 3, 1, 128)])
def test_rows_that_see_nothing_are_plus_zero(rows, Hq, Hkv, D, mx):
    """Bit for bit, beside values below zero: before their sequence begins, in a batch of one piece and of many, over pages
    out of range, and for a length out of range."""
    for longest in (70, 9000):
        p = Paged([1, rows - 1, 0, longest], rows, Hq, Hkv, D, 16, mx, seed=2)
        if mx:
            p.cache.v |= 0x80
        else:
            p.cache.v.copy_(-p.cache.v.abs())
        got = p.run().view(torch.int16)
        assert not got[0, :rows - 1].any() and not got[1, :1].any() and not got[2].any() and got[3].any()
        p.B.attention_status()
        none = p.B.moe_paged_attention(p.q, p.cache, torch.full_like(p.table, -1), p.seq_lens(), longest).view(torch.int16)
        assert not none.any()
        with pytest.raises(p.B.MoeError):
            p.B.attention_status()
        lens = torch.tensor([1, -5, 0, longest + 1], dtype=torch.int32, device="cuda")
        got = p.B.moe_paged_attention(p.q, p.cache, p.table, lens, longest).view(torch.int16)
        assert not got[1:].any()
        with pytest.raises(p.B.MoeError):
            p.B.attention_status()
