"""GPU parity: attention of packed prompts, against the float64 oracle. The tolerance is the oracle's own
(oracle.attention.attention_tolerance)."""
import numpy as np
import pytest
import torch

from oracle import attention as A

pytestmark = pytest.mark.gpu


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


class Prompts:
    def __init__(self, q_lens, Hq, Hkv, D, k_lens=None, seed=0, gap=0, q_scale=1.0, spread=0.0):
        from block_scaled_fp8_moe_gb300 import binding as B
        rng = np.random.default_rng(seed)
        self.B, self.q_lens, self.k_lens = B, q_lens, q_lens if k_lens is None else k_lens
        Tq, Tk = sum(q_lens), sum(self.k_lens)
        self.q = _bf16(rng.standard_normal((Tq, Hq + gap, D)) * q_scale)[:, :Hq]
        kv = _bf16(rng.standard_normal((Tk, 2 * Hkv + gap, D)) * np.exp(spread * rng.standard_normal((Tk, 1, 1))))
        self.k, self.v = kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
        self.cu_q, self.cu_k = _cu(q_lens), None if k_lens is None else _cu(k_lens)

    def run(self, window=0, sinks=0, **kw):
        return self.B.moe_prefill_attention(self.q, self.k, self.v, self.cu_q, self.cu_k, window=window, sinks=sinks,
                                            **kw)

    def oracle(self, window=0, sinks=0, scale=None):
        q, k, v = _np(self.q), _np(self.k), _np(self.v)
        out, mag = np.zeros(q.shape), np.zeros(q.shape)
        a = b = 0
        for n, m in zip(self.q_lens, self.k_lens):
            out[a:a + n], mag[a:a + n] = A.attend_heads(q[a:a + n], k[b:b + m], v[b:b + m], m - n,
                                                        q.shape[-1] ** -0.5 if scale is None else scale, window, sinks)
            a, b = a + n, b + m
        return out, mag

    def check(self, window=0, sinks=0, **kw):
        got = _np(self.run(window, sinks, **kw))
        want, mag = self.oracle(window, sinks, kw.get("scale"))
        bad = np.abs(got - want) > A.attention_tolerance(want, mag)
        assert not bad.any() and np.isfinite(got).all(), (int(bad.sum()), float(np.nanmax(np.abs(got - want))))
        self.B.attention_status()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (3, 1), (5, 5), (8, 1)])
def test_ragged_prompts_and_heads(Hq, Hkv, D):
    Prompts([1, 0, 130, 7, 128, 63, 0, 257, 2], Hq, Hkv, D, seed=Hq).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (3, 4), (64, 0), (100, 5), (128, 128), (129, 200), (300, 1),
                                          (200, 257), (5000, 7)])
def test_windows_and_first_tokens(window, sinks, D):
    Prompts([700, 5, 129, 1, 333], 4, 2, D, seed=window).check(window, sinks)


@pytest.mark.parametrize("n", [1, 2, 16, 127, 128, 129, 255, 256, 257, 383, 511, 640, 1025])
def test_one_prompt_of_every_tile_end(n):
    Prompts([n], 2, 1, 128, seed=n).check()


@pytest.mark.parametrize("D", [64, 128])
def test_a_prompt_that_continues(D):
    """More keys than query rows: the rows are the last ones; and fewer, where the first rows see nothing."""
    Prompts([5, 130, 1, 200, 40, 129, 3], 4, 2, D, k_lens=[300, 131, 700, 200, 0, 100, 1], seed=2).check()
    Prompts([5, 130, 1, 200, 40, 129, 3], 3, 1, D, k_lens=[300, 131, 700, 200, 0, 100, 1], seed=3).check(150, 20)


def test_growing_scores_and_other_scales():
    p = Prompts([600, 300], 4, 2, 128, seed=8, q_scale=6.0, spread=0.7)
    p.check()
    p.check(scale=-0.5)
    p.check(scale=0.0)
    p = Prompts([700], 2, 1, 128, seed=9)
    p.k *= torch.linspace(0.1, 20, 700, device="cuda").bfloat16().view(-1, 1, 1)     # later keys score far higher
    p.check()


def test_rows_of_a_wider_projection():
    Prompts([40, 300], 4, 2, 64, seed=4, gap=3).check(50, 3)
    Prompts([40, 300], 4, 2, 128, seed=4, gap=1).check()


def test_a_prompt_does_not_depend_on_its_batch():
    for Hq, Hkv in ((4, 2), (3, 1)):
        p = Prompts([200, 131, 1, 500], Hq, Hkv, 128, seed=5)
        whole = p.run(150, 9)
        a = 0
        for n in p.q_lens:
            one = p.B.moe_prefill_attention(p.q[a:a + n], p.k[a:a + n], p.v[a:a + n], _cu([n]), window=150, sinks=9)
            assert torch.equal(one, whole[a:a + n])
            a += n


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_a_row_does_not_see_does_not_reach_it(bad):
    """A later token of the same prompt, another prompt's tokens, and one between the first tokens and the window."""
    p = Prompts([300, 200], 4, 2, 64, seed=6)
    clean = _np(p.run(100, 3))
    p.k[250], p.v[250, :, ::3] = bad, bad
    p.k[330], p.v[330, :, 5] = bad, bad
    got = _np(p.run(100, 3))
    # prompt 0: the rows from 250 on see it; prompt 1: its token 30 is seen by its rows 30 to 129
    hit = np.zeros(500, dtype=bool)
    hit[250:300] = True
    hit[330:430] = True
    assert np.array_equal(got[~hit], clean[~hit])
    want, mag = p.oracle(100, 3)
    assert np.array_equal(got[~hit], clean[~hit]) and not np.isfinite(got[hit]).all(axis=(1, 2)).any()


def test_a_value_that_is_not_finite_reaches_its_column_alone():
    p = Prompts([300], 2, 1, 64, seed=6)
    p.v[10, 0, 7] = float("inf")
    got = _np(p.run())
    want, mag = p.oracle()
    keep = [d for d in range(64) if d != 7]
    assert np.all(np.abs(got - want)[:, :, keep] <= A.attention_tolerance(want, mag)[:, :, keep])
    assert np.isposinf(got[10:, :, 7]).all() and np.isfinite(got[:10]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(32, 4), (20, 4)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 1), (100, 5), (129, 200)])
def test_blocks_of_two_tiles(window, sinks, Hq, Hkv, D):
    """Enough tiles for blocks to take two at a time: two heads of a group, or 256 rows where a group's heads are odd."""
    p = Prompts([1, 0, 130, 7, 128, 63, 0, 257, 2], Hq, Hkv, D, seed=Hq)
    p.check(window, sinks)
    p.v[400, :, 5] = float("inf")                 # prompt 7's key 71
    got, (want, mag) = _np(p.run(window, sinks)), p.oracle(window, sinks)
    rows = np.isfinite(want[:, 0, 5])
    assert not rows.all() and np.array_equal(np.isfinite(got[:, :, 5]), np.isfinite(want[:, :, 5]))
    keep = [d for d in range(D) if d != 5]
    with np.errstate(invalid="ignore"):
        assert np.all(np.abs(got - want)[:, :, keep] <= A.attention_tolerance(want, mag)[:, :, keep])


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 64, 8), (128, 32, 4), (128, 33, 11)])
def test_more_work_than_the_gpu_has_room_for(D, Hq, Hkv):
    """Several times as many blocks of rows as multiprocessors, with values that are not finite here and there: sampled
    rows against the oracle, and call after call the same bits."""
    lens = [1500, 3, 2300, 700, 1]
    p = Prompts(lens, Hq, Hkv, D, seed=11)
    bad = {2: 1000, 0: 1490}                       # sequence: a key whose value is not finite
    begin = np.concatenate([[0], np.cumsum(lens)])
    for b, j in bad.items():
        p.v[int(begin[b]) + j, :, 3] = float("nan")
    for window, sinks in ((0, 0), (300, 5)):
        first = p.run(window, sinks)
        p.B.attention_status()
        for _ in range(5):
            assert torch.equal(p.run(window, sinks).view(torch.int16), first.view(torch.int16))
        q, k, v, got = _np(p.q), _np(p.k), _np(p.v), _np(first)
        for b, n in enumerate(lens):
            rows = slice(int(begin[b]), int(begin[b]) + n)
            for r in sorted({0, n // 3, n // 2, n - 1, min(n - 1, 1001), min(n - 1, 1489)}):
                with np.errstate(all="ignore"):
                    want, mag = A.attend_heads(q[rows][r:r + 1], k[rows], v[rows], r, D ** -0.5, window, sinks)
                mine = got[rows][r:r + 1]
                cols = [d for d in range(D) if d != 3]
                assert np.all(np.abs(mine - want)[..., cols] <= A.attention_tolerance(want, mag)[..., cols])
                assert np.array_equal(np.isnan(mine[..., 3]), np.isnan(want[..., 3]))


def test_other_outputs_streams_and_graphs():
    p = Prompts([129, 300], 4, 2, 128, seed=9)
    want = p.run(64, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    out = torch.empty_like(want)
    assert p.run(64, 4, stream=side, out=out) is out
    side.synchronize()
    assert torch.equal(out, want)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(64, 4, out=out, ws=ws)
    for lens in ([129, 300], [1, 428], [0, 200]):
        p.cu_q.copy_(_cu(lens))
        out.fill_(7)
        fresh = torch.full_like(out, 7)
        graph.replay()
        p.run(64, 4, out=fresh)
        torch.cuda.synchronize()
        assert torch.equal(out, fresh) and (out[sum(lens):] == 7).all()


def test_bounds_that_break_the_rule_are_left_out_and_reported():
    p = Prompts([100, 60, 90], 2, 1, 64, seed=1)
    want = p.run()
    for cu, left in (([0, 100, 90, 250], [(0, 90)]), ([0, 100, 160, 251], [(0, 100), (100, 160)]),
                     ([0, 100, 2 ** 31 - 1, 250], [(0, 100)]), ([0, -5, 160, 250], [(160, 250)])):
        p.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
        got = p.run(out=torch.full_like(want, 7))
        with pytest.raises(p.B.MoeError) as e:
            p.B.attention_status()
        assert e.value.code == p.B.MOE_ERR_DEVICE_INPUT
        for a, b in left:
            assert torch.equal(got[a:b], want[a:b])
    p.B.attention_status()


def test_refusals():
    p = Prompts([100, 60], 4, 2, 64, seed=1)
    B, f = p.B, p.B.moe_prefill_attention
    for call in (lambda: f(p.q.float(), p.k, p.v, p.cu_q), lambda: f(p.q, p.k[:50], p.v, p.cu_q),
                 lambda: f(p.q, p.k[:50], p.v[:50], p.cu_q), lambda: f(p.q, p.k, p.v, p.cu_q.long()),
                 lambda: f(p.q, p.k, p.v, p.cu_q, p.cu_q[:2]), lambda: f(p.q.cpu(), p.k, p.v, p.cu_q),
                 lambda: f(p.q, p.k, p.v, p.cu_q, out=torch.empty_like(p.q[:1])),
                 lambda: f(p.q.transpose(0, 1).contiguous().transpose(0, 1), p.k, p.v, p.cu_q)):
        with pytest.raises(ValueError):
            call()
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for call in (lambda: f(z(160, 3, 64), p.k, p.v, p.cu_q), lambda: f(z(160, 4, 96), z(160, 2, 96), z(160, 2, 96), p.cu_q),
                 lambda: f(p.q, p.k, p.v, p.cu_q, window=-1), lambda: f(p.q, p.k, p.v, p.cu_q, sinks=-3),
                 lambda: f(p.q, p.k, p.v, p.cu_q, scale=float("inf"))):
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.code == B.MOE_ERR_UNSUPPORTED_SHAPE
    with pytest.raises(B.MoeError):
        f(p.q, p.k, p.v, p.cu_q, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert f(p.q[:0], p.k[:0], p.v[:0], _cu([])).shape == (0, 4, 64)


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 128), (32, 4, 64), (20, 4, 128)])
@pytest.mark.parametrize("load", [0, 3, 10])
def test_a_wait_that_runs_out_is_reported(load, Hq, Hkv, D):
    """Blocks of one tile, of two heads and of 256 rows wait for a load that does not complete: the call ends, says so,
    and the next one is as ever."""
    p = Prompts([1100, 700], Hq, Hkv, D, seed=load)
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


def _inf_in_a_long_prompt(n, D, window, sinks, bad, clean):
    """A prompt of n tokens with values that are not finite at keys `bad` (column 3) and a short one beside it: sampled rows
    of either against the oracle, in a time far below the limit of the kernel's waits."""
    p = Prompts([n, clean], 2, 1, D, seed=n % 97)
    p.v[torch.tensor(bad, device="cuda"), 0, 3] = float("inf")
    p.run(window, sinks)
    times = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    times[0].record()
    got = _np(p.run(window, sinks))
    times[1].record()
    torch.cuda.synchronize()
    p.B.attention_status()
    assert times[0].elapsed_time(times[1]) < 400
    q, k, v = _np(p.q), _np(p.k), _np(p.v)
    cols = [d for d in range(D) if d != 3]
    for a, b, rows in ((0, n, sorted({bad[0] - 1, bad[0], bad[-1], bad[-1] + 1, n - 130, n - 2, n - 1} - {-1, n})),
                       (n, n + clean, range(0, clean, 7))):
        for r in rows:
            with np.errstate(all="ignore"):
                want, mag = A.attend_heads(q[a + r:a + r + 1], k[a:b], v[a:b], r, D ** -0.5, window, sinks)
            mine = got[a + r:a + r + 1]
            assert np.all(np.abs(mine - want)[..., cols] <= A.attention_tolerance(want, mag)[..., cols]), r
            if a:
                assert np.isfinite(mine).all()
            else:
                assert np.array_equal(np.isfinite(mine[..., 3]), np.isfinite(want[..., 3])), r


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20001, 5)])
@pytest.mark.parametrize("at", [100, -3, -140])
def test_one_infinite_value_in_a_long_prompt(at, window, sinks, D):
    n = 100_037                                  # its last tile is a partial one
    _inf_in_a_long_prompt(n, D, window, sinks, [at % n], 40)


def test_a_whole_edge_of_infinite_values_in_a_long_prompt():
    _inf_in_a_long_prompt(100_037, 128, 0, 0, list(range(99_700, 100_000)), 40)


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (20, 4), (32, 4)])
def test_infinities_of_either_sign_and_nan_together(Hq, Hkv):
    """Columns with one infinity, both, NaN and an infinity; keys in several steps of an item, first tokens and window
    ends among them; more of them than 64 at once."""
    lens, inf, nan = [700, 300], float("inf"), float("nan")
    for window, sinks in ((0, 0), (150, 20)):
        p = Prompts(lens, Hq, Hkv, 64, seed=3)
        for j, col, x in ((5, 1, inf), (6, 2, -inf), (130, 2, inf), (131, 3, nan), (132, 3, inf), (400, 4, -inf), (699, 5, inf)):
            p.v[j, :, col] = x
        p.v[700 + 100:700 + 200, :, 7] = inf
        p.v[700 + 150, :, 7] = -inf
        got = _np(p.run(window, sinks))
        with np.errstate(all="ignore"):
            want, mag = p.oracle(window, sinks)
        fine = np.isfinite(want)
        assert not fine.all() and np.array_equal(np.where(fine, 0, got), np.where(fine, 0, want), equal_nan=True)
        with np.errstate(all="ignore"):
            assert np.all((np.abs(got - want) <= A.attention_tolerance(want, mag))[fine])


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 32, 4), (128, 20, 4)])
def test_a_last_tile_does_not_depend_on_what_follows_it(D, Hq, Hkv):
    """A partial tile's rows beyond its prompt are the next prompt's: they have no part in it, however large they are."""
    p = Prompts([300, 1, 140, 700], Hq, Hkv, D, seed=4)
    want = p.run()
    p.q[441:] *= 100
    p.q[300] *= 1000
    got = p.run()
    assert torch.equal(got[:300], want[:300]) and torch.equal(got[301:441], want[301:441])


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (3, 3)])
def test_thousands_of_short_prompts(Hq, Hkv):
    """Most of them empty, bounds that break the rule among them: every block passes the bounds once."""
    rng = np.random.default_rng(3)
    lens = np.where(rng.random(5000) < 0.3, rng.integers(1, 6, 5000), 0)
    lens[[0, 31, 32, 4999]] = [300, 0, 1, 140]
    p = Prompts(lens.tolist(), Hq, Hkv, 64, seed=1)
    p.check()
    p.check(3, 1)
    want = p.run()
    cu = p.cu_q.clone()
    b = int(np.flatnonzero(lens)[500])
    p.cu_q[b + 1] += 10 ** 6                       # sequence b ends past the rows, and the next begins there
    got = p.run(out=torch.full_like(want, 7))
    with pytest.raises(p.B.MoeError):
        p.B.attention_status()
    a, z = int(cu[b]), int(cu[b + 2])
    assert torch.equal(got[:a], want[:a]) and torch.equal(got[z:], want[z:]) and (got[a:z] == 7).all()


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (128, 40, 4), (64, 64, 8)])
def test_scores_of_minus_infinity(D, Hq, Hkv):
    """A row whose scores are all minus infinity is 0 / 0; one finite score takes all; rows without keys stay zero."""
    p = Prompts([200, 5, 30], Hq, Hkv, D, k_lens=[200, 2, 30], seed=2)
    p.q[..., 0] = 1
    p.k[..., 0] = float("-inf")
    p.k[100, :, 0] = 1
    got = _np(p.run())
    with np.errstate(all="ignore"):
        want, mag = p.oracle()
        near = np.abs(got - want) <= A.attention_tolerance(want, mag)
    assert np.isnan(want[:100]).all() and (want[200:203] == 0).all() and np.isfinite(want[100:200]).all()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and near[~np.isnan(want)].all()


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (128, 40, 4), (64, 64, 8), (128, 33, 11)])
def test_rows_that_see_nothing_are_plus_zero(D, Hq, Hkv):
    """Bit for bit, beside values below zero: rows before their first key, in prompts with fewer keys than rows or none."""
    p = Prompts([300, 5, 30], Hq, Hkv, D, k_lens=[40, 0, 30], seed=2)
    p.v.copy_(-p.v.abs())
    got = p.run().view(torch.int16)
    assert not got[:260].any() and not got[300:305].any() and got[260:300].any() and got[305:].any()
