"""GPU parity where one key counts: long sequences with a key whose weight is about a half, at the first and last places of
steps, pages and pieces and at both sides of every end of the mask. A key that is lost, or counted twice, moves such a result by
a sixth of its value's size, where among thousands of random keys it would hide in the tolerance."""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import formats as F

pytestmark = pytest.mark.gpu


def _plain(q, k, v, first_pos, window, sinks):
    """The definition in 64 bits on the GPU: q [R, Hq, D] at positions first_pos ..., k and v [n, Hkv, D]. (out, mag)."""
    q, k, v = (t.double() for t in (q, k, v))
    group = q.shape[1] // k.shape[1]
    pos = torch.arange(first_pos, first_pos + q.shape[0], device="cuda").view(-1, 1)
    j = torch.arange(k.shape[0], device="cuda")
    see = j <= pos
    if window:
        see &= (pos - j < window) | (j < sinks)
    s = torch.einsum("rhd,jhd->hrj", q, k.repeat_interleave(group, 1)) * q.shape[-1] ** -0.5
    w = torch.softmax(s.masked_fill(~see, float("-inf")), -1)
    v = v.repeat_interleave(group, 1)
    return torch.einsum("hrj,jhd->rhd", w, v), torch.einsum("hrj,jhd->rhd", w, v.abs())


def _near(got, want, mag, what):
    bad = np.abs(got.double().cpu().numpy() - want.cpu().numpy()) > A.attention_tolerance(want.cpu().numpy(), mag.cpu().numpy())
    assert not bad.any(), what


def _needle(D, seen):
    """A query and a key with the score log(seen)."""
    u = torch.randn(D, generator=torch.Generator().manual_seed(D)).sign()
    return u, u * float(np.log(max(seen, 2)) * D ** -0.5)


def _places(n, rows, step, page, window, sinks, rng):
    places = set(range(0, n, step)) | set(range(step - 1, n, step)) | {n - 1 - r for r in range(rows + 1)}
    places |= {int(j) + e for j in rng.integers(1, n // page, 30) * page for e in (-1, 0)}
    if window:
        places |= {n - rows + r - window + e for r in range(rows) for e in (0, 1)} | {sinks - 1, sinks, sinks + 1}
    return sorted(j for j in places if 0 <= j < n)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,Hq,D,page,n", [(2, 4, 64, 16, 9001), (1, 8, 128, 64, 8190), (4, 4, 64, 64, 5000),
                                              (6, 8, 64, 16, 8321), (3, 8, 128, 128, 8100), (60, 3, 64, 64, 4500)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (4100, 33), (1024, 130)])
def test_one_key_in_a_paged_sequence(window, sinks, rows, Hq, D, page, n, mx):
    from block_scaled_fp8_moe_gb300 import binding as B
    rng = np.random.default_rng(n)
    places = _places(n, rows, 64 if rows * Hq <= 16 else 128, page, window, sinks, rng)
    used = -(-n // page)
    # all sequences share their pages but for the one with the key
    k = 0.3 * rng.standard_normal((used + len(places), 1, page, D))
    v = rng.standard_normal((used + len(places), 1, page, D))
    table = np.tile(rng.permutation(used).astype(np.int32), (len(places), 1))
    u, needle = _needle(D, min(n, window + sinks) if window else n)
    for b, j in enumerate(places):
        k[used + b], v[used + b] = k[table[b, j // page]], v[table[b, j // page]]
        k[used + b, 0, j % page], v[used + b, 0, j % page] = needle, 100
        table[b, j // page] = used + b
    k, v = (torch.from_numpy(t).float().bfloat16() for t in (k, v))
    if mx:
        parts = [A.quant_block_mxfp8(t.float().numpy()) for t in (k, v)]
        cache = B.KvCache(*(torch.from_numpy(p[0]).cuda() for p in parts), *(torch.from_numpy(p[1]).cuda() for p in parts))
        k, v = (torch.from_numpy(F.dequant_blocks(F.decode_e4m3(p[0]), p[1])).cuda() for p in parts)
    else:
        k, v = k.cuda(), v.cuda()
        cache = B.KvCache(k, v)
    table = torch.from_numpy(table).cuda()
    q = u.bfloat16().cuda().expand(len(places), rows, Hq, D).contiguous()
    lens = torch.full((len(places),), n, dtype=torch.int32, device="cuda")
    got = B.moe_paged_attention(q, cache, table, lens, n, window=window, sinks=sinks)
    B.attention_status()
    for b, j in enumerate(places):
        mine = table[b].long()
        kb, vb = (t[mine].transpose(1, 2).flatten(0, 1)[:n] for t in (k, v))
        _near(got[b], *_plain(q[b], kb, vb, n - rows, window, sinks), j)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (128, 1, 1), (64, 3, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 33), (300, 130)])
def test_one_key_in_a_prompt(window, sinks, D, Hq, Hkv):
    """Prompts of one length side by side, each with its key, at the ends of steps and first tokens: its rows just before and
    behind the key, at the window's end and at the prompt's."""
    from block_scaled_fp8_moe_gb300 import binding as B
    n = 1700
    rng = np.random.default_rng(n)
    places = sorted(set(range(0, n, 128)) | set(range(127, n, 128)) | {n - 1, sinks, max(sinks - 1, 0)})
    k = 0.3 * rng.standard_normal((len(places), n, Hkv, D))
    v = rng.standard_normal((len(places), n, Hkv, D))
    u, needle = _needle(D, min(n, window + sinks) if window else n // 2)
    for b, j in enumerate(places):
        k[b, j], v[b, j] = needle, 100
    k, v = (torch.from_numpy(t).float().bfloat16().cuda() for t in (k, v))
    q = u.bfloat16().cuda().expand(len(places) * n, Hq, D).contiguous()
    cu = torch.arange(len(places) + 1, dtype=torch.int32, device="cuda") * n
    got = B.moe_prefill_attention(q, k.flatten(0, 1), v.flatten(0, 1), cu, window=window, sinks=sinks).view(-1, n, Hq, D)
    B.attention_status()
    for b, j in enumerate(places):
        want, mag = _plain(q[:n], k[b], v[b], 0, window, sinks)
        rows = torch.tensor(sorted({r for r in (j - 1, j, j + 1, j + window - 1, j + window, j + window + 1, n - 1, n // 2)
                                    if 0 <= r < n}), device="cuda")
        _near(got[b, rows], want[rows], mag[rows], j)
