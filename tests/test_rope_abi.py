"""CPU-only checks of the rotary entry points and the 4-bit cache: what the host refuses before anything is launched, and the
frequencies' form, which the host works out."""
import ctypes
import math
import os
from fractions import Fraction

import numpy as np
import pytest

from oracle import attention as A
from oracle import formats as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    if not os.path.exists(os.path.join(ROOT, "block_scaled_fp8_moe_gb300", "libmoe.so")):
        from block_scaled_fp8_moe_gb300 import build
        build.build()
    from block_scaled_fp8_moe_gb300 import binding
    return binding


N = ctypes.c_void_p(0)
AT = ctypes.c_void_p(0x10000)       # an aligned address that is never followed: every call here is refused


def _rotary(lib, **kw):
    a = dict(dim=64, axes=1, interleaved=0, inverse=0, factor=1.0, turns=0x10000, axis=0)
    a.update(kw)
    return ctypes.byref(lib.MoeRotary(*a.values()))


def _cache(lib, **kw):
    a = dict(pages=8, page_size=16, Hkv=2, D=128, format=4, k=0x10000, v=0x10000, k_s=0x10000, v_s=0x10000)
    a.update(kw)
    return ctypes.byref(lib.MoeKvCache(*a.values()))


def test_turns_are_the_frequencies_as_fractions_of_a_turn(B):
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257")
    freq = np.array([1.0, 10000.0 ** -0.3, -0.25, 0.0, 1e-12, 1e6, -1e6, 123.456, 2 * math.pi, math.pi / 2, 1e-300])
    turns = np.zeros(len(freq), dtype=np.uint64)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    assert B.lib.moe_rotary_turns(len(freq), p(freq), p(turns)) == B.MOE_OK
    for w, t in zip(freq, turns):
        off = (Fraction(int(t)) - Fraction(float(w)) / two_pi * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, w
    assert B.lib.moe_rotary_turns(0, N, N) == B.MOE_OK
    assert B.lib.moe_rotary_turns(-1, p(freq), p(turns)) == B.MOE_ERR_INVALID_ARG
    assert B.lib.moe_rotary_turns(2, N, p(turns)) == B.MOE_ERR_INVALID_ARG
    for bad in (float("nan"), float("inf"), 1.5e6):
        assert B.lib.moe_rotary_turns(1, p(np.array([bad])), p(turns)) == B.MOE_ERR_INVALID_ARG


def test_rope_refusals(B):
    def call(r=None, T=4, Hq=4, Hkv=2, D=64, q=AT, qs=256, k=AT, ks=128, pos=AT, ps=4, qo=AT, qos=256, ko=AT, kos=128):
        return B.lib.moe_rope(_rotary(B) if r is None else r, T, Hq, Hkv, D, q, qs, k, ks, pos, ps, qo, qos, ko, kos, N)
    for kw in (dict(dim=0), dict(dim=4), dict(dim=72), dict(dim=63), dict(axes=0), dict(axes=5), dict(factor=float("nan")),
               dict(dim=-8)):
        assert call(_rotary(B, **kw)) == B.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(D=68), dict(D=264), dict(Hq=65536), dict(Hkv=65536), dict(T=2 ** 30 + 1, ps=2 ** 31)):
        assert call(**kw) == B.MOE_ERR_UNSUPPORTED_SHAPE, kw
    assert call(_rotary(B, dim=56), D=136) == B.MOE_ERR_UNSUPPORTED_SHAPE       # 4 values a lane: at most 128
    odd = ctypes.c_void_p(0x10008)
    for kw in (dict(T=-1), dict(Hq=-1), dict(Hkv=-1), dict(D=0), dict(q=N), dict(k=N), dict(pos=N), dict(qo=N), dict(ko=N),
               dict(q=odd), dict(k=odd), dict(qo=odd), dict(ko=odd), dict(pos=ctypes.c_void_p(0x10002)), dict(qs=248), dict(qs=260),
               dict(ks=120), dict(qos=255), dict(kos=100), dict(ps=3)):
        assert call(**kw) == B.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(turns=0), dict(turns=0x10004)):
        assert call(_rotary(B, **kw)) == B.MOE_ERR_INVALID_ARG, kw
    assert B.lib.moe_rope(None, *([0] * 4), N, 0, N, 0, N, 0, N, 0, N, 0, N) == B.MOE_ERR_INVALID_ARG
    assert call(T=0, q=N, pos=N) == B.MOE_OK and call(Hq=0, Hkv=0, q=N, k=N) == B.MOE_OK


def test_rope_append_refusals(B):
    def call(r=None, c=None, T=4, Hq=4, q=AT, qs=512, k=AT, ks=256, v=AT, vs=256, pos=AT, ps=4, slots=AT, qo=AT, qos=512, ko=N,
             kos=0, ws=AT, n=256):
        return B.lib.moe_rope_kv_append(_rotary(B) if r is None else r, _cache(B) if c is None else c, T, Hq, q, qs, k, ks, v, vs,
                                        pos, ps, slots, qo, qos, ko, kos, ws, n, N)
    for kw in (dict(page_size=12), dict(D=96), dict(pages=0), dict(Hkv=0), dict(format=2), dict(format=3), dict(pages=2 ** 30)):
        assert call(c=_cache(B, **kw)) == B.MOE_ERR_UNSUPPORTED_SHAPE, kw
    assert call(_rotary(B, dim=136)) == B.MOE_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(k=0), dict(v=0x10040), dict(k_s=0), dict(v_s=0x10010)):
        assert call(c=_cache(B, **kw)) == B.MOE_ERR_INVALID_ARG, kw
    odd = ctypes.c_void_p(0x10008)
    for kw in (dict(T=-1), dict(Hq=-1), dict(q=N), dict(k=N), dict(v=N), dict(slots=N), dict(pos=N), dict(qo=N), dict(v=odd),
               dict(ko=odd, kos=256), dict(ko=AT, kos=255), dict(vs=250), dict(vs=252), dict(ps=3),
               dict(slots=ctypes.c_void_p(0x10001))):
        assert call(**kw) == B.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(ws=N), dict(n=255), dict(ws=ctypes.c_void_p(0x10080))):
        assert call(**kw) == B.MOE_ERR_WORKSPACE, kw
    assert call(T=0, q=N, k=N, v=N, slots=N, pos=N) == B.MOE_OK


def test_a_4_bit_cache_is_checked_like_the_others(B):
    f = B.lib.moe_kv_append
    assert f(_cache(B, k_s=0), 4, AT, 256, AT, 256, AT, AT, 256, N) == B.MOE_ERR_INVALID_ARG
    assert f(_cache(B, format=3), 4, AT, 256, AT, 256, AT, AT, 256, N) == B.MOE_ERR_UNSUPPORTED_SHAPE
    a = ctypes.byref(B.MoeAttention(2, 4, 2, 128, 0, 0, 1.0))
    need = B.moe_paged_attention_workspace_bytes(2, 3, 4, 2, 128, 100)
    g = lambda c: B.lib.moe_paged_attention(a, c, 3, 100, AT, 512, AT, 8, AT, AT, AT, need, N)  # noqa: E731
    assert g(_cache(B, v_s=0)) == B.MOE_ERR_INVALID_ARG and g(_cache(B, D=64)) == B.MOE_ERR_INVALID_ARG
    assert g(_cache(B, page_size=4)) == B.MOE_ERR_UNSUPPORTED_SHAPE


def test_the_oracles_4_bit_rule():
    x = np.zeros((2, 64), dtype=np.float32)
    x[0, :8] = [.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6]
    x[0, 32:] = -6.5
    x[1, 3] = np.inf
    q, s = A.quant_block_mxfp4(x)
    assert q.shape == (2, 32) and s.tolist() == [[127, 128], [255, 0]] and not q[1].any()
    v = F.dequant_blocks(F.decode_e2m1(F.unpack_e2m1(q)), s)
    assert v[0, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, 6] and (v[0, 32:] == -6).all() and np.isnan(v[1, :32]).all()


def test_the_oracles_turn():
    x = np.arange(8, dtype=np.float64).reshape(1, 1, 8)
    out, _ = A.rope(x, [[1], [3]], [np.pi / 2, np.pi], axis=[0, 1], interleaved=True)
    assert np.allclose(out[0, 0], [-1, 0, -2, -3, 4, 5, 6, 7], atol=1e-12)
    out, mag = A.rope(x, [[1]], [np.pi / 2, 0.0], factor=2.0)
    assert np.allclose(out[0, 0], [-4, 2, 0, 6, 4, 5, 6, 7]) and mag[0, 0, 0] == 4
    back, _ = A.rope(A.rope(x, [[5]], [0.3, 0.7])[0], [[5]], [0.3, 0.7], inverse=True)
    assert np.allclose(back, x)
