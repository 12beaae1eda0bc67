"""CPU-only checks of the cache, attention and norm entry points: what the host refuses before anything is launched."""
import ctypes
import os

import pytest

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


def _cache(lib, **kw):
    a = dict(pages=8, page_size=16, Hkv=2, D=128, format=0, k=0x10000, v=0x10000, k_s=0x10000, v_s=0x10000)
    a.update(kw)
    return ctypes.byref(lib.MoeKvCache(*a.values()))


def _att(lib, **kw):
    a = dict(B=2, Hq=4, Hkv=2, D=128, window=0, sinks=0, scale=1.0)
    a.update(kw)
    return ctypes.byref(lib.MoeAttention(*a.values()))


def test_norm_refusals(B):
    f = B.lib.moe_add_rmsnorm_mxfp8
    ok = [4, 64, AT, AT, AT, 1e-6, AT, AT, AT, AT, N]
    for i, bad, code in ((0, -1, 1), (1, 0, 1), (1, 48, 2), (1, 16416, 2), (2, N, 1), (4, N, 1), (5, float("nan"), 1),
                         (5, -1.0, 1), (8, N, 1), (9, N, 1), (2, ctypes.c_void_p(0x10008), 1),
                         (3, ctypes.c_void_p(0x10002), 1), (7, ctypes.c_void_p(0x10004), 1),
                         (8, ctypes.c_void_p(0x10004), 1)):
        assert f(*(ok[:i] + [bad] + ok[i + 1:])) == code, (i, bad)
    assert f(4, 64, AT, AT, AT, 1e-6, N, N, N, N, N) == B.MOE_ERR_INVALID_ARG      # nothing to write
    assert f(0, 64, N, N, N, 1e-6, N, N, N, N, N) == B.MOE_OK


def test_append_refusals(B):
    f = B.lib.moe_kv_append
    call = lambda c=None, T=4, k=AT, ks=256, v=AT, vs=256, slots=AT, ws=AT, n=256: f(  # noqa: E731
        _cache(B) if c is None else c, T, k, ks, v, vs, slots, ws, n, N)
    assert f(None, 4, AT, 256, AT, 256, AT, AT, 256, N) == B.MOE_ERR_INVALID_ARG
    for kw in (dict(page_size=12), dict(page_size=4), dict(page_size=512), dict(D=96), dict(pages=0), dict(Hkv=0),
               dict(format=2), dict(pages=2 ** 30)):
        assert call(_cache(B, **kw)) == B.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(k=0), dict(v=0x10040), dict(format=1, k_s=0), dict(format=1, v_s=0x10010)):
        assert call(_cache(B, **kw)) == B.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(T=-1), dict(k=N), dict(v=N), dict(slots=N), dict(ks=255), dict(vs=248), dict(ks=260),
               dict(k=ctypes.c_void_p(0x10008)), dict(slots=ctypes.c_void_p(0x10001))):
        assert call(**kw) == B.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(ws=N), dict(n=255), dict(ws=ctypes.c_void_p(0x10080))):
        assert call(**kw) == B.MOE_ERR_WORKSPACE, kw
    assert call(T=0, k=N, v=N, slots=N) == B.MOE_OK


def test_paged_attention_refusals(B):
    f = B.lib.moe_paged_attention
    need = B.moe_paged_attention_workspace_bytes(2, 3, 4, 2, 128, 100)
    assert need >= 256 and need % 256 == 0

    def call(a=None, c=None, rows=3, max_len=100, q=AT, qs=512, t=AT, w=8, n=AT, out=AT, ws=AT, size=need):
        return f(_att(B) if a is None else a, _cache(B) if c is None else c, rows, max_len, q, qs, t, w, n, out, ws, size, N)
    for kw in (dict(Hq=3), dict(Hq=0), dict(Hkv=0), dict(D=80), dict(window=-1), dict(sinks=-1), dict(B=-1),
               dict(scale=float("inf"))):
        assert call(_att(B, **kw)) == B.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(rows=0), dict(rows=65)):
        assert call(**kw) == B.MOE_ERR_UNSUPPORTED_SHAPE, kw
    assert call(c=_cache(B, Hkv=1)) == B.MOE_ERR_INVALID_ARG and call(c=_cache(B, D=64)) == B.MOE_ERR_INVALID_ARG
    for kw in (dict(max_len=129), dict(max_len=-1), dict(w=6), dict(q=N), dict(t=N), dict(n=N), dict(out=N),
               dict(qs=511), dict(qs=520 - 4), dict(q=ctypes.c_void_p(0x10008)), dict(out=ctypes.c_void_p(0x10004)),
               dict(t=ctypes.c_void_p(0x10002))):
        assert call(**kw) == B.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(ws=N), dict(size=need - 1), dict(ws=ctypes.c_void_p(0x10010))):
        assert call(**kw) == B.MOE_ERR_WORKSPACE, kw
    assert call(_att(B, B=0)) == B.MOE_OK
    assert B.moe_paged_attention_workspace_bytes(2, 65, 4, 2, 128, 100) == 0
    assert B.moe_paged_attention_workspace_bytes(2, 3, 5, 2, 128, 100) == 0


def test_prefill_attention_refusals(B):
    f = B.lib.moe_prefill_attention

    def call(a=None, Tq=9, Tk=9, q=AT, qs=512, k=AT, ks=256, v=AT, vs=256, cq=AT, ck=N, out=AT, ws=AT, n=256):
        return f(_att(B) if a is None else a, Tq, Tk, q, qs, k, ks, v, vs, cq, ck, out, ws, n, N)
    for kw in (dict(Hq=3), dict(D=32), dict(window=-1), dict(scale=float("nan"))):
        assert call(_att(B, **kw)) == B.MOE_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(Tq=-1), dict(Tk=-1), dict(q=N), dict(k=N), dict(v=N), dict(cq=N), dict(out=N), dict(qs=504),
               dict(ks=252), dict(vs=257), dict(k=ctypes.c_void_p(0x10008)), dict(ck=ctypes.c_void_p(0x10001))):
        assert call(**kw) == B.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(ws=N), dict(n=8)):
        assert call(**kw) == B.MOE_ERR_WORKSPACE, kw
    assert call(Tq=0, q=N, out=N) == B.MOE_OK and call(_att(B, B=0), q=N) == B.MOE_OK


def test_lengths_whose_last_step_passes_32_bits_are_refused(B):
    for n in (2 ** 31 - 255, 2 ** 31 - 1):
        assert B.lib.moe_paged_attention_workspace_bytes(_att(B), 1, n) == 0
        assert B.lib.moe_paged_attention(_att(B), _cache(B), 1, n, AT, 512, AT, 2 ** 28, AT, AT, AT, 2 ** 60, N) == \
            B.MOE_ERR_UNSUPPORTED_SHAPE
    assert B.lib.moe_paged_attention_workspace_bytes(_att(B), 1, 2 ** 31 - 256) > 0
