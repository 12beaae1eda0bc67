"""CPU-only: the workspace that a call of the paged attention needs is its own format's, at every length."""
import ctypes

import pytest

from tests.test_attention_abi import AT, B, N, _att, _cache  # noqa: F401  (B is a fixture)


def _need(fmt, batch, rows, Hq, Hkv, D, max_len):
    """256 bytes, and where a sequence can have several pieces, D + 2 floats of every row and piece. Pieces are of 8 steps of 64
    tokens, at most 64; more than 16 rows to a key head, and MXFP4, have steps of 128, 4 of them a piece below 64 steps and 8
    from there on, at most 32 pieces."""
    small = fmt != 4 and rows * (Hq // Hkv) <= 16
    tile, most = (64, 64) if small else (128, 32)

    def pieces(steps):
        per = 8 if small or steps >= 64 else 4
        return min(max((steps + per // 2) // per, 1), most)
    steps = -(-max_len // tile)
    n = max(pieces(steps), pieces(min(steps, 63)))              # a shorter sequence can have more
    n = 0 if n == 1 else n * batch * rows * Hq
    return 256 + -(-n * D * 4 // 256) * 256 + -(-n * 8 // 256) * 256


@pytest.mark.parametrize("fmt", [0, 1, 4])
@pytest.mark.parametrize("rows,Hq", [(1, 8), (3, 10), (6, 16), (9, 30)])
def test_every_length(B, rows, Hq, fmt):  # noqa: F811
    for max_len in list(range(0, 10000, 37)) + [640, 641, 704, 705, 1153, 1216, 7809, 7872, 8192, 8193, 100000]:
        need = _need(fmt, 2, rows, Hq, 2, 128, max_len)
        assert B.moe_paged_attention_workspace_bytes(2, rows, Hq, 2, 128, max_len) >= need

        def call(size):                         # refused for its missing queries where the workspace is enough
            return B.lib.moe_paged_attention(_att(B, Hq=Hq), _cache(B, pages=8000, format=fmt), rows, max_len, N, Hq * 128, AT, 7000,
                                             AT, AT, AT, size, N)
        assert call(need) == B.MOE_ERR_INVALID_ARG, max_len
        assert call(need - 1) == B.MOE_ERR_WORKSPACE, max_len
