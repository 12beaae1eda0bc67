"""What tells a cache's format, and what says which one was meant."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_cache_is_of_the_format_that_its_caller_names():
    from block_scaled_fp8_moe_gb300 import binding as B
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    rows = lambda n: [u8(3, 2, 16, n) for _ in range(2)]  # noqa: E731
    bf16 = [t.bfloat16() for t in rows(128)]
    made = {B.MOE_KV_BF16: bf16, B.MOE_KV_MXFP8: rows(128) + rows(4), B.MOE_KV_MXFP4: rows(64) + rows(4)}
    for fmt, tensors in made.items():
        assert B.KvCache(*tensors).format == fmt
        for named in (*made, 2):
            if named == fmt:
                cache = B.KvCache(*tensors, format=named)
                assert (cache.format, cache.D) == (fmt, 128)
            else:                                # 64 bytes with four scales, say, where MXFP8 was meant
                with pytest.raises(ValueError, match="format"):
                    B.KvCache(*tensors, format=named)
