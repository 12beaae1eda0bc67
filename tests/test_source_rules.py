"""CPU-only checks of the kernels' sources for orders that no run shows reliably."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_fp8_moe_gb300", "csrc")


@pytest.mark.parametrize("name", ["attention_prefill.cu", "attention_paged_tc.cu"])
def test_tensor_memory_is_taken_before_successors_may_start(name):
    """A successor that got Tensor Memory first would wait for this grid, and this grid for columns."""
    src = re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())
    alloc, trigger = src.index("tmem_alloc("), src.index("pdl_trigger()")
    assert alloc < src.index("__syncthreads()", alloc) < trigger
