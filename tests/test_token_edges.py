"""Edges of the token operators that need no GPU: sources, refusals, the binding and its build."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_sparse_attention_35_b200", "csrc")


@pytest.mark.parametrize("name", ["kv4_attn.cu", "kv4_chunk.cu"])
def test_warps_agree_on_what_a_wait_returned(name):
    """Where a whole warp waits and goes on with shuffles, votes or matrix instructions, its lanes
    share one verdict: nothing stores a single lane's."""
    src = open(os.path.join(CSRC, name)).read()
    assert len(re.findall(r"\bmbar_wait_warp\(", src)) >= 1
    assert not re.findall(r"\bok\w*\s*=[^;]*\bmbar_wait\(", src)
    # what is left are the waits of one elected lane that asks for copies
    for m in re.finditer(r"\bmbar_wait\(", src):
        before = src[:m.start()]
        assert before.rfind("if (lane == 0)") > before.rfind("} else"), src[m.start() - 80:m.end() + 40]



def test_products_end_before_tensor_memory_is_released():
    """A softmax warp whose wait gives up leaves products in flight that the warp which issued them
    has no reason to doubt: every release stands behind the block's barrier and, where any warp
    raised the abort flag, behind a bounded wait for all products."""
    src = open(os.path.join(CSRC, "kv4_chunk.cu")).read()
    ends = [m.start() for m in re.finditer(r"\btmem_dealloc\(tmem", src)]
    assert len(ends) == 2
    for at in ends:
        tail = src[:at]
        barrier = tail.rfind("    tc_fence_before();\n    __syncthreads();")
        drain = tail[barrier:]
        assert "if (s_abort)" in drain and "umma_commit(&s_drain" in drain and "mbar_wait_drain(&s_drain" in drain
