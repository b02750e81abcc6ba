"""The order of kv_attn_chunk's stores to tensor memory, read off its source: tcgen05.st is asynchronous, and a load or an MMA
that comes after it is ordered behind it only by tcgen05.wait::st of the storing thread.  So between a store and the next
release to other threads (a fence before a barrier, or an arrival) there is a wait, in every role's code."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_fp8blk_gb300", "csrc", "kv_chunk.cuh")


def test_stores_are_waited_for_before_they_are_released():
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    stores, pending = 0, False
    for m in re.finditer(r"(void )?\b(ch_st16|ch_wait_st|t8_fence_before|mbar_arrive)\(", text):
        if m[1]:  # the definitions
            continue
        if m[2] == "ch_st16":
            stores, pending = stores + 1, True
        elif m[2] == "ch_wait_st":
            pending = False
        else:
            assert not pending, f"line {text[:m.start()].count(chr(10)) + 1}: released before tcgen05.wait::st"
    assert stores >= 4 and not pending
