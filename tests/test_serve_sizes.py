"""Workspace sizes of kv4_attention at the ends of the arguments' ranges (CPU
only: they follow from the sizes and the number of SMs)."""
import os

import pytest


@pytest.fixture(scope="module")
def clib():
    from gptq_post_weight_gb300 import _lib, build

    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,max_q", [(8, 1 << 20), (32, 1 << 20), (64, 1 << 20), (1024, 1 << 20), (1024, 4096)])
def test_the_longest_lists_of_work_do_not_overflow(clib, dim, group, max_q):
    # Rows enough for the kernel of few rows.  Once there is more work than
    # shares, more of it needs no more memory.
    size = clib.gptq_kv4_attention_call_bytes
    some = size(dim, 64, group, max_q, 64, 0, 1 << 20)
    assert 1 << 20 < some < 1 << 30
    for heads, seqs, length in ((64, 1 << 20, 1 << 20), (1024, 1024, 1 << 30), (1024, 1 << 20, 1 << 30)):
        assert size(dim, heads, group, max_q, seqs, 0, length) == some
    assert clib.gptq_kv4_attention_workspace_bytes(dim, group, max_q) == some
