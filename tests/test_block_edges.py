"""Unusual calls of a block's operators, where they can be checked without a GPU."""
import ctypes

import pytest
import torch  # noqa: F401


@pytest.fixture(scope="module")
def blk():
    import ring_allreduce_amd.block as block
    return block


@pytest.mark.parametrize("experts", [513, 1024])
def test_sort_of_no_tokens_has_a_share(blk, experts):
    """More experts than one workgroup takes: the counts of one share, also without tokens."""
    n = ctypes.c_size_t()
    assert blk._expert_sort_workspace(0, 2, experts, ctypes.byref(n)) == 0
    assert n.value == experts * 4
