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


@pytest.mark.parametrize("call", [
    lambda b, x, i, bad: b.combine_backward(x, x, i, i.reshape(-1), None, bad, True),
    lambda b, x, i, bad: b.combine_backward(x, x, i, i.reshape(-1), None, True, bad),
    lambda b, x, i, bad: b.linear(x, x, None, 0, None, None, bad)])
def test_marshalling_leaves_no_error_behind(call):
    """An option without a truth value ends the usual form of a call, which answers None; what
    was raised on the way is gone."""
    from ring_allreduce_amd import _block
    x, i = torch.zeros(4, 8).bfloat16(), torch.zeros(4, 2, dtype=torch.int32)
    assert call(_block, x, i, torch.zeros(2)) is None
