"""Unusual calls of a block's operators: nothing to do, values far from 1, infinities, bad
index tensors, against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

from tests.test_gpu_expert import check_order, make_ids, order_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_allreduce_amd
    return ring_allreduce_amd


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,experts,capacity", [
    (0, 2, 512, 0), (0, 2, 513, 0), (0, 2, 1024, 0), (0, 2, 1024, 3), (0, 8, 700, 5), (1, 2, 1024, 3)])
def test_sort_of_no_tokens(rr, dtype, tokens, k, experts, capacity):
    """A rank without tokens, with any number of experts."""
    ids = make_ids(tokens, k, experts, "any", 1)
    o = rr.expert_sort(torch.from_numpy(ids).to(dtype).cuda(), experts, capacity)
    check_order(o, order_of(ids, experts, capacity))
