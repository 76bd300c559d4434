"""The example of a mixture-of-experts step over virtual ranks: every result against the plain
step in 64 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "expert_block.py")


@pytest.mark.parametrize("argv", [[], ["--ranks", "3", "--tokens", "77", "--hidden", "264",
                                       "--inner", "136"]])
def test_step(argv):
    """Between two operators a tensor is rounded to bf16, by 2^-9 of its values at the root of the
    mean square; a result has at most 12 such roundings behind it on its longest way (norm, dispatched
    rows, z, mid, made, out; and as many back), which add up as their squares, and a slope of up to
    1.1 at the activation and the norms' own factor of 2 come on top."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("expert_block", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for name, off in example.main(argv).items():
        assert off <= 2 * 1.1 * 12 ** 0.5 * 2 ** -9, (name, off)
