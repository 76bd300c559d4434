"""Unusual calls of a block's operators, where they can be checked without a GPU."""
import ctypes
import os
import re
import subprocess
import sys

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


def test_package_without_the_marshalling_module():
    """The module is a faster way into the library, not the library: without it (not built, or
    built against another torch) the package is there, says so, and marshals in Python."""
    program = """
import sys, warnings
sys.modules["ring_allreduce_amd._block"] = None          # an import of it fails
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import ring_allreduce_amd as rr
assert any("_block" in str(w.message) for w in seen), seen
import torch
x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
for call in (lambda: rr.expert_sort(i, 4), lambda: rr.expert_dispatch(x, i, i.reshape(-1)),
             lambda: rr.expert_combine(x, i), lambda: rr.block_norm(x, x),
             lambda: rr.expert_combine_backward(x, x, i, i.reshape(-1)),
             lambda: rr.block_norm_backward(x, x, x, x), lambda: rr.block_linear(x.bfloat16(), x.bfloat16()),
             lambda: rr.block_linear_backward(x.bfloat16(), x.bfloat16(), x.bfloat16())):
    try:
        call()
    except ValueError as e:
        assert "GPU" in str(e), e
    else:
        raise AssertionError("host tensors were taken")
assert rr._abi_version() >= 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_inline_assembly_names_the_registers_it_writes():
    """A register written by an instruction of an asm block and not an operand of it has to be
    among what it clobbers: the compiler may keep a value there."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = 0
    for folder in ("csrc", "csrc_block"):
        at = os.path.join(root, "ring_allreduce_amd", folder)
        for name in sorted(os.listdir(at)):
            with open(os.path.join(at, name)) as fh:
                text = fh.read()
            for block in re.findall(r"\basm\s*(?:volatile)?\s*\(.*?\)\s*;", text, flags=re.S):
                blocks += 1
                strings = re.findall(r'"((?:[^"\\]|\\.)*)"', block)
                code = strings[0].replace("\\n", "\n").replace("\\t", " ")
                for written in re.findall(r"^\s*\w+\s+(m0|vcc|exec|s\d+|v\d+)\b", code, flags=re.M):
                    assert written in strings[1:], f"{name}: {written} in {block}"
    assert blocks >= 3
