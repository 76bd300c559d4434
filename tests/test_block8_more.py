"""More of what the operators of 8-bit rows refuse, on the host (no GPU needed; the addresses are
never dereferenced)."""
import pytest
import torch

A = 0x7F0000000000


@pytest.fixture(scope="module")
def rr():
    import ring_allreduce_amd
    return ring_allreduce_amd


@pytest.fixture(scope="module")
def blk():
    import ring_allreduce_amd.block as block
    return block


def at(n):
    return A + (n << 30)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(x=at(0) + 2), 1), (dict(out=at(1) + 2), 1), (dict(x_ld=31), 1),
    (dict(out_ld=31), 1), (dict(blocks=0), 1), (dict(k=0), 1), (dict(slots=None), 1), (dict(sources=None), 1),
    (dict(sources=at(3) + 2), 1), (dict(tokens=1 << 31), 2), (dict(rows=1 << 31), 2), (dict(out=at(0) + 128), 1),
    (dict(sources=at(1) + 4), 1), (dict(rows=0, tokens=0, x=None, out=None), 0)])
def test_dispatch_of_scales(blk, change, status):
    c = dict(dict(x=at(0), x_ld=32, tokens=8, blocks=32, k=2, slots=at(2), sources=at(3), rows=16, out=at(1),
                  out_ld=32), **change)
    assert blk._expert_dispatch_scales(blk._Rows(c["x"], c["x_ld"]), c["tokens"], c["blocks"], c["k"], c["slots"],
                                       c["sources"], c["rows"], blk._Rows(c["out"], c["out_ld"]), None) == status


@pytest.mark.parametrize("rows", [0, 1])
def test_dispatch_of_one_row_of_a_buffer_of_odd_rows(rr, rows):
    """Its distance to the next row is no reason to refuse it: that it is on no GPU is."""
    flat = torch.zeros(64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    x = rr.Quantized(flat.as_strided((rows, 6), (7, 1), 2), torch.ones(rows, 1))
    slots = torch.zeros(rows, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        rr.expert_dispatch(x, slots, slots.reshape(-1))
