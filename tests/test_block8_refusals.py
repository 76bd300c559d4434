"""What the entry points of the 8-bit format, of its products and of the gated ones refuse, on
the host, before any device work (no GPU needed; the addresses are never dereferenced)."""
import ctypes

import pytest
import torch

A = 0x7F0000000000
WORK = (A + (60 << 30), 1 << 30)


@pytest.fixture(scope="module")
def blk():
    import ring_allreduce_amd.block as block
    return block


@pytest.fixture(scope="module")
def rr():
    import ring_allreduce_amd
    return ring_allreduce_amd


def at(n):
    return A + (n << 30)


def fill(struct, blk, values):
    for k, v in values.items():
        setattr(struct, k, blk._Rows(*v) if isinstance(v, tuple) else v)
    return struct


def quantize(blk, **change):
    base = dict(groups=3, rows=130, width=300, dt=2, square=1, x=(at(0), 300), x_stride=130 * 300,
                q=(at(1), 300), q_stride=130 * 300, scales=at(2))
    return fill(blk._Quantize(), blk, dict(base, **change))


@pytest.mark.parametrize("change,status", [
    (dict(square=2), 1), (dict(dt=0), 1), (dict(dt=9), 1), (dict(width=0), 1), (dict(groups=0), 1),
    (dict(width=1 << 31, x=(at(0), 1 << 31), q=(at(1), 1 << 31)), 2), (dict(rows=1 << 31), 2),
    (dict(groups=1 << 24, rows=1 << 8), 2), (dict(x=(None, 300)), 1), (dict(q=(None, 300)), 1),
    (dict(x=(at(0) + 1, 300)), 1), (dict(x=(at(0), 299)), 1), (dict(q=(at(1), 299)), 1),
    (dict(scales=None), 1), (dict(scales=at(2) + 2), 1), (dict(q=(at(0) + 64, 300)), 1),
    (dict(scales=at(0) + 64), 1), (dict(scales=at(1) + 64), 1), (dict(x=(at(0), 1 << 41)), 2)])
def test_quantize(blk, change, status):
    a = quantize(blk, **change)
    assert blk._block_quantize(ctypes.byref(a), None) == status
    assert blk._block_dequantize(ctypes.byref(a), None) == status


def test_quantize_written_matrices_apart(blk):
    assert blk._block_quantize(ctypes.byref(quantize(blk, q_stride=130 * 300 - 1)), None) == 1
    assert blk._block_dequantize(ctypes.byref(quantize(blk, x_stride=130 * 300 - 1)), None) == 1
    assert blk._block_quantize(None, None) == 1 and blk._block_dequantize(None, None) == 1
    many = quantize(blk, groups=1 << 20, rows=128, width=1 << 13, x=(at(0), 1 << 13), x_stride=0,
                    q=(at(1) << 4, 1 << 13), q_stride=1 << 20, scales=at(2) << 5)
    assert blk._block_quantize(ctypes.byref(many), None) == 2        # 2^26 square blocks


def wide(blk, halves, eight, **change):
    """A call's struct; of 8-bit operands where ``eight``."""
    l = dict(rows=12, n=64, k=32, groups=3, dt=2, act=3, offsets=at(0), x=(at(1), 32), w=at(2),
             w_ld=32, w_stride=halves * 64 * 32, bias=at(3), z=(at(5), 64 * halves), out=(at(6), 64))
    if halves == 1:
        l["residual"] = (at(4), 64)
    scales = dict(x_scales=at(7) if eight else None, w_scales=at(8) if eight else None, z_scales=None)
    a = blk._Linear8()
    fill(a.l, blk, {k: change.pop(k, v) for k, v in l.items()})
    for k in ("reserved", "residual"):
        if k in change:
            fill(a.l, blk, {k: change.pop(k)})
    fill(a, blk, {k: change.pop(k, v) for k, v in scales.items()})
    assert not change
    return a


def calls(blk, halves):
    name = "linear8" if halves == 1 else "gated"
    return [getattr(blk, f"_block_{name}{s}") for s in ("", "_workspace", "_backward", "_backward_workspace")]


def grad(blk, halves, **change):
    base = dict(dout=(at(10), 64), dx=(at(11), 32), dw=at(12), db=at(13), dw_dt=2)
    if halves == 2:
        base["out"] = (at(14), 64)
    return fill(blk._LinearGrad() if halves == 1 else blk._GatedGrad(), blk, dict(base, **change))


@pytest.mark.parametrize("halves,eight", [(1, True), (2, True), (2, False)])
@pytest.mark.parametrize("change,status", [
    (dict(dt=0), 1), (dict(dt=1), 2), (dict(dt=9), 1), (dict(n=0), 1), (dict(k=0), 1),
    (dict(groups=0), 1), (dict(groups=1025), 2), (dict(act=5), 1), (dict(act=-1), 1),
    (dict(offsets=None, rows=13), 1), (dict(offsets=at(0) + 2), 1), (dict(w=None), 1), (dict(w_ld=31), 1),
    (dict(w_stride=64 * 32 - 1), 1), (dict(x=(None, 0)), 1), (dict(x=(at(1), 31)), 1),
    (dict(x=(at(1), 1 << 23)), 2), (dict(rows=1 << 31), 2), (dict(n=1 << 23), 1), (dict(n=1 << 33, z=(at(5), 1 << 34)), 2),
    (dict(reserved=1), 1), (dict(z=(at(5), 63)), 1), (dict(x_scales=at(7) + 2), 1)])
def test_products(blk, halves, eight, change, status):
    if eight is False and "x_scales" in change:
        change = dict(change, w_scales=at(8))
    if change.get("n") == 1 << 23:               # rows of out and z, and w, shorter than that
        change = dict(change, out=(at(6), 1 << 22))
    a, g, n = wide(blk, halves, eight, **change), grad(blk, halves), ctypes.c_size_t()
    run, size, back, back_size = calls(blk, halves)
    assert run(ctypes.byref(a), *WORK, None) == status
    assert size(ctypes.byref(a), ctypes.byref(n)) == status
    assert back(ctypes.byref(a), ctypes.byref(g), *WORK, None) == status
    assert back_size(ctypes.byref(a), ctypes.byref(g), ctypes.byref(n)) == status


def test_activations(blk):
    """The logistic function is for gates only."""
    n = ctypes.c_size_t()
    assert calls(blk, 1)[1](ctypes.byref(wide(blk, 1, True, act=4)), ctypes.byref(n)) == 1
    assert calls(blk, 2)[1](ctypes.byref(wide(blk, 2, True, act=4)), ctypes.byref(n)) == 0


@pytest.mark.parametrize("halves,eight", [(1, True), (2, True), (2, False)])
@pytest.mark.parametrize("change", [
    dict(out=(None, 0)), dict(out=(at(6), 63)), dict(out=(at(1), 64)), dict(out=(at(2), 64)),
    dict(out=(at(5), 64)), dict(out=(at(6) + 1, 64)), dict(bias=at(3) + 1), dict(out=(at(0), 64)),
    dict(out=(at(7), 64), x_scales=at(7), w_scales=at(8)), dict(z=(at(8), 128), x_scales=at(7), w_scales=at(8)),
    dict(x_scales=at(7), w_scales=None), dict(x_scales=None, w_scales=at(8)), dict(z=(at(1), 128))])
def test_forward_only(blk, halves, eight, change):
    a = wide(blk, halves, eight, **change)
    assert calls(blk, halves)[0](ctypes.byref(a), *WORK, None) == 1
    assert calls(blk, halves)[0](None, *WORK, None) == 1


def test_what_only_one_of_them_takes(blk):
    run = calls(blk, 1)[0]
    assert run(ctypes.byref(wide(blk, 1, False)), *WORK, None) == 1               # no scales
    assert run(ctypes.byref(wide(blk, 1, True, z_scales=at(9))), *WORK, None) == 1
    assert run(ctypes.byref(wide(blk, 1, True, z=(at(4), 64))), *WORK, None) == 1  # the residual's place
    gated = calls(blk, 2)[0]
    assert gated(ctypes.byref(wide(blk, 2, True, residual=(at(4), 64))), *WORK, None) == 1
    assert gated(ctypes.byref(wide(blk, 2, False, z_scales=at(9), z=(None, 0))), *WORK, None) == 1
    assert gated(ctypes.byref(wide(blk, 2, False, z_scales=at(9) + 1)), *WORK, None) == 1
    assert gated(ctypes.byref(wide(blk, 2, False, z_scales=at(6))), *WORK, None) == 1
    assert gated(ctypes.byref(wide(blk, 2, False, z_scales=at(9))), None, 0, None) == 1
    g = grad(blk, 1)
    back = calls(blk, 1)[2]
    assert back(ctypes.byref(wide(blk, 1, True, z_scales=at(9))), ctypes.byref(g), *WORK, None) == 1
    assert back(None, ctypes.byref(g), *WORK, None) == 1


@pytest.mark.parametrize("halves,eight", [(1, True), (2, True), (2, False)])
@pytest.mark.parametrize("change", [
    dict(dout=(None, 0)), dict(dout=(at(10), 63)), dict(dx=(at(11), 31)), dict(dw_dt=3), dict(reserved=1),
    dict(dw=at(12) + 1), dict(db=at(13) + 2), dict(dx=(at(10), 32)), dict(dw=at(2)), dict(db=at(12)),
    dict(dw=at(5)), dict(db=at(60) + 8)])
def test_gradients(blk, halves, eight, change):
    a, g = wide(blk, halves, eight), grad(blk, halves, **change)
    back = calls(blk, halves)[2]
    assert back(ctypes.byref(a), ctypes.byref(g), *WORK, None) == 1
    ok = grad(blk, halves)
    assert back(ctypes.byref(a), ctypes.byref(ok), None, 0, None) == 1
    assert back(ctypes.byref(a), ctypes.byref(ok), WORK[0], 64, None) == 1
    assert back(ctypes.byref(a), None, *WORK, None) == 1
    none = wide(blk, halves, eight, z=(None, 0))
    assert back(ctypes.byref(none), ctypes.byref(ok), *WORK, None) == 1


@pytest.mark.parametrize("change", [dict(out=(at(14), 63)), dict(out=(at(14) + 1, 64)), dict(out=(at(5), 64)),
                                    dict(out=(at(10), 64)), dict(out=(at(11), 64))])
def test_the_product_again(blk, change):
    a, g = wide(blk, 2, False), grad(blk, 2, **change)
    assert calls(blk, 2)[2](ctypes.byref(a), ctypes.byref(g), *WORK, None) == 1


def q(rr, rows=4, k=8, square=False, lead=(), **change):
    shape = (*lead, rows, k)
    s = (*lead, -(-rows // 128) if square else rows, -(-k // 128))
    return rr.Quantized(**dict(dict(values=torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn),
                                    scales=torch.ones(s), square=square), **change))


def test_binding(rr):
    x, b = torch.zeros(4, 8), torch.zeros(4, 8).bfloat16()
    w2 = torch.zeros(2, 4, 8).bfloat16()
    x8, w8, g8 = q(rr), q(rr, square=True), q(rr, square=True, lead=(2,))
    z8 = rr.Quantized(torch.zeros(4, 2, 4, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(4, 2, 1))
    for call in (lambda: rr.block_quantize(x), lambda: rr.block_dequantize(x8), lambda: rr.block_linear8(x8, w8),
                 lambda: rr.block_linear8_backward(b[:, :4], x8, w8), lambda: rr.block_gated(b, w2),
                 lambda: rr.block_gated(x8, g8), lambda: rr.block_gated_backward(b[:, :4], b, w2, b),
                 lambda: rr.block_gated_backward(b[:, :4], x8, w2, z8)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: rr.block_quantize(x.double()), lambda: rr.block_dequantize(x),
                 lambda: rr.block_linear8(b, w8), lambda: rr.block_linear8(x8, b),
                 lambda: rr.block_gated(x8, w2), lambda: rr.block_gated(b, g8),
                 lambda: rr.block_linear8(x8, w8, dtype=torch.float32), lambda: rr.block_gated(x, w2),
                 lambda: rr.block_linear8(q(rr, values=x), w8)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: rr.block_quantize(x.reshape(-1)), lambda: rr.block_linear8(w8, w8),
                 lambda: rr.block_linear8(x8, x8), lambda: rr.block_linear8(x8, w8, act="sigmoid"),
                 lambda: rr.block_gated(b, w2, act="tanh"), lambda: rr.block_gated(b, w2, save_preact="e5m2"),
                 lambda: rr.block_gated_backward(None, b, w2, b), lambda: rr.expert_dispatch(x8, None, None, out=x)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("halves", [1, 2])
def test_more_rows_of_weights_than_32_bits_count(blk, halves):
    n, groups = (1 << 22) // halves, 1024
    size = ctypes.c_size_t()
    for g, status in ((groups, 2), (511, 0)):
        a = wide(blk, halves, True, groups=g, n=n, k=16, x=(at(1), 32), w=1 << 40, w_ld=16, w_stride=n * halves * 16,
                 z=(at(5), 1 << 22), out=(at(6), n), residual=(None, 0), bias=None, rows=g)
        c = grad(blk, halves, dout=(at(10), n), dw=None, db=None)
        if halves == 2:
            c.out = blk._Rows(at(14), n)
        calls_ = calls(blk, halves)
        assert calls_[1](ctypes.byref(a), ctypes.byref(size)) == status
        assert calls_[3](ctypes.byref(a), ctypes.byref(c), ctypes.byref(size)) == status


def test_more_rows_of_8_bit_z_than_32_bits_count(blk):
    size = ctypes.c_size_t()
    for rows, status in ((1 << 30, 2), ((1 << 30) - 2048, 0)):
        a = wide(blk, 2, False, groups=1, rows=rows, n=1, k=1, z_scales=at(9) << 4, z=(at(5), 2), out=(at(6), 1))
        assert calls(blk, 2)[1](ctypes.byref(a), ctypes.byref(size)) == status
