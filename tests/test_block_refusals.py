"""What the entry points of a block's operators refuse, on the host, before any device
work (no GPU needed; the addresses are never dereferenced)."""
import ctypes

import pytest
import torch

A = 0x7F0000000000


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


SORT = dict(ids=at(0), id_bytes=8, id_ld=2, tokens=8192, k=2, experts=16, capacity=0, slots=at(1),
            sources=at(2), counts=at(3), offsets=at(4), work=at(5), bytes=1 << 20)


@pytest.mark.parametrize("change,status", [
    (dict(id_bytes=2), 1), (dict(k=0), 1), (dict(experts=0), 1), (dict(experts=1025), 2),
    (dict(ids=None), 1), (dict(slots=None), 1), (dict(sources=None), 1), (dict(counts=None), 1),
    (dict(offsets=None), 1), (dict(id_ld=1), 1), (dict(ids=at(0) + 4), 1), (dict(slots=at(1) + 2), 1),
    (dict(work=None), 1), (dict(bytes=16), 1), (dict(tokens=1 << 31), 2), (dict(capacity=1 << 31), 2),
    (dict(slots=at(0)), 1), (dict(sources=at(1)), 1), (dict(offsets=at(3)), 1), (dict(work=at(2)), 1)])
def test_sort(blk, change, status):
    c = dict(SORT, **change)
    assert blk._expert_sort(*c.values(), None) == status


def test_sort_workspace(blk):
    n = ctypes.c_size_t()
    assert blk._expert_sort_workspace(16, 4, 32, ctypes.byref(n)) == 0 and n.value == 0
    assert blk._expert_sort_workspace(1 << 16, 8, 256, ctypes.byref(n)) == 0 and n.value > 0
    assert blk._expert_sort_workspace(16, 4, 32, None) == 1
    assert blk._expert_sort_workspace(1 << 31, 4, 32, ctypes.byref(n)) == 2


def move(blk, kind, **change):
    c = dict(x=at(0), x_ld=64, out=at(1), out_ld=64, tokens=8, hidden=64, k=2, dt=2, slots=at(2),
             sources=at(3), rows=16, weights=at(4), dweights=at(5), drows=at(6))
    c.update(change)
    R = blk._Rows
    if kind == "dispatch":
        return blk._expert_dispatch(R(c["x"], c["x_ld"]), c["tokens"], c["hidden"], c["k"], c["dt"],
                                    c["slots"], c["sources"], c["rows"], R(c["out"], c["out_ld"]), None)
    if kind == "combine":
        return blk._expert_combine(R(c["x"], c["x_ld"]), c["rows"], c["hidden"], c["dt"], c["slots"],
                                   c["weights"], c["tokens"], c["k"], R(c["out"], c["out_ld"]), None)
    return blk._expert_combine_backward(R(c["x"], c["x_ld"]), R(c["out"], c["out_ld"]), c["rows"],
                                        c["hidden"], c["dt"], c["slots"], c["sources"], c["weights"],
                                        c["tokens"], c["k"], R(c["drows"], 64), c["dweights"], None)


@pytest.mark.parametrize("kind", ["dispatch", "combine", "backward"])
@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(x=at(0) + 1), 1), (dict(x_ld=63), 1),
    (dict(out_ld=63), 1), (dict(hidden=0), 1), (dict(k=0), 1), (dict(dt=0), 1), (dict(dt=9), 1),
    (dict(slots=None), 1), (dict(slots=at(2) + 2), 1), (dict(tokens=1 << 31), 2), (dict(rows=1 << 31), 2)])
def test_moves(blk, kind, change, status):
    assert move(blk, kind, **change) == status


def test_moves_overlap(blk):
    assert move(blk, "dispatch", out=at(0) + 128) == 1
    assert move(blk, "dispatch", sources=None) == 1
    assert move(blk, "dispatch", sources=at(1) + 4) == 1
    assert move(blk, "combine", out=at(0)) == 1
    assert move(blk, "combine", weights=at(1)) == 1
    assert move(blk, "backward", drows=at(0)) == 1
    assert move(blk, "backward", drows=at(1)) == 1
    assert move(blk, "backward", dweights=at(6)) == 1
    assert move(blk, "backward", sources=None) == 1
    assert move(blk, "dispatch", rows=0, tokens=0, x=None, out=None) == 0      # nothing to do


def norm(blk, **change):
    a = blk._Norm()
    R = blk._Rows
    base = dict(tokens=4, hidden=64, dt=2, weight_dt=2, post_norm=1, pre_norm=1, gate_kind=2,
                gate_act=3, residual_scale=1.0, branch_scale=1.0, eps=1e-6, x=R(at(0), 64),
                branch=R(at(1), 64), gate=R(at(2), 64), post_weight=at(3), pre_weight=at(4),
                h=R(at(5), 64), y=R(at(6), 64))
    for k, v in dict(base, **change).items():
        setattr(a, k, R(*v) if isinstance(v, tuple) else v)
    return a


NORM = [
    (dict(dt=0), 1), (dict(dt=7), 1), (dict(weight_dt=3), 1), (dict(hidden=0), 1),
    (dict(hidden=32769, x=(at(0), 40000), branch=(at(1), 40000), gate=(at(2), 40000),
          h=(at(5), 40000), y=(at(6), 40000)), 2),
    (dict(post_norm=2), 1), (dict(pre_norm=-1), 1), (dict(gate_kind=3), 1), (dict(gate_act=1), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(branch=(None, 0)), 1),
    (dict(branch=(at(1), 63)), 1), (dict(branch=(at(1) + 1, 64)), 1), (dict(gate=(None, 0)), 1),
    (dict(gate_kind=0), 1), (dict(gate_kind=0, gate=(None, 0)), 1), (dict(post_weight=at(3) + 1), 1),
    (dict(reserved=1), 1), (dict(tokens=1 << 31), 2)]


@pytest.mark.parametrize("change,status", NORM)
def test_norm(blk, change, status):
    a = norm(blk, **change)
    assert blk._block_norm(ctypes.byref(a), None) == status
    g, n = norm_grad(blk), ctypes.c_size_t()
    assert blk._block_norm_backward_workspace(ctypes.byref(a), ctypes.byref(g), ctypes.byref(n)) == status
    assert blk._block_norm_backward(ctypes.byref(a), ctypes.byref(g), at(20), 1 << 28, None) == status


@pytest.mark.parametrize("change", [
    dict(x=(None, 0)), dict(x=(at(0), 8)), dict(y=(None, 0)), dict(pre_norm=0), dict(h=(at(6), 64)),
    dict(h=(at(1), 64)), dict(y=(at(0), 64)), dict(h=(at(0) + 2, 64)), dict(y=(at(2), 64)),
    dict(h=(at(3), 64)), dict(pre_norm=0, y=(None, 0), h=(None, 0))])
def test_norm_forward_only(blk, change):
    a = norm(blk, **change)
    assert blk._block_norm(ctypes.byref(a), None) == 1
    assert blk._block_norm(None, None) == 1


def norm_grad(blk, **change):
    g = blk._NormGrad()
    R = blk._Rows
    base = dict(dh=(at(10), 64), dy=(at(11), 64), dx=(at(12), 64), dbranch=(at(13), 64),
                dgate=(at(14), 64), dpost_weight=at(15), dpre_weight=at(16))
    for k, v in dict(base, **change).items():
        setattr(g, k, R(*v) if isinstance(v, tuple) else v)
    return g


@pytest.mark.parametrize("change", [
    dict(dy=(None, 0)), dict(dh=(at(10), 8)), dict(dx=(at(12) + 1, 64)), dict(dgate_channel=at(17)),
    dict(dx=(at(11), 64)), dict(dbranch=(at(10), 64)), dict(dx=(at(5), 64)), dict(dgate=(at(13), 64)),
    dict(dpre_weight=at(15)), dict(dpre_weight=at(16) + 2), dict(dpost_weight=at(3))])
def test_norm_gradients(blk, change):
    a, g = norm(blk), norm_grad(blk, **change)
    assert blk._block_norm_backward(ctypes.byref(a), ctypes.byref(g), at(20), 1 << 28, None) == 1
    ok = norm_grad(blk)
    assert blk._block_norm_backward(ctypes.byref(a), ctypes.byref(ok), None, 1 << 28, None) == 1
    assert blk._block_norm_backward(ctypes.byref(a), ctypes.byref(ok), at(20), 8, None) == 1
    assert blk._block_norm_backward(ctypes.byref(a), None, at(20), 1 << 28, None) == 1


def linear(blk, **change):
    a = blk._Linear()
    R = blk._Rows
    base = dict(rows=12, n=64, k=32, groups=3, dt=2, act=3, offsets=at(0), x=(at(1), 32), w=at(2),
                w_ld=32, w_stride=64 * 32, bias=at(3), residual=(at(4), 64), z=(at(5), 64),
                out=(at(6), 64))
    for k, v in dict(base, **change).items():
        setattr(a, k, R(*v) if isinstance(v, tuple) else v)
    return a


def linear_grad(blk, **change):
    g = blk._LinearGrad()
    R = blk._Rows
    base = dict(dout=(at(10), 64), dx=(at(11), 32), dw=at(12), db=at(13), dw_dt=2)
    for k, v in dict(base, **change).items():
        setattr(g, k, R(*v) if isinstance(v, tuple) else v)
    return g


@pytest.mark.parametrize("change,status", [
    (dict(dt=0), 1), (dict(dt=1), 2), (dict(dt=9), 1), (dict(n=0), 1), (dict(k=0), 1),
    (dict(groups=0), 1), (dict(groups=1025), 2), (dict(act=4), 1), (dict(act=-1), 1),
    (dict(offsets=None, rows=13), 1), (dict(offsets=at(0) + 2), 1), (dict(w=None), 1),
    (dict(w=at(2) + 1), 1), (dict(w_ld=31), 1), (dict(w_stride=64 * 32 - 1), 1), (dict(x=(None, 0)), 1),
    (dict(x=(at(1), 31)), 1), (dict(x=(at(1), 1 << 23)), 2), (dict(rows=1 << 31), 2),
    (dict(reserved=1), 1), (dict(z=(at(5), 63)), 1)])
def test_linear(blk, change, status):
    a, g, n = linear(blk, **change), linear_grad(blk), ctypes.c_size_t()
    work = (at(30), 1 << 30)
    assert blk._block_linear(ctypes.byref(a), *work, None) == status
    assert blk._block_linear_workspace(ctypes.byref(a), ctypes.byref(n)) == status
    assert blk._block_linear_backward(ctypes.byref(a), ctypes.byref(g), *work, None) == status
    assert blk._block_linear_backward_workspace(ctypes.byref(a), ctypes.byref(g), ctypes.byref(n)) == status


@pytest.mark.parametrize("change", [
    dict(out=(None, 0)), dict(out=(at(6), 63)), dict(out=(at(1), 64)), dict(out=(at(2), 64)),
    dict(out=(at(5), 64)), dict(z=(at(4), 64)), dict(out=(at(4), 65)), dict(out=(at(4) + 2, 64)),
    dict(residual=(at(4), 8)), dict(bias=at(3) + 1), dict(out=(at(0), 64))])
def test_linear_forward_only(blk, change):
    a = linear(blk, **change)
    assert blk._block_linear(ctypes.byref(a), at(30), 1 << 30, None) == 1


@pytest.mark.parametrize("change", [
    dict(dout=(None, 0)), dict(dout=(at(10), 63)), dict(dx=(at(11), 31)), dict(dw_dt=3),
    dict(dw=at(12) + 1), dict(db=at(13) + 2), dict(dx=(at(10), 32)), dict(dw=at(2)), dict(db=at(12))])
def test_linear_gradients(blk, change):
    a, g = linear(blk), linear_grad(blk, **change)
    assert blk._block_linear_backward(ctypes.byref(a), ctypes.byref(g), at(30), 1 << 30, None) == 1
    ok = linear_grad(blk)
    assert blk._block_linear_backward(ctypes.byref(a), ctypes.byref(ok), None, 0, None) == 1
    assert blk._block_linear_backward(ctypes.byref(a), ctypes.byref(ok), at(30), 64, None) == 1
    none = linear(blk, z=(None, 0))
    assert blk._block_linear_backward(ctypes.byref(none), ctypes.byref(ok), at(30), 1 << 30, None) == 1


def test_binding_refuses_host_tensors_and_wrong_types(rr):
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: rr.expert_sort(i, 4), lambda: rr.expert_dispatch(x, i, i.reshape(-1)),
                 lambda: rr.expert_combine(x, i), lambda: rr.block_norm(x, x),
                 lambda: rr.block_linear(x.bfloat16(), x.bfloat16())):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: rr.expert_sort(x, 4), lambda: rr.block_linear(x, x),
                 lambda: rr.expert_dispatch(x.double(), i, i)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        rr.expert_sort(i, 0)
    with pytest.raises(ValueError):
        rr.expert_sort(i.reshape(-1), 4)
