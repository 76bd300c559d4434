"""A block's gated projections, in 16 and in 8 bits, dense and over groups of rows, forward and
gradients, against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

from tests.block8_util import (E4M3, gate64, gated64, gated_dz64, gradients64, per_element, quantize64, wide)
from tests.block_util import DTYPES, U, act64, assert_within, store_error, strided

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "silu", "sigmoid"]


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_allreduce_amd
    return ring_allreduce_amd


def make(rr, rows, n, k, groups, dtype, bias, eight=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * n + k)
    dt, lead = DTYPES[dtype], () if groups is None else (groups,)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d = {"x": rnd(rows, k).to(dt), "w": (rnd(*lead, 2, n, k) * k ** -0.5).to(dt),
         "bias": rnd(*lead, 2, n).to(dt) if bias else None, "dout": rnd(rows, n).to(dt),
         "z": rnd(rows, 2 * n).to(dt)}
    if eight:
        d["x"], d["w"] = rr.block_quantize(d["x"]), rr.block_quantize(d["w"], square=True)
    return d


def check_forward(rr, d, offsets, act, dt):
    out, z = rr.block_gated(d["x"], d["w"], d["bias"], act=act, offsets=offsets, save_preact=True, dtype=dt)
    ro, rz, eo, ez = gated64(d["x"], d["w"], d["bias"], offsets, act)
    assert_within(z, rz, store_error(rz, dt) + ez * (1 + 2 ** -7), "z")
    assert_within(out, ro, store_error(ro, dt) + eo * (1 + 2 ** -7), "out")
    same = dict(act=act, offsets=offsets, dtype=dt)
    assert torch.equal(rr.block_gated(d["x"], d["w"], d["bias"], **same), out)
    again, q = rr.block_gated(d["x"], d["w"], d["bias"], save_preact="e4m3", **same)
    assert torch.equal(again, out)
    # in 8 bits z is what block_quantize makes of it, each half of a row by itself
    rows, n = out.shape
    assert q.values.shape == (rows, 2, n) and q.values.dtype == E4M3 and not q.square
    if rows:
        v, s = quantize64(z.view(rows, 2, n))
        assert bool((q.values.double() == v).all()) and bool((q.scales.double() == s).all())
    return q


def check_backward(rr, d, offsets, act, dt):
    rows, n = d["dout"].shape
    z8 = rr.block_quantize(d["z"].view(rows, 2, n))
    x8, w8 = (t if not isinstance(t, torch.Tensor) else q for t, q in (
        (d["x"], rr.block_quantize(wide(d["x"]).to(dt))),
        (d["w"], rr.block_quantize(wide(d["w"]).to(dt), square=True))))
    for x, w, z in ((d["x"], d["w"], d["z"]), (x8, d["w"], z8), (x8, w8, d["z"])):
        zv = z.double() if isinstance(z, torch.Tensor) else wide(z).view(rows, 2 * n)
        got = rr.block_gated_backward(d["dout"], x, w, z, act=act, offsets=offsets, need_out=True)
        some = torch.zeros(rows, 1, dtype=torch.bool, device="cuda")
        groups = 1 if got.dw.dim() == 3 else got.dw.shape[0]
        edges = [rows * i // groups for i in range(groups + 1)] if offsets is None else offsets.tolist()
        some[edges[0]:edges[-1]] = True
        dz, e32, edz = gated_dz64(d["dout"], zv, act, dt)
        (dx, edx), (dw, edw), (db, edb) = gradients64(dz, edz, x, w, offsets, dt, e32)
        out, eo = gate64(zv, torch.zeros_like(zv), act)
        out = torch.where(some, out, 0.0)
        assert_within(got.out, out, store_error(out, dt) + eo, "out")
        assert_within(got.dx, dx, store_error(dx, dt) + edx * (1 + 2 ** -7), "dx")
        assert_within(got.dw, dw, store_error(dw, dt) + edw * (1 + 2 ** -7), "dw")
        assert_within(got.db, db, edb + U * db.abs(), "db")
    only = rr.block_gated_backward(d["dout"], x8, w8, d["z"], act=act, offsets=offsets, need_dx=False,
                                   need_db=False, dw_dtype=torch.float32)
    assert_within(only.dw, dw, edw + U * dw.abs(), "dw fp32")
    assert only.dx is None and only.db is None and only.out is None


DENSE = [  # rows, n, k
    (1, 1, 1), (1, 4096, 1024), (1, 1000, 777), (2, 64, 64), (3, 130, 4104), (4, 33, 65), (7, 515, 31),
    (16, 1024, 1040), (17, 128, 264), (33, 555, 513), (64, 1024, 80), (60, 512, 4096), (65, 65, 129),
    (128, 64, 128), (129, 50, 65), (200, 500, 1000), (255, 129, 511), (256, 128, 64), (300, 5, 2000),
    (513, 320, 320), (1024, 512, 512), (1500, 384, 1040), (2100, 1200, 272)]


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,k", DENSE)
def test_dense(rr, dtype, rows, n, k, eight):
    act = ACTS[(rows + n + k) % 5]
    d = make(rr, rows, n, k, None, dtype, n % 2 == 0, eight)
    check_forward(rr, d, None, act, DTYPES[dtype])
    check_backward(rr, d, None, act, DTYPES[dtype])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("rows", [5, 150])
def test_epilogues(rr, act, bias, rows):
    d = make(rr, rows, 200, 96, None, "bf16", bias)
    check_forward(rr, d, None, act, torch.bfloat16)
    check_backward(rr, d, None, act, torch.bfloat16)


GROUPED = [  # sizes, rows before, rows after, n, k
    ([5], 0, 0, 64, 64), ([0, 3, 0], 0, 0, 40, 144), ([1, 2, 3, 4], 2, 3, 130, 65),
    ([128, 0, 256, 1], 0, 0, 128, 128), ([300, 17, 64, 129], 5, 70, 96, 264),
    ([0, 0], 0, 9, 33, 24), ([700, 20], 0, 0, 256, 1040), ([3] * 70, 0, 1, 64, 144),
    ([40, 0, 511, 257, 90, 0, 31, 64], 0, 100, 160, 576)]


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sizes,before,after,n,k", GROUPED, ids=lambda v: str(v)[:24])
def test_groups(rr, dtype, sizes, before, after, n, k, eight):
    """Groups of any size, and rows of no group, which become zero."""
    rows = before + sum(sizes) + after
    off = torch.from_numpy(before + np.concatenate([[0], np.cumsum(sizes)])).to(torch.int32).cuda()
    d = make(rr, rows, n, k, len(sizes), dtype, True, eight)
    act = ACTS[n % 5]
    check_forward(rr, d, off, act, DTYPES[dtype])
    check_backward(rr, d, off, act, DTYPES[dtype])


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
def test_equal_groups_and_no_rows(rr, eight):
    d = make(rr, 6 * 50, 96, 80, 6, "bf16", True, eight)
    check_forward(rr, d, None, "gelu", torch.bfloat16)
    check_backward(rr, d, None, "gelu", torch.bfloat16)
    d = make(rr, 0, 96, 80, 6, "bf16", True, eight)
    out, z = rr.block_gated(d["x"], d["w"], d["bias"], save_preact="e4m3")
    assert out.shape == (0, 96) and z.values.shape == (0, 2, 96)
    for kept in (z, d["z"]):
        got = rr.block_gated_backward(d["dout"], d["x"], d["w"], kept, need_out=True)
        assert not bool(got.dw.any()) and not bool(got.db.any())
        assert got.dx.shape == (0, 80) and got.out.shape == (0, 96)


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
def test_bad_offsets_stay_in_bounds(rr, eight):
    d = make(rr, 300, 64, 128, 4, "bf16", False, eight)
    for off in ([0, 500, -7, 1 << 30, 300], [-(1 << 31), 10, 5, 400, 2], [0, 0, 0, 0, 0]):
        o = torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda()
        out, z = rr.block_gated(d["x"], d["w"], offsets=o, save_preact="e4m3")
        g = rr.block_gated_backward(d["dout"], d["x"], d["w"], z, offsets=o, need_out=True)
        torch.cuda.synchronize()
        assert out.shape == (300, 64) and g.dx.shape == (300, 128)


@pytest.mark.parametrize("rows", [3, 30, 140])
def test_strides(rr, rows):
    d = make(rr, rows, 136, 264, None, "bf16", True)
    ro, _, eo, _ = gated64(d["x"], d["w"], d["bias"], None, "silu")
    xs, _ = strided(d["x"], 9, offset=3)
    ws, _ = strided(d["w"].view(272, 264), 13, offset=5)
    ws = ws.as_strided((2, 136, 264), (136 * 277, 277, 1), ws.storage_offset())
    out, store = strided(torch.zeros_like(d["dout"]), 7, offset=1)
    rr.block_gated(xs, ws, d["bias"], out=out)
    assert_within(out, ro, store_error(ro, torch.bfloat16) + eo * (1 + 2 ** -7), "out")
    store.as_strided(out.shape, out.stride(), 1).fill_(float("nan"))
    assert bool(store.isnan().all())
    zs, _ = strided(d["z"], 5, offset=1)
    ds, _ = strided(d["dout"], 3, offset=1)
    want = rr.block_gated_backward(d["dout"], d["x"], d["w"], d["z"], need_out=True)
    got = rr.block_gated_backward(ds, xs, ws, zs, need_out=True)
    assert all(torch.equal(getattr(want, k), getattr(got, k)) for k in ("dx", "dw", "db", "out"))
    z8 = rr.block_quantize(d["z"].view(rows, 2, 136))
    apart = torch.zeros(rows, 2 * 136 + 24, dtype=torch.uint8, device="cuda").view(E4M3)
    view = apart.as_strided((rows, 2, 136), (2 * 136 + 24, 136, 1), 3)
    view.view(torch.uint8).copy_(z8.values.view(torch.uint8))
    want = rr.block_gated_backward(d["dout"], d["x"], d["w"], z8)
    got = rr.block_gated_backward(d["dout"], d["x"], d["w"], rr.Quantized(view, z8.scales))
    assert all(torch.equal(getattr(want, k), getattr(got, k)) for k in ("dx", "dw", "db"))


def test_a_matrix_of_one_row(rr):
    """One column of out, the second matrix's row further behind the first than its length."""
    d = make(rr, 70, 1, 64, None, "bf16", False)
    store = torch.zeros(2, 1, 72, device="cuda").bfloat16()
    store[:, :, :64] = d["w"]
    assert torch.equal(rr.block_gated(d["x"], store[:, :, :64]), rr.block_gated(d["x"], d["w"]))


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
@pytest.mark.parametrize("rows", [9, 150, 600])
def test_nan_stays_in_its_row(rr, rows, eight):
    d = make(rr, rows, 200, 400, None, "bf16", True, eight)
    want = rr.block_gated(d["x"], d["w"], d["bias"])
    if eight:
        d["x"].values.view(torch.uint8)[rows - 2, 333] = 0x7F
    else:
        d["x"][rows - 2, 333] = float("nan")
    got, z = rr.block_gated(d["x"], d["w"], d["bias"], save_preact="e4m3")
    keep = [r for r in range(rows) if r != rows - 2]
    assert torch.equal(got[keep], want[keep]) and bool(got[rows - 2].isnan().all())
    assert bool(z.values[rows - 2].float().isnan().all()) and bool(z.values[keep].float().isfinite().all())
    # a group's gradient does not see its neighbours' rows
    x = normal_rows(rows, 400)
    x[rows // 2:] = float("nan")
    w = wide(d["w"]).bfloat16()
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    g = rr.block_gated_backward(d["dout"], x, torch.stack([w, w]), d["z"], offsets=off, need_dx=False)
    assert bool(g.dw[0].isfinite().all()) and bool(g.dw[1].isnan().all())


def normal_rows(rows, k):
    return torch.randn(rows, k, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()


def test_gradients_match_differences(rr):
    """Along directions of x, w and bias, against central differences in 64 bits."""
    for act in ("silu", "gelu", "sigmoid"):
        d = make(rr, 40, 24, 56, None, "fp16", True)
        _, z = rr.block_gated(d["x"], d["w"], d["bias"], act=act, save_preact=True)
        got = rr.block_gated_backward(d["dout"], d["x"], d["w"], z, act=act)
        g = torch.Generator(device="cuda").manual_seed(4)
        for key, grad in (("x", got.dx), ("w", got.dw), ("bias", got.db)):
            v = torch.randn(d[key].shape, generator=g, device="cuda", dtype=torch.float64)

            def loss(step):
                p = {k: d[k].double() for k in ("x", "w", "bias")}
                p[key] = p[key] + step * v
                gate, other = (p["x"] @ p["w"][h].t() + p["bias"][h] for h in range(2))
                return float((act64(gate, act) * other * d["dout"].double()).sum())

            along = float((grad.double() * v).sum())
            size = float((grad.double() * v).abs().sum())
            # z and dz are rounded to fp16, and with them the terms
            assert abs(along - (loss(1e-5) - loss(-1e-5)) / 2e-5) <= 6 * 2 ** -11 * size, (act, key)


@pytest.mark.parametrize("rows", [1, 48, 700])
def test_graph_and_streams(rr, rows):
    d = make(rr, rows, 256, 192, 2, "bf16", True)
    off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")

    def step(stream=None):
        out, z = rr.block_gated(d["x"], d["w"], d["bias"], offsets=off, save_preact="e4m3", stream=stream)
        x8 = rr.block_quantize(d["x"], stream=stream)
        g = rr.block_gated_backward(d["dout"], x8, d["w"], z, offsets=off, need_out=True, stream=stream)
        return [out, rr.block_dequantize(z, stream=stream), g.dx, g.dw, g.db, g.out]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        d["x"].copy_(torch.randn(rows, 192, generator=torch.Generator().manual_seed(seed)))
        off.copy_(torch.tensor([0, rows * seed // 3, rows], dtype=torch.int32))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_an_expert_layer(rr):
    """The operators as they are used: rows in 8 bits to their experts and their blocks, the gated
    projections and the projection back in 8 bits, kept in 8 bits for the backward pass, and the
    sum per token: each result is what the operators give one by one on what the bits stand for."""
    tokens, hidden, inner, experts, k = 300, 256, 136, 6, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w1, w2 = rnd(tokens, hidden), rnd(experts, 2, inner, hidden) * hidden ** -0.5, \
        rnd(experts, hidden, inner) * inner ** -0.5
    ids = torch.rand(tokens, experts, generator=g, device="cuda").topk(k).indices
    weights = torch.rand(tokens, k, generator=g, device="cuda")
    order = rr.expert_sort(ids, experts)
    x8 = rr.block_quantize(x)
    rows = rr.expert_dispatch(x8, order.slots, order.sources)
    plain = rr.expert_dispatch(rr.block_dequantize(x8), order.slots, order.sources)
    assert torch.equal(rr.block_dequantize(rows), plain)
    w1q, w2q = rr.block_quantize(w1, square=True), rr.block_quantize(w2, square=True)
    mid, z = rr.block_gated(rows, w1q, offsets=order.offsets, save_preact="e4m3")
    ro, _, eo, _ = gated64(rows, w1q, None, order.offsets, "silu")
    assert_within(mid, ro, store_error(ro, torch.bfloat16) + eo * (1 + 2 ** -7), "mid")
    made = rr.block_linear8(rr.block_quantize(mid), w2q, offsets=order.offsets)
    out = rr.expert_combine(made, order.slots, weights)
    assert bool(out.isfinite().all())
    dmade, _ = rr.expert_combine_backward(x, made, order.slots, order.sources, weights)
    zv = wide(z).view(tokens * k, 2 * inner)
    dmid = rr.block_linear8_backward(dmade, mid, w2q, offsets=order.offsets, need_dw=False).dx
    back = rr.block_gated_backward(dmid, rows, w1q, z, offsets=order.offsets, need_out=True)
    dw2 = rr.block_linear_backward(dmade, back.out, rr.block_dequantize(w2q), offsets=order.offsets).dw
    assert bool(dw2.isfinite().all())
    dz, e32, edz = gated_dz64(dmid, zv, "silu", torch.bfloat16)
    (dx, edx), (dw, edw), _ = gradients64(dz, edz, rows, w1q, order.offsets, torch.bfloat16, e32)
    assert_within(back.dx, dx, store_error(dx, torch.bfloat16) + edx * (1 + 2 ** -7), "dx")
    assert_within(back.dw, dw, store_error(dw, torch.bfloat16) + edw * (1 + 2 ** -7), "dw")
    assert per_element(z.scales, z.values.shape, False).shape == z.values.shape


FORMS = [  # rows, n, k: dots, one pass, deep tiles and their parts, at any byte and in whole pieces
    (1, 4100, 4112), (1, 350, 4100), (2, 350, 1777), (4, 64, 9), (9, 257, 9000), (12, 4096, 6144), (14, 100, 8208),
    (20, 150, 1001), (24, 512, 4096), (28, 4096, 6160), (40, 256, 2048), (50, 150, 1001), (64, 500, 4112)]


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
@pytest.mark.parametrize("rows,n,k", FORMS)
def test_few_rows(rr, rows, n, k, eight):
    check_forward(rr, make(rr, rows, n, k, None, "fp16", True, eight), None, "silu", torch.float16)


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
@pytest.mark.parametrize("rows,n,k", [(4500, 2200, 2064), (4608, 2304, 2064), (2560, 2304, 1040)])
def test_large_tiles(rr, rows, n, k, eight):
    """Tiles of 256 x 256, ragged ones, and a last round cut along the contraction; z in 8 bits comes
    from the tiles themselves."""
    d = make(rr, rows, n, k, None, "bf16", True, eight)
    if eight:
        d["w"].scales[..., 9:] *= 1.25
    check_forward(rr, d, None, "gelu", torch.bfloat16)


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
def test_large_groups(rr, eight):
    sizes = [2000, 0, 1, 1500, 900]
    off = torch.from_numpy(7 + np.concatenate([[0], np.cumsum(sizes)])).to(torch.int32).cuda()
    d = make(rr, sum(sizes) + 40, 1200, 2064, len(sizes), "bf16", True, eight)
    check_forward(rr, d, off, "silu", torch.bfloat16)
    if not eight:
        check_backward(rr, d, off, "silu", torch.bfloat16)


def test_large_z_of_infinities(rr):
    """In 8 bits z's NaN and infinities become NaN and leave their block's other values theirs, also
    where fp16 makes infinities of finite sums."""
    d = make(rr, 4500, 2200, 2064, None, "fp16", False)
    d["x"][17] *= 30000.0
    d["x"][4400, 5] = float("nan")
    d["x"][18] = torch.where(d["x"][18] > 0, 20000.0, -20000.0)      # z of 20000, some 3.3 times that
    check = rr.block_gated(d["x"], d["w"], save_preact=True)[1].view(4500, 2, 2200)
    z = rr.block_gated(d["x"], d["w"], save_preact="e4m3")[1]
    v, s = quantize64(check)
    assert bool((z.scales.double() == s).all())
    assert bool(((z.values.double() == v) | (v.isnan() & z.values.double().isnan())).all())
    # row 17 is infinite itself (30000 times what is over 2.2), of both signs
    assert bool(check[17].isnan().all())
    assert bool(check[18].isinf().any()) and bool(check[18].isfinite().any())


def test_strided_z_in_8_bits(rr):
    """Through the library itself, which takes z's rows any distance apart."""
    import ctypes
    blk = rr.block
    for rows in (5, 4500):
        n, k = 256, 64
        d = make(rr, rows, n, k, None, "bf16", False)
        a = blk._Linear8()
        a.l.rows, a.l.n, a.l.k, a.l.groups, a.l.dt, a.l.act = rows, n, k, 1, 2, 3
        a.l.x, a.l.w, a.l.w_ld = blk._Rows(d["x"].data_ptr(), k), d["w"].data_ptr(), k
        out = torch.zeros(rows, n, device="cuda", dtype=torch.bfloat16)
        z = torch.full((rows, 2 * n + 40), 0x7F, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(rows, 2, 2, device="cuda")
        a.l.out, a.l.z, a.z_scales = blk._Rows(out.data_ptr(), n), blk._Rows(z.data_ptr(), 2 * n + 40), scales.data_ptr()
        size = ctypes.c_size_t()
        assert blk._block_gated_workspace(ctypes.byref(a), ctypes.byref(size)) == 0
        work = torch.zeros(size.value or 1, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream
        assert blk._block_gated(ctypes.byref(a), work.data_ptr() if size.value else None, size.value, stream) == 0
        want_out, want = rr.block_gated(d["x"], d["w"], save_preact="e4m3")
        assert torch.equal(out, want_out) and torch.equal(scales, want.scales)
        assert torch.equal(z[:, :2 * n], want.values.view(torch.uint8).view(rows, 2 * n))
        assert bool((z[:, 2 * n:] == 0x7F).all())


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
def test_two_streams_at_once(rr, eight):
    """Calls on two streams, whose scratch memory is each their own."""
    d = [make(rr, 600, 384, 1040, 2, "bf16", True, eight, seed=s) for s in (0, 1)]
    off = torch.tensor([5, 200, 590], dtype=torch.int32, device="cuda")

    def step(s, stream=None):
        out, z = rr.block_gated(d[s]["x"], d[s]["w"], d[s]["bias"], offsets=off, save_preact="e4m3", stream=stream)
        g = rr.block_gated_backward(d[s]["dout"], d[s]["x"], d[s]["w"], z, offsets=off, need_out=True, stream=stream)
        return [out, z.values.view(torch.uint8), z.scales, g.dx, g.dw, g.db, g.out]

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [step(i % 2, streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


@pytest.mark.parametrize("rows,n", [(40, 2000), (70, 100), (600, 350), (2560, 2304)])
@pytest.mark.parametrize("k", [8, 10, 150, 516, 1030])
def test_rows_of_words(rr, rows, n, k):
    """Rows that end inside 16 bytes and begin at any word, NaN before, between and behind them."""
    d = make(rr, rows, n, k, None, "bf16", True)
    ro, _, eo, _ = gated64(d["x"], d["w"], d["bias"], None, "silu")
    got = []
    for ahead, ld in ((0, (k + 7) // 8 * 8 + 8), (2, k + 2), (6, k + 6), (0, k)):
        ops = []
        for v in (d["x"], d["w"].view(2 * n, k)):
            r = v.shape[0]
            flat = torch.full((ahead + r * ld,), float("nan"), device="cuda", dtype=torch.bfloat16)
            to = flat[ahead:].view(r, ld)[:, :k]
            to.copy_(v)
            ops.append(to)
        got.append(rr.block_gated(ops[0], ops[1].view(2, n, k), d["bias"]))
    assert_within(got[0], ro, store_error(ro, torch.bfloat16) + eo * (1 + 2 ** -7), "out")
    for g in got[1:]:
        assert_within(g, ro, store_error(ro, torch.bfloat16) + eo * (1 + 2 ** -7), "out")


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
@pytest.mark.parametrize("sizes", [[2, 0, 3, 1], [9, 40, 0, 11], [30, 70, 33, 1], [130, 7, 300, 90]], ids=str)
def test_groups_of_rows_of_words(rr, sizes, eight):
    off = torch.from_numpy(3 + np.concatenate([[0], np.cumsum(sizes)])).to(torch.int32).cuda()
    d = make(rr, sum(sizes) + 7, 200, 1036 if eight else 518, len(sizes), "bf16", True, eight)
    check_forward(rr, d, off, "silu", torch.bfloat16)
