"""A block's matrix products with their epilogue, dense and over groups of rows, forward
and gradients, against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

from tests.block_util import DTYPES, U, act64, assert_within, slope64, store_error, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_allreduce_amd
    return ring_allreduce_amd


def make(rows, n, k, groups, dtype, bias, residual, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * n + k)
    dt = DTYPES[dtype]
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    grouped = groups is not None
    e = groups if grouped else 1
    lead = (e,) if grouped else ()
    return {"x": rnd(rows, k).to(dt), "w": (rnd(*lead, n, k) * k ** -0.5).to(dt),
            "bias": rnd(*lead, n).to(dt) if bias else None,
            "residual": rnd(rows, n).to(dt) if residual else None,
            "dout": rnd(rows, n).to(dt), "z": rnd(rows, n).to(dt)}


def edges_of(d, offsets):
    rows = d["x"].shape[0]
    w = d["w"] if d["w"].dim() == 3 else d["w"][None]
    if offsets is None:
        each = rows // w.shape[0]
        return w, [(i * each, (i + 1) * each) for i in range(w.shape[0])]
    off = offsets.tolist()
    return w, list(zip(off[:-1], off[1:]))


def forward64(d, offsets, act):
    """out, z and their 32-bit errors: a sum of k products (each of the matrix
    instruction's additions may be off by a step of the sum so far), the bias, the
    activation (its slope is under 1.2, its own evaluation a few steps)."""
    rows, k = d["x"].shape
    w, edges = edges_of(d, offsets)
    n = w.shape[1]
    z, size = (torch.zeros(rows, n, dtype=torch.float64, device="cuda") for _ in range(2))
    out = torch.zeros_like(z)
    for e, (lo, hi) in enumerate(edges):
        x = d["x"][lo:hi].double()
        z[lo:hi] = x @ w[e].double().t()
        size[lo:hi] = x.abs() @ w[e].double().abs().t()
        if d["bias"] is not None:
            b = d["bias"].reshape(-1, n)[e].double()
            z[lo:hi] += b
            size[lo:hi] += b.abs()
        out[lo:hi] = act64(z[lo:hi], act)
        if d["residual"] is not None:
            out[lo:hi] += d["residual"][lo:hi].double()
    err_z = (k + 2) * U * size
    extra = d["residual"].double().abs() * U if d["residual"] is not None else 0.0
    err_out = 1.2 * err_z + 8 * U * z.abs() + extra + 2 * U * out.abs()
    return out, z, err_out, err_z


def backward64(d, offsets, act, dt):
    rows, k = d["x"].shape
    w, edges = edges_of(d, offsets)
    n = w.shape[1]
    dz = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    for lo, hi in edges:
        dz[lo:hi] = d["dout"][lo:hi].double() * slope64(d["z"][lo:hi].double(), act)
    # dz in 32 bits, then (with an activation) rounded to the type as an operand; a slope near
    # its zero is a difference of terms of size 1, and an exponential carries its argument's
    # rounding, so steps count by |dout|
    edz32 = 16 * U * d["dout"].double().abs() if act != "none" else torch.zeros_like(dz)
    edz = edz32 + store_error(dz.abs() + edz32, dt) if act != "none" else edz32
    dx, edx = torch.zeros(2, rows, k, dtype=torch.float64, device="cuda")
    dw, edw = torch.zeros(2, *w.shape, dtype=torch.float64, device="cuda")
    db, edb = torch.zeros(2, w.shape[0], n, dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(edges):
        g, eg, x, we = dz[lo:hi], edz[lo:hi], d["x"][lo:hi].double(), w[e].double()
        dx[lo:hi] = g @ we
        edx[lo:hi] = (eg + (n + 2) * U * (g.abs() + eg)) @ we.abs()
        m = hi - lo
        dw[e] = g.t() @ x
        edw[e] = (eg + (m + 2) * U * (g.abs() + eg)).t() @ x.abs()
        db[e] = g.sum(0)
        edb[e] = (edz32[lo:hi] + (m + 2) * U * g.abs()).sum(0)
    return dz, (dx, edx), (dw.reshape(d["w"].shape), edw.reshape(d["w"].shape)), \
        (db.reshape(d["w"].shape[:-1]), edb.reshape(d["w"].shape[:-1]))


def check_forward(rr, d, offsets, act, dt, **kw):
    out, z = rr.block_linear(d["x"], d["w"], d["bias"], act=act, residual=d["residual"],
                             offsets=offsets, save_preact=True, **kw)
    ro, rz, eo, ez = forward64(d, offsets, act)
    assert_within(z, rz, store_error(rz, dt) + ez * (1 + 2 ** -7), "z")
    assert_within(out, ro, store_error(ro, dt) + eo * (1 + 2 ** -7), "out")
    only = rr.block_linear(d["x"], d["w"], d["bias"], act=act, residual=d["residual"],
                           offsets=offsets)
    assert torch.equal(only, out)


def check_backward(rr, d, offsets, act, dt):
    z = d["z"] if act != "none" else None
    got = rr.block_linear_backward(d["dout"], d["x"], d["w"], z, act=act, offsets=offsets)
    wide = rr.block_linear_backward(d["dout"], d["x"], d["w"], z, act=act, offsets=offsets,
                                    need_dx=False, need_db=False, dw_dtype=torch.float32)
    _, (dx, edx), (dw, edw), (db, edb) = backward64(d, offsets, act, dt)
    assert_within(got.dx, dx, store_error(dx, dt) + edx * (1 + 2 ** -7), "dx")
    assert_within(got.dw, dw, store_error(dw, dt) + edw * (1 + 2 ** -7), "dw")
    assert_within(wide.dw, dw, edw + U * dw.abs(), "dw fp32")
    assert_within(got.db, db, edb + U * db.abs(), "db")
    assert wide.dx is None and wide.db is None and got.db.dtype == torch.float32


DENSE = [  # rows, n, k
    (1, 1, 1), (1, 8192, 4096), (1, 1000, 777), (2, 64, 64), (3, 130, 4104), (7, 515, 31),
    (16, 4096, 1024), (17, 256, 264), (33, 1111, 513), (64, 2048, 72), (65, 129, 129),
    (128, 128, 128), (129, 100, 65), (200, 1000, 1000), (255, 257, 511), (256, 256, 64),
    (300, 5, 2000), (513, 640, 320), (1024, 1024, 512), (1500, 768, 1032)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,k", DENSE)
def test_dense(rr, dtype, rows, n, k):
    act = ["none", "relu", "gelu", "silu"][(rows + n + k) % 4]
    d = make(rows, n, k, None, dtype, n % 2 == 0, k % 2 == 0)
    check_forward(rr, d, None, act, DTYPES[dtype])
    check_backward(rr, d, None, act, DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("bias,residual", [(True, True), (False, False), (True, False)])
def test_epilogues(rr, dtype, act, bias, residual):
    for rows in (5, 150):
        d = make(rows, 200, 96, None, dtype, bias, residual)
        check_forward(rr, d, None, act, DTYPES[dtype])
        check_backward(rr, d, None, act, DTYPES[dtype])


GROUPED = [  # sizes, rows before, rows after, n, k
    ([5], 0, 0, 64, 64), ([0, 3, 0], 0, 0, 40, 72), ([1, 2, 3, 4], 2, 3, 130, 65),
    ([128, 0, 256, 1], 0, 0, 256, 128), ([300, 17, 64, 129], 5, 70, 192, 264),
    ([0, 0], 0, 9, 33, 24), ([700, 20], 0, 0, 512, 1000), ([3] * 70, 0, 1, 64, 136),
    ([40, 0, 511, 257, 90, 0, 31, 64], 0, 100, 320, 576)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sizes,before,after,n,k", GROUPED, ids=lambda v: str(v)[:24])
def test_groups(rr, dtype, sizes, before, after, n, k):
    """Groups of any size, and rows of no group, which become zero."""
    rows = before + sum(sizes) + after
    off = torch.from_numpy(before + np.concatenate([[0], np.cumsum(sizes)])).to(torch.int32).cuda()
    d = make(rows, n, k, len(sizes), dtype, True, True)
    act = "silu" if n % 64 else "none"
    check_forward(rr, d, off, act, DTYPES[dtype])
    check_backward(rr, d, off, act, DTYPES[dtype])


def test_equal_groups(rr):
    d = make(6 * 50, 96, 80, 6, "bf16", True, False)
    check_forward(rr, d, None, "gelu", torch.bfloat16)
    check_backward(rr, d, None, "gelu", torch.bfloat16)
    d = make(0, 96, 80, 6, "bf16", True, False)
    got = rr.block_linear_backward(d["dout"], d["x"], d["w"])
    assert not bool(got.dw.any()) and not bool(got.db.any())


def test_bad_offsets_stay_in_bounds(rr):
    """Offsets that descend or leave the rows: no access outside, and it ends."""
    d = make(300, 64, 64, 4, "bf16", False, False)
    for off in ([0, 500, -7, 1 << 30, 300], [-(1 << 31), 10, 5, 400, 2], [0, 0, 0, 0, 0]):
        o = torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda()
        out = rr.block_linear(d["x"], d["w"], offsets=o)
        g = rr.block_linear_backward(d["dout"], d["x"], d["w"], offsets=o)
        torch.cuda.synchronize()
        assert out.shape == (300, 64) and g.dx.shape == (300, 64)


@pytest.mark.parametrize("rows", [3, 140])
def test_strides_and_in_place(rr, rows):
    d = make(rows, 136, 264, None, "bf16", True, True)
    want = rr.block_linear(d["x"], d["w"], d["bias"], act="silu", residual=d["residual"])
    xs, _ = strided(d["x"], 9, offset=3)
    ws, _ = strided(d["w"], 13, offset=5)
    out, store = strided(d["residual"], 7, offset=1)
    rr.block_linear(xs, ws, d["bias"], act="silu", residual=out, out=out)
    off = (out.double() - want.double()).abs()
    assert bool((off <= 2 * store_error(want.double(), torch.bfloat16)).all())
    left = store.clone()
    left.as_strided(out.shape, out.stride(), 1).fill_(float("nan"))
    assert bool(left.isnan().all())
    wide = torch.randn(rows, 264 + 8, device="cuda").bfloat16()      # 16-byte rows apart
    a = rr.block_linear(wide[:, 8:], d["w"])
    assert torch.equal(a, rr.block_linear(wide[:, 8:].contiguous(), d["w"]))
    g = rr.block_linear_backward(d["dout"], wide[:, 8:], d["w"], need_dx=False)
    g2 = rr.block_linear_backward(d["dout"], wide[:, 8:].contiguous(), d["w"], need_dx=False)
    assert torch.equal(g.dw, g2.dw)


@pytest.mark.parametrize("k", [72, 65])
def test_nan_stays_in_its_row(rr, k):
    """Infinities and NaN of one row, or past a row's end, reach no other output."""
    d = make(150, 96, k, None, "bf16", True, False)
    want = rr.block_linear(d["x"], d["w"], d["bias"])
    xs, store = strided(d["x"], 8)           # NaN between the rows
    ws, _ = strided(d["w"], 8)
    assert bool((rr.block_linear(xs, ws, d["bias"]).isfinite()).all())
    xs[7], xs[149] = float("nan"), float("inf")
    got = rr.block_linear(xs, ws, d["bias"])
    keep = [r for r in range(150) if r not in (7, 149)]
    off = (got[keep].double() - want[keep].double()).abs()
    assert bool((off <= 2 * store_error(want[keep].double(), torch.bfloat16) + 1e-3).all())
    assert bool(got[7].isnan().all())
    # a group's gradient does not see its neighbours' rows
    x = d["x"].clone()
    x[64:] = float("nan")
    off2 = torch.tensor([0, 64, 150], dtype=torch.int32, device="cuda")
    w2 = torch.stack([d["w"], d["w"]])
    g = rr.block_linear_backward(d["dout"], x, w2, offsets=off2, need_dx=False)
    assert bool(g.dw[0].isfinite().all()) and bool(g.dw[1].isnan().all())


def test_gradients_match_differences(rr):
    """Along directions of x, w and bias, against central differences in 64 bits; the
    operands' rounding to fp16 leaves 2^-11 of the terms."""
    d = make(40, 48, 56, None, "fp16", True, False)
    _, z = rr.block_linear(d["x"], d["w"], d["bias"], act="gelu", save_preact=True)
    got = rr.block_linear_backward(d["dout"], d["x"], d["w"], z, act="gelu")
    g = torch.Generator(device="cuda").manual_seed(4)
    for key, grad in (("x", got.dx), ("w", got.dw), ("bias", got.db)):
        v = torch.randn(d[key].shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(step):
            p = {"x": d["x"].double(), "w": d["w"].double(), "bias": d["bias"].double()}
            p[key] = p[key] + step * v
            return float((act64(p["x"] @ p["w"].t() + p["bias"], "gelu") * d["dout"].double()).sum())

        along = float((grad.double() * v).sum())
        size = float((grad.double() * v).abs().sum())
        assert abs(along - (loss(1e-5) - loss(-1e-5)) / 2e-5) <= 4 * 2 ** -11 * size, key


def test_graph_and_streams(rr):
    d = make(260, 256, 192, 2, "bf16", True, True)
    off = torch.tensor([0, 100, 250], dtype=torch.int32, device="cuda")

    def step(stream=None):
        out, z = rr.block_linear(d["x"], d["w"], d["bias"], act="silu", residual=d["residual"],
                                 offsets=off, save_preact=True, stream=stream)
        g = rr.block_linear_backward(d["dout"], d["x"], d["w"], z, act="silu", offsets=off,
                                     stream=stream)
        return [out, z, g.dx, g.dw, g.db]

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
        d["x"].copy_(torch.randn(260, 192, generator=torch.Generator().manual_seed(seed)))
        off.copy_(torch.tensor([0, 10 + 80 * seed, 260 - seed], dtype=torch.int32))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))
