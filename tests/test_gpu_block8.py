"""Values in 8 bits with a scale for each block of 128, and products of them, against plain
64-bit implementations."""
import numpy as np
import pytest
import torch

from tests.block8_util import (E4M3, as_operand, e4m3_64, gradients64, linear64, per_element,
                               quantize64, wide)
from tests.block_util import DTYPES, U, assert_within, slope64, store_error, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_allreduce_amd
    return ring_allreduce_amd


def same(got, want):
    """Equal, NaN for NaN."""
    got, want = got.double(), want.double()
    return bool(((got == want) | (got.isnan() & want.isnan())).all())


def normal(shape, seed, dtype=torch.float32, spread=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(*shape, generator=g, device="cuda")
    return (v * torch.exp(2 * torch.randn(shape[-1], generator=g, device="cuda")) if spread else v).to(dtype)


# ------------------------------------------------------------------ the format --

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 127), (2, 129), (130, 260), (128, 128), (257, 1000),
                                   (1000, 8), (3, 5, 40), (2, 130, 300), (2, 2, 200, 136), (5, 0), (0, 64)],
                         ids=str)
def test_quantize(rr, dtype, square, shape):
    if shape[-1] == 0:
        with pytest.raises(ValueError):
            rr.block_quantize(torch.zeros(*shape, device="cuda"), square=square)
        return
    x = normal(shape, sum(shape), DTYPES[dtype])
    q = rr.block_quantize(x, square=square)
    assert q.values.dtype == E4M3 and q.scales.dtype == torch.float32 and q.square == square
    assert q.values.shape == x.shape
    if x.numel() == 0:
        assert rr.block_dequantize(q).shape == x.shape
        return
    v, s = quantize64(x, square)
    assert q.scales.shape == s.shape
    assert same(q.scales, s) and same(q.values, v)
    for back in (torch.bfloat16, torch.float16, torch.float32):
        b = rr.block_dequantize(q, back)
        assert b.dtype == back and same(b, (v * per_element(s, shape, square)).clamp(
            -torch.finfo(back).max, torch.finfo(back).max).to(back))


def test_every_rounding(rr):
    """Every e4m3 value, the middles between neighbours and the fp32 values beside them, both signs,
    in blocks whose scale is 1 and others."""
    grid = torch.arange(127, dtype=torch.uint8).view(E4M3).float()        # 0 .. 448
    mid = (grid[1:] + grid[:-1]) / 2
    x = torch.cat([grid, mid, torch.nextafter(mid, torch.tensor(1e9)), torch.nextafter(mid, torch.tensor(0.0))])
    x = torch.cat([x, -x])
    rows = x.reshape(-1, 1).repeat(1, 128)
    rows[:, ::2] = 448.0
    rows = torch.cat([rows, rows * 2.0 ** 20, rows * 2.0 ** -100, rows * 2.0 ** 119]).cuda()
    q = rr.block_quantize(rows)
    v, s = quantize64(rows)
    assert same(q.scales, s) and same(q.values, v)
    assert bool(q.scales[:len(x)].eq(1).all())


def test_scales_at_their_borders(rr):
    """Largest values at and beside 448 times a power of two, the smallest and largest of fp32, and
    zeros."""
    a = torch.tensor([448.0, 448.00003, 447.99997, 224.0, 224.00002, 1.0, 1.75, 1.7500001, 0.0, -0.0,
                      2.0 ** -149, 2.0 ** -126, 448 * 2.0 ** -126, 3.4028235e38, 1e-42, 896.0])
    x = torch.zeros(len(a), 128)
    x[:, 77] = -a
    q = rr.block_quantize(x.cuda())
    v, s = quantize64(x.cuda())
    assert same(q.scales, s) and same(q.values, v)
    assert float(q.scales[8]) == 1 and not bool(q.values[8].float().any())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("square", [False, True])
def test_nan_and_infinities(rr, dtype, square):
    """They become NaN, and their blocks' scales go by the finite values; blocks of nothing else
    have scale 1."""
    x = normal((140, 300), 5, DTYPES[dtype])
    x[3, 7], x[3, 8], x[4, 200], x[139, 299] = float("nan"), float("inf"), -float("inf"), float("nan")
    x[5, 128:256] = float("inf")
    x[128:, 256:] = float("nan")
    q = rr.block_quantize(x, square=square)
    v, s = quantize64(x, square)
    assert same(q.scales, s) and same(q.values, v)
    assert bool(q.values.float().isnan().eq(~x.isfinite()).all())
    assert float(q.scales[-1, -1]) == 1
    assert same(rr.block_dequantize(q, torch.float32), v * per_element(s, x.shape, square))


def test_fp16_past_its_end(rr):
    x = torch.full((1, 128), 65504.0, device="cuda", dtype=torch.float16)
    x[0, 1] = float("nan")
    b = rr.block_dequantize(rr.block_quantize(x), torch.float16)
    assert float(b[0, 0]) == 65504 and bool(b[0, 1].isnan())
    assert float(rr.block_dequantize(rr.block_quantize(x), torch.float32)[0, 0]) == 65536


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("k", [200, 201])
def test_quantize_strides(rr, square, k):
    x = normal((150, k), 9, torch.bfloat16)
    want = rr.block_quantize(x, square=square)
    for pad, offset in ((7, 1), (8, 0), (24, 8)):
        xs, store = strided(x, pad, offset=offset)
        got = rr.block_quantize(xs, square=square)
        assert same(got.values, want.values) and same(got.scales, want.scales)
        out, store = strided(torch.zeros_like(x), pad, offset=offset)
        rr.block_dequantize(want, out=out)
        assert same(out, rr.block_dequantize(want, torch.bfloat16))
        store.as_strided(out.shape, out.stride(), offset).fill_(float("nan"))
        assert bool(store.isnan().all())
    three = normal((4, 150, k), 10, torch.float16)[::2]
    got, one = rr.block_quantize(three, square=square), rr.block_quantize(three.contiguous(), square=square)
    assert same(got.values, one.values) and same(got.scales, one.scales)
    # values of rows further apart
    wide_rows = torch.zeros(150, k + 9, dtype=torch.uint8, device="cuda").view(E4M3)
    wide_rows[:, 3:k + 3].view(torch.uint8).copy_(want.values.view(torch.uint8))
    apart = rr.Quantized(wide_rows[:, 3:k + 3], want.scales, square)
    assert same(rr.block_dequantize(apart), rr.block_dequantize(want))


def test_many_rows(rr):
    """Offsets past 2^31 bytes and elements."""
    x = torch.zeros(70000, 32768, dtype=torch.bfloat16, device="cuda")
    x[-1], x[65537, 5] = 3.0, -1.5
    q = rr.block_quantize(x)
    assert float(q.scales[-1, -1]) == 2.0 ** -7 and float(q.values[-1, -1]) == 384
    assert float(q.values[65537, 5]) == -384 and float(q.scales[65537, 1]) == 1
    b = rr.block_dequantize(q)
    assert bool((b[-1] == 3).all()) and float(b[65537, 5]) == -1.5 and not bool(b[65536].any())


# ---------------------------------------------------------------- the products --

def make(rr, rows, n, k, groups, dtype, bias, residual, seed=0, foreign=False):
    dt, lead = DTYPES[dtype], () if groups is None else (groups,)
    s = seed + 7 * n + k
    d = {"x": rr.block_quantize(normal((rows, k), s, dt, False)),
         "w": rr.block_quantize(normal((*lead, n, k), s + 1, dt, False) * k ** -0.5, square=True),
         "bias": normal((*lead, n), s + 2, dt, False) if bias else None,
         "residual": normal((rows, n), s + 3, dt, False) if residual else None,
         "dout": normal((rows, n), s + 4, dt, False), "z": normal((rows, n), s + 5, dt, False)}
    if foreign:
        for q in (d["x"], d["w"]):
            q.scales *= 0.5 + torch.rand(q.scales.shape, generator=torch.Generator().manual_seed(s)).cuda()
    return d


def check_forward(rr, d, offsets, act, dt):
    out, z = rr.block_linear8(d["x"], d["w"], d["bias"], dtype=dt, act=act, residual=d["residual"],
                              offsets=offsets, save_preact=True)
    ro, rz, eo, ez = linear64(d["x"], d["w"], d["bias"], offsets, act, d["residual"])
    assert_within(z, rz, store_error(rz, dt) + ez * (1 + 2 ** -7), "z")
    assert_within(out, ro, store_error(ro, dt) + eo * (1 + 2 ** -7), "out")
    assert torch.equal(rr.block_linear8(d["x"], d["w"], d["bias"], dtype=dt, act=act, residual=d["residual"],
                                        offsets=offsets), out)


def check_backward(rr, d, offsets, act, dt):
    z = d["z"] if act != "none" else None
    dz = d["dout"].double() * (slope64(z.double(), act) if act != "none" else 1.0)
    e32 = 16 * U * d["dout"].double().abs() if act != "none" else torch.zeros_like(dz)
    edz = e32 + store_error(dz.abs() + e32, dt) if act != "none" else e32
    for x, w in ((d["x"], d["w"]), (d["x"], rr.block_dequantize(d["w"], dt)),
                 (rr.block_dequantize(d["x"], dt), d["w"])):
        got = rr.block_linear8_backward(d["dout"], x, w, z, act=act, offsets=offsets)
        (dx, edx), (dw, edw), (db, edb) = gradients64(dz, edz, x, w, offsets, dt, e32)
        assert_within(got.dx, dx, store_error(dx, dt) + edx * (1 + 2 ** -7), "dx")
        assert_within(got.dw, dw, store_error(dw, dt) + edw * (1 + 2 ** -7), "dw")
        assert_within(got.db, db, edb + U * db.abs(), "db")
    only = rr.block_linear8_backward(d["dout"], d["x"], d["w"], z, act=act, offsets=offsets, need_dx=False,
                                     need_db=False, dw_dtype=torch.float32)
    (dx, edx), (dw, edw), _ = gradients64(dz, edz, d["x"], d["w"], offsets, dt, e32)
    assert_within(only.dw, dw, edw + U * dw.abs(), "dw fp32")
    assert only.dx is None and only.db is None


DENSE = [  # rows, n, k
    (1, 1, 1), (1, 1024, 4096), (1, 1000, 777), (2, 64, 128), (3, 130, 4104), (4, 300, 144), (7, 515, 31),
    (16, 2048, 1024), (17, 256, 272), (33, 1111, 513), (64, 2048, 80), (64, 384, 4096), (65, 129, 129),
    (128, 128, 128), (129, 100, 65), (200, 1000, 1000), (255, 257, 511), (256, 256, 256), (300, 5, 2000),
    (513, 640, 1328), (1024, 1024, 512), (2100, 2304, 1040)]


@pytest.mark.parametrize("rows", [1, 40, 200])
def test_products_of_eight_neighbours(rr, rows):
    """What the 8-bit matrix instructions keep of a product: to 2^-13 of the largest among its
    eight neighbours, and all of it behind them.  A large term cancelled by one of another eight leaves
    the small one, or less."""
    x = torch.zeros(rows, 128, device="cuda")
    x[:, 0] = x[:, 64] = 256.0
    x[:, 1] = x[:, 72] = 2.0
    w = torch.zeros(14, 128, device="cuda")
    w[:, 0], w[:, 64] = 256.0, -256.0
    for j in range(14):
        w[j, 1 if j < 7 else 72] = 2.0 ** (j % 7 - 1)
    x8, w8 = x.to(E4M3), w.to(E4M3)
    out = rr.block_linear8(rr.Quantized(x8, torch.ones(rows, 1, device="cuda")),
                           rr.Quantized(w8, torch.ones(1, 1, device="cuda"), True))
    exact = torch.tensor([2.0 ** (j % 7) for j in range(14)], device="cuda")
    assert torch.equal(out[:, 7:].float(), exact[7:].expand(rows, 7))
    off = (out[:, :7].float() - exact[:7]).abs()
    assert bool((off < 2.0 ** (16 - 13)).all()) and bool((out[:, 3:7].float() == exact[3:7]).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,n,k", DENSE)
def test_dense(rr, dtype, rows, n, k):
    act = ["none", "relu", "gelu", "silu"][(rows + n + k) % 4]
    d = make(rr, rows, n, k, None, dtype, n % 2 == 0, k % 2 == 0, foreign=k % 3 == 0)
    check_forward(rr, d, None, act, DTYPES[dtype])
    check_backward(rr, d, None, act, DTYPES[dtype])


GROUPED = [  # sizes, rows before, rows after, n, k
    ([5], 0, 0, 64, 64), ([0, 3, 0], 0, 0, 40, 144), ([1, 2, 3, 4], 2, 3, 130, 65),
    ([128, 0, 256, 1], 0, 0, 256, 128), ([300, 17, 64, 129], 5, 70, 192, 264),
    ([0, 0], 0, 9, 33, 24), ([700, 20], 0, 0, 512, 1040), ([3] * 70, 0, 1, 64, 144),
    ([40, 0, 511, 257, 90, 0, 31, 64], 0, 100, 320, 576)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("sizes,before,after,n,k", GROUPED, ids=lambda v: str(v)[:24])
def test_groups(rr, dtype, sizes, before, after, n, k):
    rows = before + sum(sizes) + after
    off = torch.from_numpy(before + np.concatenate([[0], np.cumsum(sizes)])).to(torch.int32).cuda()
    d = make(rr, rows, n, k, len(sizes), dtype, True, True)
    act = "silu" if n % 64 else "none"
    check_forward(rr, d, off, act, DTYPES[dtype])
    check_backward(rr, d, off, act, DTYPES[dtype])


def test_equal_groups_and_no_rows(rr):
    d = make(rr, 6 * 50, 96, 80, 6, "bf16", True, False)
    check_forward(rr, d, None, "gelu", torch.bfloat16)
    check_backward(rr, d, None, "gelu", torch.bfloat16)
    d = make(rr, 0, 96, 80, 6, "bf16", True, False)
    assert rr.block_linear8(d["x"], d["w"], d["bias"]).shape == (0, 96)
    got = rr.block_linear8_backward(d["dout"], d["x"], d["w"])
    assert not bool(got.dw.any()) and not bool(got.db.any()) and got.dx.shape == (0, 80)


def test_bad_offsets_stay_in_bounds(rr):
    d = make(rr, 300, 64, 128, 4, "bf16", False, False)
    for off in ([0, 500, -7, 1 << 30, 300], [-(1 << 31), 10, 5, 400, 2], [0, 0, 0, 0, 0]):
        o = torch.tensor(off, dtype=torch.int64).to(torch.int32).cuda()
        out = rr.block_linear8(d["x"], d["w"], offsets=o)
        g = rr.block_linear8_backward(d["dout"], d["x"], d["w"], offsets=o)
        torch.cuda.synchronize()
        assert out.shape == (300, 64) and g.dx.shape == (300, 128)


@pytest.mark.parametrize("rows", [3, 30, 140])
def test_strides(rr, rows):
    """Rows of any byte, and outputs of any stride, in place of the residual."""
    d = make(rr, rows, 136, 264, None, "bf16", True, True)
    args = dict(act="silu", dtype=torch.bfloat16)
    ro, _, eo, _ = linear64(d["x"], d["w"], d["bias"], None, "silu", d["residual"])

    def spread(q, pad, offset, square):
        r, c = q.values.shape
        store = torch.full((r * (c + pad) + offset + 16,), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
        view = store.as_strided((r, c), (c + pad, 1), offset)
        view.view(torch.uint8).copy_(q.values.view(torch.uint8))
        return rr.Quantized(view, q.scales, square)

    for pad, offset in ((9, 3), (8, 16), (24, 5)):
        xs, ws = spread(d["x"], pad, offset, False), spread(d["w"], pad + 2, offset + 1, True)
        out, store = strided(d["residual"], 7, offset=1)
        rr.block_linear8(xs, ws, d["bias"], residual=out, out=out, **args)
        assert_within(out, ro, store_error(ro, torch.bfloat16) + eo * (1 + 2 ** -7), "out")
        store.as_strided(out.shape, out.stride(), 1).fill_(float("nan"))
        assert bool(store.isnan().all())
        g, g2 = (rr.block_linear8_backward(d["dout"], x, w) for x, w in ((xs, ws), (d["x"], d["w"])))
        assert torch.equal(g.dx, g2.dx) and torch.equal(g.dw, g2.dw)


@pytest.mark.parametrize("rows", [9, 150, 600])
def test_nan_stays_in_its_row(rr, rows):
    d = make(rr, rows, 300, 400, None, "bf16", True, False)
    want = rr.block_linear8(d["x"], d["w"], d["bias"])
    d["x"].values.view(torch.uint8)[rows - 2, 333] = 0x7F
    d["x"].scales[4, 1] = float("inf")
    got = rr.block_linear8(d["x"], d["w"], d["bias"])
    keep = [r for r in range(rows) if r not in (4, rows - 2)]
    assert torch.equal(got[keep], want[keep])
    assert bool(got[rows - 2].isnan().all()) and not bool(got[4].isfinite().any())


def test_gradients_match_differences(rr):
    """Along directions of what x and w stand for, against central differences in 64 bits."""
    d = make(rr, 40, 48, 272, None, "fp16", True, False)
    _, z = rr.block_linear8(d["x"], d["w"], d["bias"], dtype=torch.float16, act="gelu", save_preact=True)
    got = rr.block_linear8_backward(d["dout"], d["x"], d["w"], z, act="gelu")
    g = torch.Generator(device="cuda").manual_seed(4)
    from tests.block_util import act64
    base = {"x": wide(d["x"]), "w": wide(d["w"]), "bias": d["bias"].double()}
    for key, grad in (("x", got.dx), ("w", got.dw), ("bias", got.db)):
        v = torch.randn(base[key].shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(step):
            p = dict(base, **{key: base[key] + step * v})
            return float((act64(p["x"] @ p["w"].t() + p["bias"], "gelu") * d["dout"].double()).sum())

        along = float((grad.double() * v).sum())
        size = float((grad.double() * v).abs().sum())
        assert abs(along - (loss(1e-5) - loss(-1e-5)) / 2e-5) <= 4 * 2 ** -11 * size, key


def test_graph_and_streams(rr):
    d = make(rr, 260, 256, 192, 2, "bf16", True, True)
    x = normal((260, 192), 3, torch.bfloat16)
    off = torch.tensor([0, 100, 250], dtype=torch.int32, device="cuda")

    def step(stream=None):
        q = rr.block_quantize(x, stream=stream)
        out, z = rr.block_linear8(q, d["w"], d["bias"], act="silu", residual=d["residual"],
                                  offsets=off, save_preact=True, stream=stream)
        g = rr.block_linear8_backward(d["dout"], q, d["w"], z, act="silu", offsets=off, stream=stream)
        return [rr.block_dequantize(q, stream=stream), out, z, g.dx, g.dw, g.db]

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
        x.copy_(torch.randn(260, 192, generator=torch.Generator().manual_seed(seed)))
        off.copy_(torch.tensor([0, 10 + 80 * seed, 260 - seed], dtype=torch.int32))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_two_tokens_of_large_weights(rr):
    """Weights whose rows are past 2^31 bytes behind the first."""
    n, k = 70000, 32768
    w = torch.zeros(n, k, dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.ones(-(-n // 128), k // 128, device="cuda")
    w.view(torch.uint8)[n - 1] = 0x38                         # 1.0
    x = rr.block_quantize(torch.ones(2, k, device="cuda", dtype=torch.bfloat16))
    out = rr.block_linear8(x, rr.Quantized(w, scales, True))
    assert bool((out[:, n - 1] == k).all()) and not bool(out[:, :n - 1].any())
    assert float(e4m3_64(torch.tensor([448.0], dtype=torch.float64))) == 448
    assert not bool(as_operand(x, torch.bfloat16)[1].any())


def odd_scales(q, first):
    """From block ``first`` of the contraction on, scales that are no powers of two."""
    q.scales[..., first:] *= 1.0 + 0.5 * torch.rand(q.scales[..., first:].shape, generator=torch.Generator().manual_seed(1)).cuda()
    return q


FORMS = [  # rows, n, k: dots, one pass, deep tiles and their parts, at any byte and in whole pieces
    (1, 8200, 4112), (1, 700, 4100), (2, 700, 1777), (5, 64, 9), (9, 513, 9000), (12, 8192, 6144), (14, 200, 8208),
    (20, 300, 1001), (24, 1024, 4096), (30, 4112, 1040), (28, 8192, 6160), (40, 512, 2048), (50, 300, 1001), (64, 1000, 4112)]


@pytest.mark.parametrize("rows,n,k", FORMS)
def test_few_rows(rr, rows, n, k):
    d = make(rr, rows, n, k, None, "fp16", True, True, foreign=rows % 2 == 1)
    check_forward(rr, d, None, "silu", torch.float16)


@pytest.mark.parametrize("first", [0, 5, 8, 100])
@pytest.mark.parametrize("rows,n,k", [(130, 260, 1300), (1100, 1000, 1312)])
def test_scales_of_both_kinds(rr, first, rows, n, k):
    """Powers of two up to a block, which the instruction multiplies by, and others behind; in x and
    in w, and for some of the rows only."""
    for which in ("x", "w", "rows"):
        d = make(rr, rows, n, k, None, "bf16", True, False)
        if which == "rows":
            d["x"].scales[rows // 2:rows // 2 + 3, first:first + 2] *= 3.0
        else:
            odd_scales(d[which], first)
        check_forward(rr, d, None, "none", torch.bfloat16)


@pytest.mark.parametrize("rows,n,k", [(4500, 2200, 2064), (2560, 4608, 1040)])
def test_large_tiles(rr, rows, n, k):
    """Tiles of 256 x 256, ragged ones, and a last round cut along the contraction."""
    d = make(rr, rows, n, k, None, "bf16", True, True)
    odd_scales(d["w"], 9)
    check_forward(rr, d, None, "gelu", torch.bfloat16)


def test_large_groups(rr):
    sizes = [2000, 0, 1, 1500, 900]
    off = torch.from_numpy(7 + np.concatenate([[0], np.cumsum(sizes)])).to(torch.int32).cuda()
    d = make(rr, sum(sizes) + 40, 2400, 2064, len(sizes), "bf16", True, False)
    check_forward(rr, d, off, "silu", torch.bfloat16)


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_scales_of_zero(rr, rows):
    """A scale of 0 makes its block 0, whatever its values and the other operand's scale; so do the
    smallest ones there are, to what they are."""
    d = make(rr, rows, 200, 384, None, "bf16", False, False)
    d["x"].scales[:, 1] = 0.0
    d["w"].scales[:, 1] = 2.0 ** 100
    d["x"].scales[0, 0] = 2.0 ** -140
    check_forward(rr, d, None, "none", torch.bfloat16)


def test_many_rows_of_x(rr):
    """Rows whose values are past 2^31 bytes behind the first, and whose results are."""
    rows, k = 70000, 32768
    x = torch.zeros(rows, k, dtype=torch.uint8, device="cuda").view(E4M3)
    x.view(torch.uint8)[rows - 3:] = 0x38                     # 1.0
    scales = torch.full((rows, k // 128), 0.5, device="cuda")
    w = rr.block_quantize(torch.ones(40, k, device="cuda", dtype=torch.bfloat16), square=True)
    out = torch.zeros(rows, 32800, device="cuda", dtype=torch.bfloat16)[:, :40]
    rr.block_linear8(rr.Quantized(x, scales), w, out=out)
    assert bool((out[rows - 3:] == k / 2).all()) and not bool(out[:rows - 3].any())


def test_dispatch_of_8_bit_rows(rr):
    x = rr.block_quantize(normal((50, 258), 2, torch.bfloat16))
    order = rr.expert_sort(torch.randint(-1, 6, (50, 3), generator=torch.Generator().manual_seed(0)).cuda(), 6, 20)
    got = rr.expert_dispatch(x, order.slots, order.sources)
    want = rr.expert_dispatch(rr.block_dequantize(x, torch.float32), order.slots, order.sources)
    assert torch.equal(rr.block_dequantize(got, torch.float32), want)
    odd = rr.block_quantize(normal((50, 257), 2, torch.bfloat16))
    with pytest.raises(ValueError):
        rr.expert_dispatch(odd, order.slots, order.sources)


def test_dispatch_of_every_byte(rr):
    """The bits are moved, not the values: NaN of both signs stay as they are."""
    v = torch.arange(256, dtype=torch.int64).repeat(2).view(2, 256).to(torch.uint8)
    v[1] = v[0].roll(1)
    x = rr.Quantized(v.cuda().view(E4M3), torch.tensor([[1.0, 2.0], [3.0, 4.0]]).cuda())
    order = rr.expert_sort(torch.tensor([[1, 1], [0, 1]]).cuda(), 2)
    got = rr.expert_dispatch(x, order.slots, order.sources)
    rows = (order.sources // 2).long()
    assert torch.equal(got.values.view(torch.uint8), x.values.view(torch.uint8)[rows])
    assert torch.equal(got.scales, x.scales[rows])
    across = rr.Quantized(v.cuda().t().contiguous().t().view(E4M3), x.scales)
    with pytest.raises(ValueError):
        rr.expert_dispatch(across, order.slots, order.sources)


@pytest.mark.parametrize("rows", [1, 3, 20, 60, 300])
def test_scales_whose_product_is_past_the_end(rr, rows):
    """The last of an odd number of blocks: infinity times a sum, not NaN."""
    k = 384
    one = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda").view(E4M3)  # noqa: E731
    xs, ws = torch.ones(rows, 3, device="cuda"), torch.ones(2, 3, device="cuda")
    xs[:, 2] = ws[0, 2] = 1.5 * 2.0 ** 100
    out = rr.block_linear8(rr.Quantized(one(rows, k), xs), rr.Quantized(one(200, k), ws, True))
    assert bool((out[:, :128] == float("inf")).all()) and bool((out[:, 128:] > 1e32).all())


def test_two_streams_at_once(rr):
    """Calls on two streams, whose scratch memory is each their own."""
    d = [make(rr, 600, 768, 1040, 2, "bf16", True, True, seed=s) for s in (0, 1)]
    e = [make(rr, 24, 1000, 4112, None, "bf16", True, True, seed=s) for s in (0, 1)]
    off = torch.tensor([5, 200, 590], dtype=torch.int32, device="cuda")

    def step(s, stream=None):
        z = d[s]["z"]
        g = rr.block_linear8_backward(d[s]["dout"], d[s]["x"], d[s]["w"], z, act="gelu", offsets=off, stream=stream)
        return [rr.block_linear8(d[s]["x"], d[s]["w"], d[s]["bias"], act="gelu", offsets=off, stream=stream),
                rr.block_linear8(e[s]["x"], e[s]["w"], e[s]["bias"], stream=stream), g.dx, g.dw, g.db]

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [step(i % 2, streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


@pytest.mark.parametrize("rows,n,k", [(2560, 4608, 1040), (4500, 2201, 2064)])
def test_large_tiles_with_a_residual_anywhere(rr, rows, n, k):
    """At any element, rows any distance apart, and as out itself."""
    d = make(rr, rows, n, k, None, "bf16", True, True)
    want = rr.block_linear8(d["x"], d["w"], d["bias"], act="silu", residual=d["residual"])
    for ahead, ld in ((1, n), (3, n + 5), (8, n + 56)):
        flat = torch.full((ahead + rows * ld,), float("nan"), device="cuda", dtype=torch.bfloat16)
        r = flat[ahead:].view(rows, ld)[:, :n]
        r.copy_(d["residual"])
        assert torch.equal(rr.block_linear8(d["x"], d["w"], d["bias"], act="silu", residual=r), want)
        assert torch.equal(rr.block_linear8(d["x"], d["w"], d["bias"], act="silu", residual=r, out=r), want)
        assert bool(flat[:ahead].isnan().all()) and bool(flat[ahead:].view(rows, ld)[:, n:].isnan().all())


@pytest.mark.parametrize("rows,n", [(40, 6000), (70, 200), (600, 700), (2560, 4608)])
@pytest.mark.parametrize("k", [16, 20, 300, 1032, 1292, 2060])
def test_rows_of_words(rr, rows, n, k):
    """Rows that end inside 16 bytes and begin at any word, NaN before, between and behind them, give
    what copies in whole pieces give; and scales that are no powers of two."""
    d = make(rr, rows, n, k, None, "bf16", True, False)
    for foreign in (False, True):
        if foreign:
            odd_scales(d["w"], 0)
        got = []
        for ahead, ld in ((0, (k + 15) // 16 * 16 + 16), (4, k + 4), (12, k + 12), (0, k)):
            ops = []
            for q in (d["x"], d["w"]):
                r = q.values.shape[0]
                flat = torch.full((ahead + r * ld,), 0x7F, device="cuda", dtype=torch.uint8).view(E4M3)
                v = flat[ahead:].view(r, ld)[:, :k]
                v.copy_(q.values)
                ops.append(rr.Quantized(v, q.scales, q.square))
            got.append(rr.block_linear8(*ops, d["bias"]))
        ro, _, eo, _ = linear64(d["x"], d["w"], d["bias"], None, "none", None)
        assert_within(got[0], ro, store_error(ro, torch.bfloat16) + eo * (1 + 2 ** -7), "out")
        assert all(torch.equal(g, got[0]) for g in got)


@pytest.mark.parametrize("rows,n,k", [(70, 200, 1003), (600, 700, 1011), (2560, 4608, 1007)])
def test_odd_rows_that_end_a_byte_before_a_word(rr, rows, n, k):
    d = make(rr, rows, n, k, None, "fp16", True, False, foreign=True)
    check_forward(rr, d, None, "none", torch.float16)
