"""8-bit rows on their way between experts, and what sums of 8-bit products keep."""
import pytest
import torch

from tests.block8_util import E4M3, gated_dz64, gradients64, linear64, wide
from tests.block_util import U, assert_within, store_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_allreduce_amd
    ring_allreduce_amd.init()
    return ring_allreduce_amd


def normal(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def sorted_rows(rr, tokens, experts, capacity, seed=0):
    """Two experts a token, a few masked out, with room for more rows than there are."""
    ids = torch.randint(-1, experts, (tokens, 2), generator=torch.Generator().manual_seed(seed)).cuda()
    return rr.expert_sort(ids, experts, capacity)


# ------------------------------------------- rows without a source, and their products --

@pytest.mark.parametrize("rows_of", [(200, 6, 90), (5, 3, 16), (0, 2, 8), (3000, 4, 2048)], ids=str)
def test_rows_without_a_source_have_scale_one(rr, rows_of):
    """As block_quantize gives rows of zeros: a scale of 0 would cost the products of the rows beside
    them the instruction's own scales."""
    tokens, experts, capacity = rows_of
    order = sorted_rows(rr, tokens, experts, capacity)
    x = rr.block_quantize(normal((tokens, 264), 1))
    for stream in (None, torch.cuda.current_stream()):
        got = rr.expert_dispatch(x, order.slots, order.sources, stream=stream)
        none = order.sources < 0
        assert bool(none.any())
        assert bool((got.scales[none] == 1).all()) and not bool(got.values.view(torch.uint8)[none].any())
        there = (order.sources[~none] // 2).long()
        assert torch.equal(got.scales[~none], x.scales[there])
        assert torch.equal(got.values.view(torch.uint8)[~none], x.values.view(torch.uint8)[there])


@pytest.mark.parametrize("tokens,capacity,n", [(40, 16, 200), (300, 130, 320), (3000, 2048, 1152)])
def test_products_beside_rows_without_a_source(rr, tokens, capacity, n):
    """Are to the bit what they are beside rows that all have one."""
    experts, k = 4, 1024
    order = sorted_rows(rr, tokens, experts, capacity)
    rows = rr.expert_dispatch(rr.block_quantize(normal((tokens, k), 2)), order.slots, order.sources)
    there = order.sources >= 0
    assert not bool(there.all())
    filled = rr.Quantized(rows.values.clone(), rows.scales.clone())
    other = int(torch.nonzero(there)[0])
    filled.values.view(torch.uint8)[~there] = rows.values.view(torch.uint8)[other]
    filled.scales[~there] = rows.scales[other]
    w = rr.block_quantize(normal((experts, 2, n, k), 3, k ** -0.5), square=True)
    first = rr.Quantized(w.values[:, 0].contiguous(), w.scales[:, 0].contiguous(), True)
    for offsets in (None, order.offsets):
        a, b = (rr.block_gated(r, w, offsets=offsets) for r in (rows, filled))
        assert torch.equal(a[there], b[there]) and not bool(a[~there].any())
        a, b = (rr.block_linear8(r, first, offsets=offsets) for r in (rows, filled))
        assert torch.equal(a[there], b[there]) and not bool(a[~there].any())


def test_dispatch_of_one_row_of_a_buffer_of_odd_rows(rr):
    x = rr.block_quantize(normal((3, 258), 4))
    wide = torch.zeros(3, 261, dtype=torch.uint8, device="cuda")
    wide[:, 2:260] = x.values.view(torch.uint8)
    order = rr.expert_sort(torch.tensor([[1, 0]], device="cuda"), 2, 2)
    for r in range(0, 3, 2):
        one = rr.Quantized(wide.view(x.values.dtype)[r:r + 1, 2:260], x.scales[r:r + 1])
        got = rr.expert_dispatch(one, order.slots, order.sources)
        there = order.sources >= 0
        assert torch.equal(got.values.view(torch.uint8)[there], x.values.view(torch.uint8)[[r, r]])
        assert torch.equal(got.scales[there], x.scales[[r, r]])


@pytest.mark.parametrize("ranks,tokens,k", [(2, 30, 258), (4, 200, 1024), (8, 60, 264)])
def test_rows_through_the_alltoall(rr, ranks, tokens, k):
    """Values as pairs and scales go to the ranks of their experts, of which each makes the products that
    one rank with all rows would, and the results come back to their tokens."""
    n, capacity = 96, (2 * tokens // ranks + 8) // 8 * 8
    ids = [torch.rand(tokens, ranks, generator=torch.Generator().manual_seed(r)).topk(2).indices.cuda()
           for r in range(ranks)]
    orders = [rr.expert_sort(i, ranks, capacity) for i in ids]
    sent = [rr.expert_dispatch(rr.block_quantize(normal((tokens, k), 20 + r)), o.slots, o.sources)
            for r, o in enumerate(orders)]
    w = rr.block_quantize(normal((ranks, 2, n, k), 40, k ** -0.5), square=True)
    values = rr.alltoall([s.values.view(torch.bfloat16) for s in sent])
    scales = rr.alltoall([s.scales for s in sent])
    made = []
    for e in range(ranks):
        rows = rr.Quantized(values[e].view(E4M3), scales[e])
        block = slice(e * capacity, (e + 1) * capacity)
        want = rr.Quantized(torch.cat([s.values.view(torch.uint8)[block] for s in sent]).view(E4M3),
                            torch.cat([s.scales[block] for s in sent]))
        assert torch.equal(rows.values.view(torch.uint8), want.values.view(torch.uint8))
        assert torch.equal(rows.scales, want.scales)
        one = rr.Quantized(w.values[e], w.scales[e], True)
        made.append(rr.block_gated(rows, one))
        assert torch.equal(made[-1], rr.block_gated(want, one))
    for r, back in enumerate(rr.alltoall(made)):
        rr.check_kernel_error()
        out = rr.expert_combine(back, orders[r].slots)
        slots = orders[r].slots.long()
        terms = torch.where((slots >= 0)[..., None], back.double()[slots.clamp(min=0)], 0.0)
        want, error = terms.sum(1), 2 * U * terms.abs().sum(1)
        assert_within(out, want, store_error(want, torch.bfloat16) + error * (1 + 2 ** -7), "out")


# ------------------------------------------------------------------ few rows --

@pytest.mark.parametrize("rows", [17, 32])
@pytest.mark.parametrize("n,k", [(130, 1024), (130, 1025), (2100, 1009), (4096, 512), (4097, 512), (4100, 4096),
                                 (3000, 4112)])
def test_17_to_32_rows(rr, rows, n, k):
    """Both widths of a workgroup of the one-pass form, on either side of where one takes over."""
    x = rr.block_quantize(normal((rows, k), 8))
    w = rr.block_quantize(normal((n, k), 9, k ** -0.5), square=True)
    got = rr.block_linear8(x, w)
    want, _, error, _ = linear64(x, w, None, None, "none", None)
    assert_within(got, want, store_error(want, torch.bfloat16) + error * (1 + 2 ** -7), "out")


# --------------------------------------------------------- what the sums keep --

SIZES = [(1, 14), (1, 2800), (5, 70), (20, 210), (40, 700), (200, 140), (600, 700), (1024, 4200), (2560, 4620)]


@pytest.mark.parametrize("foreign", [False, True])
@pytest.mark.parametrize("rows,n", SIZES)
def test_a_small_product_beside_a_large_one(rr, rows, n, foreign):
    """Beside a product of 2^16 among the same eight neighbours, which another eight cancel, one of
    2^0 to 2^6 is there to the bit or, below 2^3, cut away; among other eight it is always there.  Of one row
    all are.  Scales by the instruction (four blocks of powers of two) and on top of its sums."""
    k = 512
    x = torch.zeros(rows, k, device="cuda")
    x[:, 0] = x[:, 64] = 256.0
    x[:, 1] = x[:, 72] = 2.0
    w = torch.zeros(14, k, device="cuda")
    w[:, 0], w[:, 64] = 256.0, -256.0
    for j in range(14):
        w[j, 1 if j < 7 else 72] = 2.0 ** (j % 7 - 1)
    w = w.repeat(n // 14, 1)
    xs, ws = torch.ones(rows, 4, device="cuda"), torch.ones(-(-n // 128), 4, device="cuda")
    if foreign:
        xs *= 3.0
    out = rr.block_linear8(rr.Quantized(x.to(E4M3), xs), rr.Quantized(w.to(E4M3), ws, True)).float()
    exact = torch.tensor([2.0 ** (j % 7) for j in range(14)], device="cuda").repeat(n // 14) * (3 if foreign else 1)
    keep = torch.tensor([j >= 3 or rows == 1 for j in range(14)], device="cuda").repeat(n // 14)
    assert torch.equal(out[:, keep], exact[keep].expand(rows, -1))
    assert bool(((out == exact) | (out == 0)).all())


@pytest.mark.parametrize("foreign", [False, True])
@pytest.mark.parametrize("rows,n", SIZES)
def test_sums_of_blocks_are_kept_in_32_bits(rr, rows, n, foreign):
    """2^23 from one block of 128, a small sum from a later one and -2^23 from another: what is left is
    the small one but for a whole step of 32 bits at the large one for each of the three."""
    k, f = 1024, 15.0 if foreign else 1.0
    small = [4.0, 16.0, 64.0, 256.0, 448.0, 32.0, 8.0]
    x = torch.ones(rows, k, device="cuda")
    w = torch.zeros(7, k, device="cuda")
    x[:, :128] = x[:, 768:896] = 256.0
    w[:, :128], w[:, 768:896] = 256.0, -256.0
    w[:, 400] = torch.tensor(small, device="cuda")
    w = w.repeat(n // 7, 1)
    xs, ws = torch.ones(rows, 8, device="cuda"), torch.ones(-(-n // 128), 8, device="cuda")
    if foreign:
        xs, ws = xs * 3.0, ws * 5.0
    out = rr.block_linear8(rr.Quantized(x.to(E4M3), xs), rr.Quantized(w.to(E4M3), ws, True)).float()
    exact = torch.tensor(small, device="cuda").repeat(n // 7) * f
    bound = 3 * 2.0 ** -23 * 2.0 ** 23 * f
    assert bool(((out - exact).abs() <= bound + 2.0 ** -8 * (exact + bound)).all())


@pytest.mark.parametrize("eight", [False, True], ids=["16", "8"])
@pytest.mark.parametrize("rows,n,k,groups", [(703, 9000, 3, 2), (2560, 2304, 40, 1), (4500, 2200, 2064, 1), (300, 300, 40, 3)])
def test_the_product_does_not_depend_on_how_z_is_kept(rr, rows, n, k, groups, eight):
    """In fp16, where the compiler may round a product and its 16-bit value in one step."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, k, generator=g, device="cuda").half()
    w = (torch.randn(groups, 2, n, k, generator=g, device="cuda") * k ** -0.5).half()
    offsets = torch.tensor([rows * (i + 1) // (groups + 2) for i in range(groups + 1)], dtype=torch.int32).cuda()
    if eight:
        x, w = rr.block_quantize(x), rr.block_quantize(w, square=True)
    for act in ("none", "sigmoid", "gelu"):
        args = dict(act=act, offsets=offsets, dtype=torch.float16)
        want = rr.block_gated(x, w, **args)
        for kept in (True, "e4m3"):
            assert torch.equal(rr.block_gated(x, w, save_preact=kept, **args)[0], want), (act, kept)


# ------------------------------------------- gradients at the ends of 16-bit types --

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("size", [3e4, 1e-2, 1e-4, 1e-5, 1e-7])
@pytest.mark.parametrize("which", ["x", "w"])
def test_gradients_of_large_and_small_operands(rr, dtype, size, which):
    """8-bit operands become dtype on their way: in bf16 exactly, in fp16 where it has what they stand
    for, else the multiple of 2^-24 next to it or, past the end, 65504.  The forward pass takes any."""
    rows, n, k = 150, 70, 200
    x = torch.randn(rows, k, generator=torch.Generator().manual_seed(1)).cuda() * (size if which == "x" else 1.0)
    w = torch.randn(2, n, k, generator=torch.Generator().manual_seed(2)).cuda() * (size if which == "w" else 1.0)
    x, w = rr.block_quantize(x), rr.block_quantize(w, square=True)
    first = rr.Quantized(w.values[0].contiguous(), w.scales[0].contiguous(), True)
    dout = normal((rows, n), 3).to(dtype)
    end = torch.finfo(dtype).max

    def check(got, dz, edz, e32, *operands):
        # as_operand's bound is for what is within the type's ends: past them the end itself is meant
        xv, wv = (q if bool((wide(q).abs() <= end).all()) else wide(q).clamp(-end, end) for q in operands)
        (dx, edx), (dw, edw), _ = gradients64(dz, edz, xv, wv, None, dtype, e32)
        assert_within(got.dw, dw, edw + U * dw.abs(), "dw")
        inside = dx.abs() + edx < end                  # fp16 results past the end are infinite
        assert_within(torch.where(inside, got.dx.double(), 0.0), torch.where(inside, dx, 0.0),
                      store_error(dx, dtype) + edx * (1 + 2 ** -7), "dx")

    zero = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    check(rr.block_linear8_backward(dout, x, first, dw_dtype=torch.float32), dout.double(), zero, zero, x, first)
    z = normal((rows, 2 * n), 4).to(dtype)
    dz, e32, edz = gated_dz64(dout, z.double(), "silu", dtype)
    check(rr.block_gated_backward(dout, x, w, z, dw_dtype=torch.float32), dz, edz, e32, x, w)
    out = rr.block_linear8(x, first, dtype=torch.bfloat16)
    want, _, error, _ = linear64(x, first, None, None, "none", None)
    assert_within(out, want, store_error(want, torch.bfloat16) + (error + 8 * U) * (1 + 2 ** -7), "out")


# ------------------------------------------------------------------- refusals --

def test_weights_of_no_matrices(rr):
    x = normal((4, 8), 5)
    for lead in ((0,), (1,), (3,), (2, 0), (2, 1), (2, 3)):
        w = torch.zeros(*lead, 6, 8, device="cuda", dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="two matrices"):
            rr.block_gated(x, w)
        with pytest.raises(ValueError, match="two matrices"):
            rr.block_gated_backward(x[:, :6], x, w, torch.zeros(4, 12, device="cuda", dtype=torch.bfloat16))


def test_what_is_no_tensor(rr):
    q = rr.block_quantize(normal((4, 8), 6))
    for call in (lambda: rr.block_quantize(None), lambda: rr.block_quantize([1.0]),
                 lambda: rr.block_dequantize(q, out=5)):
        with pytest.raises(ValueError):
            call()
