"""A block's operators at the sizes where another kernel or another way through it is taken: large
tiles, the last round of tiles cut along the contraction, operands that have to be copied, rows
of every register layout, many rows a workgroup, k beyond one batch of rows."""
import numpy as np
import pytest
import torch

from tests.block_util import DTYPES, U, assert_within, store_error, strided
from tests.test_gpu_block_linear import check_backward, check_forward, make
from tests.test_gpu_block_norm import EPS, STEPS, backward64, forward64, own_args, wide
from tests.test_gpu_block_norm import make as make_norm
from tests.test_gpu_expert import check_order, gathered64, make_ids, order_of, setup, spread64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_allreduce_amd
    return ring_allreduce_amd


@pytest.mark.parametrize("rows,n,k,dtype,act", [
    (4090, 4088, 520, "bf16", "silu"),       # one round of 256 x 256 tiles, edges in both directions
    (4350, 4090, 2048, "bf16", "none"),      # a second round of few: cut along the contraction
    (2050, 8200, 1032, "fp16", "relu"), (8200, 2056, 1040, "bf16", "gelu")])
def test_large_tiles(rr, rows, n, k, dtype, act):
    d = make(rows, n, k, None, dtype, True, True)
    check_forward(rr, d, None, act, DTYPES[dtype])
    check_backward(rr, d, None, act, DTYPES[dtype])


@pytest.mark.parametrize("sizes,before,after,n,k", [
    ([1500, 0, 2300, 700], 3, 90, 4096, 1032), ([5000, 3300], 0, 0, 2048, 2048),
    ([100] * 80, 1, 0, 1032, 520), ([4000, 4000], 0, 200, 2056, 2056)], ids=lambda v: str(v)[:24])
def test_large_groups(rr, sizes, before, after, n, k):
    rows = before + sum(sizes) + after
    off = torch.from_numpy(before + np.concatenate([[0], np.cumsum(sizes)])).to(torch.int32).cuda()
    d = make(rows, n, k, len(sizes), "bf16", True, True)
    check_forward(rr, d, off, "silu", torch.bfloat16)
    check_backward(rr, d, off, "silu", torch.bfloat16)


@pytest.mark.parametrize("act", ["none", "silu"])
def test_operands_to_copy(rr, act):
    """Odd widths, rows at odd elements and groups at odd distances, past which there is NaN."""
    rows, n, k = 700, 391, 453
    off = torch.tensor([0, 300, 333, 700], dtype=torch.int32, device="cuda")
    d = make(rows, n, k, 3, "bf16", True, False)
    want = rr.block_linear(d["x"], d["w"], d["bias"], act=act, offsets=off)
    grads = rr.block_linear_backward(d["dout"], d["x"], d["w"], d["z"], act=act, offsets=off)
    store = torch.full((3, n * (k + 4) + 7), float("nan"), dtype=torch.bfloat16, device="cuda")
    w = store.as_strided((3, n, k), (n * (k + 4) + 7, k + 4, 1), 0)
    w.copy_(d["w"])
    d2 = dict(d, x=strided(d["x"], 5, offset=3)[0], w=w, dout=strided(d["dout"], 1, offset=1)[0],
              z=strided(d["z"], 3)[0])
    assert torch.equal(rr.block_linear(d2["x"], w, d["bias"], act=act, offsets=off), want)
    again = rr.block_linear_backward(d2["dout"], d2["x"], w, d2["z"], act=act, offsets=off)
    for name in ("dx", "dw", "db"):
        assert torch.equal(getattr(again, name), getattr(grads, name)), name
    check_forward(rr, d2, off, act, torch.bfloat16)
    check_backward(rr, d2, off, act, torch.bfloat16)


def test_few_rows_long_contraction(rr):
    """The one-pass form cut along the contraction, and at the rows where it ends."""
    for rows in (1, 16, 17, 33, 64, 65):
        for n, k in ((40, 8192), (520, 4104), (33, 2051)):
            d = make(rows, n, k, None, "bf16", True, True)
            check_forward(rr, d, None, "silu", torch.bfloat16)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5])
def test_one_to_four_rows(rr, dtype, rows):
    """Dots: widths of less than a vector, of parts of a wave's stretch, of several; rows at odd
    elements."""
    for n, k in ((1, 3), (5, 8), (2051, 519), (2048, 4096), (70, 2055), (9, 6152)):
        d = make(rows, n, k, None, dtype, True, True)
        check_forward(rr, d, None, "gelu", DTYPES[dtype])
        far = dict(d, x=strided(d["x"], 3, offset=1)[0], w=strided(d["w"], 1, offset=5)[0])
        check_forward(rr, far, None, "silu", DTYPES[dtype])


def test_far_rows(rr):
    """Rows beyond 2^31 elements and 2^32 bytes: the last ones come out as they do alone."""
    tokens, hidden, last = 280_000, 8192, 279_000
    x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    x[last:].normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    x[:last] = 1.0
    w = torch.randn(hidden, device="cuda").bfloat16()
    h, y = rr.block_norm(x, post_norm=False, pre_weight=w)
    h2, y2 = rr.block_norm(x[last:].contiguous(), post_norm=False, pre_weight=w)
    assert torch.equal(h[last:], h2) and torch.equal(y[last:], y2)
    del h, h2, y2
    d = rr.block_norm_backward(None, y, x, post_norm=False, pre_weight=w, need=("dx",))
    d2 = rr.block_norm_backward(None, y[last:].contiguous(), x[last:].contiguous(), post_norm=False,
                                pre_weight=w, need=("dx",))
    assert torch.equal(d.dx[last:], d2.dx)
    del d, d2, y
    slots = torch.arange(tokens, dtype=torch.int32, device="cuda").flip(0).reshape(-1, 1).contiguous()
    sources = slots.reshape(-1).clone()
    rows = rr.expert_dispatch(x, slots, sources)
    assert torch.equal(rows[:tokens - last].flip(0), x[last:])
    back = rr.expert_combine(rows, slots)
    assert torch.equal(back[last:], x[last:]) and torch.equal(back[:5], x[:5])
    del rows, back
    wide = torch.randn(64, hidden, device="cuda").bfloat16()
    out = rr.block_linear(x, wide)
    few = rr.block_linear(x[last:].contiguous(), wide)
    # another tile or cut of the contraction adds in another order
    size = x[last:].float().abs() @ wide.float().abs().t()
    assert bool(((out[last:].double() - few.double()).abs() <= 2 * store_error(few.double(), torch.bfloat16) +
                 2 * (hidden + 2) * U * size.double()).all())


NORM = [  # tokens, hidden, gate, act, post, pre, weights
    (5000, 520, "element", "silu", True, True, "same"), (9000, 72, "channel", "sigmoid", True, True, "fp32"),
    (3000, 1030, "channel", "silu", True, True, "same"), (1500, 4104, "element", "sigmoid", True, True, "same"),
    (700, 8200, "channel", "none", True, True, "same"), (600, 12296, "channel", "silu", True, True, "fp32"),
    (40, 16383, "element", "none", True, True, "same"), (300, 9, "element", "silu", False, True, "none"),
    (11, 32767, "none", "none", True, False, "none")]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm_layouts(rr, dtype, case):
    tokens, hidden, gate, act, post, pre, weights = case
    d = make_norm(tokens, hidden, dtype, gate, weights, 2)
    c, args = own_args(d, act, post, pre)
    dt = DTYPES[dtype]
    h, y = rr.block_norm(c["x"], c["branch"], **args)
    w = wide(d)
    rh, sh, ry, sy = forward64(w, act, post, pre)
    assert_within(h.cpu(), rh, store_error(rh, dt) + STEPS * U * sh, "h")
    if pre:
        assert_within(y.cpu(), ry, store_error(ry, dt) + STEPS * U * sy, "y")
    got = rr.block_norm_backward(c["dh"], c["dy"] if pre else None, c["h"], c["branch"], **args)
    ref, size = backward64(w, act, post, pre)
    for name in ("dx", "dbranch", "dgate", "dpost_weight", "dpre_weight"):
        g = getattr(got, name)
        if g is None:
            assert name not in ref or weights == "none" and "weight" in name, name
            continue
        bound = (STEPS + tokens) * U * size[name] if g.dim() == 1 else \
            store_error(ref[name], dt) + STEPS * U * size[name]
        assert_within(g.cpu(), ref[name], bound, name)


def test_norm_without_what_is_optional(rr):
    """No gradient by the stream, no branch, no norm: what is absent counts as zero."""
    d = make_norm(50, 1000, "bf16", "none", "same")
    c, args = own_args(d, "none", True, True)
    zero = torch.zeros_like(c["dh"])
    a = rr.block_norm_backward(None, c["dy"], c["h"], c["branch"], **args)
    b = rr.block_norm_backward(zero, c["dy"], c["h"], c["branch"], **args)
    for name in ("dx", "dbranch", "dpost_weight", "dpre_weight"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    only = rr.block_norm_backward(c["dh"], None, None, None, post_norm=False, pre_norm=False,
                                  residual_scale=0.5)
    assert torch.equal(only.dx, (c["dh"].float() * 0.5).bfloat16())
    h, y = rr.block_norm(c["x"], None, post_norm=False, pre_norm=False, residual_scale=2.0, eps=EPS)
    assert y is None and torch.equal(h, (c["x"].float() * 2).bfloat16())
    c["branch"][7] = float("inf")
    h, _ = rr.block_norm(c["x"], None, post_norm=False, pre_norm=False)
    assert torch.equal(h, c["x"])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("shape", [(300, 1030, 12, 20, 0, "masked"), (90, 4104, 17, 40, 5, "any"),
                                   (500, 40, 3, 16, 300, "masked"), (70, 3, 2, 6, 90, "any")], ids=str)
def test_moves(rr, dtype, shape):
    """More rows a token than are summed at a time; many unused rows."""
    tokens, hidden, k = shape[:3]
    slots, sources, ds, dq, x, rows, weights = setup(rr, *shape, dtype)
    assert torch.equal(rr.expert_dispatch(x.cuda(), ds, dq).cpu().double(), spread64(x, sources, k))
    unused = torch.ones(len(rows), dtype=torch.bool)
    unused[torch.from_numpy(slots[slots >= 0])] = False
    rows[unused] = float("nan")                     # rows without a pair do not count
    got = rr.expert_combine(rows.cuda(), ds, weights.cuda()).cpu()
    terms = gathered64(rows, slots) * weights[..., None].double()
    assert_within(got, terms.sum(1), store_error(terms.sum(1), DTYPES[dtype]) +
                  2 * k * U * terms.abs().sum(1), "out")
    drows, dweights = rr.expert_combine_backward(x.cuda(), rows.cuda(), ds, dq, weights.cuda())
    ref = spread64(x, sources, k, weights)
    assert_within(drows.cpu(), ref, store_error(ref, DTYPES[dtype]) + U * ref.abs(), "drows")
    terms = gathered64(rows, slots) * x[:, None].double()
    steps = -(-hidden // 64) + 8 + 10
    assert_within(dweights.cpu(), terms.sum(2), steps * U * terms.abs().sum(2), "dweights")


def test_no_rows(rr):
    """Nothing to move: every pair without a slot, and no rows at all."""
    x = torch.randn(5, 72, device="cuda").bfloat16()
    slots = torch.full((5, 3), -1, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert rr.expert_dispatch(x, slots, none).shape == (0, 72)
    empty = torch.empty(0, 72, dtype=torch.bfloat16, device="cuda")
    assert not bool(rr.expert_combine(empty, slots).any())
    drows, dweights = rr.expert_combine_backward(x, empty, slots, none)
    assert drows.shape == (0, 72) and not bool(dweights.any())


@pytest.mark.parametrize("tokens,k,experts,capacity,kind", [
    (8193, 1, 1024, 9, "any"), (70000, 4, 256, 1200, "masked"), (300000, 1, 3, 0, "masked"),
    (40000, 2, 1024, 0, "one"), (2048, 4, 512, 0, "masked"), (2049, 4, 512, 17, "any")])
def test_sort_sizes(rr, tokens, k, experts, capacity, kind):
    ids = make_ids(tokens, k, experts, kind, tokens)
    check_order(rr.expert_sort(torch.from_numpy(ids).cuda(), experts, capacity),
                order_of(ids, experts, capacity))


def test_binding_refuses(rr):
    """Wrong shapes, types, layouts and places of GPU tensors, one argument at a time."""
    x = torch.zeros(6, 16, device="cuda").bfloat16()
    w, b = torch.zeros(8, 16, device="cuda").bfloat16(), torch.zeros(8, device="cuda").bfloat16()
    i = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    q = torch.zeros(12, dtype=torch.int32, device="cuda")
    values = [
        lambda: rr.expert_sort(i, 4, -1), lambda: rr.expert_dispatch(x, i[:5], q),
        lambda: rr.expert_dispatch(x, i, q.cpu()), lambda: rr.expert_dispatch(x.t(), i, q),
        lambda: rr.expert_combine(x, i, torch.zeros(6, 3, device="cuda")),
        lambda: rr.expert_combine_backward(x, x, i, q), lambda: rr.expert_combine(x, i[:, :1].expand(6, 2)),
        lambda: rr.block_norm(x, x[:5]), lambda: rr.block_norm(x, x, post_weight=x[0, :8].contiguous()),
        lambda: rr.block_norm(x, x, gate_act="silu"), lambda: rr.block_norm(x, x, gate=x[:3]),
        lambda: rr.block_norm(x, x, pre_norm=False, pre_weight=x[0].clone()),
        lambda: rr.block_norm(x), lambda: rr.block_norm(x, x.cpu()),
        lambda: rr.block_norm_backward(x, None, x, x), lambda: rr.block_norm_backward(x, x, None, x),
        lambda: rr.block_linear(x, w[:, :8]), lambda: rr.block_linear(x, w, b[:7]),
        lambda: rr.block_linear(x, w, b.cpu()), lambda: rr.block_linear(x, w, act="sigmoid"),
        lambda: rr.block_linear(x, w, residual=x), lambda: rr.block_linear(x, w, offsets=q[:3]),
        lambda: rr.block_linear(x, torch.zeros(4, 8, 16, device="cuda").bfloat16()),
        lambda: rr.block_linear_backward(x, x, w), lambda: rr.block_linear_backward(x[:, :8], x, w, act="relu")]
    types = [
        lambda: rr.expert_sort(i.to(torch.int16), 4), lambda: rr.expert_dispatch(x, i.long(), q),
        lambda: rr.expert_combine(x, i, torch.zeros(6, 2, device="cuda").bfloat16()),
        lambda: rr.block_norm(x, x.float()), lambda: rr.block_norm(x, x, post_weight=x[0].half()),
        lambda: rr.block_linear(x, w.half()), lambda: rr.block_linear(x, w, b.float()),
        lambda: rr.block_linear(x, w, offsets=q[:2].long()),
        lambda: rr.block_linear_backward(x[:, :8], x, w, dw_dtype=torch.float16)]
    for call in values:
        with pytest.raises((ValueError, rr.RRError)):
            call()
    for call in types:
        with pytest.raises(TypeError):
            call()
    with pytest.raises(rr.RRError):
        rr.expert_sort(i, 2000)
    with pytest.raises(rr.RRError):
        rr.block_norm(x, x, eps=-1.0)


def test_unusual_forms_give_the_same(rr):
    """Given outputs, another stream and strides: the same bits as the usual call."""
    d = make(90, 136, 72, None, "bf16", True, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = rr.block_linear(d["x"], d["w"], d["bias"], act="silu", residual=d["residual"])
    b = rr.block_linear(d["x"], d["w"], d["bias"], act="silu", residual=d["residual"], stream=side)
    c = rr.block_linear(d["x"], d["w"], d["bias"], act="silu", residual=d["residual"],
                        out=torch.empty_like(a))
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    one = rr.block_norm_backward(d["dout"], d["dout"], d["z"], d["residual"], need=("dbranch", "dx"))
    two = rr.block_norm_backward(d["dout"], d["dout"], d["z"], d["residual"], stream=side)
    side.synchronize()
    assert torch.equal(one.dx, two.dx) and torch.equal(one.dbranch, two.dbranch)
    assert one.dgate is None and two.dpost_weight is None


@pytest.mark.parametrize("pairs", [1024, 1025, 2049, 4095, 4097, 8192, 8193, 16385, 32768, 32769, 65537, 262144, 262145])
@pytest.mark.parametrize("experts,capacity", [(7, 0), (256, 90), (1024, 0)])
def test_sort_at_the_edges_of_its_forms(rr, pairs, experts, capacity):
    ids = make_ids(pairs, 1, experts, "masked", pairs + experts)
    check_order(rr.expert_sort(torch.from_numpy(ids).cuda(), experts, capacity),
                order_of(ids, experts, capacity))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gelu_of_single_values(rr, dtype):
    """x w^T with k = 1 and w = 1 is x itself, so this is the activation and its slope alone.
    What lies beyond z is off by the rounding of z^2 / 2 (two steps of 2^-24 of at most 18),
    the exponential's and the fit's, together 4e-6 of it."""
    dt = DTYPES[dtype]
    z = torch.cat([torch.linspace(-6, 6, 24001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 19.0, 21.0, 1e4, 6e4])])
    x = z.to(dt).cuda()[:, None]
    one = torch.ones(1, 1, dtype=dt, device="cuda")
    out, kept = rr.block_linear(x, one, act="gelu", save_preact=True)
    assert torch.equal(kept, x)
    v = x.double()
    tail = 0.5 * torch.special.erfc(v.abs() * 0.5 ** 0.5)
    want = v.clamp(min=0) - v.abs() * tail
    half = torch.finfo(dt).eps / 2
    least = torch.finfo(dt).smallest_normal * half          # half a step of the smallest values
    assert bool(((out.double() - want).abs() <= 4e-6 * v.abs() * tail + (half + 2.0 ** -23) * want.abs() + least).all())
    dz = rr.block_linear_backward(torch.ones_like(x), x, one, x, act="gelu", need_dw=False, need_db=False).dx
    density = torch.exp(-0.5 * v * v) * 0.3989422804014327
    slope = torch.where(v > 0, 1 - tail, tail) + v * density
    bound = 4e-6 * (tail + v.abs() * density) + (2 * half + 2.0 ** -22) * slope.abs() + 2 * least
    assert bool(((dz.double() - slope).abs() <= bound).all())
    far = torch.tensor([[float("inf")], [float("nan")]], dtype=dt, device="cuda")
    got = rr.block_linear(far, one, act="gelu")
    assert float(got[0]) == float("inf") and bool(got[1].isnan())


@pytest.mark.parametrize("rows,n,k,groups", [
    (16, 8192, 264, 1), (5, 8208, 264, 1), (33, 4096, 520, 1), (32, 4112, 520, 1), (7, 1000, 8200, 1),
    (3, 1000, 8192, 1), (40, 1040, 72, 5), (9, 530, 1001, 1), (64, 530, 1001, 1), (48, 5000, 999, 2)])
def test_few_rows_at_the_edges_of_the_forms(rr, rows, n, k, groups):
    d = make(rows, n, k, groups if groups > 1 else None, "bf16", True, True)
    check_forward(rr, d, None, "silu", torch.bfloat16)


@pytest.mark.parametrize("rows,n,k,groups,dtype", [
    (17, 96, 1032, 1, "bf16"), (64, 1111, 4096, 1, "fp16"), (33, 1, 1025, 1, "bf16"), (48, 4096, 8192, 1, "bf16"),
    (50, 333, 1777, 1, "bf16"), (64, 32, 20000, 1, "bf16"), (96, 264, 2048, 4, "fp16"), (160, 72, 1100, 5, "bf16"),
    (31, 40, 1280, 1, "bf16")])
def test_few_rows_of_long_contractions(rr, rows, n, k, groups, dtype):
    d = make(rows, n, k, groups if groups > 1 else None, dtype, True, True)
    check_forward(rr, d, None, "gelu", DTYPES[dtype])
    if groups > 1:                         # uneven, empty ones, rows of no group
        off = torch.tensor([3, 3] + [rows // 2 + i for i in range(groups - 2)] + [rows - 5], dtype=torch.int32, device="cuda")
        check_forward(rr, d, off, "silu", DTYPES[dtype])


@pytest.mark.parametrize("rows,n,k", [(3, 8192, 2048), (16, 8200, 1032), (9, 16384, 1096), (5, 4096, 8192), (12, 11000, 4096)])
def test_up_to_sixteen_rows_in_tiles(rr, rows, n, k):
    d = make(rows, n, k, None, "bf16", True, True)
    check_forward(rr, d, None, "none", torch.bfloat16)
    ragged = torch.empty(rows, k + 1, dtype=torch.bfloat16, device="cuda")[:, 1:]
    ragged.copy_(d["x"])
    out = rr.block_linear(ragged, d["w"], d["bias"], residual=d["residual"])
    ref = (d["x"].double() @ d["w"].double().t() + d["bias"].double() + d["residual"].double())
    assert float((out.double() - ref).norm() / ref.norm()) < 2.0 ** -8


@pytest.mark.parametrize("rows,n,k,groups", [(1, 72, 264, 64), (5, 520, 1032, 100), (200, 264, 1160, 16), (96, 40, 2048, 6)])
def test_few_rows_over_many_groups(rr, rows, n, k, groups):
    d = make(rows, n, k, groups, "bf16", True, True)
    g = torch.Generator().manual_seed(rows)
    edges = torch.randint(0, rows + 1, (groups + 1,), generator=g).sort().values.int().cuda()
    check_forward(rr, d, edges, "silu", torch.bfloat16)
    check_backward(rr, d, edges, "silu", torch.bfloat16)
