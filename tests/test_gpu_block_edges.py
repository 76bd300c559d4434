"""Unusual calls of a block's operators: nothing to do, values far from 1, infinities, bad
index tensors, against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

from tests.block_util import DTYPES, U, assert_within, store_error
from tests.test_gpu_block_norm import STEPS
from tests.test_gpu_expert import check_order, make_ids, order_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_allreduce_amd
    return ring_allreduce_amd


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,experts,capacity", [
    (0, 2, 512, 0), (0, 2, 513, 0), (0, 2, 1024, 0), (0, 2, 1024, 3), (0, 8, 700, 5), (1, 2, 1024, 3)])
def test_sort_of_no_tokens(rr, dtype, tokens, k, experts, capacity):
    """A rank without tokens, with any number of experts."""
    ids = make_ids(tokens, k, experts, "any", 1)
    o = rr.expert_sort(torch.from_numpy(ids).to(dtype).cuda(), experts, capacity)
    check_order(o, order_of(ids, experts, capacity))


def pullback64(grad, v, w, eps):
    """Gradient of N(v) * w by v, the magnitude its error is counted in, and by w."""
    r = (v.square().mean(1, keepdim=True) + eps).rsqrt()
    u, p = v * r, grad * w
    d = r * (p - u * (p * u).mean(1, keepdim=True))
    return d, r * (p.abs() + u.abs() * (p * u).abs().mean(1, keepdim=True)), (grad * u).sum(0)


@pytest.mark.parametrize("hidden", [96, 1030, 4099, 12296])
@pytest.mark.parametrize("dtype,scale,eps", [
    ("bf16", 1e14, 1e-6), ("bf16", 1e15, 1e-6), ("bf16", 1e16, 1e-6), ("fp32", 1e15, 1e-6),
    ("fp32", 1e-13, 0.0), ("fp32", 1e-15, 0.0), ("bf16", 1e-13, 0.0)])
def test_norm_gradients_of_rows_far_from_one(rr, dtype, scale, eps, hidden):
    """The gradients scale with 1 / size, down to where the squares leave 32 bits: no power of it
    beyond that may be formed on the way."""
    g, dt, tokens = torch.Generator().manual_seed(hidden), DTYPES[dtype], 40
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    h, u = ((rnd(tokens, hidden) * scale).to(dt) for _ in range(2))
    dy, wn, wp = rnd(tokens, hidden).to(dt), (1 + 0.3 * rnd(hidden)).to(dt), (1 + 0.3 * rnd(hidden)).to(dt)
    got = rr.block_norm_backward(None, dy.cuda(), h.cuda(), u.cuda(), post_weight=wp.cuda(),
                                 pre_weight=wn.cuda(), eps=eps)
    dx, size, dpre = pullback64(dy.double(), h.double(), wn.double(), eps)
    assert_within(got.dx.cpu(), dx, store_error(dx, dt) + STEPS * U * size, "dx")
    assert_within(got.dpre_weight.cpu(), dpre, (STEPS + tokens) * U *
                  (dy.double() * h.double() / h.double().square().mean(1, keepdim=True).sqrt()).abs().sum(0), "dpre")
    du, size_u, dpost = pullback64(dx, u.double(), wp.double(), eps)
    more = pullback64(size, u.double().abs(), wp.double().abs(), eps)[1]      # dx's own error, carried on
    assert_within(got.dbranch.cpu(), du, store_error(du, dt) + STEPS * U * (size_u + more), "dbranch")
    unit_u = (u.double() / u.double().square().mean(1, keepdim=True).sqrt()).abs()
    assert_within(got.dpost_weight.cpu(), dpost, (STEPS + tokens) * U * (size * unit_u).sum(0), "dpost")


@pytest.mark.parametrize("hidden", [72, 1030, 4099])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_gradient_by_an_infinite_branch(rr, gate, hidden):
    """Without a norm of the branch its gradient is the stream's times scale and gate, whatever
    the branch holds."""
    g, tokens = torch.Generator().manual_seed(hidden), 20
    u, dh, z = (torch.randn(tokens, hidden, generator=g).bfloat16() for _ in range(3))
    u[3, 5], u[7, 0], u[11, hidden - 1] = float("inf"), float("nan"), float("-inf")
    args = dict(gate=z.cuda(), gate_act="sigmoid") if gate else {}
    got = rr.block_norm_backward(dh.cuda(), None, None, u.cuda(), post_norm=False, pre_norm=False,
                                 branch_scale=1.5, **args)
    want = 1.5 * dh.double() * (torch.sigmoid(z.double()) if gate else 1.0)
    # the exponential's argument is under 8: its rounding counts as many steps
    assert_within(got.dbranch.cpu(), want, store_error(want, torch.bfloat16) + 16 * U * want.abs(), "dbranch")


def test_options_without_a_truth_value(rr):
    """They raise what their bool() raises, and the next call is as it was."""
    x, w = torch.randn(6, 16, device="cuda").bfloat16(), torch.randn(8, 16, device="cuda").bfloat16()
    i = torch.zeros(6, 1, dtype=torch.int32, device="cuda")
    q, bad = torch.full((1,), -1, dtype=torch.int32, device="cuda"), torch.zeros(2)
    want = rr.block_linear(x, w)
    for call in (lambda: rr.block_norm(x, x, post_norm=bad), lambda: rr.block_norm(x, x, pre_norm=bad),
                 lambda: rr.block_norm_backward(x, x, x, x, post_norm=bad),
                 lambda: rr.block_linear(x, w, save_preact=bad),
                 lambda: rr.block_linear_backward(want, x, w, need_dx=bad),
                 lambda: rr.block_linear_backward(want, x, w, need_dw=bad),
                 lambda: rr.block_linear_backward(want, x, w, need_db=bad),
                 lambda: rr.expert_combine_backward(x, x[:1], i, q, need_rows=bad),
                 lambda: rr.expert_combine_backward(x, x[:1], i, q, need_weights=bad)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()
    assert torch.equal(rr.block_linear(x, w), want)


def test_weights_and_bias_in_another_order_are_refused(rr):
    """As many elements are not enough: they are read in the order of [tokens, k] and [groups, n]."""
    x, i = torch.randn(6, 16, device="cuda"), torch.arange(12, dtype=torch.int32, device="cuda").reshape(6, 2)
    q, rows = torch.arange(12, dtype=torch.int32, device="cuda"), torch.randn(12, 16, device="cuda")
    w = torch.rand(6, 2, device="cuda")
    xs, ws = torch.randn(9, 16, device="cuda").bfloat16(), torch.randn(3, 8, 16, device="cuda").bfloat16()
    b = torch.randn(3, 8, device="cuda").bfloat16()
    out = torch.empty(9, 8, dtype=torch.bfloat16, device="cuda")
    bad_w, bad_b = w.t().contiguous(), b.t().contiguous()
    for call in (lambda: rr.expert_combine(rows, i, bad_w), lambda: rr.expert_combine(rows, i, bad_w, out=torch.empty_like(x)),
                 lambda: rr.expert_combine(rows, i, w.reshape(3, 4)),
                 lambda: rr.expert_combine_backward(x, rows, i, q, bad_w),
                 lambda: rr.expert_combine_backward(x, rows, i, q, bad_w, out=torch.empty_like(rows)),
                 lambda: rr.block_linear(xs, ws, bad_b), lambda: rr.block_linear(xs, ws, bad_b, out=out),
                 lambda: rr.block_linear(xs, ws, b.reshape(2, 12))):
        with pytest.raises(ValueError, match="must be"):
            call()
    want, grads = rr.expert_combine(rows, i, w), rr.expert_combine_backward(x, rows, i, q, w)
    made = rr.block_linear(xs, ws, b)
    for same in (lambda t: t.reshape(-1), lambda t: t[..., None], lambda t: t[None]):     # the same order
        assert torch.equal(rr.expert_combine(rows, i, same(w)), want)
        assert torch.equal(rr.expert_combine(rows, i, same(w), out=torch.empty_like(x)), want)
        assert all(torch.equal(*ab) for ab in zip(rr.expert_combine_backward(x, rows, i, q, same(w)), grads))
        assert torch.equal(rr.block_linear(xs, ws, same(b)), made)
        assert torch.equal(rr.block_linear(xs, ws, same(b), out=out), made)
    one = rr.block_linear(xs, ws[0], b[0])
    assert torch.equal(rr.block_linear(xs, ws[0], b[:1]), one) and torch.equal(rr.block_linear(xs, ws[:1], b[0]), one)


def test_marshalled_in_python(rr, monkeypatch):
    """The same bits from every call without the C++ marshalling."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, u, dh, dy, gate, w = rnd(70, 96), rnd(70, 96), rnd(70, 96), rnd(70, 96), rnd(70, 96), rnd(96)
    ws, b, dout, z = rnd(3, 40, 96), rnd(3, 40), rnd(70, 40), rnd(70, 40)
    ids = torch.from_numpy(make_ids(70, 2, 3, "masked", 3)).cuda()
    weights, rows = torch.rand(70, 2, generator=g, device="cuda"), rnd(60, 96)
    off = torch.tensor([0, 30, 31, 68], dtype=torch.int32, device="cuda")

    def step():
        o = rr.expert_sort(ids, 3, 20)
        n = rr.block_norm_backward(dh, dy, x, u, post_weight=w, pre_weight=w, gate=gate, gate_act="silu")
        m = rr.block_linear_backward(dout, x, ws, z, act="gelu", offsets=off)
        return [o.slots, o.sources, o.counts, o.offsets, rr.expert_dispatch(x, o.slots, o.sources),
                rr.expert_combine(rows, o.slots, weights),
                *rr.expert_combine_backward(x, rows, o.slots, o.sources, weights),
                *rr.block_norm(x, u, post_weight=w, pre_weight=w, gate=gate, gate_act="silu"),
                n.dx, n.dbranch, n.dgate, n.dpost_weight, n.dpre_weight,
                *rr.block_linear(x, ws, b, act="gelu", offsets=off, save_preact=True), m.dx, m.dw, m.db]

    want = step()
    monkeypatch.setattr(rr.block, "_block", rr.block._Absent())
    assert all(torch.equal(p, q) for p, q in zip(want, step(), strict=True))


def test_combine_backward_of_many_tokens(rr):
    """More tokens than a launch has workgroups: four short rows share one."""
    tokens, hidden = (1 << 24) + 9, 8
    at = torch.tensor([0, 1, 77, 1 << 20, (1 << 24) - 1, 1 << 24, tokens - 1], device="cuda")
    slots = torch.full((tokens, 1), -1, dtype=torch.int32, device="cuda")
    slots[at, 0] = torch.arange(len(at), dtype=torch.int32, device="cuda")
    sources = torch.cat([at.int(), torch.full((3,), -1, dtype=torch.int32, device="cuda")])
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randint(-4, 5, (len(sources), hidden), generator=g, device="cuda").bfloat16()
    dout = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    dout[at] = torch.randint(-4, 5, (len(at), hidden), generator=g, device="cuda").bfloat16()
    drows, dweights = rr.expert_combine_backward(dout, rows, slots, sources)
    assert torch.equal(drows[:len(at)], dout[at]) and not bool(drows[len(at):].any())
    want = torch.zeros(tokens, 1, device="cuda")            # sums of few small integers: exact
    want[at, 0] = (dout[at].float() * rows[:len(at)].float()).sum(1)
    assert torch.equal(dweights, want)
    assert torch.equal(rr.expert_combine_backward(dout, rows, slots, sources, need_rows=False)[1], want)


def test_overlapping_groups_of_many_rows(rr):
    """Offsets that descend, over so many rows that the tiles of all ranges are more than 2^31.
    The first group has every row and all groups have the same weights, so that the result is
    known; nothing around it is written."""
    rows, groups, guard = 1 << 28, 1024, 512
    value = (torch.arange(rows, dtype=torch.int32, device="cuda") % 7).bfloat16()
    x = value[:, None].expand(rows, 8).contiguous()
    w = torch.ones(groups, 8, 8, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[1::2] = rows
    store = torch.full((rows + 2 * guard, 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = rr.block_linear(x, w, offsets=off, out=store[guard:-guard])
    torch.cuda.synchronize()
    del x
    assert bool(store[:guard].isnan().all()) and bool(store[-guard:].isnan().all())
    assert bool((out == (8 * value)[:, None]).all())           # 8 products of up to 6: exact


class Guarded:
    """Tensors in one allocation, with 4 KiB of a pattern before, between and behind them."""
    GAP, PATTERN = 4096, 0xA5

    def __init__(self, size):
        self.store = torch.full((size,), self.PATTERN, dtype=torch.uint8, device="cuda")
        self.at, self.spans = self.GAP, []

    def make(self, *shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        lo, self.at = self.at, -(-(self.at + n) // 256) * 256 + self.GAP
        assert self.at <= self.store.numel()
        self.spans.append((lo, lo + n))
        return self.store[lo:lo + n].view(dtype).view(shape)

    def whole(self):
        """Whether nothing around the tensors was written."""
        left = self.store == self.PATTERN
        for lo, hi in self.spans:
            left[lo:hi] = True
        return bool(left.all())


def bad_offsets(rows, groups):
    g = torch.Generator().manual_seed(rows)
    wild = torch.randint(-rows, 2 * rows, (groups + 1,), generator=g)
    wild[groups // 2], wild[-1] = -(1 << 31), (1 << 31) - 1
    full = torch.zeros(groups + 1, dtype=torch.int64)
    full[1::2] = rows
    return [torch.arange(groups, -1, -1) * rows // groups, full, wild]


# rows, groups, n, k: one pass over rows of 16 (whole, and cut along k), 32 and 64; four parts in a
# workgroup; parts joined by a second launch; a last round of tiles cut along k; copied operands
@pytest.mark.parametrize("rows,groups,n,k", [
    (48, 4, 264, 520), (40, 4, 40, 4096), (100, 4, 264, 264), (200, 4, 264, 264), (160, 4, 264, 4096),
    (300, 3, 128, 8192), (4400, 3, 4096, 2048), (300, 5, 131, 77), (900, 70, 200, 136)])
def test_bad_offsets_write_nothing_else(rr, rows, groups, n, k):
    """Whatever the offsets hold, the calls end, and write nothing but their outputs and scratch."""
    blk, dt = rr.block, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(k)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, w, bias, res, dout = rnd(rows, k), rnd(groups, n, k), rnd(groups, n), rnd(rows, n), rnd(rows, n)
    stream, size = torch.cuda.current_stream().cuda_stream, blk._sz()
    for offsets in bad_offsets(rows, groups):
        off = offsets.to(torch.int32).cuda()
        a = blk._linear_args(x, w, off, "silu")
        a.bias, a.residual = bias.data_ptr(), blk._Rows(res.data_ptr(), n)
        assert blk._block_linear_workspace(a, size) == 0
        room = Guarded(size.value + 8 * rows * n + (1 << 16))
        out, z, work = room.make(rows, n, dtype=dt), room.make(rows, n, dtype=dt), room.make(size.value, dtype=torch.uint8)
        a.out, a.z = blk._Rows(out.data_ptr(), n), blk._Rows(z.data_ptr(), n)
        assert blk._block_linear(a, work.data_ptr(), size.value, stream) == 0
        assert room.whole(), offsets
        zs, grad = rnd(rows, n), blk._LinearGrad()
        a.z = blk._Rows(zs.data_ptr(), n)
        grad.dout, grad.dw_dt = blk._Rows(dout.data_ptr(), n), blk.FLOAT_DTYPES[torch.float32]
        grad.dx, grad.dw, grad.db = blk._Rows(1 << 20, k), 1 << 20, 1 << 20      # wanted; where to, below
        assert blk._block_linear_backward_workspace(a, grad, size) == 0
        room = Guarded(size.value + 4 * rows * k + 4 * groups * n * (k + 1) + (1 << 17))
        dx, dw = room.make(rows, k, dtype=dt), room.make(groups, n, k, dtype=torch.float32)
        db, work = room.make(groups, n, dtype=torch.float32), room.make(size.value, dtype=torch.uint8)
        grad.dx, grad.dw, grad.db = blk._Rows(dx.data_ptr(), k), dw.data_ptr(), db.data_ptr()
        assert blk._block_linear_backward(a, grad, work.data_ptr(), size.value, stream) == 0
        assert room.whole(), offsets
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act,value,slope", [
    ("none", [np.inf, -np.inf, np.nan], [1, 1, 1]), ("relu", [np.inf, 0, np.nan], [1, 0, 0]),
    ("gelu", [np.inf, 0, np.nan], [1, 0, np.nan]), ("silu", [np.inf, np.nan, np.nan], [np.nan] * 3)])
def test_activations_at_infinities(rr, dtype, act, value, slope):
    """x w^T with k = 1 and w = 1 is x itself, so this is the activation and its slope alone."""
    x = torch.tensor([[np.inf], [-np.inf], [np.nan]]).to(DTYPES[dtype]).cuda()
    one = torch.ones(1, 1, dtype=x.dtype, device="cuda")
    for rows in (1, 3, 40, 300):                   # a wave's dots, one pass, tiles
        z = x.repeat(rows, 1)[:rows]
        out = rr.block_linear(z, one, act=act)
        d = rr.block_linear_backward(torch.ones_like(z), z, one, z, act=act, need_dw=False)
        want = [torch.tensor(v, dtype=torch.float64).repeat(rows)[:rows, None] for v in (value, slope)]
        torch.testing.assert_close(out.cpu().double(), want[0], rtol=0, atol=0, equal_nan=True)
        torch.testing.assert_close(d.dx.cpu().double(), want[1], rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hidden", [515, 1025, 1027, 1543, 2049, 4099, 8193, 16385])
def test_norm_in_place_at_odd_widths(rr, dtype, hidden):
    """A row's last vector is read so that it ends with the row, over elements that other waves
    own and, without a norm in between, may have written by then: those do not count."""
    g, dt, tokens = torch.Generator(device="cuda").manual_seed(hidden), DTYPES[dtype], 300
    x, u, z = (torch.randn(tokens, hidden, generator=g, device="cuda").to(dt) for _ in range(3))
    args = dict(post_norm=False, pre_norm=False, gate=z, gate_act="sigmoid", residual_scale=1.5)
    h, _ = rr.block_norm(x, u, **args)
    in_place = x.clone()
    rr.block_norm(in_place, u, **args, h=in_place)
    assert torch.equal(in_place, h)
    want = rr.block_norm_backward(x, None, None, u, **args)
    blk, dh = rr.block, x.clone()
    a = blk._norm_args(x, u, False, None, z, "sigmoid", 1.5, 1.0, False, None, 1e-6)
    grad, du, dz = blk._NormGrad(), torch.empty_like(x), torch.empty_like(x)
    grad.dh = grad.dx = blk._Rows(dh.data_ptr(), hidden)
    grad.dbranch, grad.dgate = blk._Rows(du.data_ptr(), hidden), blk._Rows(dz.data_ptr(), hidden)
    assert blk._block_norm_backward(a, grad, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(dh, want.dx) and torch.equal(du, want.dbranch) and torch.equal(dz, want.dgate)
