"""Tokens sorted by expert, moved to their experts' rows and summed back, with the
gradients, against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

from tests.block_util import DTYPES, U, assert_within, store_error, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_allreduce_amd
    return ring_allreduce_amd


def order_of(ids, experts, capacity):
    """slots, sources, counts, offsets, one pair at a time."""
    flat = ids.reshape(-1)
    counts = np.zeros(experts, np.int64)
    for e in range(experts):
        counts[e] = int((flat == e).sum())
    first = np.concatenate([[0], np.cumsum(counts)])
    offsets = np.arange(experts + 1) * capacity if capacity else first
    rows = experts * capacity if capacity else flat.size
    slots, sources = np.full(flat.size, -1), np.full(rows, -1)
    seen = np.zeros(experts, np.int64)
    for p, e in enumerate(flat):
        if 0 <= e < experts:
            if not capacity or seen[e] < capacity:
                slots[p] = offsets[e] + seen[e]
                sources[slots[p]] = p
            seen[e] += 1
    return slots.reshape(ids.shape), sources, counts, offsets


def make_ids(tokens, k, experts, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((tokens, k), experts - 1)
    if kind == "none":
        return np.full((tokens, k), -1)
    ids = rng.integers(0, experts, (tokens, k))
    if kind == "masked":
        ids[rng.random((tokens, k)) < 0.3] = -1
        ids[rng.random((tokens, k)) < 0.1] = experts
    return ids


def check_order(o, want):
    for name, w in zip(("slots", "sources", "counts", "offsets"), want):
        assert np.array_equal(getattr(o, name).cpu().numpy(), w), name


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,experts,capacity,kind", [
    (0, 2, 8, 0, "any"), (0, 2, 8, 3, "any"), (1, 1, 1, 0, "any"), (1, 8, 64, 0, "any"),
    (1, 3, 5, 2, "masked"), (16, 4, 32, 0, "any"), (63, 1, 7, 0, "any"), (65, 1, 7, 9, "masked"),
    (511, 2, 60, 0, "masked"), (513, 1, 3, 100, "any"), (4096, 2, 512, 0, "any"),
    (4097, 2, 8, 0, "any"), (1000, 3, 1024, 2, "masked"), (3001, 8, 256, 90, "masked"),
    (9000, 1, 1, 5000, "any"), (5000, 3, 129, 0, "one"), (300, 2, 16, 7, "one"),
    (700, 2, 16, 0, "none"), (9000, 2, 16, 4, "none"), (20011, 6, 513, 0, "masked")])
def test_sort(rr, dtype, tokens, k, experts, capacity, kind):
    ids = make_ids(tokens, k, experts, kind, tokens + k)
    o = rr.expert_sort(torch.from_numpy(ids).to(dtype).cuda(), experts, capacity)
    check_order(o, order_of(ids, experts, capacity))


def test_sort_of_a_wider_tensor_and_far_ids(rr):
    """Ids with a row stride; int64 ids whose low 32 bits look like an expert."""
    ids = make_ids(777, 4, 24, "any", 3)
    wide = torch.from_numpy(np.concatenate([ids, ids + 1], 1)).cuda()
    check_order(rr.expert_sort(wide[:, :4], 24), order_of(ids, 24, 0))
    far = ids.astype(np.int64)
    far[::5] += 1 << 32
    far[1::5] -= 1 << 40
    check_order(rr.expert_sort(torch.from_numpy(far).cuda(), 24, 90), order_of(far, 24, 90))


SHAPES = [  # tokens, hidden, k, experts, capacity, kind
    (1, 1, 1, 1, 0, "any"), (1, 4096, 8, 64, 0, "any"), (5, 7, 3, 4, 2, "masked"),
    (33, 64, 2, 8, 0, "any"), (130, 1025, 4, 16, 40, "masked"), (64, 2050, 6, 12, 0, "masked"),
    (257, 4099, 2, 8, 50, "any"), (40, 8192, 1, 3, 20, "one"), (20, 96, 5, 9, 3, "none"),
    (0, 32, 2, 4, 3, "any"), (300, 520, 9, 16, 0, "any"), (3, 20000, 2, 4, 0, "masked")]


def setup(rr, tokens, hidden, k, experts, capacity, kind, dtype, seed=0, pad=0):
    ids = make_ids(tokens, k, experts, kind, seed + tokens)
    slots, sources, _, _ = order_of(ids, experts, capacity)
    g = torch.Generator().manual_seed(seed + hidden)
    x = torch.randn(tokens, hidden, generator=g).to(DTYPES[dtype])
    rows = torch.randn(len(sources), hidden, generator=g).to(DTYPES[dtype])
    weights = torch.rand(tokens, k, generator=g)
    dev = lambda a: torch.from_numpy(a).to(torch.int32).cuda()  # noqa: E731
    return slots, sources, dev(slots), dev(sources), x, rows, weights


def spread64(x, sources, k, weights=None):
    out = torch.zeros(len(sources), x.shape[1], dtype=torch.float64)
    for r, p in enumerate(sources):
        if p >= 0:
            w = 1.0 if weights is None else float(weights.reshape(-1)[p])
            out[r] = w * x[p // k].double()
    return out


def gathered64(rows, slots):
    got = torch.zeros(*slots.shape, rows.shape[1], dtype=torch.float64)
    for t, j in np.ndindex(*slots.shape):
        if slots[t, j] >= 0:
            got[t, j] = rows[slots[t, j]].double()
    return got


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dispatch(rr, dtype, shape):
    slots, sources, ds, dq, x, _, _ = setup(rr, *shape, dtype)
    got = rr.expert_dispatch(x.cuda(), ds, dq).cpu()
    assert torch.equal(got.double(), spread64(x, sources, shape[2]))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_combine(rr, dtype, weighted, shape):
    """A sum of k products in order: k fused steps, one rounding at the end."""
    slots, _, ds, _, _, rows, weights = setup(rr, *shape, dtype)
    unused = torch.ones(len(rows), dtype=torch.bool)
    unused[torch.from_numpy(slots[slots >= 0])] = False
    rows[unused] = float("nan")                     # rows without a pair are not read
    w = weights.cuda() if weighted else None
    got = rr.expert_combine(rows.cuda(), ds, w).cpu()
    terms = gathered64(rows, slots) * (weights[..., None].double() if weighted else 1.0)
    ref = terms.sum(1)
    bound = store_error(ref, DTYPES[dtype]) + 2 * shape[2] * U * terms.abs().sum(1)
    assert_within(got, ref, bound, "out")
    if not weighted:
        same = rr.expert_dispatch_backward(rows.cuda(), ds).cpu()
        assert torch.equal(got, same)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_combine_backward(rr, dtype, shape):
    tokens, hidden, k = shape[:3]
    slots, sources, ds, dq, dout, rows, weights = setup(rr, *shape, dtype)
    drows, dweights = rr.expert_combine_backward(dout.cuda(), rows.cuda(), ds, dq, weights.cuda())
    ref = spread64(dout, sources, k, weights)
    assert_within(drows.cpu(), ref, store_error(ref, DTYPES[dtype]) +
                  U * ref.abs() + 0.0 * ref, "drows")
    terms = gathered64(rows, slots) * dout[:, None].double()
    ref = terms.sum(2)
    # a thread adds ceil(hidden / 64 lanes) products at most, then 6 lane and 4 wave steps
    steps = -(-hidden // 64) + 8 + 10
    assert_within(dweights.cpu(), ref, steps * U * terms.abs().sum(2), "dweights")
    only_w = rr.expert_combine_backward(dout.cuda(), rows.cuda(), ds, dq, weights.cuda(),
                                        need_rows=False)
    assert only_w[0] is None and torch.equal(only_w[1], dweights)
    only_r = rr.expert_combine_backward(dout.cuda(), None, ds, dq, weights.cuda(),
                                        need_weights=False)
    assert only_r[1] is None and torch.equal(only_r[0], drows)


def test_row_strides_and_guards(rr):
    """Rows apart in memory, starting at an odd element; nothing between them is written."""
    slots, sources, ds, dq, x, rows, weights = setup(rr, 37, 131, 3, 5, 20, "masked", "bf16")
    xs, _ = strided(x, 13, offset=3)
    out, store = strided(rows, 5, offset=1)
    rr.expert_dispatch(xs, ds, dq, out=out)
    assert torch.equal(out.cpu().double(), spread64(x, sources, 3))
    left = store.clone()
    left.as_strided(out.shape, out.stride(), 1).fill_(float("nan"))
    assert bool(left.isnan().all())
    rs, _ = strided(rows, 9, offset=5)
    back, store = strided(x, 3, offset=7)
    rr.expert_combine(rs, ds, weights.cuda(), out=back)
    assert torch.equal(back.cpu(), rr.expert_combine(rows.cuda(), ds, weights.cuda()).cpu())
    left = store.clone()
    left.as_strided(back.shape, back.stride(), 7).fill_(float("nan"))
    assert bool(left.isnan().all())


def test_bad_indexes_stay_in_bounds(rr):
    """Slots and sources outside the tensors count as none."""
    x = torch.randn(4, 64, device="cuda")
    slots = torch.tensor([[0, 9], [-5, 1], [1 << 30, -(1 << 31)], [2, 3]], dtype=torch.int32).cuda()
    sources = torch.tensor([0, 3, 6, 7, 8, 1 << 30, -9], dtype=torch.int32).cuda()
    got = rr.expert_dispatch(x, slots, sources)
    want = torch.zeros(7, 64, device="cuda")
    want[0], want[1], want[2], want[3] = x[0], x[1], x[3], x[3]
    assert torch.equal(got, want)
    back = rr.expert_combine(got, slots)
    assert torch.equal(back, torch.stack([x[0], x[1], 0 * x[2], 2 * x[3]]))


def test_gradients_match_differences(rr):
    """The gradients along a direction against central differences of the 64-bit sums."""
    slots, sources, ds, dq, x, rows, weights = setup(rr, 24, 40, 3, 6, 10, "masked", "fp32")
    dout = x
    drows, dweights = rr.expert_combine_backward(dout.cuda(), rows.cuda(), ds, dq, weights.cuda())
    g = torch.Generator().manual_seed(5)
    vr = torch.randn(rows.shape, generator=g, dtype=torch.float64)
    vw = torch.randn(weights.shape, generator=g, dtype=torch.float64)

    def loss(step):
        got = gathered64(rows.double() + step * vr, slots)
        return float(((got * (weights.double() + step * vw)[..., None]).sum(1) * dout.double()).sum())

    used = torch.from_numpy(sources >= 0)
    along = float((drows.cpu().double() * vr)[used].sum() + (dweights.cpu().double() * vw).sum())
    step = 1e-4
    # the loss is quadratic in the step: central differences are exact but for 64-bit rounding
    assert abs(along - (loss(step) - loss(-step)) / (2 * step)) <= 1e-5 * max(1.0, abs(along))


def test_other_stream_and_repeats(rr):
    """The same bits on another stream, and every time."""
    slots, sources, ds, dq, x, rows, weights = setup(rr, 500, 1000, 4, 16, 0, "masked", "bf16")
    x, rows, weights = x.cuda(), rows.cuda(), weights.cuda()
    ids = torch.from_numpy(make_ids(6000, 4, 16, "masked", 1)).cuda()
    first = [rr.expert_dispatch(x, ds, dq), rr.expert_combine(rows, ds, weights),
             *rr.expert_combine_backward(x, rows, ds, dq, weights), rr.expert_sort(ids, 16).slots]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        for _ in range(2):
            again = [rr.expert_dispatch(x, ds, dq, stream=stream),
                     rr.expert_combine(rows, ds, weights, stream=stream),
                     *rr.expert_combine_backward(x, rows, ds, dq, weights, stream=stream),
                     rr.expert_sort(ids, 16, stream=stream).slots]
            side.synchronize()
            for a, b in zip(first, again):
                assert torch.equal(a, b)


def test_graph(rr):
    """Captured once, replayed on changed inputs, between eager calls."""
    tokens, k, experts, cap, hidden = 3000, 4, 32, 400, 256
    ids = torch.zeros(tokens, k, dtype=torch.int64, device="cuda")
    x = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(tokens, k, device="cuda")

    def step():
        o = rr.expert_sort(ids, experts, cap)
        rows = rr.expert_dispatch(x, o.slots, o.sources)
        out = rr.expert_combine(rows, o.slots, w)
        return [o.slots, o.sources, o.counts, rows, out,
                *rr.expert_combine_backward(out, rows, o.slots, o.sources, w)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(4):
        ids.copy_(torch.from_numpy(make_ids(tokens, k, experts, "masked", seed)))
        x.copy_(torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(seed)))
        w.copy_(torch.rand(tokens, k, generator=torch.Generator().manual_seed(seed)))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)
