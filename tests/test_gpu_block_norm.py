"""The norms around a block with gate and scaled residual, forward and gradients, against
plain 64-bit implementations."""
import pytest
import torch

from tests.block_util import DTYPES, U, act64, assert_within, slope64, store_error, strided

pytestmark = pytest.mark.gpu

RS, BS, EPS = 0.75, 1.25, 1e-5
# 32-bit steps behind a value: a row's sums (at most 32 products in a thread, 6 lane and 16
# wave additions), the root, the products with weights, gate and scales, and the exponential of
# the gate (its argument's rounding counts as many steps as the argument is large, under 32)
STEPS = 256


@pytest.fixture(scope="module")
def rr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_allreduce_amd
    return ring_allreduce_amd


def make(tokens, hidden, dtype, gate, weights, seed=0):
    g = torch.Generator().manual_seed(seed + hidden)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DTYPES[dtype]
    wt = {"same": dt, "fp32": torch.float32, "none": None}[weights]
    d = {"x": (3 * rnd(tokens, hidden)).to(dt), "branch": rnd(tokens, hidden).to(dt),
         "dh": rnd(tokens, hidden).to(dt), "dy": rnd(tokens, hidden).to(dt),
         "h": (3 * rnd(tokens, hidden)).to(dt),
         "post_weight": None if wt is None else (1 + 0.3 * rnd(hidden)).to(wt),
         "pre_weight": None if wt is None else (1 + 0.3 * rnd(hidden)).to(wt), "gate": None}
    if gate == "channel":
        d["gate"] = rnd(hidden).to(wt or dt)
    elif gate == "element":
        d["gate"] = (2 * rnd(tokens, hidden)).to(dt)
    return d


def wide(d):
    return {k: None if v is None else v.double() for k, v in d.items()}


def unit(v):
    r = (v.square().mean(1, keepdim=True) + EPS).rsqrt()
    return v * r, r


def forward64(d, act, post, pre):
    """h, y and the magnitudes their errors are counted in."""
    n = unit(d["branch"])[0] if post else d["branch"]
    if post and d["post_weight"] is not None:
        n = n * d["post_weight"]
    a = act64(d["gate"], act) if d["gate"] is not None else 1.0
    h = RS * d["x"] + BS * a * n
    size_h = (RS * d["x"]).abs() + (BS * a * n).abs()
    if not pre:
        return h, size_h, None, None
    y, r = unit(h)
    w = d["pre_weight"] if d["pre_weight"] is not None else 1.0
    return h, size_h, y * w, (size_h * r * w).abs() + (y * w).abs() * (1 + (size_h * r).square().mean(1, keepdim=True))


def backward64(d, act, post, pre):
    """Gradients and the magnitudes their errors are counted in."""
    one = torch.ones(d["branch"].shape[1], dtype=torch.float64)
    wp = d["post_weight"] if d["post_weight"] is not None else one
    wn = d["pre_weight"] if d["pre_weight"] is not None else one
    out, size = {}, {}
    g, m = d["dh"], d["dh"].abs()
    if pre:
        hu, q = unit(d["h"])
        p = d["dy"] * wn
        g = g + q * p - q * hu * (p * hu).mean(1, keepdim=True)
        m = m + (q * p).abs() + (q * hu).abs() * (p * hu).abs().mean(1, keepdim=True)
        out["dpre_weight"], size["dpre_weight"] = (d["dy"] * hu).sum(0), (d["dy"] * hu).abs().sum(0)
    out["dx"], size["dx"] = RS * g, RS * m
    bu, r = unit(d["branch"]) if post else (d["branch"], torch.ones(1, 1, dtype=torch.float64))
    e, me = BS * g, BS * m
    n = bu * wp if post else bu
    if d["gate"] is not None:
        dg, mg = e * n * slope64(d["gate"], act), me * (n.abs() * 1.2)
        if d["gate"].dim() == 1:
            dg, mg = dg.sum(0), mg.sum(0)
        out["dgate"], size["dgate"] = dg, mg
        a = act64(d["gate"], act)
        e, me = e * a, me * a.abs()
    if post:
        out["dpost_weight"], size["dpost_weight"] = (e * bu).sum(0), (me * bu.abs()).sum(0)
        p, mp = e * wp, me * wp.abs()
        out["dbranch"] = r * (p - bu * (p * bu).mean(1, keepdim=True))
        size["dbranch"] = r * (mp + bu.abs() * (mp * bu.abs()).mean(1, keepdim=True))
    else:
        out["dbranch"], size["dbranch"] = e, me
    return out, size


def own_args(d, act, post, pre):
    c = {k: None if v is None else v.cuda() for k, v in d.items()}
    args = dict(post_norm=post, post_weight=c["post_weight"] if post else None, gate=c["gate"],
                gate_act=act, residual_scale=RS, branch_scale=BS, pre_norm=pre,
                pre_weight=c["pre_weight"] if pre else None, eps=EPS)
    return c, args


CASES = [  # tokens, hidden, gate, act, post, pre, weights
    (1, 1, "none", "none", True, True, "same"), (1, 8192, "none", "none", True, True, "same"),
    (3, 7, "element", "silu", True, True, "fp32"), (5, 512, "channel", "none", True, True, "same"),
    (130, 513, "element", "sigmoid", True, True, "same"), (17, 1000, "none", "none", False, True, "same"),
    (9, 1024, "channel", "sigmoid", True, False, "fp32"), (40, 2049, "element", "none", False, True, "none"),
    (33, 4096, "element", "sigmoid", True, True, "same"), (7, 4099, "channel", "silu", True, True, "same"),
    (2100, 64, "element", "silu", True, True, "same"), (6, 8200, "element", "sigmoid", True, True, "same"),
    (3, 16384, "element", "silu", True, True, "fp32"), (2, 20001, "channel", "none", True, True, "same"),
    (2, 32768, "element", "sigmoid", True, True, "same"), (0, 96, "channel", "none", True, True, "same"),
    (5, 300, "element", "silu", False, False, "none")]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(rr, dtype, case):
    tokens, hidden, gate, act, post, pre, weights = case
    d = make(tokens, hidden, dtype, gate, weights)
    c, args = own_args(d, act, post, pre)
    h, y = rr.block_norm(c["x"], c["branch"], **args)
    rh, sh, ry, sy = forward64(wide(d), act, post, pre)
    dt = DTYPES[dtype]
    assert_within(h.cpu(), rh, store_error(rh, dt) + STEPS * U * sh, "h")
    if pre:
        assert_within(y.cpu(), ry, store_error(ry, dt) + STEPS * U * sy, "y")
    else:
        assert y is None


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(rr, dtype, case):
    tokens, hidden, gate, act, post, pre, weights = case
    d = make(tokens, hidden, dtype, gate, weights, 1)
    c, args = own_args(d, act, post, pre)
    got = rr.block_norm_backward(c["dh"], c["dy"] if pre else None, c["h"], c["branch"], **args)
    w = wide(d)
    if weights == "none":
        w["post_weight"] = w["pre_weight"] = None
    ref, size = backward64(w, act, post, pre)
    dt = DTYPES[dtype]
    for name in ("dx", "dbranch", "dgate", "dpost_weight", "dpre_weight"):
        g = getattr(got, name)
        if name not in ref or (weights == "none" and "weight" in name):
            assert g is None, name
            continue
        if g.dim() == 2:
            bound = store_error(ref[name], dt) + STEPS * U * size[name]
        else:       # fp32 sums over the tokens, added in turn by a workgroup, then over them
            assert g.dtype == torch.float32
            bound = (STEPS + tokens) * U * size[name]
        assert_within(g.cpu(), ref[name], bound, name)


def test_no_branch(rr):
    """The first norm of a model: h = residual_scale * x, y = N(h)."""
    d = make(21, 700, "bf16", "none", "same")
    x, w = d["x"].cuda(), d["pre_weight"].cuda()
    h, y = rr.block_norm(x, post_norm=False, pre_weight=w, eps=EPS)
    assert torch.equal(h, x)
    ref = unit(d["x"].double())[0] * d["pre_weight"].double()
    assert_within(y.cpu(), ref, store_error(ref, torch.bfloat16) + STEPS * U * ref.abs(), "y")
    got = rr.block_norm_backward(None, d["dy"].cuda(), x, post_norm=False, pre_weight=w, eps=EPS)
    dw = wide(d)
    hu, q = unit(dw["x"])
    p = dw["dy"] * dw["pre_weight"]
    ref = q * (p - hu * (p * hu).mean(1, keepdim=True))
    size = q * (p.abs() + hu.abs() * (p * hu).abs().mean(1, keepdim=True))
    assert_within(got.dx.cpu(), ref, store_error(ref, torch.bfloat16) + STEPS * U * size, "dx")
    assert got.dbranch is None and got.dgate is None and got.dpost_weight is None


def test_strides_and_in_place(rr):
    d = make(19, 515, "bf16", "element", "same")
    c, args = own_args(d, "silu", True, True)
    h, y = rr.block_norm(c["x"], c["branch"], **args)
    xs, _ = strided(d["x"], 11, offset=3)
    us, _ = strided(d["branch"], 7, offset=1)
    gs, _ = strided(d["gate"], 2)
    h2, store = strided(d["x"], 5, offset=1)
    rr.block_norm(xs, us, **dict(args, gate=gs), h=h2)
    assert torch.equal(h2, h)
    left = store.clone()
    left.as_strided(h2.shape, h2.stride(), 1).fill_(float("nan"))
    assert bool(left.isnan().all())
    rr.block_norm(xs, us, **args, h=xs, y=us)
    assert torch.equal(xs, h) and torch.equal(us, y)


def test_rows_are_apart(rr):
    """A row of NaN or infinities leaves every other row as it was."""
    d = make(64, 1536, "bf16", "element", "same")
    c, args = own_args(d, "sigmoid", True, True)
    h, y = rr.block_norm(c["x"], c["branch"], **args)
    g = rr.block_norm_backward(c["dh"], c["dy"], c["h"], c["branch"], **args)
    for t in (c["x"], c["branch"], c["dh"], c["h"]):
        t[5], t[40] = float("nan"), float("inf")
    h2, y2 = rr.block_norm(c["x"], c["branch"], **args)
    g2 = rr.block_norm_backward(c["dh"], c["dy"], c["h"], c["branch"], **args)
    keep = [t for t in range(64) if t not in (5, 40)]
    for a, b in ((h, h2), (y, y2), (g.dx, g2.dx), (g.dbranch, g2.dbranch), (g.dgate, g2.dgate)):
        assert torch.equal(a[keep], b[keep])
    assert bool(y2[5].isnan().all())


def test_gradients_match_differences(rr):
    d = make(12, 96, "fp32", "element", "same", 3)
    c, args = own_args(d, "silu", True, True)
    h, _ = rr.block_norm(c["x"], c["branch"], **args)
    got = rr.block_norm_backward(c["dh"], c["dy"], h, c["branch"], **args)
    g = torch.Generator().manual_seed(9)
    names = {"x": "dx", "branch": "dbranch", "gate": "dgate", "post_weight": "dpost_weight",
             "pre_weight": "dpre_weight"}
    base = wide(d)
    for key, grad in names.items():
        v = torch.randn(base[key].shape, generator=g, dtype=torch.float64)

        def loss(step):
            hh, _, yy, _ = forward64({**base, key: base[key] + step * v}, "silu", True, True)
            return float((hh * base["dh"]).sum() + (yy * base["dy"]).sum())

        along = float((getattr(got, grad).cpu().double() * v).sum())
        diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
        # the difference's own error is of the order step^2; the gradient's is counted in
        # 32-bit steps of its terms, about 1e-5 of their absolute sum
        size = float((getattr(got, grad).cpu().double() * v).abs().sum())
        assert abs(along - diff) <= 1e-4 * size, grad


def test_graph_and_streams(rr):
    d = make(300, 2048, "bf16", "element", "same")
    c, args = own_args(d, "sigmoid", True, True)

    def step(stream=None):
        h, y = rr.block_norm(c["x"], c["branch"], **args, stream=stream)
        g = rr.block_norm_backward(c["dh"], c["dy"], h, c["branch"], **args, stream=stream)
        return [h, y, g.dx, g.dbranch, g.dgate, g.dpost_weight, g.dpre_weight]

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
        c["x"].copy_(torch.randn(300, 2048, generator=torch.Generator().manual_seed(seed)))
        c["dy"].copy_(torch.randn(300, 2048, generator=torch.Generator().manual_seed(seed + 9)))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))
