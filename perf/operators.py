"""Cases and plain forms of the operators of a transformer block around the collectives.

The operators are what a rank computes between two collectives of this library:

* ``sort``      tokens counted and ordered by the expert each of their k choices names
                (``expert_sort``);
* ``dispatch``  token rows copied to their experts' slots, and the gradient back
                (``expert_dispatch``, ``expert_dispatch_backward``);
* ``combine``   the experts' rows summed back per token with the router's weights, and the
                gradients of rows and weights (``expert_combine``, ``expert_combine_backward``);
* ``norm``      the norm after a block with its gate, the scaled residual, and the norm before
                the next block, in one pass, and all gradients (``block_norm``,
                ``block_norm_backward``);
* ``linear``    the matrix product with bias, activation and residual in its epilogue, dense or
                over the sorted rows of experts, and all gradients (``block_linear``,
                ``block_linear_backward``).

``run`` computes an operator in its plain form, elementary torch operations in 32 bits rounded
once at the end, or, where ``own`` is true, by the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoding step of a small batch: 16 requests, 4 of 32 experts each
        {"name": "sort decode", "op": "sort", "tokens": 16, "k": 4, "experts": 32, "capacity": 0,
         "masked": 0.0},
        # a training batch of many small experts, some choices masked out, with a capacity
        {"name": "sort train", "op": "sort", "tokens": 65536, "k": 8, "experts": 256,
         "capacity": 2304, "masked": 0.02},
        # equal blocks for an all-to-all: odd token count and row length, tokens dropped
        {"name": "dispatch odd", "op": "dispatch", "dtype": "fp16", "tokens": 1037, "hidden": 2050,
         "k": 2, "experts": 16, "capacity": 120, "masked": 0.0, "train": False},
        # a training step: rows out to packed experts, and their gradient back
        {"name": "dispatch train", "op": "dispatch", "dtype": "bf16", "tokens": 16384,
         "hidden": 4096, "k": 4, "experts": 64, "capacity": 0, "masked": 0.0, "train": True},
        # one token being decoded
        {"name": "combine token", "op": "combine", "dtype": "bf16", "tokens": 1, "hidden": 4096,
         "k": 8, "experts": 64, "capacity": 0, "masked": 0.0, "train": False},
        # a training step with dropped choices: the sum, the rows' and the weights' gradients
        {"name": "combine train", "op": "combine", "dtype": "bf16", "tokens": 16384,
         "hidden": 4096, "k": 4, "experts": 64, "capacity": 1100, "masked": 0.02, "train": True},
        # a few tokens being decoded, between two blocks
        {"name": "norm decode", "op": "norm", "dtype": "bf16", "tokens": 4, "hidden": 8192,
         "gate": "none", "gate_act": "none", "post": True, "pre": True, "train": False},
        # a training step between two blocks, with a gate for each element
        {"name": "norm train", "op": "norm", "dtype": "bf16", "tokens": 16384, "hidden": 4096,
         "gate": "element", "gate_act": "sigmoid", "post": True, "pre": True, "train": True},
        # one token being decoded: the weights are read once
        {"name": "linear token", "op": "linear", "dtype": "bf16", "rows": 1, "n": 8192, "k": 8192,
         "groups": 1, "act": "none", "bias": True, "residual": True, "train": False},
        # a short prompt through odd sizes
        {"name": "linear odd", "op": "linear", "dtype": "fp16", "rows": 1001, "n": 1111, "k": 1777,
         "groups": 1, "act": "gelu", "bias": True, "residual": False, "train": False},
        # a long prompt or one accumulation step's forward
        {"name": "linear prefill", "op": "linear", "dtype": "bf16", "rows": 8192, "n": 8192,
         "k": 4096, "groups": 1, "act": "silu", "bias": True, "residual": True, "train": False},
        # a training step over the sorted rows of 8 experts of uneven load
        {"name": "linear experts", "op": "linear", "dtype": "bf16", "rows": 16384, "n": 8192,
         "k": 2048, "groups": 8, "act": "silu", "bias": True, "residual": False, "train": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "norm", "linear"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    masked = rng.choice([0.0, 0.0, 0.05])
    if op == "linear":
        groups = rng.choice([1, 1, 1, 3, 16])
        rows, train = _log(rng, 1, 16384), rng.random() < 0.4
        n, k = _log(rng, 64, 8192), _log(rng, 64, 8192)
        if rng.random() < 0.7:                      # most layers have round widths
            n, k = (n + 7) // 8 * 8, (k + 7) // 8 * 8
        while rows * n * k > 16384 * 8192 * 2048:
            rows = rows // 2 + 1
        return {"op": op, "dtype": dtype if dtype != "fp32" else "bf16", "rows": rows, "n": n,
                "k": k, "groups": groups, "act": rng.choice(["none", "relu", "gelu", "silu"]),
                "bias": rng.random() < 0.7, "residual": rng.random() < 0.5, "train": train}
    if op == "norm":
        hidden, train = _log(rng, 64, 16384), rng.random() < 0.5
        if rng.random() < 0.7:
            hidden = (hidden + 7) // 8 * 8
        tokens = min(_log(rng, 1, 65536), 16384 * 4096 * 2 // BYTES[dtype] // hidden)
        gate = rng.choice(["none", "channel", "element"])
        act = rng.choice(["none", "sigmoid", "silu"]) if gate == "element" else "none"
        post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        return {"op": op, "dtype": dtype, "tokens": tokens, "hidden": hidden, "gate": gate,
                "gate_act": act, "post": post, "pre": pre, "train": train}
    k, experts = rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([8, 12, 16, 60, 64, 128, 256])
    if op == "sort":
        tokens = _log(rng, 1, 65536)
        capacity = rng.choice([0, (tokens * k * 5 // 4 + experts - 1) // experts])
        return {"op": op, "tokens": tokens, "k": k, "experts": experts, "capacity": capacity,
                "masked": masked}
    hidden = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        hidden = (hidden + 7) // 8 * 8
    tokens = min(_log(rng, 1, 32768), 16384 * 4 * 4096 * 2 // BYTES[dtype] // hidden // k)
    capacity = rng.choice([0, (tokens * k * 5 // 4 + experts - 1) // experts])
    return {"op": op, "dtype": dtype, "tokens": tokens, "hidden": hidden, "k": k,
            "experts": experts, "capacity": capacity, "masked": masked,
            "train": rng.random() < 0.5}


def work(case):
    c = case
    if c["op"] == "sort":
        pairs = c["tokens"] * c["k"]
        rows = c["experts"] * c["capacity"] if c["capacity"] else pairs
        return {"bytes": 8 * pairs + 4 * pairs + 4 * rows + 4 * (2 * c["experts"] + 1), "flops": 0}
    if c["op"] in ("dispatch", "combine"):
        row = c["hidden"] * BYTES[c["dtype"]]
        pairs = c["tokens"] * c["k"]
        slots = c["experts"] * c["capacity"] if c["capacity"] else pairs
        used = min(slots, pairs * (1.0 - c["masked"]))
        t = c["tokens"]
        if c["op"] == "dispatch":                   # x in, rows out; rows' gradient in, dx out
            b = t * row + slots * row + 4 * (pairs + slots)
            if c["train"]:
                b += used * row + t * row + 4 * pairs
            return {"bytes": b, "flops": pairs * c["hidden"] if c["train"] else 0}
        b = used * row + t * row + 8 * pairs        # rows in, sums out
        if c["train"]:                              # rows and dout in, rows' gradient out
            b += used * row + t * row + slots * row + 4 * (3 * pairs + slots)
        return {"bytes": b, "flops": (6 if c["train"] else 2) * pairs * c["hidden"]}
    if c["op"] == "norm":
        e = c["tokens"] * c["hidden"] * BYTES[c["dtype"]]
        gate = c["gate"] == "element"
        b = e * (2 + gate + 1 + c["pre"])           # x, branch, gate in; stream, y out
        if c["train"]:                              # dh, dy, h, branch, gate in; dx, dbranch, dgate out
            b += e * (1 + 2 * c["pre"] + 1 + gate + 2 + gate)
        return {"bytes": b + 8 * c["hidden"],
                "flops": (40 if c["train"] else 15) * c["tokens"] * c["hidden"]}
    m, n, k, e = c["rows"], c["n"], c["k"], BYTES[c["dtype"]]
    b = e * (m * k + c["groups"] * n * k + m * n * (1 + c["residual"]))
    if c["train"]:                                  # z out; dout, x, w, z in; dx, dw out
        b += e * (2 * m * n + 2 * m * k + 2 * c["groups"] * n * k)
        b += e * m * n if c["act"] != "none" else 0
    return {"bytes": b, "flops": 2 * m * n * k * (3 if c["train"] else 1)}


# ----------------------------------------------------------------- inputs --

def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _choices(case, g):
    """k different experts for each token, experts of uneven load; -1: masked out."""
    c = case
    lean = torch.randn(c["experts"], generator=g, device="cuda") * 0.5
    keys = torch.rand(c["tokens"], c["experts"], generator=g, device="cuda").log_().neg_().log_()
    ids = torch.topk(lean - keys, c["k"], dim=1).indices
    if c["masked"]:
        lost = torch.rand(c["tokens"], c["k"], generator=g, device="cuda") < c["masked"]
        ids = ids.masked_fill(lost, -1)
    return ids


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "sort":
        s["ids"] = _choices(c, g)
        return s
    dt = DTYPES[c["dtype"]]
    if c["op"] in ("dispatch", "combine"):
        slots, sources, _, _ = _plain_sort(_choices(c, g), c["experts"], c["capacity"])
        s.update(slots=slots, sources=sources)
        t, h, rows = c["tokens"], c["hidden"], sources.numel()
        if c["op"] == "dispatch":
            s["x"] = _normal(g, t, h, dtype=dt)
            if c["train"]:
                s["drows"] = _normal(g, rows, h, dtype=dt)
        else:
            s["rows"] = _normal(g, rows, h, dtype=dt)
            s["weights"] = torch.softmax(_normal(g, t, c["k"]), 1)
            if c["train"]:
                s["dout"] = _normal(g, t, h, dtype=dt)
        return s
    if c["op"] == "norm":
        t, h = c["tokens"], c["hidden"]
        spread = torch.exp(_normal(g, h, scale=0.5))       # channels of uneven size
        s["x"] = (_normal(g, t, h) * spread * 2).to(dt)
        s["branch"] = (_normal(g, t, h) * spread).to(dt)
        s["post_weight"] = (1 + _normal(g, h, scale=0.2)).to(dt) if c["post"] else None
        s["pre_weight"] = (1 + _normal(g, h, scale=0.2)).to(dt) if c["pre"] else None
        s["gate"] = None
        if c["gate"] != "none":
            s["gate"] = _normal(g, *((t, h) if c["gate"] == "element" else (h,)), dtype=dt)
        if c["train"]:
            s["dh"] = _normal(g, t, h, dtype=dt)
            s["dy"] = _normal(g, t, h, dtype=dt) if c["pre"] else None
            s["h"] = (_normal(g, t, h) * spread * 2).to(dt)     # the stream an earlier pass stored
        return s
    m, n, k, e = c["rows"], c["n"], c["k"], c["groups"]
    s["x"] = _normal(g, m, k, dtype=dt)
    s["w"] = _normal(g, *((e, n, k) if e > 1 else (n, k)), dtype=dt, scale=k ** -0.5)
    s["bias"] = _normal(g, *((e, n) if e > 1 else (n,)), dtype=dt, scale=0.5) if c["bias"] else None
    s["residual"] = _normal(g, m, n, dtype=dt) if c["residual"] else None
    s["dout"] = _normal(g, m, n, dtype=dt) if c["train"] else None
    # the pre-activation an earlier pass stored
    s["z"] = _normal(g, m, n, dtype=dt) if c["train"] and c["act"] != "none" else None
    s["offsets"], s["largest"] = None, m
    if e > 1:                                       # rows of each expert, uneven, some maybe none
        r = np.random.RandomState(seed % (1 << 31))
        sizes = r.multinomial(m, r.dirichlet([3.0] * e))
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        s["offsets"], s["largest"] = torch.from_numpy(off).cuda(), max(1, int(sizes.max()))
    return s


# ------------------------------------------------------------ plain forms --

def _plain_sort(ids, experts, capacity):
    flat = ids.reshape(-1)
    none = (flat < 0) | (flat >= experts)
    key = torch.where(none, experts, flat)
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    count = count.scatter_add_(0, key, torch.ones_like(key))[:experts]
    start = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    start[1:] = torch.cumsum(count, 0)
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=ids.device)
    safe = torch.where(none, 0, flat)
    if capacity:
        rank = place - start[safe]
        kept = ~none & (rank < capacity)
        slot = safe * capacity + rank
        rows = experts * capacity
        offsets = torch.arange(experts + 1, device=ids.device) * capacity
    else:
        kept, slot, rows, offsets = ~none, place, flat.numel(), start
    slots = torch.where(kept, slot, -1)
    spare = torch.full((rows + 1,), -1, dtype=torch.int64, device=ids.device)
    spare[torch.where(kept, slot, rows)] = torch.arange(flat.numel(), device=ids.device)
    return (slots.to(torch.int32).reshape(ids.shape), spare[:rows].to(torch.int32),
            count.to(torch.int32), offsets.to(torch.int32))


def _gather(rows, slots):
    """The rows of each token's slots in 32 bits, [tokens, k, hidden]; zeros where there is none."""
    got = rows[slots.clamp(min=0).long()].float()
    return torch.where((slots >= 0)[..., None], got, 0.0)


def _spread(values, sources, k):
    """values [tokens, hidden] at each row's token; zeros in rows without one."""
    got = values[sources.clamp(min=0).long() // k]
    return torch.where((sources >= 0)[:, None], got, torch.zeros((), dtype=got.dtype, device=got.device))


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if act == "sigmoid":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 - q)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


RESIDUAL_SCALE, BRANCH_SCALE = 0.75, 1.25


def _norm_forward(s):
    """stream = rs * x + bs * act(gate) * N(branch) * w_post; y = N(stream) * w_pre."""
    c, dt = s["case"], s["x"].dtype
    b = s["branch"].float()
    if c["post"]:
        b = b * torch.rsqrt((b * b).mean(1, keepdim=True) + EPS) * s["post_weight"].float()
    if s["gate"] is not None:
        b = b * _act(s["gate"].float(), c["gate_act"])
    h = RESIDUAL_SCALE * s["x"].float() + BRANCH_SCALE * b
    out = {"h": h.to(dt)}
    if c["pre"]:
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["pre_weight"].float()
        out["y"] = y.to(dt)
    return out


def _norm_pullback(grad, x, w):
    """Gradients of N(x) * w = x * r * w, r = (mean(x^2) + eps)^-1/2, by x and by w."""
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    p = grad * w
    return r * p - x * r * r * r * (p * x).mean(1, keepdim=True), (grad * x * r).sum(0)


def _norm_backward(s):
    c, dt, out = s["case"], s["x"].dtype, {}
    d = s["dh"].float()
    if c["pre"]:
        more, out["dpre_weight"] = _norm_pullback(s["dy"].float(), s["h"].float(), s["pre_weight"].float())
        d = d + more
    out["dx"] = (RESIDUAL_SCALE * d).to(dt)
    d = BRANCH_SCALE * d
    b = s["branch"].float()
    n = b
    if c["post"]:
        n = b * torch.rsqrt((b * b).mean(1, keepdim=True) + EPS) * s["post_weight"].float()
    if s["gate"] is not None:
        z = s["gate"].float()
        dg = d * n * _act_slope(z, c["gate_act"])
        out["dgate"] = dg.to(dt) if c["gate"] == "element" else dg.sum(0)
        d = d * _act(z, c["gate_act"])
    if c["post"]:
        d, out["dpost_weight"] = _norm_pullback(d, b, s["post_weight"].float())
    out["dbranch"] = d.to(dt)
    return out


def _groups(s):
    """(group, place within it) of each row, from the groups' first rows."""
    r = torch.arange(s["x"].shape[0], device="cuda", dtype=torch.int32)
    group = torch.searchsorted(s["offsets"][1:].contiguous(), r, right=True)
    return group, r - s["offsets"][group]


def _apart(s, v):
    """Sorted rows v as [groups, largest, columns] in 32 bits, zeros after each group's rows."""
    group, place = _groups(s)
    out = torch.zeros(s["case"]["groups"], s["largest"], v.shape[1], device="cuda")
    out[group, place] = v.float()
    return out


def _plain_linear(s):
    c, dt = s["case"], s["x"].dtype
    if s["offsets"] is None:
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
    else:
        group, place = _groups(s)
        z = torch.bmm(_apart(s, s["x"]), s["w"].float().transpose(1, 2))[group, place]
        if s["bias"] is not None:
            z = z + s["bias"].float()[group]
    out = _act(z, c["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    got = {"out": out.to(dt)}
    if not c["train"]:
        return got
    if c["act"] != "none":
        got["z"] = z.to(dt)
    dz = s["dout"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), c["act"])
    if s["offsets"] is None:
        got["dx"] = (dz @ s["w"].float()).to(dt)
        got["dw"] = (dz.t() @ s["x"].float()).to(dt)
        if s["bias"] is not None:
            got["db"] = dz.sum(0)
    else:
        dzs = _apart(s, dz)
        got["dx"] = torch.bmm(dzs, s["w"].float())[group, place].to(dt)
        got["dw"] = torch.bmm(dzs.transpose(1, 2), _apart(s, s["x"])).to(dt)
        if s["bias"] is not None:
            got["db"] = dzs.sum(1)
    return got


def _run_plain(s):
    c = s["case"]
    if c["op"] == "sort":
        slots, sources, counts, offsets = _plain_sort(s["ids"], c["experts"], c["capacity"])
        return {"slots": slots, "sources": sources, "counts": counts, "offsets": offsets}
    if c["op"] == "dispatch":
        out = {"rows": _spread(s["x"], s["sources"], c["k"])}
        if c["train"]:
            out["dx"] = _gather(s["drows"], s["slots"]).sum(1).to(s["x"].dtype)
        return out
    if c["op"] == "combine":
        dt, got = s["rows"].dtype, _gather(s["rows"], s["slots"])
        out = {"out": (got * s["weights"][..., None]).sum(1).to(dt)}
        if c["train"]:
            d = s["dout"].float()
            out["dweights"] = (got * d[:, None]).sum(2)
            at = s["sources"].clamp(min=0).long()
            w = torch.where(s["sources"] >= 0, s["weights"].reshape(-1)[at], 0.0)
            out["drows"] = (_spread(d, s["sources"], c["k"]) * w[:, None]).to(dt)
        return out
    if c["op"] == "norm":
        out = _norm_forward(s)
        if c["train"]:
            out.update(_norm_backward(s))
        return out
    return _plain_linear(s)


# ------------------------------------------------- the library's operators --

def _run_own(s):
    import ring_allreduce_amd as rr
    c = s["case"]
    if c["op"] == "sort":
        o = rr.expert_sort(s["ids"], c["experts"], c["capacity"])
        return {"slots": o.slots, "sources": o.sources, "counts": o.counts, "offsets": o.offsets}
    if c["op"] == "dispatch":
        out = {"rows": rr.expert_dispatch(s["x"], s["slots"], s["sources"])}
        if c["train"]:
            out["dx"] = rr.expert_dispatch_backward(s["drows"], s["slots"])
        return out
    if c["op"] == "combine":
        out = {"out": rr.expert_combine(s["rows"], s["slots"], s["weights"])}
        if c["train"]:
            out["drows"], out["dweights"] = rr.expert_combine_backward(
                s["dout"], s["rows"], s["slots"], s["sources"], s["weights"])
        return out
    if c["op"] == "norm":
        same = dict(post_norm=c["post"], post_weight=s["post_weight"], gate=s["gate"],
                    gate_act=c["gate_act"], residual_scale=RESIDUAL_SCALE,
                    branch_scale=BRANCH_SCALE, pre_norm=c["pre"], pre_weight=s["pre_weight"],
                    eps=EPS)
        h, y = rr.block_norm(s["x"], s["branch"], **same)
        out = {"h": h, "y": y} if c["pre"] else {"h": h}
        if c["train"]:
            d = rr.block_norm_backward(s["dh"], s["dy"], s["h"], s["branch"], **same)
            out.update({k: getattr(d, k) for k in ("dx", "dbranch", "dgate", "dpost_weight",
                                                   "dpre_weight") if getattr(d, k) is not None})
        return out
    keep = c["train"] and c["act"] != "none"
    got = rr.block_linear(s["x"], s["w"], s["bias"], act=c["act"], residual=s["residual"],
                          offsets=s["offsets"], save_preact=keep)
    out = {"out": got[0], "z": got[1]} if keep else {"out": got}
    if c["train"]:
        d = rr.block_linear_backward(s["dout"], s["x"], s["w"], s["z"], act=c["act"],
                                     offsets=s["offsets"], need_db=s["bias"] is not None)
        out.update(dx=d.dx, dw=d.dw)
        if d.db is not None:
            out["db"] = d.db
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- 64 bits --

def _exact_pairs(sources):
    """The rows in use, and the (token, choice) pair of each."""
    row = torch.nonzero(sources >= 0)[:, 0]
    return row, sources[row].long()


def _exact_rms(v):
    return torch.sqrt(torch.linalg.vecdot(v, v)[:, None] / v.shape[1] + EPS)


def _logistic(z):
    return torch.special.expit(z)


_CURVES = {
    "none": (lambda z: z, lambda z: torch.ones_like(z)),
    "relu": (lambda z: torch.maximum(z, torch.zeros_like(z)), lambda z: torch.heaviside(z, torch.zeros_like(z))),
    "sigmoid": (_logistic, lambda z: _logistic(z) * _logistic(-z)),
    "silu": (lambda z: z * _logistic(z), lambda z: _logistic(z) + z * _logistic(z) * _logistic(-z)),
    "gelu": (lambda z: z * torch.special.ndtr(z),
             lambda z: torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)),
}


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "sort":
        flat = s["ids"].cpu().numpy().reshape(-1)
        count = np.array([int((flat == e).sum()) for e in range(c["experts"])])
        slots = np.full(flat.size, -1, np.int32)
        first = np.concatenate([[0], np.cumsum(count)])
        for e in range(c["experts"]):
            at = np.flatnonzero(flat == e)
            if c["capacity"]:
                at = at[:c["capacity"]]
            slots[at] = (e * c["capacity"] if c["capacity"] else first[e]) + np.arange(at.size)
        sources = np.full(c["experts"] * c["capacity"] if c["capacity"] else flat.size, -1, np.int32)
        sources[slots[slots >= 0]] = np.flatnonzero(slots >= 0)
        offsets = np.arange(c["experts"] + 1) * c["capacity"] if c["capacity"] else first
        return {"slots": slots.reshape(-1, c["k"]), "sources": sources,
                "counts": count.astype(np.int32), "offsets": offsets.astype(np.int32)}
    if c["op"] in ("dispatch", "combine"):
        row, pair = _exact_pairs(s["sources"])
        token = pair // c["k"]
        big = lambda n: torch.zeros(n, c["hidden"], dtype=torch.float64, device="cuda")  # noqa: E731
        if c["op"] == "dispatch":
            rows = big(s["sources"].numel())
            rows[row] = s["x"].double()[token]
            out = {"rows": rows}
            if c["train"]:
                out["dx"] = big(c["tokens"]).index_add_(0, token, s["drows"].double()[row])
            return out
        w = s["weights"].double().reshape(-1)[pair]
        y = s["rows"].double()[row]
        out = {"out": big(c["tokens"]).index_add_(0, token, y * w[:, None])}
        if c["train"]:
            d = s["dout"].double()[token]
            drows = big(s["sources"].numel())
            drows[row] = d * w[:, None]
            dw = torch.zeros(c["tokens"] * c["k"], dtype=torch.float64, device="cuda")
            dw[pair] = torch.linalg.vecdot(d, y)
            out.update(drows=drows, dweights=dw.reshape(c["tokens"], c["k"]))
        return out
    if c["op"] == "norm":
        return _exact_norm(c, s)
    return _exact_linear(c, s)


def _exact_norm(c, s):
    wide = lambda v: None if v is None else v.double()  # noqa: E731
    x, b, g = wide(s["x"]), wide(s["branch"]), wide(s["gate"])
    wp, wn = wide(s["post_weight"]), wide(s["pre_weight"])
    curve, slope = _CURVES[c["gate_act"]]
    scale = _exact_rms(b) if c["post"] else 1.0
    unit = b / scale
    n = unit * wp if c["post"] else unit
    open_ = curve(g) if g is not None else 1.0
    h = RESIDUAL_SCALE * x + BRANCH_SCALE * open_ * n
    out = {"h": h}
    if c["pre"]:
        out["y"] = h / _exact_rms(h) * wn
    if not c["train"]:
        return out
    dh = wide(s["dh"])
    if c["pre"]:
        h = wide(s["h"])
        size = _exact_rms(h)
        unit_h, p = h / size, wide(s["dy"]) * wn
        out["dpre_weight"] = torch.linalg.vecdot(wide(s["dy"]), unit_h, dim=0)
        dh = dh + (p - unit_h * torch.linalg.vecdot(p, unit_h)[:, None] / c["hidden"]) / size
    out["dx"] = RESIDUAL_SCALE * dh
    if g is not None:
        dg = BRANCH_SCALE * dh * n
        out["dgate"] = dg * slope(g) if c["gate"] == "element" else (dg * slope(g)).sum(0)
    dn = BRANCH_SCALE * dh * open_
    if c["post"]:
        out["dpost_weight"] = torch.linalg.vecdot(dn, unit, dim=0)
        p = dn * wp
        dn = (p - unit * torch.linalg.vecdot(p, unit)[:, None] / c["hidden"]) / scale
    out["dbranch"] = dn
    return out


def _exact_linear(c, s):
    if work(c)["flops"] > 4e12:
        return None
    edges = [0, c["rows"]] if s["offsets"] is None else s["offsets"].tolist()
    ws = s["w"].reshape(-1, c["n"], c["k"])
    bs = None if s["bias"] is None else s["bias"].reshape(-1, c["n"]).double()
    curve, slope = _CURVES[c["act"]]
    parts = []
    for e, (lo, hi) in enumerate(zip(edges[:-1], edges[1:])):
        w, x = ws[e].double(), s["x"][lo:hi].double()
        z = torch.mm(x, w.t().contiguous())
        if bs is not None:
            z += bs[e]
        p = {"out": curve(z)}
        if s["residual"] is not None:
            p["out"] = p["out"] + s["residual"][lo:hi].double()
        if c["train"]:
            d = s["dout"][lo:hi].double()
            if c["act"] != "none":
                p["z"] = z
                d = d * slope(s["z"][lo:hi].double())
            p["dx"], p["dw"], p["db"] = torch.mm(d, w), torch.mm(d.t().contiguous(), x)[None], d.sum(0)[None]
        parts.append(p)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if c["train"]:
        out["dw"] = out["dw"].reshape(s["w"].shape)
        out["db"] = out["db"].reshape(s["w"].shape[:-1])
        if s["bias"] is None:
            del out["db"]
    return out
