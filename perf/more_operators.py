"""Cases and plain forms of a block's gated projections and of its 8-bit operators.

The 8-bit format: e4m3 values with a 32-bit scale for each block of 128, 128 columns of a row for
activations, 128 x 128 of a matrix for weights; an element stands for its value times its scale.

* ``quantize``    values to the 8-bit format and back (``block_quantize``, ``block_dequantize``);
* ``linear8``     activations to 8 bits and their product with 8-bit weights, with bias, activation
                  and residual, dense or over the sorted rows of experts, and all gradients
                  (``block_linear8``, ``block_linear8_backward``);
* ``gated``       act(x Wg^T + bg) * (x Wu^T + bu), dense or over the sorted rows of experts, in 16 or
                  8 bits, and all gradients (``block_gated``, ``block_gated_backward``);
* ``checkpoint``  the same in training with what the backward pass reads kept in 8 bits: x, and both
                  projections; the backward pass makes the product again from them.

``run`` computes an operator in its plain form, elementary torch operations in 32 bits rounded
once at the end, or, where ``own`` is true, by the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
BLOCK = 128
LARGEST = 448.0                                     # of e4m3


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the activations of a few requests, one decoding step
        {"name": "quantize decode", "op": "quantize", "dtype": "bf16", "groups": 1, "rows": 16,
         "k": 4096, "square": False},
        # a training batch's activations
        {"name": "quantize train", "op": "quantize", "dtype": "bf16", "groups": 1, "rows": 16384,
         "k": 8192, "square": False},
        # one token being decoded: the weights are read once
        {"name": "linear8 token", "op": "linear8", "dtype": "bf16", "rows": 1, "n": 8192, "k": 8192,
         "groups": 1, "act": "none", "bias": True, "residual": True, "train": False},
        # a short prompt through odd sizes
        {"name": "linear8 odd", "op": "linear8", "dtype": "fp16", "rows": 1001, "n": 1111, "k": 1777,
         "groups": 1, "act": "gelu", "bias": True, "residual": False, "train": False},
        # a long prompt or one accumulation step's forward
        {"name": "linear8 prefill", "op": "linear8", "dtype": "bf16", "rows": 8192, "n": 8192,
         "k": 4096, "groups": 1, "act": "silu", "bias": True, "residual": True, "train": False},
        # a training step over the sorted rows of 8 experts of uneven load
        {"name": "linear8 experts", "op": "linear8", "dtype": "bf16", "rows": 16384, "n": 8192,
         "k": 2048, "groups": 8, "act": "silu", "bias": True, "residual": False, "train": True},
        # one token being decoded
        {"name": "gated token", "op": "gated", "dtype": "bf16", "bits": 16, "rows": 1, "n": 8192,
         "k": 4096, "groups": 1, "act": "silu", "bias": False, "train": False},
        # a decoding step of 64 requests, 4 of 32 experts each, weights in 8 bits
        {"name": "gated decode", "op": "gated", "dtype": "bf16", "bits": 8, "rows": 256, "n": 2048,
         "k": 4096, "groups": 32, "act": "silu", "bias": False, "train": False},
        # a short training step through odd sizes
        {"name": "gated odd", "op": "gated", "dtype": "fp16", "bits": 16, "rows": 777, "n": 1111,
         "k": 1777, "groups": 1, "act": "gelu", "bias": True, "train": True},
        # a training step over the sorted rows of 8 experts of uneven load
        {"name": "gated experts", "op": "gated", "dtype": "bf16", "bits": 16, "rows": 16384,
         "n": 4096, "k": 2048, "groups": 8, "act": "silu", "bias": True, "train": True},
        # a small training step that keeps its activations in 8 bits, ragged columns
        {"name": "checkpoint small", "op": "checkpoint", "dtype": "bf16", "rows": 520, "n": 1000,
         "k": 1032, "groups": 1, "act": "gelu"},
        # the step over experts, its activations kept in 8 bits
        {"name": "checkpoint experts", "op": "checkpoint", "dtype": "bf16", "rows": 16384, "n": 4096,
         "k": 2048, "groups": 8, "act": "silu"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear8", "linear8", "gated", "gated", "checkpoint"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "quantize":
        square = rng.random() < 0.4
        groups, rows, k = rng.choice([1, 1, 5]) if square else 1, _log(rng, 1, 65536), _log(rng, 64, 16384)
        if rng.random() < 0.7:                      # most layers have round widths
            k = (k + 7) // 8 * 8
        while groups * rows * k > 16384 * 8192:
            rows = rows // 2 + 1
        return {"op": op, "dtype": rng.choice([dtype, dtype, "fp32"]), "groups": groups, "rows": rows,
                "k": k, "square": square}
    groups = rng.choice([1, 1, 1, 3, 16])
    rows = _log(rng, 32 if op == "checkpoint" else 1, 16384)
    n, k = _log(rng, 64, 8192 if op == "linear8" else 4096), _log(rng, 64, 8192)
    if rng.random() < 0.7:
        n, k = (n + 7) // 8 * 8, (k + 7) // 8 * 8
    halves = 1 if op == "linear8" else 2
    while rows * n * halves * k > 16384 * 8192 * 2048:
        rows = rows // 2 + 1
    c = {"op": op, "dtype": dtype, "rows": rows, "n": n, "k": k, "groups": groups}
    if op == "linear8":
        return {**c, "act": rng.choice(["none", "relu", "gelu", "silu"]), "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.5, "train": rng.random() < 0.4}
    c["act"] = rng.choice(["silu", "silu", "gelu", "relu", "sigmoid", "none"])
    if op == "checkpoint":
        return c
    bits = rng.choice([16, 16, 8])
    return {**c, "bits": bits, "bias": rng.random() < 0.4, "train": rng.random() < 0.4}


def _columns(c):
    return c["n"] if c["op"] == "linear8" else 2 * c["n"]


def work(case):
    c = case
    e = BYTES[c["dtype"]]
    if c["op"] == "quantize":                       # values in; 8 bits out, and in again; values out
        v = c["groups"] * c["rows"] * c["k"]
        return {"bytes": v * (e + 1 + 1 + 2) + v // (BLOCK if not c["square"] else BLOCK * BLOCK) * 8,
                "flops": 0}
    m, n, k, g = c["rows"], c["n"], c["k"], c["groups"]
    wide, train = _columns(c), c.get("train", True)
    x_out = 0                                       # the 8-bit form of x, where it is kept
    if c["op"] == "linear8" or c.get("bits") == 8:
        w_bytes = g * wide * k
        x_out = m * k if train else 0
    else:
        w_bytes = g * wide * k * e
    if c["op"] == "checkpoint":
        x_out = m * k
    b = e * m * k + x_out + w_bytes + e * m * n * (1 + c.get("residual", False))
    if train:
        kept = 1 if c["op"] == "checkpoint" else e if c["op"] == "gated" or c["act"] != "none" else 0
        b += 2 * kept * m * wide                    # z out, and in again
        b += e * m * n                              # dout
        b += x_out if x_out else e * m * k          # x again
        b += w_bytes + e * m * k + e * g * wide * k     # w again; dx, dw out
        b += e * m * n if c["op"] == "checkpoint" else 0    # the product again
    return {"bytes": b, "flops": 2 * m * wide * k * (3 if train else 1)}


# ----------------------------------------------------------------- inputs --

def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _padded(x, dim):
    """x in 32 bits, zeros behind up to whole blocks along ``dim``."""
    extra = -x.shape[dim] % BLOCK
    if not extra:
        return x.float()
    shape = list(x.shape)
    shape[dim] = extra
    return torch.cat([x.float(), x.new_zeros(shape, dtype=torch.float32)], dim)


def _blocks(x, square):
    """x as [..., row blocks, rows of a block, column blocks, 128], and its largest finite
    magnitudes, one for each block."""
    p = _padded(_padded(x, -2), -1) if square else _padded(x, -1)
    high = BLOCK if square else 1
    b = p.reshape(*p.shape[:-2], p.shape[-2] // high, high, p.shape[-1] // BLOCK, BLOCK)
    a = torch.where(torch.isfinite(b), b.abs(), 0.0).amax((-3, -1))
    return b, a


def _two_power(a):
    """The least power of two p, from 2^-126, with a / p <= 448; 1 for a = 0."""
    m, e = torch.frexp(a)                           # a = m 2^e, 1/2 <= m < 1; 448 = 7/8 2^9
    p = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    return torch.where(a == 0, 1.0, ((p + 127) << 23).view(torch.float32))


def _plain_quantize(x, square=False, two_power=True):
    """(values, scales) of x: e4m3, and 32 bits a block."""
    b, a = _blocks(x, square)
    scale = _two_power(a) if two_power else torch.where(a == 0, 1.0, a / LARGEST)
    v = torch.where(torch.isfinite(b), b, math.nan) / scale[..., :, None, :, None]
    v = v.reshape(*v.shape[:-4], v.shape[-4] * v.shape[-3], -1)[..., :x.shape[-2], :x.shape[-1]]
    return v.to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


def _plain_back(q, square=False):
    """What (values, scales) stands for, in 32 bits."""
    v, s = q
    high = s.repeat_interleave(BLOCK, -2)[..., :v.shape[-2], :] if square else s
    return v.float() * high.repeat_interleave(BLOCK, -1)[..., :v.shape[-1]]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    dt = DTYPES[c["dtype"]]
    if c["op"] == "quantize":
        shape = (c["groups"], c["rows"], c["k"]) if c["groups"] > 1 else (c["rows"], c["k"])
        spread = torch.exp(_normal(g, c["k"]))             # channels of uneven size
        s["x"] = (_normal(g, *shape) * spread).to(dt)
        return s
    m, n, k, e = c["rows"], c["n"], c["k"], c["groups"]
    lead = ((e,) if e > 1 else ()) + (() if c["op"] == "linear8" else (2,))
    s["x"] = _normal(g, m, k, dtype=dt)
    w = _normal(g, *lead, n, k, dtype=dt, scale=k ** -0.5)
    if c["op"] == "linear8" or c.get("bits") == 8:
        # a training step makes its 8-bit weights itself, a file of weights brings scales of its own
        w = _plain_quantize(w, True, c["train"])
    s["w"] = w
    s["bias"] = _normal(g, *lead, n, dtype=dt, scale=0.5) if c.get("bias") else None
    s["residual"] = _normal(g, m, n, dtype=dt) if c.get("residual") else None
    s["dout"] = _normal(g, m, n, dtype=dt) if c.get("train", True) else None
    # the pre-activation an earlier pass stored
    keep = c["op"] != "checkpoint" and c["train"] and (c["op"] == "gated" or c["act"] != "none")
    s["z"] = _normal(g, m, _columns(c), dtype=dt) if keep else None
    s["offsets"], s["largest"] = None, m
    if e > 1:                                       # rows of each expert, uneven, some maybe none
        r = np.random.RandomState(seed % (1 << 31))
        sizes = r.multinomial(m, r.dirichlet([3.0] * e))
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        s["offsets"], s["largest"] = torch.from_numpy(off).cuda(), max(1, int(sizes.max()))
    return s


# ------------------------------------------------------------ plain forms --

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
    if act in ("silu", "sigmoid"):
        q = 1 / (1 + torch.exp(-z))
        return q * (1 - q) if act == "sigmoid" else q * (1 + z * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _apart(s, v):
    """Sorted rows v as [groups, largest, columns] in 32 bits, zeros after each group's rows, and
    the place of each row there; one group without offsets as it is."""
    if s["offsets"] is None:
        return v.float()[None], None
    r = torch.arange(v.shape[0], device="cuda", dtype=torch.int32)
    group = torch.searchsorted(s["offsets"][1:].contiguous(), r, right=True)
    place = group, r - s["offsets"][group]
    out = torch.zeros(s["case"]["groups"], s["largest"], v.shape[1], device="cuda")
    out[place] = v.float()
    return out, place


def _together(v, place):
    return v[0] if place is None else v[place]


def _forward(s, x, w):
    """x w^T + bias in 32 bits, of x [rows, k] and w [groups, columns, k] in 32 bits."""
    apart, place = _apart(s, x)
    z = torch.bmm(apart, w.transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"].float().reshape(w.shape[0], 1, -1)
    return _together(z, place)


def _backward(s, dz, x, w, shape):
    """dx, dw and db in 32 bits; dw and db of the weights' shape."""
    apart, place = _apart(s, dz)
    out = {"dx": _together(torch.bmm(apart, w), place).to(s["x"].dtype),
           "dw": torch.bmm(apart.transpose(1, 2), _apart(s, x)[0]).reshape(shape).to(s["x"].dtype)}
    if s["bias"] is not None:
        out["db"] = apart.sum(1).reshape(shape[:-1])
    return out


def _weights(s):
    """The weights in 32 bits as [groups, columns, k], and their shape."""
    w = s["w"]
    shape = w[0].shape if isinstance(w, tuple) else w.shape
    wide = _plain_back(w, True) if isinstance(w, tuple) else w.float()
    return wide.reshape(s["case"]["groups"], -1, shape[-1]), shape


def _run_plain(s):
    c, x = s["case"], s["x"]
    dt = x.dtype
    if c["op"] == "quantize":
        q = _plain_quantize(x, c["square"])
        return {"back": _plain_back(q, c["square"]).to(torch.bfloat16), "scales": q[1]}
    w, shape = _weights(s)
    n, act = c["n"], c["act"]
    kept = _plain_back(_plain_quantize(x)) if c["op"] in ("linear8", "checkpoint") or c["bits"] == 8 else x
    z = _forward(s, x if c["op"] == "checkpoint" else kept, w)
    if c["op"] == "linear8":
        out = _act(z, act)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        got = {"out": out.to(dt)}
        if c["train"]:
            dz = s["dout"].float()
            if act != "none":
                got["z"] = z.to(dt)
                dz = dz * _act_slope(s["z"].float(), act)
            got.update(_backward(s, dz, kept, w, shape))
        return got
    got = {"out": (_act(z[:, :n], act) * z[:, n:]).to(dt)}
    if not c.get("train", True):
        return got
    if c["op"] == "checkpoint":
        z = z.to(dt).reshape(-1, 2, n)               # each half of a row by itself
        z = _plain_back(_plain_quantize(z)).reshape(-1, 2 * n)
    else:
        got["z"] = z.to(dt)
        z = s["z"].float()
    g, u, d = z[:, :n], z[:, n:], s["dout"].float()
    if c["op"] == "checkpoint":
        got["again"] = (_act(g, act) * u).to(dt)
    dz = torch.cat([d * u * _act_slope(g, act), d * _act(g, act)], 1)
    got.update(_backward(s, dz, kept, w, shape))
    return got


# ------------------------------------------------- the library's operators --

def _run_own(s):
    import ring_allreduce_amd as rr
    c, x, w = s["case"], s["x"], s["w"] if "w" in s else None
    if c["op"] == "quantize":
        q = rr.block_quantize(x, square=c["square"])
        return {"back": rr.block_dequantize(q, torch.bfloat16), "scales": q.scales}
    if isinstance(w, tuple):
        w = rr.Quantized(w[0], w[1], square=True)
    same = dict(act=c["act"], offsets=s["offsets"])
    if c["op"] == "linear8":
        kept = rr.block_quantize(x)
        keep = c["train"] and c["act"] != "none"
        got = rr.block_linear8(kept, w, s["bias"], residual=s["residual"], save_preact=keep,
                               dtype=x.dtype, **same)
        out = {"out": got[0], "z": got[1]} if keep else {"out": got}
        if c["train"]:
            d = rr.block_linear8_backward(s["dout"], kept, w, s["z"], need_db=s["bias"] is not None,
                                          **same)
            out.update(dx=d.dx, dw=d.dw)
            if d.db is not None:
                out["db"] = d.db
        return out
    if c["op"] == "checkpoint":
        out, z = rr.block_gated(x, w, save_preact="e4m3", **same)
        kept = rr.block_quantize(x)
        d = rr.block_gated_backward(s["dout"], kept, w, z, need_db=False, need_out=True, **same)
        return {"out": out, "again": d.out, "dx": d.dx, "dw": d.dw}
    kept = rr.block_quantize(x) if c["bits"] == 8 else x
    if not c["train"]:
        return {"out": rr.block_gated(kept, w, s["bias"], dtype=x.dtype, **same)}
    out, z = rr.block_gated(kept, w, s["bias"], save_preact=True, dtype=x.dtype, **same)
    d = rr.block_gated_backward(s["dout"], kept, w, s["z"], need_db=s["bias"] is not None, **same)
    got = {"out": out, "z": z, "dx": d.dx, "dw": d.dw}
    if d.db is not None:
        got["db"] = d.db
    return got


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- 64 bits --

def _exact_power(p):
    """2^p in 64 bits, to the bit (exp2 and pow may be a step off)."""
    return ((p.long() + 1023) << 52).view(torch.float64)


def _exact_scales(x, square):
    """The scale of each block, in 64 bits."""
    size = x.double().abs()
    size = size.masked_fill(~(size < math.inf), 0.0)
    area = (BLOCK if square else 1, BLOCK)
    top = torch.nn.functional.max_pool2d(size.reshape(-1, 1, *size.shape[-2:]), area, ceil_mode=True)
    top = top.reshape(*size.shape[:-2], *top.shape[-2:])
    p = torch.ceil(torch.log2(top.clamp(min=LARGEST * 2.0 ** -126) / LARGEST))
    p = torch.where(LARGEST * _exact_power(p - 1) >= top, p - 1, p)       # where log2 was rounded up
    return torch.where(top > 0, _exact_power(p.clamp(min=-126.0)), 1.0)


def _exact_e4m3(v):
    """v, up to 448 in size, at e4m3's steps: 2^-3 of its power of two, from 2^-9."""
    step = _exact_power(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_kept(x, square=False):
    """(what the 8 bits of x stand for, its scales) in 64 bits."""
    s = _exact_scales(x, square)
    r = torch.arange(x.shape[-2], device="cuda") // (BLOCK if square else 1)
    each = s[..., r, :][..., torch.arange(x.shape[-1], device="cuda") // BLOCK]
    return _exact_e4m3(x.double() / each) * each, s


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


def _exact_weights(w, groups):
    if isinstance(w, tuple):
        v, s = w
        r = torch.arange(v.shape[-2], device="cuda") // BLOCK
        w = v.double() * s.double()[..., r, :][..., torch.arange(v.shape[-1], device="cuda") // BLOCK]
    return w.double().reshape(groups, -1, w.shape[-1])


def exact(case, seed):
    c = dict(case)
    if c["op"] != "quantize" and work(c)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    x = s["x"]
    if c["op"] == "quantize":
        back, scales = _exact_kept(x, c["square"])
        return {"back": back, "scales": scales}
    dt, n, train = x.dtype, c["n"], c.get("train", True)
    curve, slope = _CURVES[c["act"]]
    shape = s["w"][0].shape if isinstance(s["w"], tuple) else s["w"].shape
    ws = _exact_weights(s["w"], c["groups"])
    kept = _exact_kept(x)[0] if c["op"] in ("linear8", "checkpoint") or c["bits"] == 8 else x.double()
    seen = x.double() if c["op"] == "checkpoint" else kept
    bs = None if s["bias"] is None else s["bias"].double().reshape(c["groups"], -1)
    edges = [0, c["rows"]] if s["offsets"] is None else s["offsets"].tolist()
    parts = []
    for e, (lo, hi) in enumerate(zip(edges[:-1], edges[1:])):
        z = torch.mm(seen[lo:hi], ws[e].t().contiguous())
        if bs is not None:
            z += bs[e]
        d = s["dout"][lo:hi].double() if train else None
        if c["op"] == "linear8":
            p = {"out": curve(z)}
            if s["residual"] is not None:
                p["out"] = p["out"] + s["residual"][lo:hi].double()
            if train and c["act"] != "none":
                p["z"] = z
                d = d * slope(s["z"][lo:hi].double())
        else:
            p = {"out": curve(z[:, :n]) * z[:, n:]}
            if train:
                if c["op"] == "checkpoint":
                    if hi > lo:
                        z = _exact_kept(z.to(dt).unflatten(1, (2, n)))[0].flatten(1)
                    p["again"] = curve(z[:, :n]) * z[:, n:]
                else:
                    p["z"], z = z, s["z"][lo:hi].double()
                d = torch.cat([d * z[:, n:] * slope(z[:, :n]), d * curve(z[:, :n])], 1)
        if train:
            p["dx"], p["db"] = torch.mm(d, ws[e]), d.sum(0)[None]
            p["dw"] = torch.mm(d.t().contiguous(), kept[lo:hi])[None]
        parts.append(p)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if train:
        out["dw"] = out["dw"].reshape(shape)
        out["db"] = out["db"].reshape(shape[:-1])
        if s["bias"] is None:
            del out["db"]
    return out
