"""A block's operators between two collectives -- Python binding.

Tokens sorted by expert and moved to the AlltoAll's blocks and back, the norms
around a block, and a block's matrix products, plain and gated, in 16 and in 8 bits,
with their gradients, as declared in ``include/rr.h``.  Like the rest of the binding this only marshals: it checks
shapes and types, makes output and scratch tensors, and calls the library; there
is no fallback.  Calls in their usual form (on the current device and stream, new
outputs) are marshalled by the module ``_block``, in C++, which is bound to the torch it
was built with; what it does not take it leaves to the Python here, which also says what
is wrong with a call.

Every call runs on ``stream`` (default: torch's current stream of the tensors'
device); the outputs and scratch it allocates belong to that stream, and inputs of
another stream are the caller's to keep until it is done.  Matrices may have any row
stride (of the products: up to 2^22 elements) as long as the elements of a row are
neighbours.

There is no autograd here: outputs have no history, whether or not an input requires a
gradient, and each operator's gradients are a function of their own, ``*_backward``.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import warnings
from dataclasses import dataclass

import torch

_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t

FLOAT_DTYPES = {torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "sigmoid": 4}
GATES = {"none": 0, "channel": 1, "element": 2}


class _Rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("ld", _sz)]


class _Norm(ctypes.Structure):
    _fields_ = [("tokens", _sz), ("hidden", _sz), ("dt", ctypes.c_int32),
                ("weight_dt", ctypes.c_int32), ("post_norm", ctypes.c_int32),
                ("pre_norm", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("gate_act", ctypes.c_int32), ("residual_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("x", _Rows), ("branch", _Rows), ("gate", _Rows),
                ("post_weight", _vp), ("pre_weight", _vp), ("h", _Rows), ("y", _Rows)]


class _NormGrad(ctypes.Structure):
    _fields_ = [("dh", _Rows), ("dy", _Rows), ("dx", _Rows), ("dbranch", _Rows),
                ("dgate", _Rows), ("dgate_channel", _vp), ("dpost_weight", _vp),
                ("dpre_weight", _vp)]


class _Linear(ctypes.Structure):
    _fields_ = [("rows", _sz), ("n", _sz), ("k", _sz), ("groups", ctypes.c_int32),
                ("dt", ctypes.c_int32), ("act", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("offsets", _vp), ("x", _Rows), ("w", _vp), ("w_ld", _sz), ("w_stride", _sz),
                ("bias", _vp), ("residual", _Rows), ("z", _Rows), ("out", _Rows)]


class _LinearGrad(ctypes.Structure):
    _fields_ = [("dout", _Rows), ("dx", _Rows), ("dw", _vp), ("db", _vp),
                ("dw_dt", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _Linear8(ctypes.Structure):
    _fields_ = [("l", _Linear), ("x_scales", _vp), ("w_scales", _vp), ("z_scales", _vp)]


class _GatedGrad(ctypes.Structure):
    _fields_ = [("dout", _Rows), ("dx", _Rows), ("dw", _vp), ("db", _vp), ("out", _Rows),
                ("dw_dt", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _Quantize(ctypes.Structure):
    _fields_ = [("groups", _sz), ("rows", _sz), ("width", _sz), ("dt", ctypes.c_int32),
                ("square", ctypes.c_int32), ("x", _Rows), ("x_stride", _sz), ("q", _Rows),
                ("q_stride", _sz), ("scales", _vp)]


class _Absent:
    """In the place of the module ``_block``: takes no call, so that all are marshalled here."""

    def __getattr__(self, name):
        return lambda *args: None


def _bind(sig):
    """Declares the library's functions with the binding's ``sig``; called once, when
    librr.so is loaded."""
    p = ctypes.POINTER
    g = globals()
    try:
        from . import _block
    except ImportError as e:
        warnings.warn(f"{__package__}._block cannot be loaded ({e}); the calls of a block's "
                      "operators are marshalled in Python", RuntimeWarning, stacklevel=3)
        _block = _Absent()
    g["_block"] = _block
    g["_expert_sort"] = sig("expert_sort", _i, _vp, _i, _sz, _sz, _i, _i, _sz, _vp, _vp, _vp, _vp,
                            _vp, _sz, _vp)
    g["_expert_sort_workspace"] = sig("expert_sort_workspace", _i, _sz, _i, _i, p(_sz))
    g["_expert_dispatch"] = sig("expert_dispatch", _i, _Rows, _sz, _sz, _i, _i, _vp, _vp, _sz,
                                _Rows, _vp)
    g["_expert_dispatch_scales"] = sig("expert_dispatch_scales", _i, _Rows, _sz, _sz, _i, _vp, _vp, _sz,
                                       _Rows, _vp)
    g["_expert_combine"] = sig("expert_combine", _i, _Rows, _sz, _sz, _i, _vp, _vp, _sz, _i, _Rows,
                               _vp)
    g["_expert_combine_backward"] = sig("expert_combine_backward", _i, _Rows, _Rows, _sz, _sz, _i,
                                        _vp, _vp, _vp, _sz, _i, _Rows, _vp, _vp)
    g["_block_norm"] = sig("block_norm", _i, p(_Norm), _vp)
    g["_block_norm_backward"] = sig("block_norm_backward", _i, p(_Norm), p(_NormGrad), _vp, _sz,
                                    _vp)
    g["_block_norm_backward_workspace"] = sig("block_norm_backward_workspace", _i, p(_Norm),
                                              p(_NormGrad), p(_sz))
    g["_block_linear"] = sig("block_linear", _i, p(_Linear), _vp, _sz, _vp)
    g["_block_linear_workspace"] = sig("block_linear_workspace", _i, p(_Linear), p(_sz))
    g["_block_linear_backward"] = sig("block_linear_backward", _i, p(_Linear), p(_LinearGrad), _vp,
                                      _sz, _vp)
    g["_block_linear_backward_workspace"] = sig("block_linear_backward_workspace", _i, p(_Linear),
                                                p(_LinearGrad), p(_sz))
    g["_block_quantize"] = sig("block_quantize", _i, p(_Quantize), _vp)
    g["_block_dequantize"] = sig("block_dequantize", _i, p(_Quantize), _vp)
    for name, grad in (("linear8", _LinearGrad), ("gated", _GatedGrad)):
        name = "block_" + name
        g["_" + name] = sig(name, _i, p(_Linear8), _vp, _sz, _vp)
        g[f"_{name}_workspace"] = sig(name + "_workspace", _i, p(_Linear8), p(_sz))
        g[f"_{name}_backward"] = sig(name + "_backward", _i, p(_Linear8), p(grad), _vp, _sz, _vp)
        g[f"_{name}_backward_workspace"] = sig(name + "_backward_workspace", _i, p(_Linear8), p(grad),
                                               p(_sz))


EXPORTED = ["expert_sort", "expert_sort_workspace", "expert_dispatch",
            "expert_dispatch_scales", "expert_combine",
            "expert_combine_backward", "block_norm", "block_norm_backward",
            "block_norm_backward_workspace", "block_linear", "block_linear_workspace",
            "block_linear_backward", "block_linear_backward_workspace", "block_quantize",
            "block_dequantize", "block_linear8", "block_linear8_workspace",
            "block_linear8_backward", "block_linear8_backward_workspace", "block_gated",
            "block_gated_workspace", "block_gated_backward", "block_gated_backward_workspace"]


def _check(status, what):
    if status != 0:
        from . import RRError
        raise RRError(status, what)


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device


class _Current:
    """The current stream of the current device: nothing to set, nothing to restore."""
    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *_):
        return False


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield _raw_stream(device.index)
            return
        s = stream
        if isinstance(s, int):
            s = torch.cuda.ExternalStream(s, device=device) if s else \
                torch.cuda.default_stream(device)
        with torch.cuda.stream(s):
            yield s.cuda_stream


def _on(device, stream):
    """The device and stream of a call, for its allocations and its launch; a context that
    gives the stream's handle.  A call on the current ones enters nothing: a small call's
    time is the host's, and torch's contexts are 4 us of it."""
    if stream is None and device.index == _current_device():
        return _Current(_raw_stream(device.index))
    return _switched(device, stream)


def _need(cond, what):
    if not cond:
        raise ValueError(what)


# Messages are made where a check fails: made beforehand they cost more than the checks.
def _matrix(t, name, device=None, dtype=None, rows=None, width=None):
    """``t`` as a matrix of neighbouring elements in a row; returns its _Rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on the same GPU")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    r, w = t.shape
    if rows is not None and r != rows:
        raise ValueError(f"{name} must have {rows} rows, not {r}")
    if width is not None and w != width:
        raise ValueError(f"{name} must have {width} columns, not {w}")
    if r == 0 or w == 0:
        return _Rows(t.data_ptr(), w or 1)
    ld, step = t.stride()
    if step != 1 and w != 1:
        raise ValueError(f"{name}: the elements of a row must be neighbours")
    if r == 1:
        ld = w
    elif ld < w:
        raise ValueError(f"{name}: rows overlap")
    return _Rows(t.data_ptr(), ld)


def _float_type(t, name):
    dt = FLOAT_DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}; use float32, bfloat16 or float16")
    return dt


def _vector(t, name, device, dtype, numel):
    """The address of a contiguous tensor of ``numel`` elements (None: any number)."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be on the same GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous() or (numel is not None and t.numel() != numel):
        raise ValueError(f"{name} must be contiguous" +
                         ("" if numel is None else f", with {numel} elements"))
    return t.data_ptr()


def _ints(t, name, device, numel=None):
    return _vector(t, name, device, torch.int32, numel)


def _row(t, name, device, dtype, numel):
    """A contiguous vector, or None."""
    return None if t is None else _vector(t, name, device, dtype, numel)


def _ordered(t, name, device, dtype, *shape):
    """A contiguous tensor of ``shape``, but for dimensions of 1, or flat; or None."""
    if t is None:
        return None
    at = _vector(t, name, device, dtype, math.prod(shape))
    if t.dim() != 1 and [n for n in t.shape if n != 1] != [n for n in shape if n != 1]:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    return at


def _new(rows, width, like):
    """A new matrix of ``like``'s type on its device, and its _Rows."""
    t = torch.empty((rows, width), dtype=like.dtype, device=like.device)
    return t, _Rows(t.data_ptr(), width or 1)


def _scratch(size, device):
    """``size`` bytes of scratch memory: (tensor or None, its address or None)."""
    if not size:
        return None, None
    t = torch.empty(size, dtype=torch.uint8, device=device)
    return t, t.data_ptr()


# ------------------------------------------------ tokens sorted by expert, and back

@dataclass
class ExpertOrder:
    """What ``expert_sort`` found: ``slots`` [tokens, k] (-1: none), ``sources`` [rows]
    (pair t * k + j, or -1), ``counts`` [experts], ``offsets`` [experts + 1]."""
    slots: torch.Tensor
    sources: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor


def expert_sort(ids, experts: int, capacity: int = 0, *, stream=None) -> ExpertOrder:
    """Orders the pairs (token, choice) of ``ids`` [tokens, k] (int32 or int64) by expert,
    stably.  Ids outside [0, experts) are masked out.  ``capacity`` 0 packs the experts'
    rows one after another (tokens * k rows); otherwise every expert has ``capacity``
    rows and later pairs are dropped."""
    if stream is None:
        done = _block.sort(ids, experts, capacity)
        if done is not None:
            return ExpertOrder(*done)
    _need(isinstance(ids, torch.Tensor) and ids.dim() == 2, "ids must be a matrix")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, not {ids.dtype}")
    _need(experts >= 1 and capacity >= 0, "experts must be positive and capacity not negative")
    at = _matrix(ids, "ids")
    tokens, k = ids.shape
    dev = ids.device
    with _on(dev, stream) as s:
        need = _sz()
        _check(_expert_sort_workspace(tokens, k, experts, need), "expert_sort")
        rows = experts * capacity if capacity else tokens * k
        slots = torch.empty((tokens, k), dtype=torch.int32, device=dev)
        sources = torch.empty(rows, dtype=torch.int32, device=dev)
        counts = torch.empty(experts, dtype=torch.int32, device=dev)
        offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
        work, wp = _scratch(need.value, dev)
        _check(_expert_sort(at.data, ids.element_size(), at.ld, tokens, k, experts, capacity,
                            slots.data_ptr(), sources.data_ptr(), counts.data_ptr(),
                            offsets.data_ptr(), wp, need.value, s), "expert_sort")
    return ExpertOrder(slots, sources, counts, offsets)


def _pairs(slots, name="slots"):
    if not isinstance(slots, torch.Tensor) or slots.dim() != 2:
        raise ValueError(f"{name} must be [tokens, k]")
    return slots.shape


def expert_dispatch(x, slots, sources, *, out=None, stream=None):
    """Copies each token's row to the rows of its slots: [len(sources), hidden].  Rows
    without a source become zero.  A Quantized ``x`` (a scale for each 128 of a row, an even
    number of columns) is dispatched as values and scales; rows without a source are zeros with
    scales of 1, as ``block_quantize`` gives them."""
    if isinstance(x, Quantized):
        _need(out is None, "out is for tensors only")
        _quantized(x, "x", False)
        v = x.values
        _need(v.dim() == 2 and v.shape[1] % 2 == 0 and v.stride(1) == 1 and
              (v.shape[0] < 2 or v.stride(0) % 2 == 0) and
              v.storage_offset() % 2 == 0, "x must be a matrix whose rows are whole pairs of values")
        _scales(x, "x", v.device)
        if v.shape[0] < 2:              # no distance between rows to speak of, odd or not
            v = v.as_strided(v.shape, (v.shape[1], 1))
        return Quantized(_dispatch(v.view(torch.bfloat16), slots, sources, None, stream).view(E4M3),
                         _dispatch(x.scales, slots, sources, None, stream, True))
    return _dispatch(x, slots, sources, out, stream)


def _dispatch(x, slots, sources, out, stream, scales=False):
    if stream is None and out is None:
        done = _block.dispatch(x, slots, sources, scales)
        if done is not None:
            return done
    dt = _float_type(x, "x")
    xr = _matrix(x, "x")
    tokens, k = _pairs(slots)
    _need(tokens == x.shape[0], "slots must have a row for each token")
    rows, hidden = sources.numel(), x.shape[1]
    with _on(x.device, stream) as s:
        sp, so = _ints(slots, "slots", x.device), _ints(sources, "sources", x.device)
        if out is None:
            out, o = _new(rows, hidden, x)
        else:
            o = _matrix(out, "out", x.device, x.dtype, rows, hidden)
        if scales:
            _check(_expert_dispatch_scales(xr, tokens, hidden, k, sp, so, rows, o, s), "expert_dispatch")
        else:
            _check(_expert_dispatch(xr, tokens, hidden, k, dt, sp, so, rows, o, s), "expert_dispatch")
    return out


def expert_combine(rows, slots, weights=None, *, out=None, stream=None):
    """Sum of each token's rows, times ``weights`` [tokens, k] (fp32; None: all 1), in the
    order of its choices: [tokens, hidden]."""
    if stream is None and out is None:
        done = _block.combine(rows, slots, weights)
        if done is not None:
            return done
    dt = _float_type(rows, "rows")
    r = _matrix(rows, "rows")
    tokens, k = _pairs(slots)
    hidden = rows.shape[1]
    with _on(rows.device, stream) as s:
        sp = _ints(slots, "slots", rows.device)
        wp = _ordered(weights, "weights", rows.device, torch.float32, tokens, k)
        if out is None:
            out, o = _new(tokens, hidden, rows)
        else:
            o = _matrix(out, "out", rows.device, rows.dtype, tokens, hidden)
        _check(_expert_combine(r, rows.shape[0], hidden, dt, sp, wp, tokens, k, o, s),
               "expert_combine")
    return out


def expert_dispatch_backward(drows, slots, *, out=None, stream=None):
    """Gradient of ``expert_dispatch`` by x: the sum of each token's rows of ``drows``."""
    return expert_combine(drows, slots, None, out=out, stream=stream)


def expert_combine_backward(dout, rows, slots, sources, weights=None, *, need_rows=True,
                            need_weights=True, out=None, stream=None):
    """Gradients of ``expert_combine``: (drows [len(sources), hidden] in the rows' type,
    dweights [tokens, k] in fp32); what is not needed is None."""
    if stream is None and out is None:
        done = _block.combine_backward(dout, rows, slots, sources, weights, need_rows, need_weights)
        if done is not None:
            return done
    dt = _float_type(dout, "dout")
    tokens, k = _pairs(slots)
    d = _matrix(dout, "dout", None, None, tokens)
    n, hidden = sources.numel(), dout.shape[1]
    dev = dout.device
    with _on(dev, stream) as s:
        r = _matrix(rows, "rows", dev, dout.dtype, n, hidden) if need_weights else _Rows()
        sp, so = _ints(slots, "slots", dev), _ints(sources, "sources", dev)
        wp = _ordered(weights, "weights", dev, torch.float32, tokens, k)
        drows = dweights = None
        o = _Rows()
        if need_rows:
            if out is None:
                drows, o = _new(n, hidden, dout)
            else:
                drows, o = out, _matrix(out, "out", dev, dout.dtype, n, hidden)
        if need_weights:
            dweights = torch.empty((tokens, k), dtype=torch.float32, device=dev)
        _check(_expert_combine_backward(d, r, n, hidden, dt, sp, so, wp, tokens, k, o,
                                        dweights.data_ptr() if need_weights else None, s),
               "expert_combine_backward")
    return drows, dweights


# ------------------------------------------------------------- the norms around a block

def _norm_args(like, branch, post_norm, post_weight, gate, gate_act, residual_scale, branch_scale,
               pre_norm, pre_weight, eps):
    a = _Norm()
    tokens, hidden = like.shape
    dev = like.device
    a.tokens, a.hidden, a.dt = tokens, hidden, _float_type(like, "x")
    a.post_norm, a.pre_norm = int(bool(post_norm)), int(bool(pre_norm))
    _need(gate_act in ("none", "sigmoid", "silu"), "gate_act must be none, sigmoid or silu")
    a.gate_act = ACTS[gate_act]
    a.residual_scale, a.branch_scale, a.eps = residual_scale, branch_scale, eps
    if branch is not None:
        a.branch = _matrix(branch, "branch", dev, like.dtype, tokens, hidden)
    _need(post_norm or post_weight is None, "post_weight without post_norm")
    _need(pre_norm or pre_weight is None, "pre_weight without pre_norm")
    _need(branch is not None or not (post_norm or gate is not None),
          "post_norm and gate need a branch")
    kinds = [w.dtype for w in (post_weight, pre_weight) if w is not None]
    if gate is not None and gate.dim() == 1:
        kinds.append(gate.dtype)
    wt = kinds[0] if kinds else like.dtype
    if any(w != wt for w in kinds) or wt not in (like.dtype, torch.float32):
        raise TypeError("weights and channel gate must share x's dtype or float32")
    a.weight_dt = FLOAT_DTYPES[wt]
    a.post_weight = _row(post_weight, "post_weight", dev, wt, hidden)
    a.pre_weight = _row(pre_weight, "pre_weight", dev, wt, hidden)
    if gate is None:
        _need(gate_act == "none", "gate_act without a gate")
    elif gate.dim() == 1:
        a.gate_kind = GATES["channel"]
        a.gate = _Rows(_row(gate, "gate", dev, wt, hidden), hidden)
    else:
        a.gate_kind = GATES["element"]
        a.gate = _matrix(gate, "gate", dev, like.dtype, tokens, hidden)
    return a


def block_norm(x, branch=None, *, post_norm=True, post_weight=None, gate=None, gate_act="none",
               residual_scale=1.0, branch_scale=1.0, pre_norm=True, pre_weight=None, eps=1e-6,
               h=None, y=None, stream=None):
    """The stream after a block and the next block's input.

    n = N(branch) * post_weight (post_norm) or branch; h = residual_scale * x +
    branch_scale * gate_act(gate) * n; y = N(h) * pre_weight (pre_norm), with N(v) =
    v / sqrt(mean(v^2) + eps).  ``gate`` is [hidden] or [tokens, hidden].  Returns (h, y);
    y is None without pre_norm.  Without a branch, pass post_norm=False; h is then
    residual_scale * x.  ``h`` may be x itself and ``y`` the branch (in place)."""
    if stream is None and h is None and y is None:
        done = _block.norm(x, branch, post_norm, post_weight, gate, ACTS.get(gate_act, -1),
                           residual_scale, branch_scale, pre_norm, pre_weight, eps)
        if done is not None:
            return done
    xr = _matrix(x, "x")
    a = _norm_args(x, branch, post_norm, post_weight, gate, gate_act, residual_scale, branch_scale,
                   pre_norm, pre_weight, eps)
    a.x = xr
    with _on(x.device, stream) as s:
        if h is None:
            h, a.h = _new(*x.shape, x)
        else:
            a.h = _matrix(h, "h", x.device, x.dtype, *x.shape)
        if pre_norm:
            if y is None:
                y, a.y = _new(*x.shape, x)
            else:
                a.y = _matrix(y, "y", x.device, x.dtype, *x.shape)
        else:
            _need(y is None, "y without pre_norm")
        _check(_block_norm(a, s), "block_norm")
    return h, y


@dataclass
class NormGrads:
    """Gradients of ``block_norm``; what does not apply or is not needed is None.  The
    weights' and the channel gate's gradients are fp32."""
    dx: torch.Tensor | None = None
    dbranch: torch.Tensor | None = None
    dgate: torch.Tensor | None = None
    dpost_weight: torch.Tensor | None = None
    dpre_weight: torch.Tensor | None = None


NORM_GRADS = ("dx", "dbranch", "dgate", "dpost_weight", "dpre_weight")


def block_norm_backward(dh, dy, h, branch=None, *, post_norm=True, post_weight=None, gate=None,
                        gate_act="none", residual_scale=1.0, branch_scale=1.0, pre_norm=True,
                        pre_weight=None, eps=1e-6, need=NORM_GRADS, stream=None) -> NormGrads:
    """Gradients of ``block_norm`` with the same arguments.  ``dh`` and ``dy`` are the
    gradients by h and y (dh None: zero; dy None without pre_norm); ``h`` is the stream
    that block_norm returned (not read without pre_norm)."""
    if stream is None:
        wanted = 31 if need is NORM_GRADS else sum(1 << i for i, n in enumerate(NORM_GRADS) if n in need)
        done = _block.norm_backward(dh, dy, h, branch, post_norm, post_weight, gate,
                                    ACTS.get(gate_act, -1), residual_scale, branch_scale, pre_norm,
                                    pre_weight, eps, wanted)
        if done is not None:
            return NormGrads(*done)
    like = next((t for t in (dh, dy, h, branch) if t is not None), None)
    _need(like is not None and like.dim() == 2, "dh, dy or h must be given")
    a = _norm_args(like, branch, post_norm, post_weight, gate, gate_act, residual_scale,
                   branch_scale, pre_norm, pre_weight, eps)
    dev, dtype, shape = like.device, like.dtype, like.shape
    g, out = _NormGrad(), NormGrads()
    _need(pre_norm == (dy is not None), "dy is given exactly with pre_norm")
    if dh is not None:
        g.dh = _matrix(dh, "dh", dev, dtype, *shape)
    if pre_norm:
        _need(h is not None, "pre_norm needs h")
        g.dy = _matrix(dy, "dy", dev, dtype, *shape)
        a.h = _matrix(h, "h", dev, dtype, *shape)
    with _on(dev, stream) as s:
        def rows(name):
            t, r = _new(*shape, like)
            setattr(out, name, t)
            return r

        def sums(name):
            t = torch.empty(shape[1], dtype=torch.float32, device=dev)
            setattr(out, name, t)
            return t.data_ptr()

        if "dx" in need:
            g.dx = rows("dx")
        if "dbranch" in need and branch is not None:
            g.dbranch = rows("dbranch")
        if "dgate" in need and a.gate_kind == GATES["element"]:
            g.dgate = rows("dgate")
        if "dgate" in need and a.gate_kind == GATES["channel"]:
            g.dgate_channel = sums("dgate")
        if "dpost_weight" in need and post_weight is not None:
            g.dpost_weight = sums("dpost_weight")
        if "dpre_weight" in need and pre_weight is not None:
            g.dpre_weight = sums("dpre_weight")
        size = _sz()
        _check(_block_norm_backward_workspace(a, g, size), "block_norm_backward")
        work, wp = _scratch(size.value, dev)
        _check(_block_norm_backward(a, g, wp, size.value, s), "block_norm_backward")
    return out


# ------------------------------------------------------------- a block's matrix products

def _linear_args(x, w, offsets, act):
    a = _Linear()
    dev, dtype = x.device, x.dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x: unsupported dtype {dtype}; use bfloat16 or float16")
    a.x = _matrix(x, "x")
    a.rows, a.k, a.dt = x.shape[0], x.shape[1], FLOAT_DTYPES[dtype]
    _need(isinstance(w, torch.Tensor) and w.dim() in (2, 3), "w must be [n, k] or [groups, n, k]")
    _need(w.device == dev, "w must be on the same GPU")
    if w.dtype != dtype:
        raise TypeError(f"w must be {dtype}, not {w.dtype}")
    _need(w.shape[-1] == a.k, f"w must have {a.k} columns, not {w.shape[-1]}")
    a.groups = w.shape[0] if w.dim() == 3 else 1
    _need(a.groups >= 1, "w must have at least one group")
    a.n = w.shape[-2]
    first = w[0] if w.dim() == 3 else w
    r = _matrix(first, "w")
    a.w, a.w_ld = r.data, r.ld
    a.w_stride = w.stride(0) if w.dim() == 3 else 0
    _need(act in ("none", "relu", "gelu", "silu"), "act must be none, relu, gelu or silu")
    a.act = ACTS[act]
    if offsets is not None:
        a.offsets = _ints(offsets, "offsets", dev, a.groups + 1)
    else:
        _need(a.rows % a.groups == 0, "without offsets the groups must divide the rows")
    return a


def block_linear(x, w, bias=None, *, act="none", residual=None, offsets=None, save_preact=False,
                 out=None, stream=None):
    """act(x w^T + bias) + residual, for x [rows, k] and w [n, k], or the rows of each group
    with its own w [groups, n, k] and bias [groups, n]: ``offsets`` (int32, groups + 1) as
    ``expert_sort`` gives them, or None for equal groups.  Rows of no group become zero.
    Returns out, or (out, z) with the pre-activation z = x w^T + bias that
    ``block_linear_backward`` needs if save_preact.  ``residual`` may be ``out``."""
    if stream is None and out is None:
        done = _block.linear(x, w, bias, ACTS.get(act, -1), residual, offsets, save_preact)
        if done is not None:
            return done
    a = _linear_args(x, w, offsets, act)
    dev, shape = x.device, (x.shape[0], a.n)
    a.bias = _ordered(bias, "bias", dev, x.dtype, a.groups, a.n)
    if residual is not None:
        a.residual = _matrix(residual, "residual", dev, x.dtype, *shape)
    with _on(dev, stream) as s:
        if out is None:
            out, a.out = _new(*shape, x)
        else:
            a.out = _matrix(out, "out", dev, x.dtype, *shape)
        z = None
        if save_preact:
            z, a.z = _new(*shape, x)
        size = _sz()
        _check(_block_linear_workspace(a, size), "block_linear")
        work, wp = _scratch(size.value, dev)
        _check(_block_linear(a, wp, size.value, s), "block_linear")
    return (out, z) if save_preact else out


@dataclass
class LinearGrads:
    """Gradients of ``block_linear``; what is not needed is None.  db is fp32."""
    dx: torch.Tensor | None = None
    dw: torch.Tensor | None = None
    db: torch.Tensor | None = None


def block_linear_backward(dout, x, w, z=None, *, act="none", offsets=None, need_dx=True,
                          need_dw=True, need_db=True, dw_dtype=None, stream=None) -> LinearGrads:
    """Gradients of ``block_linear`` by x, w and bias (the residual's is dout itself).
    ``z`` is the saved pre-activation, needed if act is set; ``dw_dtype`` x's dtype
    (default) or float32."""
    if stream is None and dw_dtype in (None, torch.float32):
        done = _block.linear_backward(dout, x, w, z, ACTS.get(act, -1), offsets, need_dx, need_dw,
                                      need_db, dw_dtype is not None)
        if done is not None:
            return LinearGrads(*done)
    a = _linear_args(x, w, offsets, act)
    dev = x.device
    g, out = _LinearGrad(), LinearGrads()
    g.dout = _matrix(dout, "dout", dev, x.dtype, x.shape[0], a.n)
    if act != "none":
        _need(z is not None, "act needs the pre-activation z")
        a.z = _matrix(z, "z", dev, x.dtype, x.shape[0], a.n)
    dw_dtype = dw_dtype or x.dtype
    if dw_dtype not in (x.dtype, torch.float32):
        raise TypeError(f"dw_dtype must be {x.dtype} or float32")
    g.dw_dt = FLOAT_DTYPES[dw_dtype]
    with _on(dev, stream) as s:
        if need_dx:
            out.dx, g.dx = _new(*x.shape, x)
        if need_dw:
            out.dw = torch.empty(w.shape, dtype=dw_dtype, device=dev)
            g.dw = out.dw.data_ptr()
        if need_db:
            out.db = torch.empty(w.shape[:-1], dtype=torch.float32, device=dev)
            g.db = out.db.data_ptr()
        size = _sz()
        _check(_block_linear_backward_workspace(a, g, size), "block_linear_backward")
        work, wp = _scratch(size.value, dev)
        _check(_block_linear_backward(a, g, wp, size.value, s), "block_linear_backward")
    return out


# ------------------------------------- 8-bit values with a scale for each block of 128

BLOCK = 128
E4M3 = torch.float8_e4m3fn


@dataclass
class Quantized:
    """8-bit values and the fp32 scales of their blocks: an element stands for its value times
    its block's scale.  ``values`` [..., rows, k] (float8_e4m3fn); ``scales`` [..., rows,
    ceil(k / 128)], one for 128 columns of a row, or, ``square``, [..., ceil(rows / 128),
    ceil(k / 128)], one for 128 rows by 128 columns."""
    values: torch.Tensor
    scales: torch.Tensor
    square: bool = False


def _blocks(n):
    return -(-n // BLOCK)


def _scales_shape(shape, square):
    return (*shape[:-2], _blocks(shape[-2]) if square else shape[-2], _blocks(shape[-1]))


def _scales(q, name, device):
    """The address of a Quantized's scales, their shape and place checked."""
    shape, s = _scales_shape(q.values.shape, q.square), q.scales
    if not isinstance(s, torch.Tensor) or s.device != device:
        raise ValueError(f"{name}.scales must be on the same GPU")
    if s.dtype != torch.float32:
        raise TypeError(f"{name}.scales must be torch.float32, not {s.dtype}")
    if tuple(s.shape) != shape or not s.is_contiguous():
        raise ValueError(f"{name}.scales must be contiguous, of shape {list(shape)}")
    return s.data_ptr()


def _quantized(q, name, square):
    if not isinstance(q.values, torch.Tensor) or q.values.dtype != E4M3:
        raise TypeError(f"{name}.values must be {E4M3}")
    _need(bool(q.square) == square, f"{name} must have " +
          ("square blocks" if square else "a scale for each 128 of a row, not square blocks"))


def _stack(t, name):
    """``t`` [..., rows, width] as matrices a stride apart: (groups, _Rows, stride)."""
    if not isinstance(t, torch.Tensor) or t.dim() < 2:
        raise ValueError(f"{name} must be a matrix, or matrices")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the same GPU")
    if t.dim() == 2:
        return 1, _matrix(t, name), 0
    try:
        s = t.view(-1, *t.shape[-2:]) if t.numel() else t.new_empty((0, *t.shape[-2:]))
    except RuntimeError:
        raise ValueError(f"{name}: its matrices must be one stride apart") from None
    if not s.shape[0]:
        return 0, _Rows(), 0
    return s.shape[0], _matrix(s[0], name), s.stride(0)


def _quantize_args(wide, q, dt):
    a = _Quantize()
    groups, a.x, a.x_stride = _stack(wide, "x")
    n, a.q, a.q_stride = _stack(q.values, "values")
    a.groups, a.rows, a.width = groups, wide.shape[-2], wide.shape[-1]
    a.dt, a.square = dt, int(q.square)
    a.scales = q.scales.data_ptr()
    return a


def block_quantize(x, *, square=False, stream=None) -> Quantized:
    """``x`` [..., rows, k] in e4m3 with a scale for each 128 columns of a row, or, ``square``,
    128 x 128 of a matrix: the least power of two with which the block's largest finite value is
    at most 448 (1 for zeros).  Values are rounded to the nearest, ties to even; NaN and
    infinities become NaN."""
    if stream is None:
        done = _block.quantize(x, square)
        if done is not None:
            return Quantized(*done, bool(square))
    _need(isinstance(x, torch.Tensor), "x must be a matrix, or matrices")
    dt = _float_type(x, "x")
    _need(x.dim() >= 2, "x must be a matrix, or matrices")
    _need(x.is_cuda, "x must be on a GPU")
    _need(x.shape[-1] > 0, "x must have columns")
    square = bool(square)
    with _on(x.device, stream) as s:
        q = Quantized(torch.empty(x.shape, dtype=E4M3, device=x.device),
                      torch.empty(_scales_shape(x.shape, square), device=x.device), square)
        if x.numel():
            _check(_block_quantize(_quantize_args(x, q, dt), s), "block_quantize")
    return q


def block_dequantize(q, dtype=torch.bfloat16, *, out=None, stream=None):
    """What ``q`` stands for, in ``dtype``, or in ``out``'s; a finite value beyond float16's largest becomes that."""
    if stream is None and out is None and isinstance(q, Quantized):
        done = _block.dequantize(q.values, q.scales, q.square, FLOAT_DTYPES.get(dtype, -1))
        if done is not None:
            return done
    if not isinstance(q, Quantized):
        raise TypeError("q must be Quantized")
    _quantized(q, "q", bool(q.square))
    _need(q.values.dim() >= 2 and q.values.is_cuda, "q must be matrices on a GPU")
    _need(q.values.shape[-1] > 0, "q must have columns")
    dev = q.values.device
    _scales(q, "q", dev)
    if out is not None:
        _need(isinstance(out, torch.Tensor), "out must be a tensor")
        dtype = out.dtype
        _need(out.device == dev and out.shape == q.values.shape, "out must have q's shape and GPU")
    if dtype not in FLOAT_DTYPES:
        raise TypeError(f"unsupported dtype {dtype}; use float32, bfloat16 or float16")
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty(q.values.shape, dtype=dtype, device=dev)
        if q.values.numel():
            _check(_block_dequantize(_quantize_args(out, q, FLOAT_DTYPES[dtype]), s), "block_dequantize")
    return out


_NOWHERE = 16       # in the place of an empty tensor's address: there, and read by nothing


def _operand(t, name, dev, dtype, rows=None, width=None):
    """The matrix x, in ``dtype`` or Quantized: (its _Rows, its scales' address or None)."""
    if not isinstance(t, Quantized):
        return _matrix(t, name, dev, dtype, rows, width), None
    _quantized(t, name, False)
    return _matrix(t.values, name, dev, E4M3, rows, width), \
        _scales(t, name, t.values.device if dev is None else dev) or _NOWHERE


def _wide_args(x, w, offsets, act, dtype, halves):
    """The _Linear8 of x [rows, k] and w [n, k] or [groups, n, k], with ``halves`` 2 [2, n, k] or
    [groups, 2, n, k], each in ``dtype`` or Quantized."""
    a = _Linear8()
    l = a.l
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"unsupported dtype {dtype}; use bfloat16 or float16")
    xv, wv = (t.values if isinstance(t, Quantized) else t for t in (x, w))
    if not isinstance(xv, torch.Tensor) or xv.dim() != 2:
        raise ValueError("x must be a matrix")
    dev = xv.device
    l.x, a.x_scales = _operand(x, "x", None, dtype)
    l.rows, l.k, l.dt = xv.shape[0], xv.shape[1], FLOAT_DTYPES[dtype]
    d = 2 if halves == 1 else 3
    _need(isinstance(wv, torch.Tensor) and wv.dim() in (d, d + 1),
          "w must be [n, k] or [groups, n, k]" if halves == 1 else "w must be [2, n, k] or [groups, 2, n, k]")
    _need(wv.device == dev, "w must be on the same GPU")
    if isinstance(w, Quantized):
        _quantized(w, "w", True)
        a.w_scales = _scales(w, "w", dev)
    elif wv.dtype != dtype:
        raise TypeError(f"w must be {dtype}, not {wv.dtype}")
    _need(wv.shape[-1] == l.k, f"w must have {l.k} columns, not {wv.shape[-1]}")
    l.groups = wv.shape[0] if wv.dim() > d else 1
    _need(l.groups >= 1, "w must have at least one group")
    l.n = wv.shape[-2]
    first = wv[0] if wv.dim() > d else wv
    if halves == 2:
        _need(first.shape[0] == 2, "w must hold two matrices, the gate's and the other projection's")
    r = _matrix(first[0] if halves == 2 else first, "w")
    l.w, l.w_ld = r.data, r.ld
    if halves == 2:
        if l.n == 1:
            l.w_ld = first.stride(0)
        _need(first.stride(0) == l.n * l.w_ld, "w: the second matrix must follow the first")
    l.w_stride = wv.stride(0) if wv.dim() > d else 0
    l.act = ACTS[act]
    if offsets is not None:
        l.offsets = _ints(offsets, "offsets", dev, l.groups + 1)
    else:
        _need(l.rows % l.groups == 0, "without offsets the groups must divide the rows")
    return a, dev


def _act_of(act, allowed):
    _need(act in allowed, "act must be " + ", ".join(allowed[:-1]) + " or " + allowed[-1])


_LINEAR_ACTS = ("none", "relu", "gelu", "silu")
_GATED_ACTS = ("none", "relu", "gelu", "silu", "sigmoid")


def block_linear8(x, w, bias=None, *, dtype=torch.bfloat16, act="none", residual=None, offsets=None,
                  save_preact=False, out=None, stream=None):
    """``block_linear`` of 8-bit operands: ``x`` Quantized [rows, k] with a scale for each 128 of a
    row, ``w`` Quantized [n, k] or [groups, n, k] with square blocks (``block_quantize``'s, or any
    others with finite fp32 scales).  ``dtype`` (bfloat16 or float16) is the type of bias, residual, z
    and out.  Sums are held in 32 bits, but for more rows than one the matrix instructions cut each
    of eight neighbouring products at 2^-13 of the power of two of the largest before they add them
    (``include/rr.h`` has the bound)."""
    if stream is None and out is None and isinstance(x, Quantized) and isinstance(w, Quantized) and \
            w.square and not x.square:
        done = _block.linear8(x.values, x.scales, w.values, w.scales, bias, ACTS.get(act, -1),
                              residual, offsets, save_preact, FLOAT_DTYPES.get(dtype, -1))
        if done is not None:
            return done
    if not isinstance(x, Quantized) or not isinstance(w, Quantized):
        raise TypeError("x and w must be Quantized")
    _act_of(act, _LINEAR_ACTS)
    a, dev = _wide_args(x, w, offsets, act, dtype, 1)
    l, shape = a.l, (x.values.shape[0], a.l.n)
    l.bias = _ordered(bias, "bias", dev, dtype, l.groups, l.n)
    if residual is not None:
        l.residual = _matrix(residual, "residual", dev, dtype, *shape)
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=dev)
        l.out = _matrix(out, "out", dev, dtype, *shape)
        z = None
        if save_preact:
            z = torch.empty(shape, dtype=dtype, device=dev)
            l.z = _matrix(z, "z", dev, dtype, *shape)
        size = _sz()
        _check(_block_linear8_workspace(a, size), "block_linear8")
        work, wp = _scratch(size.value, dev)
        _check(_block_linear8(a, wp, size.value, s), "block_linear8")
    return (out, z) if save_preact else out


def _dw_type(dw_dtype, dtype):
    dw_dtype = dw_dtype or dtype
    if dw_dtype not in (dtype, torch.float32):
        raise TypeError(f"dw_dtype must be {dtype} or float32")
    return dw_dtype


def _values(t):
    return t.values if isinstance(t, Quantized) else t


def block_linear8_backward(dout, x, w, z=None, *, act="none", offsets=None, need_dx=True, need_dw=True,
                           need_db=True, dw_dtype=None, stream=None) -> LinearGrads:
    """Gradients of ``block_linear8`` or ``block_linear`` by x, w and bias, at what ``x`` and ``w``
    stand for: each Quantized, as a forward pass used or kept it, or a tensor of ``dout``'s
    dtype.  A Quantized becomes that dtype on its way into the products: float16 has multiples of 2^-24
    up to 65504, and what is smaller or larger than its values becomes the nearest one."""
    if not isinstance(dout, torch.Tensor):
        raise ValueError("dout must be a matrix")
    dtype = dout.dtype
    if stream is None and dw_dtype in (None, torch.float32):
        done = _block.linear8_backward(
            dout, *_pair(x, False), *_pair(w, True), z, ACTS.get(act, -1), offsets, need_dx, need_dw,
            need_db, dw_dtype is not None)
        if done is not None:
            return LinearGrads(*done)
    _act_of(act, _LINEAR_ACTS)
    a, dev = _wide_args(x, w, offsets, act, dtype, 1)
    l, g, out = a.l, _LinearGrad(), LinearGrads()
    g.dout = _matrix(dout, "dout", dev, dtype, l.rows, l.n)
    if act != "none":
        _need(z is not None, "act needs the pre-activation z")
        l.z = _matrix(z, "z", dev, dtype, l.rows, l.n)
    dw_dtype = _dw_type(dw_dtype, dtype)
    g.dw_dt = FLOAT_DTYPES[dw_dtype]
    with _on(dev, stream) as s:
        _make_grads(g, out, _values(x), _values(w), dtype, dw_dtype, dev, need_dx, need_dw, need_db)
        size = _sz()
        _check(_block_linear8_backward_workspace(a, g, size), "block_linear8_backward")
        work, wp = _scratch(size.value, dev)
        _check(_block_linear8_backward(a, g, wp, size.value, s), "block_linear8_backward")
    return out


def _pair(t, square):
    """A Quantized's tensors, or a tensor and None, for the module ``_block``."""
    if isinstance(t, Quantized):
        return (t.values, t.scales) if bool(t.square) == square else (False, False)
    return t, None


def _make_grads(g, out, x, w, dtype, dw_dtype, dev, need_dx, need_dw, need_db):
    if need_dx:
        out.dx = torch.empty(x.shape, dtype=dtype, device=dev)
        g.dx = _Rows(out.dx.data_ptr(), x.shape[1] or 1)
    if need_dw:
        out.dw = torch.empty(w.shape, dtype=dw_dtype, device=dev)
        g.dw = out.dw.data_ptr()
    if need_db:
        out.db = torch.empty(w.shape[:-1], dtype=torch.float32, device=dev)
        g.db = out.db.data_ptr()


# ------------------------------------------------------- a block's gated projections

def block_gated(x, w, bias=None, *, act="silu", offsets=None, save_preact=False, dtype=None, out=None,
                stream=None):
    """act(g) * u for [g | u] = x w^T + bias: x [rows, k], w [2, n, k] (the gate's matrix, then
    the other projection's) and bias [2, n], or the rows of each group with its own w [groups, 2, n,
    k] and bias [groups, 2, n]; ``offsets`` as ``block_linear`` takes them.  act: none, relu, gelu,
    silu or sigmoid.  x and w are tensors of ``dtype``, or both Quantized (then ``dtype`` says the
    type of bias, z and out: bfloat16 by default; sums as ``block_linear8`` says).  Returns out, or
    (out, z) if save_preact: z [rows, 2 n] is g and u, and with save_preact="e4m3" a Quantized [rows,
    2, n].  Rows of no group become zero."""
    eight = save_preact == "e4m3"
    if stream is None and out is None:
        kind = FLOAT_DTYPES.get(dtype, -1 if dtype is not None else 0)
        done = _block.gated(*_pair(x, False), *_pair(w, True), bias, ACTS.get(act, -1), offsets,
                            2 if eight else 1 if save_preact is True else 0 if save_preact is False else -1, kind)
        if done is not None:
            if eight:
                return done[0], Quantized(done[1], done[2])
            return done
    _need(save_preact in (False, True, "e4m3"), 'save_preact must be False, True or "e4m3"')
    _act_of(act, _GATED_ACTS)
    if isinstance(x, Quantized) != isinstance(w, Quantized):
        raise TypeError("x and w must both be Quantized, or neither")
    if dtype is None:
        dtype = torch.bfloat16 if isinstance(x, Quantized) else getattr(x, "dtype", None)
    a, dev = _wide_args(x, w, offsets, act, dtype, 2)
    l = a.l
    l.bias = _ordered(bias, "bias", dev, dtype, l.groups, 2, l.n)
    with _on(dev, stream) as s:
        if out is None:
            out = torch.empty((l.rows, l.n), dtype=dtype, device=dev)
        l.out = _matrix(out, "out", dev, dtype, l.rows, l.n)
        z = None
        if eight:
            z = Quantized(torch.empty((l.rows, 2, l.n), dtype=E4M3, device=dev),
                          torch.empty((l.rows, 2, _blocks(l.n)), device=dev))
            l.z, a.z_scales = _Rows(z.values.data_ptr(), 2 * l.n), z.scales.data_ptr()
        elif save_preact:
            z = torch.empty((l.rows, 2 * l.n), dtype=dtype, device=dev)
            l.z = _Rows(z.data_ptr(), 2 * l.n)
        size = _sz()
        _check(_block_gated_workspace(a, size), "block_gated")
        work, wp = _scratch(size.value, dev)
        _check(_block_gated(a, wp, size.value, s), "block_gated")
    return (out, z) if save_preact else out


@dataclass
class GatedGrads:
    """Gradients of ``block_gated``; what is not needed is None.  db is fp32.  ``out`` is the
    forward pass's result, made again from z."""
    dx: torch.Tensor | None = None
    dw: torch.Tensor | None = None
    db: torch.Tensor | None = None
    out: torch.Tensor | None = None


def block_gated_backward(dout, x, w, z, *, act="silu", offsets=None, need_dx=True, need_dw=True,
                         need_db=True, need_out=False, dw_dtype=None, stream=None) -> GatedGrads:
    """Gradients of ``block_gated`` by x, w and bias, of w's shape.  ``z`` is what save_preact
    gave, in either form; x and w are tensors of ``dout``'s dtype or Quantized, each by itself: the
    gradients are those at what they stand for, in that dtype as ``block_linear8_backward`` says.
    ``need_out`` makes the forward pass's out again, which the next product's backward pass reads, so
    that nobody has to keep it."""
    if not isinstance(dout, torch.Tensor):
        raise ValueError("dout must be a matrix")
    dtype = dout.dtype
    if stream is None and dw_dtype in (None, torch.float32):
        done = _block.gated_backward(
            dout, *_pair(x, False), *_pair(w, True), *_pair(z, False), ACTS.get(act, -1), offsets,
            need_dx, need_dw, need_db, need_out, dw_dtype is not None)
        if done is not None:
            return GatedGrads(*done)
    _act_of(act, _GATED_ACTS)
    a, dev = _wide_args(x, w, offsets, act, dtype, 2)
    l, g, out = a.l, _GatedGrad(), GatedGrads()
    g.dout = _matrix(dout, "dout", dev, dtype, l.rows, l.n)
    if isinstance(z, Quantized):
        _quantized(z, "z", False)
        v = z.values
        _need(v.device == dev and tuple(v.shape) == (l.rows, 2, l.n), f"z must be [{l.rows}, 2, {l.n}]")
        _need(not v.numel() or (v.stride(2) == 1 or l.n == 1) and v.stride(1) == l.n and
              (l.rows == 1 or v.stride(0) >= 2 * l.n), "z: the halves of a row must be neighbours")
        l.z = _Rows(v.data_ptr(), v.stride(0) if l.rows > 1 else 2 * l.n)
        a.z_scales = _scales(z, "z", dev) or _NOWHERE
    else:
        l.z = _matrix(z, "z", dev, dtype, l.rows, 2 * l.n)
    dw_dtype = _dw_type(dw_dtype, dtype)
    g.dw_dt = FLOAT_DTYPES[dw_dtype]
    with _on(dev, stream) as s:
        _make_grads(g, out, _values(x), _values(w), dtype, dw_dtype, dev, need_dx, need_dw, need_db)
        if need_out:
            out.out = torch.empty((l.rows, l.n), dtype=dtype, device=dev)
            g.out = _Rows(out.out.data_ptr(), l.n or 1)
        size = _sz()
        _check(_block_gated_backward_workspace(a, g, size), "block_gated_backward")
        work, wp = _scratch(size.value, dev)
        _check(_block_gated_backward(a, g, wp, size.value, s), "block_gated_backward")
    return out
