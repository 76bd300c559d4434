// blk_binding.cpp -- the Python module ring_allreduce_amd._block: calls of a block's operators in
// their usual form, marshalled without Python.
//
// A call of a small operator costs what the host spends on it.  In Python, checks, output
// tensors and ctypes took 10 us of the 13 of a norm between two blocks, 6 of the 9 of a
// combine; here they take 2 to 3.  Every function takes a call's arguments as they came, and
// answers None if it is anything but the usual form: not all tensors on the current device, another
// type, shape or layout, an empty tensor, a status other than RR_OK.  block.py then goes
// through the checks one by one, and raises or makes the call itself.
#include <Python.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>

#include "rr.h"

namespace {

using at::Tensor;

struct Call {
    int device = -1;
    rr_stream_t stream = nullptr;

    // The call's first matrix: decides device and stream.
    bool begin(const Tensor& t) {
        if (!t.is_cuda() || t.get_device() != c10::hip::current_device()) return false;
        device = t.get_device();
        stream = (rr_stream_t)c10::hip::getCurrentHIPStream(device).stream();
        return true;
    }
    bool here(const Tensor& t) const { return t.is_cuda() && t.get_device() == device; }

    bool matrix(const Tensor& t, at::ScalarType type, int64_t rows, int64_t width, rr_rows_t& r) const {
        if (t.dim() != 2 || !here(t) || t.scalar_type() != type) return false;
        if (t.size(0) != rows || t.size(1) != width || rows < 1 || width < 1) return false;
        if (t.stride(1) != 1 || (rows > 1 && t.stride(0) < width)) return false;
        r = {t.data_ptr(), (size_t)(rows > 1 ? t.stride(0) : width)};
        return true;
    }
    bool vector(const Tensor& t, at::ScalarType type, int64_t numel) const {
        return here(t) && t.scalar_type() == type && t.numel() == numel && t.is_contiguous();
    }
    // A vector whose elements are in the order of a tensor of `sizes`: that tensor, but for
    // dimensions of 1, or a flat one.
    bool ordered(const Tensor& t, at::ScalarType type, at::IntArrayRef sizes) const {
        if (!vector(t, type, c10::multiply_integers(sizes))) return false;
        if (t.dim() == 1) return true;
        size_t at = 0;
        for (const int64_t n : t.sizes()) {
            if (n == 1) continue;
            while (at < sizes.size() && sizes[at] == 1) ++at;
            if (at == sizes.size() || sizes[at++] != n) return false;
        }
        return true;
    }
    Tensor make(at::IntArrayRef sizes, at::ScalarType type) const {
        return at::empty(sizes, at::TensorOptions().dtype(type).device(c10::DeviceType::CUDA, (c10::DeviceIndex)device));
    }
    Tensor make_rows(int64_t rows, int64_t width, at::ScalarType type, rr_rows_t& r) const {
        Tensor t = make({rows, width}, type);
        r = {t.data_ptr(), (size_t)width};
        return t;
    }
    Tensor scratch(size_t bytes, void*& at) const {
        at = nullptr;
        if (!bytes) return Tensor();
        Tensor t = make({(int64_t)bytes}, at::kByte);
        at = t.data_ptr();
        return t;
    }
};

// The arguments: nothing, or a tensor; anything else ends the usual form.
struct Args {
    PyObject* const* a;
    bool good = true;
    const Tensor* tensor(int i) {
        if (a[i] == Py_None) return nullptr;
        if (!THPVariable_Check(a[i])) {
            good = false;
            return nullptr;
        }
        return &THPVariable_Unpack(a[i]);
    }
    const Tensor* needed(int i) {
        const Tensor* t = tensor(i);
        if (!t) good = false;
        return t;
    }
    long number(int i) {
        const long v = PyLong_Check(a[i]) ? PyLong_AsLong(a[i]) : (good = false, 0L);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            good = false;
        }
        return v;
    }
    float real(int i) {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            good = false;
        }
        return (float)v;
    }
    bool flag(int i) {
        const int v = PyObject_IsTrue(a[i]);
        if (v < 0) {
            PyErr_Clear();
            good = false;
        }
        return v == 1;
    }
};

rr_dtype_t type_of(at::ScalarType t) {
    return t == at::kFloat ? RR_FP32 : t == at::kBFloat16 ? RR_BF16 : t == at::kHalf ? RR_FP16 : (rr_dtype_t)-1;
}
bool known(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16 || t == at::kHalf; }

PyObject* none() { Py_RETURN_NONE; }
PyObject* wrap(const Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : none(); }
PyObject* tuple(std::initializer_list<Tensor> all) {
    PyObject* out = PyTuple_New((Py_ssize_t)all.size());
    Py_ssize_t i = 0;
    for (const Tensor& t : all) PyTuple_SET_ITEM(out, i++, wrap(t));
    return out;
}
const int32_t* ints(const Tensor& t) { return (const int32_t*)t.data_ptr(); }

// ids, experts, capacity
PyObject* sort(Args& a) {
    const Tensor* ids = a.needed(0);
    const long experts = a.number(1), capacity = a.number(2);
    Call c;
    if (!a.good || experts < 1 || experts > RR_MAX_EXPERTS || capacity < 0 || !c.begin(*ids) || ids->dim() != 2)
        return none();
    const auto type = ids->scalar_type();
    const int64_t tokens = ids->size(0), k = ids->size(1);
    rr_rows_t in;
    if ((type != at::kInt && type != at::kLong) || !c.matrix(*ids, type, tokens, k, in)) return none();
    if (capacity > INT32_MAX / experts || tokens > INT32_MAX / k) return none();
    size_t need = 0;
    if (expert_sort_workspace((size_t)tokens, (int)k, (int)experts, &need) != RR_OK) return none();
    const int64_t rows = capacity ? experts * capacity : tokens * k;
    Tensor slots = c.make({tokens, k}, at::kInt), sources = c.make({rows}, at::kInt);
    Tensor counts = c.make({experts}, at::kInt), offsets = c.make({experts + 1}, at::kInt);
    void* at;
    Tensor work = c.scratch(need, at);
    if (expert_sort(in.data, type == at::kInt ? 4 : 8, in.ld, (size_t)tokens, (int)k, (int)experts, (size_t)capacity,
                    (int32_t*)slots.data_ptr(), (int32_t*)sources.data_ptr(), (int32_t*)counts.data_ptr(),
                    (int32_t*)offsets.data_ptr(), at, need, c.stream) != RR_OK)
        return none();
    return tuple({slots, sources, counts, offsets});
}

// x, slots, sources, whether x is scales of 8-bit rows
PyObject* dispatch(Args& a) {
    const Tensor *x = a.needed(0), *slots = a.needed(1), *sources = a.needed(2);
    const bool scales = a.flag(3);
    Call c;
    if (!a.good || !c.begin(*x) || x->dim() != 2 || slots->dim() != 2 || !known(x->scalar_type())) return none();
    if (scales && x->scalar_type() != at::kFloat) return none();
    const int64_t tokens = x->size(0), hidden = x->size(1), k = slots->size(1), rows = sources->numel();
    rr_rows_t in, to;
    if (!c.matrix(*x, x->scalar_type(), tokens, hidden, in) || slots->size(0) != tokens || rows < 1 || k < 1 ||
        !c.vector(*slots, at::kInt, tokens * k) || !c.vector(*sources, at::kInt, rows))
        return none();
    Tensor out = c.make_rows(rows, hidden, x->scalar_type(), to);
    const rr_status_t st =
        scales ? expert_dispatch_scales(in, (size_t)tokens, (size_t)hidden, (int)k, ints(*slots), ints(*sources),
                                        (size_t)rows, to, c.stream)
               : expert_dispatch(in, (size_t)tokens, (size_t)hidden, (int)k, type_of(x->scalar_type()), ints(*slots),
                                 ints(*sources), (size_t)rows, to, c.stream);
    if (st != RR_OK) return none();
    return wrap(out);
}

// rows, slots, weights
PyObject* combine(Args& a) {
    const Tensor *rows = a.needed(0), *slots = a.needed(1), *weights = a.tensor(2);
    Call c;
    if (!a.good || !c.begin(*rows) || rows->dim() != 2 || slots->dim() != 2 || !known(rows->scalar_type())) return none();
    const int64_t n = rows->size(0), hidden = rows->size(1), tokens = slots->size(0), k = slots->size(1);
    rr_rows_t in, to;
    if (!c.matrix(*rows, rows->scalar_type(), n, hidden, in) || tokens < 1 || k < 1 ||
        !c.vector(*slots, at::kInt, tokens * k) || (weights && !c.ordered(*weights, at::kFloat, {tokens, k})))
        return none();
    Tensor out = c.make_rows(tokens, hidden, rows->scalar_type(), to);
    if (expert_combine(in, (size_t)n, (size_t)hidden, type_of(rows->scalar_type()), ints(*slots),
                       weights ? (const float*)weights->data_ptr() : nullptr, (size_t)tokens, (int)k, to,
                       c.stream) != RR_OK)
        return none();
    return wrap(out);
}

// dout, rows, slots, sources, weights, need_rows, need_weights
PyObject* combine_backward(Args& a) {
    const Tensor *dout = a.needed(0), *rows = a.tensor(1), *slots = a.needed(2), *sources = a.needed(3);
    const Tensor* weights = a.tensor(4);
    const bool need_rows = a.flag(5), need_weights = a.flag(6);
    Call c;
    if (!a.good || !c.begin(*dout) || dout->dim() != 2 || slots->dim() != 2 || !known(dout->scalar_type())) return none();
    const auto type = dout->scalar_type();
    const int64_t tokens = dout->size(0), hidden = dout->size(1), k = slots->size(1), n = sources->numel();
    rr_rows_t d, r = {nullptr, 0}, to = {nullptr, 0};
    if (!c.matrix(*dout, type, tokens, hidden, d) || slots->size(0) != tokens || k < 1 || n < 1 ||
        !c.vector(*slots, at::kInt, tokens * k) || !c.vector(*sources, at::kInt, n) ||
        (weights && !c.ordered(*weights, at::kFloat, {tokens, k})))
        return none();
    if (need_weights && (!rows || !c.matrix(*rows, type, n, hidden, r))) return none();
    Tensor drows, dweights;
    if (need_rows) drows = c.make_rows(n, hidden, type, to);
    if (need_weights) dweights = c.make({tokens, k}, at::kFloat);
    if (expert_combine_backward(d, r, (size_t)n, (size_t)hidden, type_of(type), ints(*slots), ints(*sources),
                                weights ? (const float*)weights->data_ptr() : nullptr, (size_t)tokens, (int)k, to,
                                need_weights ? (float*)dweights.data_ptr() : nullptr, c.stream) != RR_OK)
        return none();
    return tuple({drows, dweights});
}

// branch, post_norm, post_weight, gate, gate_act, residual_scale, branch_scale, pre_norm,
// pre_weight, eps from argument `i` on
bool norm_args(Args& a, int i, const Call& c, const Tensor& like, rr_norm_t& n) {
    const Tensor *branch = a.tensor(i), *post = a.tensor(i + 2), *gate = a.tensor(i + 3), *pre = a.tensor(i + 8);
    const long act = a.number(i + 4);
    n.post_norm = a.flag(i + 1);
    n.pre_norm = a.flag(i + 7);
    n.residual_scale = a.real(i + 5);
    n.branch_scale = a.real(i + 6);
    n.eps = a.real(i + 9);
    if (!a.good || act < 0 || (post && !n.post_norm) || (pre && !n.pre_norm) || (!gate && act != RR_ACT_NONE)) return false;
    const int64_t tokens = like.size(0), hidden = like.size(1);
    const auto type = like.scalar_type();
    n.tokens = (size_t)tokens;
    n.hidden = (size_t)hidden;
    n.dt = type_of(type);
    n.gate_act = (int32_t)act;
    if (branch ? !c.matrix(*branch, type, tokens, hidden, n.branch) : (n.post_norm || gate)) return false;
    const bool channel = gate && gate->dim() == 1;
    const Tensor* first = post ? post : pre ? pre : channel ? gate : nullptr;
    const auto weight = first ? first->scalar_type() : type;
    if (weight != type && weight != at::kFloat) return false;
    n.weight_dt = type_of(weight);
    for (const Tensor* w : {post, pre, channel ? gate : nullptr})
        if (w && !c.vector(*w, weight, hidden)) return false;
    n.post_weight = post ? post->data_ptr() : nullptr;
    n.pre_weight = pre ? pre->data_ptr() : nullptr;
    if (channel) {
        n.gate_kind = RR_GATE_CHANNEL;
        n.gate = {gate->data_ptr(), (size_t)hidden};
    } else if (gate) {
        n.gate_kind = RR_GATE_ELEMENT;
        if (!c.matrix(*gate, type, tokens, hidden, n.gate)) return false;
    }
    return true;
}

// x, then norm_args
PyObject* norm(Args& a) {
    const Tensor* x = a.needed(0);
    Call c;
    rr_norm_t n = {};
    if (!a.good || !c.begin(*x) || x->dim() != 2 || !known(x->scalar_type())) return none();
    if (!c.matrix(*x, x->scalar_type(), x->size(0), x->size(1), n.x) || !norm_args(a, 1, c, *x, n)) return none();
    Tensor h = c.make_rows(x->size(0), x->size(1), x->scalar_type(), n.h), y;
    if (n.pre_norm) y = c.make_rows(x->size(0), x->size(1), x->scalar_type(), n.y);
    if (block_norm(&n, c.stream) != RR_OK) return none();
    return tuple({h, y});
}

// dh, dy, h, then norm_args, then what is needed: 1 dx, 2 dbranch, 4 dgate, 8 dpost, 16 dpre
PyObject* norm_backward(Args& a) {
    const Tensor *dh = a.tensor(0), *dy = a.tensor(1), *h = a.tensor(2), *branch = a.tensor(3);
    const long need = a.number(13);
    const Tensor* like = dh ? dh : dy ? dy : h ? h : branch;
    Call c;
    rr_norm_t n = {};
    rr_norm_grad_t g = {};
    if (!a.good || !like || like->dim() != 2 || !known(like->scalar_type()) || !c.begin(*like) ||
        !norm_args(a, 3, c, *like, n))
        return none();
    const auto type = like->scalar_type();
    const int64_t tokens = like->size(0), hidden = like->size(1);
    if (tokens < 1 || hidden < 1 || (n.pre_norm != 0) != (dy != nullptr) || (n.pre_norm && !h)) return none();
    if (dh && !c.matrix(*dh, type, tokens, hidden, g.dh)) return none();
    if (n.pre_norm && (!c.matrix(*dy, type, tokens, hidden, g.dy) || !c.matrix(*h, type, tokens, hidden, n.h)))
        return none();
    Tensor dx, dbranch, dgate, dpost, dpre;
    const auto sums = [&](Tensor& t) {
        t = c.make({hidden}, at::kFloat);
        return (float*)t.data_ptr();
    };
    if (need & 1) dx = c.make_rows(tokens, hidden, type, g.dx);
    if ((need & 2) && branch) dbranch = c.make_rows(tokens, hidden, type, g.dbranch);
    if ((need & 4) && n.gate_kind == RR_GATE_ELEMENT) dgate = c.make_rows(tokens, hidden, type, g.dgate);
    if ((need & 4) && n.gate_kind == RR_GATE_CHANNEL) g.dgate_channel = sums(dgate);
    if ((need & 8) && n.post_weight) g.dpost_weight = sums(dpost);
    if ((need & 16) && n.pre_weight) g.dpre_weight = sums(dpre);
    size_t bytes = 0;
    if (block_norm_backward_workspace(&n, &g, &bytes) != RR_OK) return none();
    void* at;
    Tensor work = c.scratch(bytes, at);
    if (block_norm_backward(&n, &g, at, bytes, c.stream) != RR_OK) return none();
    return tuple({dx, dbranch, dgate, dpost, dpre});
}

bool linear_args(const Call& c, const Tensor& x, const Tensor& w, const Tensor* offsets, long act, rr_linear_t& l) {
    const auto type = x.scalar_type();
    if (x.dim() != 2 || (type != at::kBFloat16 && type != at::kHalf)) return false;
    const int64_t rows = x.size(0), k = x.size(1);
    if (!c.matrix(x, type, rows, k, l.x)) return false;
    const int d = (int)w.dim();
    if ((d != 2 && d != 3) || !c.here(w) || w.scalar_type() != type || w.numel() == 0 || w.size(d - 1) != k) return false;
    const int64_t groups = d == 3 ? w.size(0) : 1, n = w.size(d - 2);
    const int64_t ld = n > 1 ? w.stride(d - 2) : k;
    if (groups > RR_MAX_EXPERTS || w.stride(d - 1) != 1 || ld < k) return false;
    if (act < RR_ACT_NONE || act > RR_ACT_SILU) return false;
    if (offsets ? !c.vector(*offsets, at::kInt, groups + 1) : rows % groups != 0) return false;
    l.rows = (size_t)rows;
    l.n = (size_t)n;
    l.k = (size_t)k;
    l.groups = (int32_t)groups;
    l.dt = type_of(type);
    l.act = (int32_t)act;
    l.offsets = offsets ? ints(*offsets) : nullptr;
    l.w = w.data_ptr();
    l.w_ld = (size_t)ld;
    l.w_stride = d == 3 ? (size_t)w.stride(0) : 0;
    return d != 3 || w.stride(0) >= 0;
}

// x, w, bias, act, residual, offsets, save_preact
PyObject* linear(Args& a) {
    const Tensor *x = a.needed(0), *w = a.needed(1), *bias = a.tensor(2), *residual = a.tensor(4), *offsets = a.tensor(5);
    const long act = a.number(3);
    const bool save = a.flag(6);
    Call c;
    rr_linear_t l = {};
    if (!a.good || !c.begin(*x) || !linear_args(c, *x, *w, offsets, act, l)) return none();
    const auto type = x->scalar_type();
    const int64_t rows = (int64_t)l.rows, n = (int64_t)l.n;
    if (bias && !c.ordered(*bias, type, {l.groups, n})) return none();
    l.bias = bias ? bias->data_ptr() : nullptr;
    if (residual && !c.matrix(*residual, type, rows, n, l.residual)) return none();
    Tensor out = c.make_rows(rows, n, type, l.out), z;
    if (save) z = c.make_rows(rows, n, type, l.z);
    size_t bytes = 0;
    if (block_linear_workspace(&l, &bytes) != RR_OK) return none();
    void* at;
    Tensor work = c.scratch(bytes, at);
    if (block_linear(&l, at, bytes, c.stream) != RR_OK) return none();
    return save ? tuple({out, z}) : wrap(out);
}

// dout, x, w, z, act, offsets, need_dx, need_dw, need_db, dw in fp32
PyObject* linear_backward(Args& a) {
    const Tensor *dout = a.needed(0), *x = a.needed(1), *w = a.needed(2), *z = a.tensor(3), *offsets = a.tensor(5);
    const long act = a.number(4);
    const bool need_dx = a.flag(6), need_dw = a.flag(7), need_db = a.flag(8), wide_dw = a.flag(9);
    Call c;
    rr_linear_t l = {};
    rr_linear_grad_t g = {};
    if (!a.good || !c.begin(*x) || !linear_args(c, *x, *w, offsets, act, l)) return none();
    const auto type = x->scalar_type(), wide = wide_dw ? at::kFloat : type;
    const int64_t rows = (int64_t)l.rows, n = (int64_t)l.n;
    if (!c.matrix(*dout, type, rows, n, g.dout)) return none();
    if (act != RR_ACT_NONE && (!z || !c.matrix(*z, type, rows, n, l.z))) return none();
    Tensor dx, dw, db;
    if (need_dx) dx = c.make_rows(rows, (int64_t)l.k, type, g.dx);
    if (need_dw) {
        dw = c.make(w->sizes(), wide);
        g.dw = dw.data_ptr();
    }
    if (need_db) {
        db = c.make(w->sizes().slice(0, (size_t)w->dim() - 1), at::kFloat);
        g.db = (float*)db.data_ptr();
    }
    g.dw_dt = type_of(wide);
    size_t bytes = 0;
    if (block_linear_backward_workspace(&l, &g, &bytes) != RR_OK) return none();
    void* at;
    Tensor work = c.scratch(bytes, at);
    if (block_linear_backward(&l, &g, at, bytes, c.stream) != RR_OK) return none();
    return tuple({dx, dw, db});
}

// ------------------------------------------------- 8-bit values and gated projections

constexpr auto kE4M3 = at::kFloat8_e4m3fn;
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

// The shape of the scales of values of shape `s`.
std::vector<int64_t> scales_shape(at::IntArrayRef s, bool square) {
    std::vector<int64_t> v(s.begin(), s.end());
    const size_t d = v.size();
    v[d - 1] = blocks_of(v[d - 1]);
    if (square) v[d - 2] = blocks_of(v[d - 2]);
    return v;
}
bool scales_fit(const Call& c, const Tensor& values, const Tensor& scales, bool square) {
    return c.here(scales) && scales.scalar_type() == at::kFloat && scales.is_contiguous() &&
           scales.sizes().equals(scales_shape(values.sizes(), square));
}

// t [..., rows, width], not empty, as contiguous matrices or one of any row stride.
bool stack(const Call& c, const Tensor& t, rr_rows_t& r, size_t& stride, rr_quantize_t& q) {
    const int64_t d = t.dim();
    if (d < 2 || t.numel() < 1 || !c.here(t)) return false;
    q.rows = (size_t)t.size(d - 2);
    q.width = (size_t)t.size(d - 1);
    q.groups = (size_t)t.numel() / q.rows / q.width;
    stride = q.rows * q.width;
    r = {t.data_ptr(), q.width};
    if (t.is_contiguous()) return true;
    if (d != 2 || t.stride(1) != 1 || (t.size(0) > 1 && t.stride(0) < t.size(1))) return false;
    if (t.size(0) > 1) r.ld = (size_t)t.stride(0);
    return true;
}

// x, square
PyObject* quantize(Args& a) {
    const Tensor* x = a.needed(0);
    const bool square = a.flag(1);
    Call c;
    rr_quantize_t q = {};
    if (!a.good || !c.begin(*x) || !known(x->scalar_type()) || !stack(c, *x, q.x, q.x_stride, q)) return none();
    Tensor values = c.make(x->sizes(), kE4M3), scales = c.make(scales_shape(x->sizes(), square), at::kFloat);
    q.dt = type_of(x->scalar_type());
    q.square = square;
    q.q = {values.data_ptr(), q.width};
    q.q_stride = q.rows * q.width;
    q.scales = (float*)scales.data_ptr();
    if (block_quantize(&q, c.stream) != RR_OK) return none();
    return tuple({values, scales});
}

at::ScalarType type_named(long dt) {
    return dt == RR_FP32 ? at::kFloat : dt == RR_BF16 ? at::kBFloat16 : dt == RR_FP16 ? at::kHalf : at::kByte;
}

// values, scales, square, dtype
PyObject* dequantize(Args& a) {
    const Tensor *values = a.needed(0), *scales = a.needed(1);
    const bool square = a.flag(2);
    const auto type = type_named(a.number(3));
    Call c;
    rr_quantize_t q = {};
    if (!a.good || !known(type) || values->scalar_type() != kE4M3 || !c.begin(*values) ||
        !stack(c, *values, q.q, q.q_stride, q) || !scales_fit(c, *values, *scales, square))
        return none();
    Tensor out = c.make(values->sizes(), type);
    q.dt = type_of(type);
    q.square = square;
    q.x = {out.data_ptr(), q.width};
    q.x_stride = q.rows * q.width;
    q.scales = (float*)scales->data_ptr();
    if (block_dequantize(&q, c.stream) != RR_OK) return none();
    return wrap(out);
}

// x and w, each with its scales or none, of a product of `halves` matrices a group
bool wide_args(const Call& c, const Tensor& x, const Tensor* xs, const Tensor& w, const Tensor* ws, const Tensor* offsets,
               long act, at::ScalarType type, int halves, rr_linear8_t& a) {
    rr_linear_t& l = a.l;
    if (x.dim() != 2 || (type != at::kBFloat16 && type != at::kHalf)) return false;
    const int64_t rows = x.size(0), k = x.size(1);
    if (!c.matrix(x, xs ? kE4M3 : type, rows, k, l.x) || (xs && !scales_fit(c, x, *xs, false))) return false;
    const int d = (int)w.dim(), one = halves == 1 ? 2 : 3;
    if ((d != one && d != one + 1) || !c.here(w) || w.scalar_type() != (ws ? kE4M3 : type) || w.numel() == 0 ||
        w.size(d - 1) != k || (halves == 2 && w.size(d - 3) != 2) || (ws && !scales_fit(c, w, *ws, true)))
        return false;
    const int64_t groups = d > one ? w.size(0) : 1, n = w.size(d - 2);
    const int64_t ld = n > 1 ? w.stride(d - 2) : halves == 2 ? w.stride(d - 3) : k;
    if (groups > RR_MAX_EXPERTS || (w.stride(d - 1) != 1 && k > 1) || ld < k) return false;
    if (halves == 2 && w.stride(d - 3) != n * ld) return false;
    if (act < RR_ACT_NONE || act > (halves == 2 ? RR_ACT_SIGMOID : RR_ACT_SILU)) return false;
    if (offsets ? !c.vector(*offsets, at::kInt, groups + 1) : rows % groups != 0) return false;
    l.rows = (size_t)rows;
    l.n = (size_t)n;
    l.k = (size_t)k;
    l.groups = (int32_t)groups;
    l.dt = type_of(type);
    l.act = (int32_t)act;
    l.offsets = offsets ? ints(*offsets) : nullptr;
    l.w = w.data_ptr();
    l.w_ld = (size_t)ld;
    l.w_stride = d > one ? (size_t)w.stride(0) : 0;
    a.x_scales = xs ? (const float*)xs->data_ptr() : nullptr;
    a.w_scales = ws ? (const float*)ws->data_ptr() : nullptr;
    return d == one || w.stride(0) >= 0;
}

// x, x's scales, w, w's scales, bias, act, residual, offsets, save_preact, dtype
PyObject* linear8(Args& a) {
    const Tensor *x = a.needed(0), *xs = a.needed(1), *w = a.needed(2), *ws = a.needed(3), *bias = a.tensor(4);
    const Tensor *residual = a.tensor(6), *offsets = a.tensor(7);
    const long act = a.number(5);
    const bool save = a.flag(8);
    const auto type = type_named(a.number(9));
    Call c;
    rr_linear8_t l = {};
    if (!a.good || !c.begin(*x) || !wide_args(c, *x, xs, *w, ws, offsets, act, type, 1, l)) return none();
    const int64_t rows = (int64_t)l.l.rows, n = (int64_t)l.l.n;
    if (bias && !c.ordered(*bias, type, {l.l.groups, n})) return none();
    l.l.bias = bias ? bias->data_ptr() : nullptr;
    if (residual && !c.matrix(*residual, type, rows, n, l.l.residual)) return none();
    Tensor out = c.make_rows(rows, n, type, l.l.out), z;
    if (save) z = c.make_rows(rows, n, type, l.l.z);
    size_t bytes = 0;
    if (block_linear8_workspace(&l, &bytes) != RR_OK) return none();
    void* at;
    Tensor work = c.scratch(bytes, at);
    if (block_linear8(&l, at, bytes, c.stream) != RR_OK) return none();
    return save ? tuple({out, z}) : wrap(out);
}

// The gradients by x, w and bias that are wanted.
template <typename G>
void make_grads(const Call& c, const Tensor& x, const Tensor& w, at::ScalarType type, at::ScalarType wide, bool need_dx,
                bool need_dw, bool need_db, G& g, Tensor& dx, Tensor& dw, Tensor& db) {
    if (need_dx) dx = c.make_rows(x.size(0), x.size(1), type, g.dx);
    if (need_dw) {
        dw = c.make(w.sizes(), wide);
        g.dw = dw.data_ptr();
    }
    if (need_db) {
        db = c.make(w.sizes().slice(0, (size_t)w.dim() - 1), at::kFloat);
        g.db = (float*)db.data_ptr();
    }
    g.dw_dt = type_of(wide);
}

// dout, x, x's scales, w, w's scales, z, act, offsets, need_dx, need_dw, need_db, dw in fp32
PyObject* linear8_backward(Args& a) {
    const Tensor *dout = a.needed(0), *x = a.needed(1), *xs = a.tensor(2), *w = a.needed(3), *ws = a.tensor(4);
    const Tensor *z = a.tensor(5), *offsets = a.tensor(7);
    const long act = a.number(6);
    const bool need_dx = a.flag(8), need_dw = a.flag(9), need_db = a.flag(10), wide_dw = a.flag(11);
    Call c;
    rr_linear8_t l = {};
    rr_linear_grad_t g = {};
    if (!a.good || !c.begin(*x)) return none();
    const auto type = dout->scalar_type(), wide = wide_dw ? at::kFloat : type;
    if (!wide_args(c, *x, xs, *w, ws, offsets, act, type, 1, l)) return none();
    const int64_t rows = (int64_t)l.l.rows, n = (int64_t)l.l.n;
    if (!c.matrix(*dout, type, rows, n, g.dout)) return none();
    if (act != RR_ACT_NONE && (!z || !c.matrix(*z, type, rows, n, l.l.z))) return none();
    Tensor dx, dw, db;
    make_grads(c, *x, *w, type, wide, need_dx, need_dw, need_db, g, dx, dw, db);
    size_t bytes = 0;
    if (block_linear8_backward_workspace(&l, &g, &bytes) != RR_OK) return none();
    void* at;
    Tensor work = c.scratch(bytes, at);
    if (block_linear8_backward(&l, &g, at, bytes, c.stream) != RR_OK) return none();
    return tuple({dx, dw, db});
}

// x, x's scales, w, w's scales, bias, act, offsets, z (0 none, 1 in 16 bits, 2 in 8), dtype (0: x's)
PyObject* gated(Args& a) {
    const Tensor *x = a.needed(0), *xs = a.tensor(1), *w = a.needed(2), *ws = a.tensor(3), *bias = a.tensor(4);
    const Tensor* offsets = a.tensor(6);
    const long act = a.number(5), save = a.number(7), named = a.number(8);
    Call c;
    rr_linear8_t l = {};
    if (!a.good || !c.begin(*x) || save < 0 || save > 2 || !xs != !ws) return none();
    const auto type = named ? type_named(named) : xs ? at::kBFloat16 : x->scalar_type();
    if (!wide_args(c, *x, xs, *w, ws, offsets, act, type, 2, l)) return none();
    const int64_t rows = (int64_t)l.l.rows, n = (int64_t)l.l.n;
    if (bias && !c.ordered(*bias, type, {l.l.groups, 2, n})) return none();
    l.l.bias = bias ? bias->data_ptr() : nullptr;
    Tensor out = c.make_rows(rows, n, type, l.l.out), z, scales;
    if (save == 1) z = c.make_rows(rows, 2 * n, type, l.l.z);
    if (save == 2) {
        z = c.make({rows, 2, n}, kE4M3);
        scales = c.make({rows, 2, blocks_of(n)}, at::kFloat);
        l.l.z = {z.data_ptr(), (size_t)(2 * n)};
        l.z_scales = (float*)scales.data_ptr();
    }
    size_t bytes = 0;
    if (block_gated_workspace(&l, &bytes) != RR_OK) return none();
    void* at;
    Tensor work = c.scratch(bytes, at);
    if (block_gated(&l, at, bytes, c.stream) != RR_OK) return none();
    return save == 2 ? tuple({out, z, scales}) : save ? tuple({out, z}) : wrap(out);
}

// dout, x, x's scales, w, w's scales, z, z's scales, act, offsets, need_dx, need_dw, need_db,
// need_out, dw in fp32
PyObject* gated_backward(Args& a) {
    const Tensor *dout = a.needed(0), *x = a.needed(1), *xs = a.tensor(2), *w = a.needed(3), *ws = a.tensor(4);
    const Tensor *z = a.needed(5), *zs = a.tensor(6), *offsets = a.tensor(8);
    const long act = a.number(7);
    const bool need_dx = a.flag(9), need_dw = a.flag(10), need_db = a.flag(11), need_out = a.flag(12), wide_dw = a.flag(13);
    Call c;
    rr_linear8_t l = {};
    rr_gated_grad_t g = {};
    if (!a.good || !c.begin(*x)) return none();
    const auto type = dout->scalar_type(), wide = wide_dw ? at::kFloat : type;
    if (!wide_args(c, *x, xs, *w, ws, offsets, act, type, 2, l)) return none();
    const int64_t rows = (int64_t)l.l.rows, n = (int64_t)l.l.n;
    if (!c.matrix(*dout, type, rows, n, g.dout)) return none();
    if (!zs) {
        if (!c.matrix(*z, type, rows, 2 * n, l.l.z)) return none();
    } else {
        if (!c.here(*z) || z->scalar_type() != kE4M3 || !z->sizes().equals({rows, 2, n}) || !z->is_contiguous() ||
            !scales_fit(c, *z, *zs, false))
            return none();
        l.l.z = {z->data_ptr(), (size_t)(2 * n)};
        l.z_scales = (float*)zs->data_ptr();
    }
    Tensor dx, dw, db, out;
    make_grads(c, *x, *w, type, wide, need_dx, need_dw, need_db, g, dx, dw, db);
    if (need_out) out = c.make_rows(rows, n, type, g.out);
    size_t bytes = 0;
    if (block_gated_backward_workspace(&l, &g, &bytes) != RR_OK) return none();
    void* at;
    Tensor work = c.scratch(bytes, at);
    if (block_gated_backward(&l, &g, at, bytes, c.stream) != RR_OK) return none();
    return tuple({dx, dw, db, out});
}

// No C++ exception leaves the module: what torch throws becomes the Python error it stands for.
template <PyObject* (*F)(Args&), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, not %zd", N, n);
        return nullptr;
    }
    Args a{args};
    return F(a);
    END_HANDLE_TH_ERRORS
}
#define BLK_ENTRY(name, f, n) \
    {name, (PyCFunction)(void (*)(void))(entry<f, n>), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {BLK_ENTRY("sort", sort, 3),
                         BLK_ENTRY("dispatch", dispatch, 4),
                         BLK_ENTRY("combine", combine, 3),
                         BLK_ENTRY("combine_backward", combine_backward, 7),
                         BLK_ENTRY("norm", norm, 11),
                         BLK_ENTRY("norm_backward", norm_backward, 14),
                         BLK_ENTRY("linear", linear, 7),
                         BLK_ENTRY("linear_backward", linear_backward, 10),
                         BLK_ENTRY("quantize", quantize, 2),
                         BLK_ENTRY("dequantize", dequantize, 4),
                         BLK_ENTRY("linear8", linear8, 10),
                         BLK_ENTRY("linear8_backward", linear8_backward, 12),
                         BLK_ENTRY("gated", gated, 9),
                         BLK_ENTRY("gated_backward", gated_backward, 14),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
