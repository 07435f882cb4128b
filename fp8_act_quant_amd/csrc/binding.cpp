// binding.cpp -- the Python calls of the routed-expert, 8-bit integer and dense-block operators: argument
// checks, outputs and workspaces from torch's allocator, one call of the C ABI (fp8q.h) on the
// tensors' device and torch's current stream there.
//
// Native because these calls are small: a decode step's kernel takes 3 us, and checks, allocations
// and ctypes in Python took 6 us a call around the 3 us that the launch itself takes; here they
// take about 1 us (gated_linear_backward 2 to 4: the choice of its tiles, for the workspace and for the
// launch, is 0.1 to 1.4 us each). Names, defaults and documentation are in moe.py, int8.py and block.py.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <fp8q.h>

namespace {

using at::ScalarType;
using at::Tensor;

// ---- errors: Python exceptions of the kinds that the Python checks raise ------------------

struct Raised {};   // a Python exception is set

template <class... A>
[[noreturn]] void raise(PyObject *kind, const char *format, A... args) {
    PyErr_Format(kind, format, args...);
    throw Raised{};
}

const char *type_name(ScalarType t) {
    switch (t) {
    case ScalarType::Float: return "torch.float32";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Double: return "torch.float64";
    case ScalarType::Char: return "torch.int8";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    default: return c10::toString(t);
    }
}

// A status of the library becomes its Python error
void check(const char *call, int status) {
    if (status == FP8Q_OK) return;
    PyObject *lib = PyImport_ImportModule("fp8_act_quant_amd._lib");
    if (lib) {
        PyObject *r = PyObject_CallMethod(lib, "check", "si", call, status);
        Py_XDECREF(r);
        Py_DECREF(lib);
    }
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s failed with status %d", call, status);
    throw Raised{};
}

// ---- arguments -----------------------------------------------------------------------------

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a GPU tensor", name);
    return t;
}

void placed(const Tensor &t, const char *name, uintptr_t align, const Tensor *beside) {
    if (beside && t.device() != beside->device())
        raise(PyExc_ValueError, "%s must be on %s, got %s", name, beside->device().str().c_str(),
              t.device().str().c_str());
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    if (reinterpret_cast<uintptr_t>(t.data_ptr()) % align)
        raise(PyExc_ValueError, "%s must be %zu-byte aligned", name, (size_t)align);
}

// a contiguous GPU tensor of one type, on `beside`'s device
const Tensor &need(PyObject *o, const char *name, ScalarType type, uintptr_t align, const Tensor *beside = nullptr) {
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != type)
        raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
    placed(t, name, align, beside);
    return t;
}

// float32 or bfloat16, aligned to its elements
const Tensor &need_float(PyObject *o, const char *name, const Tensor *beside = nullptr) {
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != ScalarType::Float && t.scalar_type() != ScalarType::BFloat16)
        raise(PyExc_TypeError, "%s must be torch.float32 or torch.bfloat16, got %s", name, type_name(t.scalar_type()));
    placed(t, name, t.element_size(), beside);
    return t;
}

void shaped(const Tensor &t, const char *name, at::IntArrayRef shape) {
    if (t.sizes() != shape) {
        std::string want, got;
        for (int64_t s : shape) want += (want.empty() ? "" : ", ") + std::to_string(s);
        for (int64_t s : t.sizes()) got += (got.empty() ? "" : ", ") + std::to_string(s);
        raise(PyExc_ValueError, "%s must have shape (%s), got (%s)", name, want.c_str(), got.c_str());
    }
}

int64_t integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        if (PyErr_ExceptionMatches(PyExc_OverflowError)) {
            PyErr_Clear();
            raise(PyExc_ValueError, "%s is out of range", name);
        }
        throw Raised{};
    }
    return v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v == 1;
}

float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}

int code_of(const Tensor &t) { return t.scalar_type() == ScalarType::BFloat16 ? FP8Q_OUT_BF16 : FP8Q_OUT_F32; }

const void *data(const Tensor *t) { return t && t->defined() ? t->data_ptr() : nullptr; }
template <class T>
T *ptr(const Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}

// Straight from the GPU allocator: at::empty's way through the dispatcher takes 0.25 us more, with one
// to four outputs a call (calls one after another: moe_place of 48 x 8 6.0 -> 5.3 us). With deterministic algorithms it is taken: it then
// fills the memory, which shows a reader of rows that no expert owns.
Tensor like(const Tensor &t, at::IntArrayRef shape, ScalarType type) {
    if (at::globalContext().deterministicAlgorithms()) return at::empty(shape, t.options().dtype(type));
    return at::detail::empty_cuda(shape, type, t.device(), std::nullopt);
}

int64_t rows_of(const Tensor &t) {   // of a [..., K] tensor
    int64_t n = 1;
    for (int64_t s : t.sizes().slice(0, t.dim() - 1)) n *= s;
    return n;
}

// A bf16 or fp32 output: the caller's (checked), or a new one of type `code` (FP8Q_OUT_*)
Tensor output(PyObject *out, at::IntArrayRef shape, ScalarType type, uintptr_t align, const Tensor &beside) {
    if (out == Py_None) return like(beside, shape, type);
    const Tensor &t = need(out, "out", type, align, &beside);
    shaped(t, "out", shape);
    return t;
}
// `out` written while `t` is still read: refused where they share memory
void apart(const Tensor &out, const Tensor *t, const char *name) {
    if (!t || !t->numel() || !out.numel()) return;
    const char *a = static_cast<const char *>(out.data_ptr()), *b = static_cast<const char *>(t->data_ptr());
    if (a < b + t->nbytes() && b < a + out.nbytes()) raise(PyExc_ValueError, "out must not overlap %s", name);
}
ScalarType type_of_code(PyObject *o) {
    return integer(o, "out_dtype") == FP8Q_OUT_BF16 ? ScalarType::BFloat16 : ScalarType::Float;
}

// The tensors' device made current, and torch's current stream there
struct On {
    int before, device;
    explicit On(const Tensor &t) : before(c10::hip::current_device()), device(t.get_device()) {
        if (device != before) c10::hip::set_device((c10::DeviceIndex)device);
    }
    ~On() {
        if (device != before) c10::hip::set_device((c10::DeviceIndex)before);
    }
    void *stream() const { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }
};

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *pack(std::initializer_list<Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw Raised{};
    Py_ssize_t i = 0;
    for (const Tensor &t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));   // (an undefined tensor is None)
    return r;
}

constexpr int64_t kMinNormH = 8, kMaxNormH = 16384, kDenseStep = 8, kMaxRank = 256;
constexpr int64_t kMaxExperts = 1024, kMaxTopK = 32, kMaxGroups = 64, kStep = 16, kMaxK = (int64_t)1 << 17;

// ---- routing -------------------------------------------------------------------------------

// (logits, top_k, bias or None, groups, topk_groups, scale, flags)
PyObject *route(PyObject *const *a) {
    const Tensor &x = need_float(a[0], "logits");
    if (x.dim() < 1) raise(PyExc_ValueError, "logits must be [..., E]");
    const int64_t E = x.size(-1), k = integer(a[1], "top_k"), groups = integer(a[3], "groups"),
                  kept = integer(a[4], "topk_groups");
    if (E < 1 || E > kMaxExperts) raise(PyExc_ValueError, "1 to %d experts are supported, got %lld", (int)kMaxExperts, (long long)E);
    if (groups < 1 || groups > kMaxGroups || E % groups || kept < 1 || kept > groups)
        raise(PyExc_ValueError, "groups must divide the experts (at most %d) and be at least topk_groups", (int)kMaxGroups);
    if (k < 1 || k > kMaxTopK || k > kept * (E / groups))
        raise(PyExc_ValueError, "top_k must be 1 to %d and at most the experts of the topk_groups groups", (int)kMaxTopK);
    const Tensor *bias = nullptr;
    if (a[2] != Py_None) {
        bias = &need(a[2], "bias", ScalarType::Float, 4, &x);
        shaped(*bias, "bias", {E});
    }
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = k;
    const Tensor w = like(x, shape, ScalarType::Float), e = like(x, shape, ScalarType::Int);
    const On on(x);
    check("moe_route", moe_route(x.data_ptr(), code_of(x), static_cast<const float *>(data(bias)), ptr<float>(w),
                                 ptr<int32_t>(e), x.numel() / E, E, k, groups, kept, real(a[5]),
                                 (int)integer(a[6], "flags"), on.stream()));
    return pack({w, e});
}

// (dweights, logits, experts, scale, flags)
PyObject *route_backward(PyObject *const *a) {
    const Tensor &x = need_float(a[1], "logits");
    if (x.dim() < 1 || x.size(-1) < 1 || x.size(-1) > kMaxExperts)
        raise(PyExc_ValueError, "logits must be [..., E] with 1 to %d experts", (int)kMaxExperts);
    const Tensor &e = need(a[2], "experts", ScalarType::Int, 4, &x);
    if (e.dim() != x.dim() || e.sizes().slice(0, e.dim() - 1) != x.sizes().slice(0, x.dim() - 1) || e.size(-1) < 1 ||
        e.size(-1) > kMaxTopK)
        raise(PyExc_ValueError, "experts must be [..., k] for the logits' tokens, k at most %d", (int)kMaxTopK);
    const Tensor &dw = need(a[0], "dweights", ScalarType::Float, 4, &x);
    shaped(dw, "dweights", e.sizes());
    const Tensor dx = like(x, x.sizes(), x.scalar_type());
    const On on(x);
    check("moe_route_backward",
          moe_route_backward(ptr<float>(dw), x.data_ptr(), code_of(x), ptr<int32_t>(e), dx.data_ptr(),
                             x.numel() / x.size(-1), x.size(-1), e.size(-1), real(a[3]), (int)integer(a[4], "flags"),
                             on.stream()));
    return wrap(dx);
}

// ---- placement -----------------------------------------------------------------------------

// (experts, n_experts, first)
PyObject *place(PyObject *const *a) {
    const Tensor &e = need(a[0], "experts", ScalarType::Int, 4);
    if (e.dim() != 2 || e.size(1) < 1 || e.size(1) > kMaxTopK)
        raise(PyExc_ValueError, "experts must be [T, k], k at most %d", (int)kMaxTopK);
    const int64_t n = integer(a[1], "n_experts"), first = integer(a[2], "first"), T = e.size(0), k = e.size(1);
    if (n < 1 || n > kMaxExperts || first < 0)
        raise(PyExc_ValueError, "n_experts must be 1 to %d and first not negative", (int)kMaxExperts);
    const Tensor offsets = like(e, {n + 1}, ScalarType::Long), rows = like(e, {T * k}, ScalarType::Int),
                 slots = like(e, {T, k}, ScalarType::Int);
    // (a workspace from torch's allocator is kept from calls on other streams until this one is done)
    const size_t bytes = moe_place_workspace_bytes(T, k, n);
    const Tensor ws = bytes ? like(e, {(int64_t)bytes}, ScalarType::Byte) : Tensor();
    const On on(e);
    check("moe_place", moe_place(ptr<int32_t>(e), ptr<int64_t>(offsets), ptr<int32_t>(rows), ptr<int32_t>(slots), T, k,
                                 n, first, bytes ? ws.data_ptr() : nullptr, bytes, on.stream()));
    return pack({offsets, rows, slots});
}

struct Rows {
    const Tensor &h, &slots;
};
Rows rows_and_slots(PyObject *ho, PyObject *so) {
    const Tensor &h = need_float(ho, "h");
    if (h.dim() != 2) raise(PyExc_ValueError, "h must be [rows, H]");
    const Tensor &slots = need(so, "slots", ScalarType::Int, 4, &h);
    if (slots.dim() != 2 || slots.size(1) < 1 || slots.size(1) > kMaxTopK)
        raise(PyExc_ValueError, "slots must be [T, k], k at most %d", (int)kMaxTopK);
    return {h, slots};
}

// (h, slots, weights or None, out or None)
PyObject *combine(PyObject *const *a) {
    const auto [h, slots] = rows_and_slots(a[0], a[1]);
    const Tensor *w = nullptr;
    if (a[2] != Py_None) {
        w = &need(a[2], "weights", ScalarType::Float, 4, &h);
        shaped(*w, "weights", slots.sizes());
    }
    const Tensor y = output(a[3], {slots.size(0), h.size(1)}, h.scalar_type(), h.element_size(), h);
    const On on(h);
    check("moe_combine", moe_combine(h.data_ptr(), code_of(h), ptr<int32_t>(slots), static_cast<const float *>(data(w)),
                                     y.data_ptr(), slots.size(0), slots.size(1), h.size(0), h.size(1), on.stream()));
    return wrap(y);
}

// (dy, h, slots, weights)
PyObject *combine_backward(PyObject *const *a) {
    const auto [h, slots] = rows_and_slots(a[1], a[2]);
    const Tensor &w = need(a[3], "weights", ScalarType::Float, 4, &h);
    shaped(w, "weights", slots.sizes());
    const Tensor &dy = need(a[0], "dy", h.scalar_type(), h.element_size(), &h);
    shaped(dy, "dy", {slots.size(0), h.size(1)});
    const Tensor dh = like(h, h.sizes(), h.scalar_type()), dw = like(h, w.sizes(), ScalarType::Float);
    const On on(h);
    check("moe_combine_backward",
          moe_combine_backward(dy.data_ptr(), h.data_ptr(), code_of(h), ptr<int32_t>(slots), ptr<float>(w),
                               dh.data_ptr(), ptr<float>(dw), slots.size(0), slots.size(1), h.size(0), h.size(1),
                               on.stream()));
    return pack({dh, dw});
}

// ---- 8-bit integers ------------------------------------------------------------------------

void depth(int64_t K) {
    if (K % kStep || K >= kMaxK)
        raise(PyExc_ValueError, "the last dimension must be a multiple of %d below %d", (int)kStep, (int)kMaxK);
}

const Tensor *bias_of(PyObject *o, int64_t N, const Tensor &beside) {
    if (o == Py_None) return nullptr;
    const Tensor &b = need(o, "bias", ScalarType::Float, 4, &beside);
    shaped(b, "bias", {N});
    return &b;
}

// (x)
PyObject *quant(PyObject *const *a) {
    const Tensor &x = need(a[0], "x", ScalarType::BFloat16, 16);
    if (x.dim() < 1 || x.size(-1) % kStep)
        raise(PyExc_ValueError, "the last dimension must be a multiple of %d", (int)kStep);
    const int64_t K = x.size(-1);
    const Tensor q = like(x, x.sizes(), ScalarType::Char);
    const auto shape = x.sizes().slice(0, x.dim() - 1);
    // (rows of no elements have the scale of a zero row)
    const Tensor s = K ? like(x, shape, ScalarType::Float) : at::zeros(shape, x.options().dtype(ScalarType::Float));
    const On on(x);
    check("int8_quant", int8_quant(ptr<uint16_t>(x), ptr<int8_t>(q), ptr<float>(s), rows_of(x), K, on.stream()));
    return pack({q, s});
}

// (a, a_s, w, w_s, bias or None, dtype code, out or None)
PyObject *gemm(PyObject *const *a) {
    const Tensor &x = need(a[0], "a", ScalarType::Char, 16), &w = need(a[2], "w", ScalarType::Char, 16, &x);
    if (x.dim() < 1 || w.dim() != 2 || w.size(1) != x.size(-1))
        raise(PyExc_ValueError, "w must be [N, K] with the activation's K");
    const int64_t N = w.size(0), K = w.size(1);
    depth(K);
    const Tensor &xs = need(a[1], "a_s", ScalarType::Float, 4, &x), &ws = need(a[3], "w_s", ScalarType::Float, 4, &x);
    shaped(xs, "a_s", x.sizes().slice(0, x.dim() - 1));
    shaped(ws, "w_s", {N});
    const Tensor *bias = bias_of(a[4], N, x);
    const ScalarType type = type_of_code(a[5]);
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = N;
    const Tensor y = output(a[6], shape, type, 4, x);
    const On on(x);
    check("int8_gemm", int8_gemm(ptr<int8_t>(x), ptr<float>(xs), ptr<int8_t>(w), ptr<float>(ws),
                                 static_cast<const float *>(data(bias)), y.data_ptr(), code_of(y), rows_of(x), N, K,
                                 on.stream()));
    return wrap(y);
}

// (x, weight, weight_scale, bias or None, dtype code)
PyObject *linear(PyObject *const *a) {
    const Tensor &x = need(a[0], "x", ScalarType::BFloat16, 16), &w = need(a[1], "weight", ScalarType::Char, 16, &x);
    if (x.dim() < 1 || w.dim() != 2 || w.size(1) != x.size(-1))
        raise(PyExc_ValueError, "weight must be [N, K] with the activation's K");
    const int64_t N = w.size(0), K = w.size(1), M = rows_of(x);
    depth(K);
    const Tensor &ws = need(a[2], "weight_scale", ScalarType::Float, 4, &x);
    shaped(ws, "weight_scale", {N});
    const Tensor *bias = bias_of(a[3], N, x);
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = N;
    const Tensor y = like(x, shape, type_of_code(a[4]));
    const size_t bytes = int8_linear_workspace_bytes(M, N, K);
    const Tensor work = bytes ? like(x, {(int64_t)bytes}, ScalarType::Byte) : Tensor();
    const On on(x);
    check("int8_linear", int8_linear(ptr<uint16_t>(x), ptr<int8_t>(w), ptr<float>(ws),
                                     static_cast<const float *>(data(bias)), y.data_ptr(), code_of(y), M, N, K,
                                     bytes ? work.data_ptr() : nullptr, bytes, on.stream()));
    return wrap(y);
}

// (a, a_s, w, w_s, offsets, rows or None, dtype code, out or None)
PyObject *grouped_gemm(PyObject *const *a) {
    const Tensor &x = need(a[0], "a", ScalarType::Char, 16), &w = need(a[2], "w", ScalarType::Char, 16, &x);
    if (x.dim() != 2 || w.dim() != 3 || w.size(2) != x.size(1))
        raise(PyExc_ValueError, "a must be [tokens, K] and w [E, N, K]");
    const int64_t tokens = x.size(0), K = x.size(1), E = w.size(0), N = w.size(1);
    depth(K);
    const Tensor &xs = need(a[1], "a_s", ScalarType::Float, 4, &x), &ws = need(a[3], "w_s", ScalarType::Float, 4, &x);
    shaped(xs, "a_s", {tokens});
    shaped(ws, "w_s", {E, N});
    const Tensor &offsets = need(a[4], "offsets", ScalarType::Long, 8, &x);
    shaped(offsets, "offsets", {E + 1});
    const Tensor *rows = nullptr;
    if (a[5] != Py_None) {
        rows = &need(a[5], "rows", ScalarType::Int, 4, &x);
        if (rows->dim() != 1) raise(PyExc_ValueError, "rows must be [R]");
    }
    const int64_t R = rows ? rows->size(0) : tokens;
    const Tensor y = output(a[7], {R, N}, type_of_code(a[6]), 4, x);
    const On on(x);
    check("int8_grouped_gemm",
          int8_grouped_gemm(ptr<int8_t>(x), ptr<float>(xs), ptr<int8_t>(w), ptr<float>(ws), ptr<int64_t>(offsets),
                            static_cast<const int32_t *>(data(rows)), y.data_ptr(), code_of(y), E, R, tokens, N, K,
                            on.stream()));
    return wrap(y);
}

// ---- the dense block -----------------------------------------------------------------------

struct Norm {   // the arguments that residual_norm and its gradient share
    const Tensor *weight = nullptr, *post = nullptr, *gate = nullptr;
    int flags = 0;
    float scale, eps;
    int64_t H;
    Norm(const Tensor &x, const char *name, PyObject *w, PyObject *p, PyObject *g, PyObject *s, PyObject *e)
        : scale(real(s)), eps(real(e)) {
        if (x.dim() < 1 || x.size(-1) < kMinNormH || x.size(-1) > kMaxNormH)
            raise(PyExc_ValueError, "%s must be [..., H] with H from %d to %d", name, (int)kMinNormH, (int)kMaxNormH);
        if (!(eps >= 0.0f)) raise(PyExc_ValueError, "eps must not be negative");
        H = x.size(-1);
        if (w != Py_None) shaped(*(weight = &need(w, "weight", ScalarType::Float, 4, &x)), "weight", {H});
        if (p != Py_None) shaped(*(post = &need(p, "post", ScalarType::Float, 4, &x)), "post", {H});
        if (g == Py_None) return;
        // one per channel, or per element
        if (tensor(g, "gate").dim() == 1 && THPVariable_Unpack(g).scalar_type() == ScalarType::Float) {
            shaped(*(gate = &need(g, "gate", ScalarType::Float, 4, &x)), "gate", {H});
        } else {
            shaped(*(gate = &need(g, "gate", x.scalar_type(), x.element_size(), &x)), "gate", x.sizes());
            flags = FP8Q_NORM_GATES;
        }
    }
};
const Tensor *beside_of(PyObject *o, const char *name, const Tensor &x) {   // of x's type and shape, or None
    if (o == Py_None) return nullptr;
    const Tensor &t = need(o, name, x.scalar_type(), x.element_size(), &x);
    shaped(t, name, x.sizes());
    return &t;
}
void *out_of(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// (x, y or None, weight or None, post or None, gate or None, scale, eps)
PyObject *norm(PyObject *const *a) {
    const Tensor &x = need_float(a[0], "x");
    const Tensor *y = beside_of(a[1], "y", x);
    const Norm n(x, "x", a[2], a[3], a[4], a[5], a[6]);
    if (!y && !n.weight) raise(PyExc_ValueError, "weight must be given");
    const Tensor t = y ? like(x, x.sizes(), x.scalar_type()) : Tensor(),
                 z = n.weight ? like(x, x.sizes(), x.scalar_type()) : Tensor();
    const On on(x);
    check("residual_norm",
          residual_norm(x.data_ptr(), data(y), code_of(x), static_cast<const float *>(data(n.weight)),
                        static_cast<const float *>(data(n.post)), data(n.gate), n.flags, n.scale, n.eps, out_of(t),
                        out_of(z), rows_of(x), n.H, on.stream()));
    return y ? pack({t, z}) : wrap(z);
}

// (dt or None, dz or None, t, y or None, weight or None, post or None, gate or None, scale, eps)
PyObject *norm_backward(PyObject *const *a) {
    const Tensor &t = need_float(a[2], "t");
    const Tensor *y = beside_of(a[3], "y", t), *dt = beside_of(a[0], "dt", t), *dz = beside_of(a[1], "dz", t);
    const Norm n(t, "t", a[4], a[5], a[6], a[7], a[8]);
    if ((dz != nullptr) != (n.weight != nullptr)) raise(PyExc_ValueError, "dz and weight go together");
    if (!dt && !dz) raise(PyExc_ValueError, "dt or dz must be given");
    const int64_t T = rows_of(t);
    const Tensor dx = like(t, t.sizes(), t.scalar_type()), dy = y ? like(t, t.sizes(), t.scalar_type()) : Tensor(),
                 dw = n.weight ? like(t, {n.H}, ScalarType::Float) : Tensor(),
                 dp = y && n.post ? like(t, {n.H}, ScalarType::Float) : Tensor(),
                 dg = y && n.gate ? like(t, n.gate->sizes(), n.gate->scalar_type()) : Tensor();
    const size_t bytes = residual_norm_backward_workspace_bytes(T, n.H);
    const Tensor ws = bytes ? like(t, {(int64_t)bytes}, ScalarType::Byte) : Tensor();
    const On on(t);
    check("residual_norm_backward",
          residual_norm_backward(data(dt), data(dz), t.data_ptr(), data(y), code_of(t),
                                 static_cast<const float *>(data(n.weight)), static_cast<const float *>(data(n.post)),
                                 data(n.gate), n.flags, n.scale, n.eps, dx.data_ptr(), out_of(dy),
                                 static_cast<float *>(out_of(dw)), static_cast<float *>(out_of(dp)), out_of(dg), T, n.H,
                                 out_of(ws), bytes, on.stream()));
    return pack({dx, dy, dw, dp, dg});
}

struct Gated {
    const Tensor &x, &w;
    int64_t M, F, K;
    Gated(PyObject *xo, PyObject *wo)
        : x(need(xo, "x", ScalarType::BFloat16, 16)), w(need(wo, "w", ScalarType::BFloat16, 16, &x)) {
        if (x.dim() < 1 || w.dim() != 2 || w.size(1) != x.size(-1) || w.size(0) % 2)
            raise(PyExc_ValueError, "w must be [2 F, K] with the activation's K");
        M = rows_of(x), F = w.size(0) / 2, K = w.size(1);
        if (F % kDenseStep || K % kDenseStep) raise(PyExc_ValueError, "F and K must be multiples of %d", (int)kDenseStep);
    }
    c10::SmallVector<int64_t, 6> shape(int64_t last) const {
        c10::SmallVector<int64_t, 6> s(x.sizes().begin(), x.sizes().end());
        s.back() = last;
        return s;
    }
};

// (x, w, act, keep, dtype code)
PyObject *gated(PyObject *const *a) {
    const Gated g(a[0], a[1]);
    const int act = (int)integer(a[2], "act");
    const bool keep = truth(a[3]);
    const Tensor h = like(g.x, g.shape(g.F), type_of_code(a[4])),
                 gu = keep ? like(g.x, g.shape(2 * g.F), ScalarType::BFloat16) : Tensor();
    const On on(g.x);
    check("gated_linear", gated_linear(ptr<uint16_t>(g.x), ptr<uint16_t>(g.w), h.data_ptr(), code_of(h),
                                       static_cast<uint16_t *>(out_of(gu)), act, g.M, g.F, g.K, on.stream()));
    return keep ? pack({h, gu}) : wrap(h);
}

// (dh, x, w, gu or None, act and flags, dx dtype code, dw dtype code)
PyObject *gated_backward(PyObject *const *a) {
    const Gated g(a[1], a[2]);
    const Tensor &dh = need(a[0], "dh", ScalarType::BFloat16, 16, &g.x);
    shaped(dh, "dh", g.shape(g.F));
    const Tensor *gu = nullptr;
    if (a[3] != Py_None) shaped(*(gu = &need(a[3], "gu", ScalarType::BFloat16, 16, &g.x)), "gu", g.shape(2 * g.F));
    const Tensor dx = like(g.x, g.x.sizes(), type_of_code(a[5])), dw = like(g.x, g.w.sizes(), type_of_code(a[6]));
    const int act = (int)integer(a[4], "act");
    const size_t bytes = act & FP8Q_GATED_WIDE ? gated_linear_backward_wide_workspace_bytes(g.M, g.F, g.K)
                                               : gated_linear_backward_workspace_bytes(g.M, g.F, g.K);
    const Tensor ws = bytes ? like(g.x, {(int64_t)bytes}, ScalarType::Byte) : Tensor();
    const On on(g.x);
    check("gated_linear_backward",
          gated_linear_backward(ptr<uint16_t>(dh), ptr<uint16_t>(g.x), ptr<uint16_t>(g.w),
                                static_cast<const uint16_t *>(data(gu)), act, dx.data_ptr(),
                                code_of(dx), dw.data_ptr(), code_of(dw), g.M, g.F, g.K, out_of(ws), bytes, on.stream()));
    return pack({dx, dw});
}

// (x, w or None, a, b, ids, scales or None, bias or None, base or None, dtype code, out or None): w or base
PyObject *adapter(PyObject *const *a) {
    const Tensor &x = need(a[0], "x", ScalarType::BFloat16, 16);
    const Tensor &la = need(a[2], "a", ScalarType::BFloat16, 16, &x), &lb = need(a[3], "b", ScalarType::BFloat16, 16, &x);
    if (x.dim() < 1 || la.dim() != 3 || lb.dim() != 3 || la.size(0) != lb.size(0) || la.size(1) != lb.size(2) ||
        la.size(2) != x.size(-1))
        raise(PyExc_ValueError, "a must be [adapters, rank, K] with the activation's K and b [adapters, N, rank]");
    const int64_t M = rows_of(x), K = x.size(-1), L = la.size(0), r = la.size(1), N = lb.size(1);
    if (K % kDenseStep) raise(PyExc_ValueError, "the last dimension must be a multiple of %d", (int)kDenseStep);
    if (r < kDenseStep || r % kDenseStep || r > kMaxRank)
        raise(PyExc_ValueError, "the rank must be a multiple of %d from %d to %d", (int)kDenseStep, (int)kDenseStep, (int)kMaxRank);
    const Tensor &ids = need(a[4], "ids", ScalarType::Int, 4, &x);
    shaped(ids, "ids", x.sizes().slice(0, x.dim() - 1));
    const Tensor *scales = nullptr, *w = nullptr, *base = nullptr;
    if (a[5] != Py_None) shaped(*(scales = &need(a[5], "scales", ScalarType::Float, 4, &x)), "scales", {L});
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = N;
    if (a[1] != Py_None) shaped(*(w = &need(a[1], "w", ScalarType::BFloat16, 16, &x)), "w", {N, K});
    else shaped(*(base = &need_float(a[7], "y", &x)), "y", shape);
    const Tensor *bias = bias_of(a[6], N, x);
    if (base && reinterpret_cast<uintptr_t>(base->data_ptr()) % 4) raise(PyExc_ValueError, "y must be 4-byte aligned");
    const Tensor y = output(a[9], shape, base ? base->scalar_type() : type_of_code(a[8]), 4, x);
    if (a[9] != Py_None) {   // (x, a and scales are read by the first launch; beside w x is read by the second too)
        if (w) apart(y, &x, "x"), apart(y, w, "w");
        else if (y.data_ptr() != base->data_ptr()) apart(y, base, "y but as a whole");
        apart(y, &lb, "b"), apart(y, &ids, "ids"), apart(y, bias, "bias");
    }
    const size_t bytes = L ? adapter_linear_workspace_bytes(M, K, r) : 0;
    const Tensor ws = bytes ? like(x, {(int64_t)bytes}, ScalarType::Byte) : Tensor();
    const On on(x);
    check("adapter_linear",
          adapter_linear(ptr<uint16_t>(x), static_cast<const uint16_t *>(data(w)), static_cast<const float *>(data(bias)),
                         ptr<uint16_t>(la), ptr<uint16_t>(lb), static_cast<const float *>(data(scales)), ptr<int32_t>(ids),
                         data(base), y.data_ptr(), code_of(y), M, N, K, L, r, out_of(ws), bytes, on.stream()));
    return wrap(y);
}

// ---- module --------------------------------------------------------------------------------

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    HANDLE_TH_ERRORS
    try {
        return F(args);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define ENTRY(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<&name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(route, 7),    ENTRY(route_backward, 5), ENTRY(place, 3),
                         ENTRY(combine, 4),  ENTRY(combine_backward, 4), ENTRY(quant, 1),
                         ENTRY(gemm, 7),     ENTRY(linear, 5),         ENTRY(grouped_gemm, 8),
                         ENTRY(norm, 7),     ENTRY(norm_backward, 9),  ENTRY(gated, 5),
                         ENTRY(gated_backward, 7), ENTRY(adapter, 10),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "Calls of the routed-expert, 8-bit integer and dense-block operators", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
