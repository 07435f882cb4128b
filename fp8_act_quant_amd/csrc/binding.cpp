// binding.cpp -- the Python calls of the routed-expert and 8-bit integer operators: argument
// checks, outputs and workspaces from torch's allocator, one call of the C ABI (fp8q.h) on the
// tensors' device and torch's current stream there.
//
// Native because these calls are small: a decode step's kernel takes 3 us, and checks, allocations
// and ctypes in Python took 6 us a call around the 3 us that the launch itself takes; here they
// take about 1 us. Names, defaults and documentation are in moe.py and int8.py.
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
    for (const Tensor &t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}

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
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "Calls of the routed-expert and 8-bit integer operators", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
