// Python side of the operators around the layer: checks torch tensors,
// allocates the outputs that were not given and calls the C ABI.  These calls
// stand between two small kernels of a decode step, where ctypes and checks in
// Python cost more than the kernels (RMSNorm of 64 x 4096 with its residual:
// 9.2 us a call that way, 4.3 us of it the ctypes call and the launch; 4.0 us
// here, about 3 us of it the launch).
//
// The library's entry points come in as addresses (bind), so this module works
// on whichever build of the library the package loaded.  A wrong argument is
// an AssertionError, a status of the library is returned as a number.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

namespace {

// the C ABI (include/moe.h); a stream is passed as the pointer it is
using NormFn = int (*)(const void*, const void*, const void*, float, int32_t, int32_t, int32_t, void*, void*, uint8_t*,
                       void*, void*);
using ActFn = int (*)(const void*, int32_t, int32_t, float, int32_t, void*, uint8_t*, void*, void*);
using DenseFn = int (*)(const void*, const void*, const void*, const void*, int32_t, int32_t, int32_t, void*, void*);
using GroupedFn = int (*)(const void*, const void*, const void*, const void*, const void*, int32_t, int32_t, int32_t,
                          int32_t, int32_t, void*, void*);
NormFn g_norm;
ActFn g_act;
DenseFn g_dense;
GroupedFn g_grouped;

constexpr int kBf16 = 0, kFp8 = 1, kMx = 2;   // MOE_WDTYPE_*

// (an empty text where a Python exception is set already)
struct Wrong : std::runtime_error {
    using std::runtime_error::runtime_error;
};
void need(bool ok, const char* what, const char* why) {
    if (!ok) throw Wrong(std::string(what) + ": " + why);
}

// one tensor argument, or the place of an output
struct Arg {
    PyObject* obj;             // borrowed; None for a missing one
    const at::Tensor* t;       // null for None
    const char* what;
    Arg(PyObject* o, const char* w) : obj(o), t(nullptr), what(w) {
        if (o == Py_None) return;
        need(THPVariable_Check(o), w, "must be a tensor");
        t = &THPVariable_Unpack(o);
    }
    void type(std::initializer_list<at::ScalarType> types) const {
        for (at::ScalarType s : types)
            if (t->scalar_type() == s) return;
        throw Wrong(std::string(what) + ": dtype " + c10::toString(t->scalar_type()) + ", expected " +
                    c10::toString(*types.begin()));
    }
    void is(std::initializer_list<at::ScalarType> types, at::IntArrayRef shape) const {
        need(t != nullptr, what, "must be a tensor");
        type(types);
        if (t->sizes() != shape) {
            std::string s = std::string(what) + ": shape [";
            for (int64_t v : t->sizes()) s += std::to_string(v) + " ";
            s += "], expected [";
            for (int64_t v : shape) s += std::to_string(v) + " ";
            throw Wrong(s + "]");
        }
        need(t->is_contiguous(), what, "must be contiguous");
    }
    void on(const at::Tensor& first) const {
        if (t) need(t->device() == first.device(), what, "must be on the device of the first operand");
    }
    void* ptr() const { return t ? t->data_ptr() : nullptr; }
};

// an output: the given tensor, or a new one when `want`
struct Out {
    Arg arg;
    at::Tensor fresh;
    Out(PyObject* o, const char* w) : arg(o, w) {}
    void make(bool want, at::ScalarType as, std::initializer_list<at::ScalarType> types, at::IntArrayRef shape,
              const at::Tensor& like) {
        if (!want) {
            need(!arg.t, arg.what, "given, but not asked for");
        } else if (arg.t) {
            arg.is(types, shape);
        } else {
            fresh = at::empty(shape, like.options().dtype(as));
        }
    }
    void* ptr() const { return fresh.defined() ? fresh.data_ptr() : arg.ptr(); }
    PyObject* result() const {
        if (fresh.defined()) return THPVariable_Wrap(fresh);
        Py_INCREF(arg.obj);
        return arg.obj;
    }
};

constexpr auto BF16 = at::ScalarType::BFloat16;
constexpr auto F32 = at::ScalarType::Float;
constexpr auto U8 = at::ScalarType::Byte;
constexpr auto E4M3 = at::ScalarType::Float8_e4m3fn;
constexpr auto I32 = at::ScalarType::Int;

int32_t size32(int64_t v, const char* what) {
    need(v <= INT32_MAX, what, "a size beyond 2^31 - 1");
    return int32_t(v);
}
void on_gpu(const at::Tensor& first, std::initializer_list<const Arg*> others) {
    need(first.is_cuda(), "operands", "must be on a GPU");
    for (const Arg* a : others) a->on(first);
}
long number(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Wrong("");
    return v;
}
void* stream_of(PyObject* o) { return PyLong_AsVoidPtr(o); }
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Wrong("");
    return float(v);
}
// with_y: None (whether y is given or there is no quantisation), or a truth value
bool wants_y(PyObject* with_y, PyObject* y, int quant) {
    if (with_y == Py_None) return y != Py_None || quant == kBf16;
    const int yes = PyObject_IsTrue(with_y);
    if (yes < 0) throw Wrong("");   // with the exception that its truth value raised
    return yes == 1;
}
void make_codes(int quant, int64_t rows, int64_t cols, const at::Tensor& like, Out& codes, Out& scales) {
    const bool mx = quant == kMx;
    codes.make(quant != kBf16, U8, {U8, E4M3}, {rows, cols}, like);
    scales.make(quant != kBf16, mx ? U8 : F32, {mx ? U8 : F32}, {rows, std::max<int64_t>(cols / (mx ? 32 : 128), 1)},
                like);
}

template <typename F>
int call(F f) {
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return st;
}

// run a call's body; wrong arguments become AssertionError, torch's errors (out
// of memory) the exceptions they are in Python
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
    HANDLE_TH_ERRORS
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return body();
    } catch (const Wrong& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_AssertionError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// rmsnorm(x, weight, eps, residual, quant, with_y, y, residual_out, codes, scales, stream)
PyObject* py_rmsnorm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        Arg x(v[0], "x"), weight(v[1], "weight"), residual(v[3], "residual");
        const int quant = int(number(v[4]));
        Out y(v[6], "y"), res(v[7], "residual_out"), codes(v[8], "codes"), scales(v[9], "scales");
        need(x.t && x.t->dim() == 2, "x", "must be [rows, cols]");
        const int64_t rows = x.t->size(0), cols = x.t->size(1);
        x.is({BF16}, {rows, cols});
        weight.is({BF16}, {cols});
        if (residual.t) residual.is({BF16}, {rows, cols});
        y.make(wants_y(v[5], v[6], quant), BF16, {BF16}, {rows, cols}, *x.t);
        res.make(residual.t != nullptr, BF16, {BF16}, {rows, cols}, *x.t);
        make_codes(quant, rows, cols, *x.t, codes, scales);
        on_gpu(*x.t, {&weight, &residual, &y.arg, &res.arg, &codes.arg, &scales.arg});
        const int32_t r = size32(rows, "x"), c = size32(cols, "x");
        const float eps = real(v[2]);
        void* s = stream_of(v[10]);
        const int st = call([&] {
            return g_norm(x.ptr(), residual.ptr(), weight.ptr(), eps, r, c, quant, res.ptr(), y.ptr(),
                          static_cast<uint8_t*>(codes.ptr()), scales.ptr(), s);
        });
        if (st != 0) return PyLong_FromLong(st);
        return Py_BuildValue("(NNNN)", y.result(), res.result(), codes.result(), scales.result());
    });
}

// silu_mul(h, quant, clamp_limit, with_y, y, codes, scales, stream)
PyObject* py_silu_mul(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        Arg h(v[0], "h");
        const int quant = int(number(v[1]));
        Out y(v[4], "y"), codes(v[5], "codes"), scales(v[6], "scales");
        need(h.t && h.t->dim() == 2 && h.t->size(1) % 2 == 0, "h", "must be [rows, 2 * cols]");
        const int64_t rows = h.t->size(0), cols = h.t->size(1) / 2;
        h.is({BF16}, {rows, 2 * cols});
        y.make(wants_y(v[3], v[4], quant), BF16, {BF16}, {rows, cols}, *h.t);
        make_codes(quant, rows, cols, *h.t, codes, scales);
        on_gpu(*h.t, {&y.arg, &codes.arg, &scales.arg});
        const int32_t r = size32(rows, "h"), c = size32(cols, "h");
        const float limit = real(v[2]);
        void* s = stream_of(v[7]);
        const int st = call([&] {
            return g_act(h.ptr(), r, c, limit, quant, y.ptr(), static_cast<uint8_t*>(codes.ptr()), scales.ptr(), s);
        });
        if (st != 0) return PyLong_FromLong(st);
        return Py_BuildValue("(NNN)", y.result(), codes.result(), scales.result());
    });
}

// gemm_fp8(a, a_scale, w, w_scale, out, stream)
PyObject* py_gemm_fp8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        Arg a(v[0], "a"), as(v[1], "a_scale"), w(v[2], "w"), ws(v[3], "w_scale");
        Out out(v[4], "out");
        need(a.t && a.t->dim() == 2, "a", "must be [M, K]");
        need(w.t && w.t->dim() == 2, "w", "must be [N, K]");
        const int64_t M = a.t->size(0), K = a.t->size(1), N = w.t->size(0);
        a.is({U8, E4M3}, {M, K});
        w.is({U8, E4M3}, {N, K});
        as.is({F32}, {M, K / 128});
        ws.is({F32}, {(N + 127) / 128, K / 128});
        out.make(true, BF16, {BF16}, {M, N}, *a.t);
        on_gpu(*a.t, {&as, &w, &ws, &out.arg});
        const int32_t m = size32(M, "a"), k = size32(K, "a"), nn = size32(N, "w");
        void* s = stream_of(v[5]);
        const int st = call([&] { return g_dense(a.ptr(), as.ptr(), w.ptr(), ws.ptr(), m, nn, k, out.ptr(), s); });
        return st != 0 ? PyLong_FromLong(st) : out.result();
    });
}

// grouped_gemm(a, w, offsets, a_scale, w_scale, out, stream)
PyObject* py_grouped_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        Arg a(v[0], "a"), w(v[1], "w"), off(v[2], "offsets"), as(v[3], "a_scale"), ws(v[4], "w_scale");
        Out out(v[5], "out");
        need(a.t && a.t->dim() == 2, "a", "must be [rows, K]");
        need(w.t && w.t->dim() == 3, "w", "must be [E, N, K]");
        const int64_t rows = a.t->size(0), K = a.t->size(1), E = w.t->size(0), N = w.t->size(1);
        const bool fp8 = a.t->scalar_type() == U8 || a.t->scalar_type() == E4M3;
        if (fp8) {
            a.is({U8, E4M3}, {rows, K});
            w.is({U8, E4M3}, {E, N, K});
            as.is({F32}, {rows, K / 128});
            ws.is({F32}, {E, (N + 127) / 128, K / 128});
        } else {
            a.is({BF16}, {rows, K});
            w.is({BF16}, {E, N, K});
            need(!as.t && !ws.t, "a_scale, w_scale", "bf16 operands take no scales");
        }
        off.is({I32}, {E + 1});
        out.make(true, BF16, {BF16}, {rows, N}, *a.t);
        on_gpu(*a.t, {&w, &off, &as, &ws, &out.arg});
        const int32_t r = size32(rows, "a"), k = size32(K, "a"), e = size32(E, "w"), nn = size32(N, "w");
        void* s = stream_of(v[6]);
        const int st = call([&] {
            return g_grouped(a.ptr(), as.ptr(), w.ptr(), ws.ptr(), off.ptr(), r, e, nn, k, fp8 ? kFp8 : kBf16,
                             out.ptr(), s);
        });
        return st != 0 ? PyLong_FromLong(st) : out.result();
    });
}

// bind(rmsnorm, silu_mul, gemm_fp8, grouped_gemm): addresses of the entry points
PyObject* py_bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        g_norm = reinterpret_cast<NormFn>(PyLong_AsVoidPtr(v[0]));
        g_act = reinterpret_cast<ActFn>(PyLong_AsVoidPtr(v[1]));
        g_dense = reinterpret_cast<DenseFn>(PyLong_AsVoidPtr(v[2]));
        g_grouped = reinterpret_cast<GroupedFn>(PyLong_AsVoidPtr(v[3]));
        Py_RETURN_NONE;
    });
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_bind)), METH_FASTCALL, nullptr},
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_rmsnorm)), METH_FASTCALL, nullptr},
    {"silu_mul", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_silu_mul)), METH_FASTCALL, nullptr},
    {"gemm_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_gemm_fp8)), METH_FASTCALL, nullptr},
    {"grouped_gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_grouped_gemm)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
