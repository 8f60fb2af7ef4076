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
using SortFn = int (*)(const void*, const void*, const void*, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t,
                       void*, void*, void*, void*, void*, int64_t, void*);
using SortBytesFn = int64_t (*)(int32_t, int32_t, int32_t);
using CombineFn = int (*)(const void*, const void*, const void*, int32_t, int32_t, int32_t, int32_t, void*, void*);
using CombineBwdFn = int (*)(const void*, const void*, const void*, const void*, int32_t, int32_t, int32_t, int32_t,
                             void*, void*, void*);
using QuantInt8Fn = int (*)(const void*, int32_t, int32_t, void*, void*, void*);
using ActInt8Fn = int (*)(const void*, int32_t, int32_t, float, void*, void*, void*);
NormFn g_norm;
ActFn g_act;
DenseFn g_dense, g_dense_int8;
GroupedFn g_grouped;
SortFn g_sort;
SortBytesFn g_sort_bytes;
CombineFn g_combine;
CombineBwdFn g_combine_bwd;
QuantInt8Fn g_quant_int8;
ActInt8Fn g_act_int8;

constexpr int kBf16 = 0, kFp8 = 1, kMx = 2, kInt8 = 4;   // MOE_WDTYPE_*

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
constexpr auto I8 = at::ScalarType::Char;

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
        } else if (a.t->scalar_type() == I8) {
            w.is({I8}, {E, N, K});
            a.is({I8}, {rows, K});
            as.is({F32}, {rows});
            ws.is({F32}, {E, N});
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
            return g_grouped(a.ptr(), as.ptr(), w.ptr(), ws.ptr(), off.ptr(), r, e, nn, k,
                             fp8 ? kFp8 : a.t->scalar_type() == I8 ? kInt8 : kBf16, out.ptr(), s);
        });
        return st != 0 ? PyLong_FromLong(st) : out.result();
    });
}

// gemm_int8(a, a_scale, w, w_scale, out, stream)
PyObject* py_gemm_int8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject* {
        Arg a(v[0], "a"), as(v[1], "a_scale"), w(v[2], "w"), ws(v[3], "w_scale");
        Out out(v[4], "out");
        need(a.t && a.t->dim() == 2, "a", "must be [M, K]");
        need(w.t && w.t->dim() == 2, "w", "must be [N, K]");
        const int64_t M = a.t->size(0), K = a.t->size(1), N = w.t->size(0);
        a.is({I8}, {M, K});
        w.is({I8}, {N, K});
        as.is({F32}, {M});
        ws.is({F32}, {N});
        out.make(true, BF16, {BF16}, {M, N}, *a.t);
        on_gpu(*a.t, {&as, &w, &ws, &out.arg});
        const int32_t m = size32(M, "a"), k = size32(K, "a"), nn = size32(N, "w");
        void* s = stream_of(v[5]);
        const int st = call([&] { return g_dense_int8(a.ptr(), as.ptr(), w.ptr(), ws.ptr(), m, nn, k, out.ptr(), s); });
        return st != 0 ? PyLong_FromLong(st) : out.result();
    });
}

// quant_act_int8(x, codes, scales, stream)
PyObject* py_quant_act_int8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        Arg x(v[0], "x");
        Out codes(v[1], "codes"), scales(v[2], "scales");
        need(x.t && x.t->dim() == 2, "x", "must be [rows, cols]");
        const int64_t rows = x.t->size(0), cols = x.t->size(1);
        x.is({BF16}, {rows, cols});
        codes.make(true, I8, {I8}, {rows, cols}, *x.t);
        scales.make(true, F32, {F32}, {rows}, *x.t);
        on_gpu(*x.t, {&codes.arg, &scales.arg});
        const int32_t r = size32(rows, "x"), c = size32(cols, "x");
        void* s = stream_of(v[3]);
        const int st = call([&] { return g_quant_int8(x.ptr(), r, c, codes.ptr(), scales.ptr(), s); });
        if (st != 0) return PyLong_FromLong(st);
        return Py_BuildValue("(NN)", codes.result(), scales.result());
    });
}

// silu_mul_int8(h, clamp_limit, codes, scales, stream)
PyObject* py_silu_mul_int8(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        Arg h(v[0], "h");
        Out codes(v[2], "codes"), scales(v[3], "scales");
        need(h.t && h.t->dim() == 2 && h.t->size(1) % 2 == 0, "h", "must be [rows, 2 * cols]");
        const int64_t rows = h.t->size(0), cols = h.t->size(1) / 2;
        h.is({BF16}, {rows, 2 * cols});
        codes.make(true, I8, {I8}, {rows, cols}, *h.t);
        scales.make(true, F32, {F32}, {rows}, *h.t);
        on_gpu(*h.t, {&codes.arg, &scales.arg});
        const int32_t r = size32(rows, "h"), c = size32(cols, "h");
        const float limit = real(v[1]);
        void* s = stream_of(v[4]);
        const int st = call([&] { return g_act_int8(h.ptr(), r, c, limit, codes.ptr(), scales.ptr(), s); });
        if (st != 0) return PyLong_FromLong(st);
        return Py_BuildValue("(NN)", codes.result(), scales.result());
    });
}

// sort_rows(x, topk_ids, E, x_scale, rowtype or -1 for x's own, rows, scales, offsets, inv, scratch, stream)
PyObject* py_sort_rows(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        Arg x(v[0], "x"), ids(v[1], "topk_ids"), xs(v[3], "x_scale"), scratch(v[9], "scratch");
        Out rows(v[5], "rows"), scales(v[6], "scales"), offsets(v[7], "offsets"), inv(v[8], "inv");
        const long E = number(v[2]), asked = number(v[4]);
        need(x.t && x.t->dim() == 2, "x", "must be [T, cols]");
        need(ids.t && ids.t->dim() == 2, "topk_ids", "must be [T, topk]");
        need(E >= 1 && E <= INT32_MAX, "E", "must be a number of experts");
        const int64_t T = x.t->size(0), cols = x.t->size(1), topk = ids.t->size(1);
        const bool bf16 = x.t->scalar_type() == BF16, int8 = x.t->scalar_type() == I8;
        const int xtype = bf16 ? kBf16 : int8 ? kInt8 : kFp8;
        const int type = asked < 0 ? xtype : int(asked);
        need(bf16 || asked < 0, "quant", "x holds codes already");
        ids.is({I32}, {T, topk});
        if (bf16) {
            x.is({BF16}, {T, cols});
            need(!xs.t, "x_scale", "bf16 rows take no scales");
        } else if (int8) {
            x.is({I8}, {T, cols});
            xs.is({F32}, {T});
        } else {
            x.is({E4M3, U8}, {T, cols});
            xs.is({F32}, {T, cols / 128});
        }
        const int32_t t = size32(T, "x"), c = size32(cols, "x"), k = size32(topk, "topk_ids");
        const int64_t bytes = g_sort_bytes(t, k, int32_t(E));   // (and its checks, before anything is allocated)
        if (bytes < 0) return PyLong_FromLong(long(bytes));
        const int64_t R = T * topk;
        // fp8 rows made from bf16 ones are uint8 as moe_quant_act's are, copied ones of x's own type
        const auto as = type == kBf16 ? BF16 : type == kInt8 ? I8 : bf16 ? U8 : x.t->scalar_type();
        if (type == kFp8) rows.make(true, as, {U8, E4M3}, {R, cols}, *x.t);
        else rows.make(true, as, {as}, {R, cols}, *x.t);
        if (type == kInt8) scales.make(true, F32, {F32}, {R}, *x.t);
        else scales.make(type != kBf16, F32, {F32}, {R, cols / 128}, *x.t);
        offsets.make(true, I32, {I32}, {E + 1}, *x.t);
        inv.make(true, I32, {I32}, {T, topk}, *x.t);
        if (scratch.t) {
            scratch.type({U8});
            need(scratch.t->is_contiguous(), "scratch", "must be contiguous");
        }
        on_gpu(*x.t, {&ids, &xs, &rows.arg, &scales.arg, &offsets.arg, &inv.arg, &scratch});
        at::Tensor own;
        if (!scratch.t && bytes > 0) own = at::empty({bytes}, x.t->options().dtype(U8));
        void* ws = own.defined() ? own.data_ptr() : scratch.ptr();
        const int64_t room = own.defined() ? bytes : scratch.t ? scratch.t->numel() : 0;
        void* s = stream_of(v[10]);
        const int st = call([&] {
            return g_sort(x.ptr(), xs.ptr(), ids.ptr(), t, k, int32_t(E), c, xtype, type, rows.ptr(), scales.ptr(),
                          offsets.ptr(), inv.ptr(), ws, room, s);
        });
        if (st != 0) return PyLong_FromLong(st);
        return Py_BuildValue("(NNNN)", rows.result(), scales.result(), offsets.result(), inv.result());
    });
}

// combine_rows(rows, inv, weights, out, stream)
PyObject* py_combine_rows(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        Arg rows(v[0], "rows"), inv(v[1], "inv"), weights(v[2], "weights");
        Out out(v[3], "out");
        need(rows.t && rows.t->dim() == 2, "rows", "must be [num_rows, cols]");
        need(inv.t && inv.t->dim() == 2, "inv", "must be [T, topk]");
        const int64_t num = rows.t->size(0), cols = rows.t->size(1), T = inv.t->size(0), topk = inv.t->size(1);
        rows.is({BF16}, {num, cols});
        inv.is({I32}, {T, topk});
        if (weights.t) weights.is({F32}, {T, topk});
        out.make(true, BF16, {BF16}, {T, cols}, *rows.t);
        on_gpu(*rows.t, {&inv, &weights, &out.arg});
        const int32_t t = size32(T, "inv"), k = size32(topk, "inv"), c = size32(cols, "rows"), m = size32(num, "rows");
        void* s = stream_of(v[4]);
        const int st = call([&] { return g_combine(rows.ptr(), inv.ptr(), weights.ptr(), t, k, c, m, out.ptr(), s); });
        return st != 0 ? PyLong_FromLong(st) : out.result();
    });
}

// combine_rows_bwd(grad_out, inv, rows, weights, grad_rows, grad_weights, stream)
PyObject* py_combine_rows_bwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        Arg grad(v[0], "grad_out"), inv(v[1], "inv"), rows(v[2], "rows"), weights(v[3], "weights");
        Out grad_rows(v[4], "grad_rows"), grad_weights(v[5], "grad_weights");
        need(grad.t && grad.t->dim() == 2, "grad_out", "must be [T, cols]");
        need(inv.t && inv.t->dim() == 2, "inv", "must be [T, topk]");
        const int64_t T = grad.t->size(0), cols = grad.t->size(1), topk = inv.t->size(1);
        grad.is({BF16}, {T, cols});
        inv.is({I32}, {T, topk});
        if (weights.t) weights.is({F32}, {T, topk});
        const at::Tensor* sized = rows.t ? rows.t : grad_rows.arg.t;
        need(!sized || sized->dim() == 2, rows.t ? "rows" : "grad_rows", "must be [num_rows, cols]");
        const int64_t num = sized ? sized->size(0) : T * topk;
        if (rows.t) rows.is({BF16}, {num, cols});
        grad_rows.make(true, BF16, {BF16}, {num, cols}, *grad.t);
        grad_weights.make(rows.t != nullptr, F32, {F32}, {T, topk}, *grad.t);
        on_gpu(*grad.t, {&inv, &rows, &weights, &grad_rows.arg, &grad_weights.arg});
        const int32_t t = size32(T, "grad_out"), k = size32(topk, "inv"), c = size32(cols, "grad_out"),
                      m = size32(num, "grad_rows");
        void* s = stream_of(v[6]);
        const int st = call([&] {
            return g_combine_bwd(grad.ptr(), rows.ptr(), inv.ptr(), weights.ptr(), t, k, c, m, grad_rows.ptr(),
                                 grad_weights.ptr(), s);
        });
        if (st != 0) return PyLong_FromLong(st);
        return Py_BuildValue("(NN)", grad_rows.result(), grad_weights.result());
    });
}

// bind(rmsnorm, silu_mul, gemm_fp8, grouped_gemm, gemm_int8, quant_act_int8, silu_mul_int8, sort_rows,
// sort_scratch_bytes, combine_rows, combine_rows_bwd): addresses of the entry points
PyObject* py_bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        g_norm = reinterpret_cast<NormFn>(PyLong_AsVoidPtr(v[0]));
        g_act = reinterpret_cast<ActFn>(PyLong_AsVoidPtr(v[1]));
        g_dense = reinterpret_cast<DenseFn>(PyLong_AsVoidPtr(v[2]));
        g_grouped = reinterpret_cast<GroupedFn>(PyLong_AsVoidPtr(v[3]));
        g_dense_int8 = reinterpret_cast<DenseFn>(PyLong_AsVoidPtr(v[4]));
        g_quant_int8 = reinterpret_cast<QuantInt8Fn>(PyLong_AsVoidPtr(v[5]));
        g_act_int8 = reinterpret_cast<ActInt8Fn>(PyLong_AsVoidPtr(v[6]));
        g_sort = reinterpret_cast<SortFn>(PyLong_AsVoidPtr(v[7]));
        g_sort_bytes = reinterpret_cast<SortBytesFn>(PyLong_AsVoidPtr(v[8]));
        g_combine = reinterpret_cast<CombineFn>(PyLong_AsVoidPtr(v[9]));
        g_combine_bwd = reinterpret_cast<CombineBwdFn>(PyLong_AsVoidPtr(v[10]));
        Py_RETURN_NONE;
    });
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_bind)), METH_FASTCALL, nullptr},
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_rmsnorm)), METH_FASTCALL, nullptr},
    {"silu_mul", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_silu_mul)), METH_FASTCALL, nullptr},
    {"gemm_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_gemm_fp8)), METH_FASTCALL, nullptr},
    {"grouped_gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_grouped_gemm)), METH_FASTCALL, nullptr},
    {"gemm_int8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_gemm_int8)), METH_FASTCALL, nullptr},
    {"quant_act_int8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_quant_act_int8)), METH_FASTCALL,
     nullptr},
    {"silu_mul_int8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_silu_mul_int8)), METH_FASTCALL, nullptr},
    {"sort_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_sort_rows)), METH_FASTCALL, nullptr},
    {"combine_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_combine_rows)), METH_FASTCALL, nullptr},
    {"combine_rows_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_combine_rows_bwd)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
