// sfar_tensors.cpp -- the Python calls of include/sfar_kv.h and sfar_fp8.h:
// checks torch tensors, takes their pointers, sizes and strides, and makes the
// C call on the stream.
//
// A call has up to ten tensors, or a pointer for each rank; read through
// Python attributes and marshalled by ctypes they cost 9 to 12 us a call,
// above the GPU time of a decode step's kernels.  Here a call costs 2.7 to 2.9,
// most of it the launch.
//
// The C functions come in by address (bind), so that this module is linked
// with torch alone.  Every function returns the call's status; wrong tensors
// are a ValueError.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "sfar_fp8.h"
#include "sfar_kv.h"

namespace {

constexpr int kMostRanks = 16;

decltype(&sfar_kv_plan) c_plan;
decltype(&sfar_kv_append) c_append;
decltype(&sfar_kv_attention) c_attention;
decltype(&sfar_quantize_fp8) c_quantize;
decltype(&sfar_rowpar_gemm_fp8) c_gemm;

struct PythonError {};                  // an exception is set already

[[noreturn]] void wrong(const std::string &what) { throw std::invalid_argument(what); }

const at::Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o))
        wrong(std::string(what) + ": need a tensor");
    return THPVariable_Unpack(o);
}

enum Type { kBf16, kF32, kByte };
bool is(at::ScalarType t, Type want)
{
    switch (want) {
    case kBf16: return t == at::kBFloat16;
    case kF32: return t == at::kFloat;
    default: return t == at::kFloat8_e4m3fn || t == at::kByte;
    }
}
const char *name(Type t) { return t == kBf16 ? "bfloat16" : t == kF32 ? "float32" : "float8_e4m3fn or uint8"; }

// R tensors of one form: a list or tuple of them, or one tensor [R, ...] whose
// slices they are.  Strides of dimensions of one entry are 0, whatever torch
// keeps there.
struct Ranks {
    void *ptr[kMostRanks] = {};
    int64_t shape[4] = {}, stride[4] = {};
    bool dense = true;

    Ranks(PyObject *x, int R, int ndim, Type type, const char *what)
    {
        if (R < 1 || R > kMostRanks)
            wrong(std::string(what) + ": need 1 to 16 ranks");
        const bool list = PyList_Check(x), tuple = PyTuple_Check(x);
        if (list || tuple) {
            const Py_ssize_t n = list ? PyList_GET_SIZE(x) : PyTuple_GET_SIZE(x);
            if (n != R)
                wrong(std::string(what) + ": need " + std::to_string(R) + " tensors, one per rank");
            auto at = [&](int i) -> const at::Tensor & { return tensor(list ? PyList_GET_ITEM(x, i) : PyTuple_GET_ITEM(x, i), what); };
            const at::Tensor &t = at(0);
            for (int i = 0; i < R; ++i) {
                const at::Tensor &o = at(i);
                if (i && (o.sizes() != t.sizes() || o.strides() != t.strides() || o.scalar_type() != t.scalar_type()))
                    wrong(std::string(what) + ": the ranks' tensors differ in shape, strides or type");
                if (!o.is_cuda())
                    wrong(std::string(what) + ": must be on the GPU");
                ptr[i] = o.data_ptr();
            }
            form(t, 0, ndim, type, what);
            return;
        }
        const at::Tensor &t = tensor(x, what);
        if (t.dim() == 0 || t.size(0) != R)
            wrong(std::string(what) + ": need [" + std::to_string(R) + ", ...], a slice per rank");
        form(t, 1, ndim, type, what);
        char *base = static_cast<char *>(t.data_ptr());
        const int64_t step = t.stride(0) * (int64_t)t.element_size();
        for (int i = 0; i < R; ++i)
            ptr[i] = base + i * step;
    }
    bool same(std::initializer_list<int64_t> want) const { return std::equal(want.begin(), want.end(), shape); }

  private:
    void form(const at::Tensor &t, int skip, int ndim, Type type, const char *what)
    {
        if (t.dim() != ndim + skip || !is(t.scalar_type(), type))
            wrong(std::string(what) + ": need " + std::to_string(ndim) + " dimensions of " + name(type) + " per rank");
        if (!t.is_cuda())
            wrong(std::string(what) + ": must be on the GPU");
        int64_t n = 1;
        for (int i = ndim - 1; i >= 0; --i) {
            shape[i] = t.size(i + skip);
            stride[i] = shape[i] > 1 ? t.stride(i + skip) : 0;
            dense = dense && (shape[i] <= 1 || stride[i] == n);
            n *= shape[i];
        }
        if (shape[ndim - 1] > 1 && stride[ndim - 1] != 1)
            wrong(std::string(what) + ": the last dimension must be contiguous");
    }
};

// a contiguous int32 tensor of this shape
int32_t *ints(PyObject *x, std::initializer_list<int64_t> shape, const char *what)
{
    const at::Tensor &t = tensor(x, what);
    if (t.scalar_type() != at::kInt || t.sizes() != at::IntArrayRef(shape.begin(), shape.size()) || !t.is_contiguous() || !t.is_cuda()) {
        std::string s;
        for (int64_t n : shape)
            s += (s.empty() ? "" : ", ") + std::to_string(n);
        wrong(std::string(what) + ": need a contiguous int32 tensor of shape [" + s + "] on the GPU");
    }
    return static_cast<int32_t *>(t.data_ptr());
}
int64_t size(PyObject *x, int dims, int dim, const char *what)
{
    const at::Tensor &t = tensor(x, what);
    if (t.dim() != dims)
        wrong(std::string(what) + ": need " + std::to_string(dims) + " dimensions");
    return t.size(dim);
}

// None: torch's current stream
sfar_stream_t stream_of(PyObject *s)
{
    if (s == Py_None)
        return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *n = PyNumber_Long(s);
    void *p = n ? PyLong_AsVoidPtr(n) : nullptr;
    Py_XDECREF(n);
    if (PyErr_Occurred())
        throw PythonError();
    return static_cast<sfar_stream_t>(p);
}
void *handle_of(PyObject *h)
{
    if (h == Py_None)
        return nullptr;                 // closed: refused by the call
    void *p = PyLong_AsVoidPtr(h);
    if (PyErr_Occurred())
        throw PythonError();
    return p;
}
long long number(PyObject *x)
{
    PyObject *n = PyNumber_Index(x);
    const long long v = n ? PyLong_AsLongLong(n) : -1;
    Py_XDECREF(n);
    if (PyErr_Occurred())
        throw PythonError();
    return v;
}
size_t natural(PyObject *x, const char *what)
{
    const long long v = number(x);
    if (v < 0)
        wrong(std::string(what) + ": must not be negative");
    return (size_t)v;
}

template <class F> PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F body)
{
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "need %zd arguments", want);
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)body());
    } catch (const PythonError &) {
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
template <class F> sfar_status released(F call)
{
    sfar_status r;
    Py_BEGIN_ALLOW_THREADS
    r = call();
    Py_END_ALLOW_THREADS
    return r;
}

// (handle, pages, lens, delta, table, ring, state, lens_out, state_out, starts, slots, taken, stream)
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&] {
        const auto h = static_cast<sfar_kv_t *>(handle_of(a[0]));
        const int64_t pages = number(a[1]), B = size(a[2], 1, 0, "lens"), W = size(a[4], 2, 1, "table"), T = size(a[10], 1, 0, "slots");
        int32_t *lens = ints(a[2], {B}, "lens"), *delta = ints(a[3], {B}, "delta"), *table = ints(a[4], {B, W}, "table"),
                *ring = ints(a[5], {pages}, "ring"), *state = ints(a[6], {2}, "state"), *lens_out = ints(a[7], {B}, "lens_out"),
                *state_out = ints(a[8], {2}, "state_out"), *starts = ints(a[9], {B + 1}, "starts"), *slots = ints(a[10], {T}, "slots"),
                *taken = ints(a[11], {B}, "taken");
        const sfar_stream_t s = stream_of(a[12]);
        return released([&] { return c_plan(h, lens, delta, table, ring, state, lens_out, state_out, starts, slots, taken, B, W, T, s); });
    });
}

// (handle, R, kv_heads, head_dim, k, v, slots, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const auto h = static_cast<sfar_kv_t *>(handle_of(a[0]));
        const int R = (int)number(a[1]);
        const int64_t H = number(a[2]), D = number(a[3]), T = size(a[6], 1, 0, "slots");
        const Ranks k(a[4], R, 3, kBf16, "k"), v(a[5], R, 3, kBf16, "v");
        if (!k.same({T, H, D}) || !v.same({T, H, D}))
            wrong("append: need k and v of shape [" + std::to_string(T) + ", " + std::to_string(H) + ", " + std::to_string(D) + "] per rank");
        const int32_t *slots = ints(a[6], {T}, "slots");
        const sfar_stream_t s = stream_of(a[7]);
        return released([&] { return c_append(h, k.ptr, v.ptr, slots, T, k.stride[0], k.stride[1], v.stride[0], v.stride[1], s); });
    });
}

// (handle, R, q_heads, head_dim, q, out, table, lens, starts, max_q, scale, window, stream)
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&] {
        const auto h = static_cast<sfar_kv_t *>(handle_of(a[0]));
        const int R = (int)number(a[1]);
        const int64_t H = number(a[2]), D = number(a[3]);
        const size_t max_q = natural(a[9], "max_q"), window = natural(a[11], "window");
        const Ranks q(a[4], R, 3, kBf16, "q"), out(a[5], R, 3, kBf16, "out");
        const int64_t T = q.shape[0];
        if (!q.same({T, H, D}) || !out.same({T, H, D}))
            wrong("attention: need q and out of shape [tokens, " + std::to_string(H) + ", " + std::to_string(D) + "] per rank");
        const int64_t B = size(a[6], 2, 0, "table"), W = size(a[6], 2, 1, "table");
        const int32_t *table = ints(a[6], {B, W}, "table"), *lens = ints(a[7], {B}, "lens"), *starts = ints(a[8], {B + 1}, "starts");
        const double scale = PyFloat_AsDouble(a[10]);
        if (PyErr_Occurred())
            throw PythonError();
        const sfar_stream_t s = stream_of(a[12]);
        return released([&] {
            return c_attention(h, q.ptr, const_cast<void *const *>(out.ptr), table, lens, starts, B, W, T, q.stride[0], q.stride[1],
                               out.stride[0], out.stride[1], max_q, (float)scale, window, s);
        });
    });
}

// The row stride of a matrix of rows of k.  A single row has none, and gets one that every call takes; that of an expanded
// matrix, 0, is passed on and refused.
size_t row_stride(const Ranks &x) { return x.shape[0] == 1 ? (size_t)(x.shape[1] + 15) / 16 * 16 : (size_t)x.stride[0]; }

// (handle, R, x, x8, sx, stream)
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        const auto h = static_cast<sfar_t *>(handle_of(a[0]));
        const int R = (int)number(a[1]);
        const Ranks x(a[2], R, 2, kBf16, "x"), x8(a[3], R, 2, kByte, "x8"), sx(a[4], R, 2, kF32, "sx");
        const int64_t m = x.shape[0], k = x.shape[1];
        if (!x8.same({m, k}) || !sx.same({(k + 127) / 128, m}) || !sx.dense)
            wrong("quantize_fp8: x8 must be [m, k], sx a contiguous [ceil(k / 128), m]");
        const sfar_stream_t s = stream_of(a[5]);
        return released([&] {
            return c_quantize(h, x.ptr, const_cast<void *const *>(x8.ptr), reinterpret_cast<float *const *>(sx.ptr), m, k,
                              row_stride(x), row_stride(x8), s);
        });
    });
}

// (handle, R, x8, sx, w8, sw, y, stream)
PyObject *gemm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&] {
        const auto h = static_cast<sfar_t *>(handle_of(a[0]));
        const int R = (int)number(a[1]);
        const Ranks x8(a[2], R, 2, kByte, "x8"), sx(a[3], R, 2, kF32, "sx"), w8(a[4], R, 2, kByte, "w8"), sw(a[5], R, 2, kF32, "sw"),
            y(a[6], R, 2, kBf16, "y");
        const int64_t m = x8.shape[0], k = x8.shape[1], N = w8.shape[0], kb = (k + 127) / 128;
        if (w8.shape[1] != k || !y.same({m, N}) || !sx.same({kb, m}) || !sw.same({(N + 127) / 128, kb}) || !(y.dense && sx.dense && sw.dense))
            wrong("rowpar_gemm_fp8: need x8 [m, k], w8 [hidden, k], contiguous sx [ceil(k / 128), m], sw [ceil(hidden / 128), "
                  "ceil(k / 128)] and y [m, hidden]");
        const sfar_stream_t s = stream_of(a[7]);
        return released([&] {
            return c_gemm(h, x8.ptr, reinterpret_cast<const float *const *>(sx.ptr), w8.ptr, reinterpret_cast<const float *const *>(sw.ptr),
                          const_cast<void *const *>(y.ptr), m, k, N, row_stride(x8), row_stride(w8), s);
        });
    });
}

// (tensors, R, dimensions, "bf16" | "fp32" | "byte", what) -> (pointers, shape, contiguous)
PyObject *ranks(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    PyObject *result = nullptr;
    PyObject *status = guarded(n, 5, [&] {
        const int R = (int)number(a[1]), ndim = (int)number(a[2]);
        const char *type = PyUnicode_AsUTF8(a[3]), *what = PyUnicode_AsUTF8(a[4]);
        if (!type || !what)
            throw PythonError();
        if (ndim < 1 || ndim > 4)
            wrong("need 1 to 4 dimensions");
        const Ranks x(a[0], R, ndim, type[1] == 'f' ? kBf16 : type[0] == 'f' ? kF32 : kByte, what);
        PyObject *p = PyTuple_New(R), *s = PyTuple_New(ndim);
        for (int i = 0; p && i < R; ++i)
            PyTuple_SET_ITEM(p, i, PyLong_FromVoidPtr(x.ptr[i]));
        for (int i = 0; s && i < ndim; ++i)
            PyTuple_SET_ITEM(s, i, PyLong_FromLongLong(x.shape[i]));
        result = p && s ? Py_BuildValue("(NNO)", p, s, x.dense ? Py_True : Py_False) : nullptr;
        if (!result)
            throw PythonError();
        return 0;
    });
    if (!status)
        return nullptr;
    Py_DECREF(status);
    return result;
}

// the addresses of the five C functions
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 5, [&] {
        c_plan = reinterpret_cast<decltype(c_plan)>(handle_of(a[0]));
        c_append = reinterpret_cast<decltype(c_append)>(handle_of(a[1]));
        c_attention = reinterpret_cast<decltype(c_attention)>(handle_of(a[2]));
        c_quantize = reinterpret_cast<decltype(c_quantize)>(handle_of(a[3]));
        c_gemm = reinterpret_cast<decltype(c_gemm)>(handle_of(a[4]));
        return 0;
    });
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"ranks", fast(ranks), METH_FASTCALL, nullptr},
                         {"plan", fast(plan), METH_FASTCALL, nullptr},
                         {"append", fast(append), METH_FASTCALL, nullptr},
                         {"attention", fast(attention), METH_FASTCALL, nullptr},
                         {"quantize_fp8", fast(quantize), METH_FASTCALL, nullptr},
                         {"rowpar_gemm_fp8", fast(gemm), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "sfar_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit_sfar_tensors() { return PyModule_Create(&module); }
