// Native marshalling of the binding's small calls (tq.rmsnorm, tq.moe_*,
// tq.gemm_dense_i8): checks of the tensors and the C call, with no step of the
// computation.  Through ctypes such a call took 6 to 8 us on the host, more
// than its kernel on small inputs; here it takes 3 to 4, the launch itself.
//
// Every function takes the arguments of the C call in its order, with tensors
// (or addresses, or None) for arrays, and returns the status.  Of a tensor it
// checks what the C call cannot see: type, layout, length and device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/tq.h"

namespace {

// The library's functions (set by setup(), so that the one library that the
// binding has loaded is called) and torch's getters.
decltype(&tq_rmsnorm) p_rmsnorm;
decltype(&tq_moe_dispatch) p_dispatch;
decltype(&tq_moe_combine) p_combine;
decltype(&tq_moe_combine_grad) p_grad;
decltype(&tq_gemm_dense_i8) p_dense;
PyObject *get_device, *get_stream;

enum { KIND_I32 = 100, KIND_ANY = 101 };      // besides the values of tq_dtype

bool type_fits(at::ScalarType t, int64_t kind)
{
    switch (kind) {
    case TQ_F32: return t == at::kFloat;
    case TQ_BF16: return t == at::kBFloat16 || t == at::kShort || t == at::kUInt16;   // or the bits
    case TQ_I8: return t == at::kChar;
    case KIND_I32: return t == at::kInt;
    default: return true;                     // a type that the C call turns down
    }
}

const char* type_name(int64_t kind)
{
    return kind == TQ_F32    ? "torch.float32"
           : kind == TQ_BF16 ? "torch.bfloat16"
           : kind == TQ_I8   ? "torch.int8"
                             : "torch.int32";
}

// a * b elements; past 64 bits more than any tensor has.
int64_t count_of(int64_t a, int64_t b)
{
    int64_t v;
    return __builtin_mul_overflow(a, b, &v) ? INT64_MAX : v;
}

// One call's arguments, in order; `bad` once a Python error is set.
struct Call {
    PyObject* const* args;
    Py_ssize_t n, at = 0;
    bool bad = false;
    long device = -1;

    Call(PyObject* const* a, Py_ssize_t count, Py_ssize_t want) : args(a), n(count)
    {
        if (n != want) {
            PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, want);
            bad = true;
        }
    }
    int64_t integer()
    {
        if (bad) return 0;
        const long long v = PyLong_AsLongLong(args[at++]);
        if (v == -1 && PyErr_Occurred()) bad = true;
        return v;
    }
    int32_t integer32()
    {
        const int64_t v = integer();
        if (!bad && v != (int32_t)v) {
            PyErr_Format(PyExc_OverflowError, "%lld does not fit 32 bits", (long long)v);
            bad = true;
        }
        return (int32_t)v;
    }
    float real()
    {
        if (bad) return 0.0f;
        const double v = PyFloat_AsDouble(args[at++]);
        if (v == -1.0 && PyErr_Occurred()) bad = true;
        return (float)v;
    }
    bool present() const { return !bad && args[at] != Py_None; }
    long current_device()
    {
        if (device < 0) {
            PyObject* d = PyObject_CallNoArgs(get_device);
            device = d ? PyLong_AsLong(d) : -1;
            Py_XDECREF(d);
            if (device < 0) bad = true;
        }
        return device;
    }
    template <typename T = void>
    T* array(const char* name, int64_t kind, int64_t count)
    {
        if (bad) return nullptr;
        PyObject* o = args[at++];
        if (o == Py_None) return nullptr;
        if (PyLong_Check(o)) {
            void* p = PyLong_AsVoidPtr(o);
            bad = !p && PyErr_Occurred();
            return (T*)p;
        }
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s: a tensor, an address or None, not %s", name, Py_TYPE(o)->tp_name);
            bad = true;
            return nullptr;
        }
        const at::Tensor& t = THPVariable_Unpack(o);
        const bool is_gpu = t.is_cuda();
        if (type_fits(t.scalar_type(), kind) && t.is_contiguous() && t.numel() >= count && is_gpu &&
            t.get_device() == current_device())
            return bad ? nullptr : (T*)t.data_ptr();
        if (!bad) {
            if (!type_fits(t.scalar_type(), kind)) {
                PyObject* d = PyObject_GetAttrString(o, "dtype");
                if (d) PyErr_Format(PyExc_ValueError, "%s: %S, not %s", name, d, type_name(kind));
                Py_XDECREF(d);
            } else if (!t.is_contiguous()) {
                PyObject* s = PyObject_CallMethod(o, "stride", nullptr);
                if (s) PyErr_Format(PyExc_ValueError, "%s: not contiguous (strides %S)", name, s);
                Py_XDECREF(s);
            } else if (t.numel() < count) {
                PyErr_Format(PyExc_ValueError, "%s: %lld elements, needs %lld", name, (long long)t.numel(),
                             (long long)count);
            } else if (!is_gpu) {
                PyErr_Format(PyExc_ValueError, "%s: not a GPU tensor", name);
            } else {
                PyErr_Format(PyExc_ValueError, "%s: on device %d, the current one is %ld", name, (int)t.get_device(),
                             device);
            }
        }
        bad = true;
        return nullptr;
    }
    // None: torch's current stream; a number; or an object with `cuda_stream`
    void* stream()
    {
        if (bad) return nullptr;
        PyObject* o = args[at++];
        PyObject* v;
        if (o == Py_None) {
            const long d = current_device();
            PyObject* index = bad ? nullptr : PyLong_FromLong(d);
            v = index ? PyObject_CallOneArg(get_stream, index) : nullptr;
            Py_XDECREF(index);
        } else if (PyLong_Check(o)) {
            Py_INCREF(o);
            v = o;
        } else {
            v = PyObject_GetAttrString(o, "cuda_stream");
        }
        void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
        Py_XDECREF(v);
        if (PyErr_Occurred()) bad = true;
        return p;
    }
};

// `body(call)` with C++ exceptions as Python errors; the status as a number.
template <typename F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, F body)
{
    try {
        Call c(args, n, want);
        int status = 0;
        if (!c.bad) status = body(c);
        return c.bad ? nullptr : PyLong_FromLong(status);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// The C call without the interpreter's lock, if no argument was bad.
template <typename F>
int unlocked(const Call& c, F f)
{
    if (c.bad) return 0;
    int s;
    Py_BEGIN_ALLOW_THREADS
    s = f();
    Py_END_ALLOW_THREADS
    return s;
}

PyObject* rmsnorm(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(args, n, 13, [](Call& c) {
        const int64_t M = c.integer(), K = c.integer(), e = count_of(M, K);
        const int32_t xt = c.integer32();
        const void* x = c.array("x", xt, e);
        const int32_t rt = c.integer32();
        const void* res = c.array("residual", rt, e);
        void* out = c.array("residual_out", rt, e);
        const float* w = c.array<float>("weight", TQ_F32, K);
        const float eps = c.real();
        const int32_t yt = c.integer32();
        void* y = c.array("y", yt, e);
        float* s = c.array<float>("y_scale", TQ_F32, yt == TQ_I8 ? M : 0);
        void* st = c.stream();
        return unlocked(c, [=] { return (int)p_rmsnorm(M, K, xt, x, rt, res, out, w, eps, yt, y, s, st); });
    });
}

PyObject* dispatch(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(args, n, 16, [](Call& c) {
        const int64_t T = c.integer();
        const int32_t k = c.integer32(), E = c.integer32();
        const int64_t P = count_of(T, k);
        const int32_t* ids = c.array<int32_t>("experts", KIND_I32, P);
        int32_t* rows = c.array<int32_t>("rows", KIND_I32, P);
        int32_t* pairs = c.array<int32_t>("pairs", KIND_I32, P);
        int32_t* offsets = c.array<int32_t>("offsets", KIND_I32, (int64_t)E + 1);
        const int64_t H = c.integer();
        const int32_t xt = c.integer32();
        const bool scales = c.present() && xt == TQ_I8;
        const void* x = c.array("x", xt, count_of(T, H));
        const float* xsc = c.array<float>("x_scale", TQ_F32, scales ? T : 0);
        void* xs = c.array("xs", xt, count_of(P, H));
        float* xss = c.array<float>("xs_scale", TQ_F32, scales ? P : 0);
        const int64_t nws = c.integer();                   // before the workspace, whose length it is
        if (nws < 0 && !c.bad) {
            PyErr_Format(PyExc_ValueError, "workspace_bytes = %lld", (long long)nws);
            c.bad = true;
        }
        void* ws = c.array("workspace", KIND_ANY, nws);
        void* st = c.stream();
        return unlocked(c, [=] {
            return (int)p_dispatch(T, k, E, ids, rows, pairs, offsets, H, xt, x, xsc, xs, xss, ws, (size_t)nws, st);
        });
    });
}

PyObject* combine(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(args, n, 11, [](Call& c) {
        const int64_t T = c.integer();
        const int32_t k = c.integer32();
        const int64_t H = c.integer(), R = c.integer(), P = count_of(T, k);
        const int32_t* rows = c.array<int32_t>("rows", KIND_I32, P);
        const float* w = c.array<float>("weights", TQ_F32, P);
        const int32_t st_ = c.integer32();
        const void* ys = c.array("ys", st_, count_of(R, H));
        const int32_t yt = c.integer32();
        void* y = c.array("y", yt, count_of(T, H));
        void* st = c.stream();
        return unlocked(c, [=] { return (int)p_combine(T, k, H, R, rows, w, st_, ys, yt, y, st); });
    });
}

PyObject* combine_grad(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(args, n, 13, [=](Call& c) {
        const int64_t T = c.integer();
        const int32_t k = c.integer32();
        const int64_t H = c.integer(), R = c.integer(), P = count_of(T, k);
        const int32_t* rows = c.array<int32_t>("rows", KIND_I32, P);
        const float* w = c.array<float>("weights", TQ_F32, P);
        const int32_t dt = c.integer32();
        const void* dy = c.array("dy", dt, count_of(T, H));
        const int32_t st_ = c.integer32();
        const void* ys = c.array("ys", st_, args[11] != Py_None ? count_of(R, H) : 0);      // read for d_weights only
        void* dys = c.array("d_ys", st_, count_of(R, H));
        float* dw = c.array<float>("d_weights", TQ_F32, P);
        void* st = c.stream();
        return unlocked(c, [=] { return (int)p_grad(T, k, H, R, rows, w, dt, dy, st_, ys, dys, dw, st); });
    });
}

PyObject* gemm_dense_i8(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(args, n, 10, [](Call& c) {
        const int64_t M = c.integer(), N = c.integer(), K = c.integer();
        const int8_t* x = c.array<int8_t>("xq", TQ_I8, count_of(M, K));
        const float* xs = c.array<float>("x_scale", TQ_F32, M);
        const int8_t* w = c.array<int8_t>("w", TQ_I8, count_of(N, K));
        const float* ws = c.array<float>("w_scale", TQ_F32, N);
        const int32_t yt = c.integer32();
        void* y = c.array("y", yt, count_of(M, N));
        void* st = c.stream();
        return unlocked(c, [=] { return (int)p_dense(M, N, K, x, xs, w, ws, yt, y, st); });
    });
}

// setup(addresses of the five functions, torch's current-device and current-stream getters)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != 7) return PyErr_Format(PyExc_TypeError, "setup takes 7 arguments, got %zd", n);
    void* p[5];
    for (int i = 0; i < 5; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(args[i])))
            return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "function %d has no address", i);
    p_rmsnorm = (decltype(p_rmsnorm))p[0];
    p_dispatch = (decltype(p_dispatch))p[1];
    p_combine = (decltype(p_combine))p[2];
    p_grad = (decltype(p_grad))p[3];
    p_dense = (decltype(p_dense))p[4];
    for (int i = 0; i < 2; ++i) {
        Py_INCREF(args[5 + i]);
        (i ? get_stream : get_device) = args[5 + i];
    }
    Py_RETURN_NONE;
}

#define TQ_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TQ_METHOD(setup),        TQ_METHOD(rmsnorm),       TQ_METHOD(dispatch), TQ_METHOD(combine),
                         TQ_METHOD(combine_grad), TQ_METHOD(gemm_dense_i8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tqbind", "Native marshalling of small calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tqbind(void) { return PyModule_Create(&module); }
