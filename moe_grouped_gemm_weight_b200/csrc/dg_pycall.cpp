/*
 * dg_pycall.cpp -- argument marshalling for the calls that a decoding step
 * makes every few microseconds: CPython vector calls that take tensors and
 * numbers and call the C ABI of include/dg.h, and the check of a call's tensors
 * in one go.  Measured for 15 arguments with four tensors: 0.4 us, against 1.9
 * us through ctypes and 1.8 us of checks in Python.  The functions' addresses
 * are given by the Python side, which has loaded libdg.so; it is not linked
 * here.  Each returns the dg_status as an int.  The interpreter lock is released
 * during the call, as ctypes does.
 */
#define PY_SSIZE_T_CLEAN
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "dg.h"

static void *g_entry[15];

enum { ROUTE, ROUTE_BWD, LAYOUT, DISPATCH, COMBINE, COMBINE_BWD, SWIGLU, SWIGLU_BWD, RECAST,
       EPILOGUE, EPILOGUE_BWD, NORM, NORM_BWD, BALANCE, BALANCE_BWD };

/*
 * Argument i as a pointer (a tensor's data, None as null, or a number) or an
 * int; *bad is set where it is none.  Nothing is looked at once an error is
 * pending: the tensor test itself throws then.
 */
static void *ptr_at(PyObject *const *a, int i) {
    if (a[i] == Py_None || PyErr_Occurred()) return nullptr;
    if (PyLong_Check(a[i])) return PyLong_AsVoidPtr(a[i]);
    if (THPVariable_Check(a[i])) return THPVariable_Unpack(a[i]).data_ptr();
    PyErr_Format(PyExc_TypeError, "argument %d is neither a tensor nor an address", i);
    return nullptr;
}
static int int_at(PyObject *const *a, int i, int *bad) {
    int over = 0;
    if (PyErr_Occurred()) return 0;
    const long v = PyLong_AsLongAndOverflow(a[i], &over);
    if (over || v > 0x7FFFFFFFL || v < -0x7FFFFFFFL - 1) {
        *bad = 1;
        return 0;
    }
    return (int)v;
}

/* Converts to whatever pointer the header's prototype asks for. */
struct Ptr {
    void *p;
    template <typename T>
    operator T *() const {
        return static_cast<T *>(p);
    }
};

#define P(i) ptr_at(a, i)
#define I(i) int_at(a, i, &bad)

/* What torch throws becomes a Python error: no exception leaves an entry. */
#define NO_THROW_BEGIN try {
#define NO_THROW_END                                                                              \
    }                                                                                             \
    catch (python_error & e) {                                                                    \
        e.restore();                                                                              \
        return NULL;                                                                              \
    }                                                                                             \
    catch (const std::exception &e) {                                                             \
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());                     \
        return NULL;                                                                              \
    }

/* Defines a vector call of `count` arguments; `call` uses P(i), I(i) and `fn`. */
#define ENTRY(name, slot, count, call)                                                            \
    static PyObject *py_##name(PyObject *self, PyObject *const *a, Py_ssize_t n) {                     \
        int bad = 0;                                                                              \
        dg_status s;                                                                              \
        (void)self;                                                                               \
        if (n != (count)) return PyErr_Format(PyExc_TypeError, #name " takes %d arguments", count); \
        if (!g_entry[slot]) return PyErr_Format(PyExc_RuntimeError, #name " is not bound");       \
        NO_THROW_BEGIN                                                                            \
        call;                                                                                     \
        return PyLong_FromLong((long)s);                                                          \
        NO_THROW_END                                                                              \
    }
#define CHECKED                                                                                   \
    if (PyErr_Occurred()) return NULL;                                                            \
    if (bad) return PyErr_Format(PyExc_OverflowError, "a size or stride does not fit in 32 bits")
/* The function's type is the header's own, so a call that no longer fits it does not compile. */
#define RUN(name, slot, ...)                                                                      \
    do {                                                                                          \
        decltype(&name) fn = reinterpret_cast<decltype(&name)>(g_entry[slot]);                    \
        CHECKED;                                                                                  \
        Py_BEGIN_ALLOW_THREADS s = fn(__VA_ARGS__);                                               \
        Py_END_ALLOW_THREADS                                                                      \
    } while (0)

ENTRY(dg_route_topk, ROUTE, 15, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p4{P(4)}; Ptr st{P(14)};
    int dt = I(3); int T = I(5); int E = I(6); int k = I(7); int ng = I(8); int tg = I(9); int gt = I(10);
    int sc = I(11); int rn = I(12);
    float f = PyErr_Occurred() ? 0.f : (float)PyFloat_AsDouble(a[13]);
    RUN(dg_route_topk, ROUTE, p0, p1, p2, dt, p4, T, E, k, ng, tg, gt, sc, rn, f, st);
})
ENTRY(dg_route_topk_bwd, ROUTE_BWD, 12, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p4{P(4)}; Ptr st{P(11)};
    int dt = I(3); int T = I(5); int E = I(6); int k = I(7); int sc = I(8); int rn = I(9);
    float f = PyErr_Occurred() ? 0.f : (float)PyFloat_AsDouble(a[10]);
    RUN(dg_route_topk_bwd, ROUTE_BWD, p0, p1, p2, dt, p4, T, E, k, sc, rn, f, st);
})
ENTRY(dg_route_layout, LAYOUT, 12, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p3{P(3)}; Ptr p4{P(4)}; Ptr p5{P(5)};
    Ptr st{P(11)};
    int T = I(6); int k = I(7); int E = I(8); int rows = I(9); int mr = I(10);
    RUN(dg_route_layout, LAYOUT, p0, p1, p2, p3, p4, p5, T, k, E, rows, mr, st);
})
ENTRY(dg_dispatch_fp8_1x128, DISPATCH, 11, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p3{P(3)}; Ptr p4{P(4)}; Ptr st{P(10)};
    int str = I(2); int T = I(5); int k = I(6); int K = I(7); int rows = I(8); int gr = I(9);
    RUN(dg_dispatch_fp8_1x128, DISPATCH, p0, p1, str, p3, p4, T, k, K, rows, gr, st);
})
ENTRY(dg_combine, COMBINE, 9, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p3{P(3)}; Ptr st{P(8)};
    int T = I(4); int k = I(5); int N = I(6); int rows = I(7);
    RUN(dg_combine, COMBINE, p0, p1, p2, p3, T, k, N, rows, st);
})
ENTRY(dg_combine_bwd, COMBINE_BWD, 17, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p4{P(4)}; Ptr p5{P(5)}; Ptr p7{P(7)};
    Ptr p8{P(8)}; Ptr p9{P(9)}; Ptr p10{P(10)}; Ptr p11{P(11)}; Ptr st{P(16)};
    int rs = I(3); int cs = I(6); int T = I(12); int k = I(13); int N = I(14); int rows = I(15);
    RUN(dg_combine_bwd, COMBINE_BWD, p0, p1, p2, rs, p4, p5, cs, p7, p8, p9, p10, p11, T, k, N, rows, st);
})
ENTRY(dg_swiglu_fp8, SWIGLU, 12, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p3{P(3)}; Ptr p4{P(4)}; Ptr p6{P(6)}; Ptr p7{P(7)};
    Ptr st{P(11)};
    int sa = I(2); int cs = I(5); int rows = I(8); int F = I(9); int gr = I(10);
    RUN(dg_swiglu_fp8, SWIGLU, p0, p1, sa, p3, p4, cs, p6, p7, rows, F, gr, st);
})
ENTRY(dg_swiglu_fp8_bwd, SWIGLU_BWD, 16, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p3{P(3)}; Ptr p4{P(4)}; Ptr p6{P(6)}; Ptr p7{P(7)};
    Ptr p8{P(8)}; Ptr p9{P(9)}; Ptr p10{P(10)}; Ptr p12{P(12)}; Ptr st{P(15)};
    int rs = I(2); int cs = I(5); int ks = I(11); int rows = I(13); int F = I(14);
    RUN(dg_swiglu_fp8_bwd, SWIGLU_BWD, p0, p1, rs, p3, p4, cs, p6, p7, p8, p9, p10, ks, p12, rows, F, st);
})
ENTRY(dg_fp8_1x128_to_128x128, RECAST, 9, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p3{P(3)}; Ptr p5{P(5)}; Ptr st{P(8)};
    int sa = I(4); int rows = I(6); int K = I(7);
    RUN(dg_fp8_1x128_to_128x128, RECAST, p0, p1, p2, p3, sa, p5, rows, K, st);
})

ENTRY(dg_fp8_gemm_nt_epilogue, EPILOGUE, 17, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p3{P(3)}; Ptr p5{P(5)}; Ptr p6{P(6)};
    Ptr p8{P(8)}; Ptr p9{P(9)}; Ptr p10{P(10)}; Ptr p12{P(12)}; Ptr st{P(16)};
    int qs = I(4); int as = I(7); int act = I(11); int M = I(13); int N = I(14); int K = I(15);
    RUN(dg_fp8_gemm_nt_epilogue, EPILOGUE, p0, p1, p2, p3, qs, p5, p6, as, p8, p9, p10, act, p12, M, N, K, st);
})
ENTRY(dg_epilogue_bwd, EPILOGUE_BWD, 14, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p3{P(3)}; Ptr p4{P(4)}; Ptr p6{P(6)}; Ptr p7{P(7)};
    Ptr p8{P(8)}; Ptr p9{P(9)}; Ptr st{P(13)};
    int rs = I(2); int cs = I(5); int act = I(10); int M = I(11); int N = I(12);
    RUN(dg_epilogue_bwd, EPILOGUE_BWD, p0, p1, rs, p3, p4, cs, p6, p7, p8, p9, act, M, N, st);
})
ENTRY(dg_norm_residual, NORM, 18, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p3{P(3)}; Ptr p5{P(5)}; Ptr p6{P(6)};
    Ptr p8{P(8)}; Ptr p9{P(9)}; Ptr p10{P(10)}; Ptr p11{P(11)}; Ptr st{P(17)};
    int qs = I(4); int dt = I(7); int T = I(12); int N = I(13); int pn = I(14);
    float scale = PyErr_Occurred() ? 0.f : (float)PyFloat_AsDouble(a[15]);
    float eps = PyErr_Occurred() ? 0.f : (float)PyFloat_AsDouble(a[16]);
    RUN(dg_norm_residual, NORM, p0, p1, p2, p3, qs, p5, p6, dt, p8, p9, p10, p11, T, N, pn, scale, eps, st);
})
ENTRY(dg_norm_residual_bwd, NORM_BWD, 20, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p3{P(3)}; Ptr p4{P(4)}; Ptr p5{P(5)};
    Ptr p6{P(6)}; Ptr p7{P(7)}; Ptr p8{P(8)}; Ptr p10{P(10)}; Ptr p11{P(11)}; Ptr p12{P(12)};
    Ptr p13{P(13)}; Ptr p14{P(14)};
    int dt = I(9); int T = I(15); int N = I(16); int pn = I(17);
    float scale = PyErr_Occurred() ? 0.f : (float)PyFloat_AsDouble(a[18]);
    Ptr st{P(19)};
    RUN(dg_norm_residual_bwd, NORM_BWD, p0, p1, p2, p3, p4, p5, p6, p7, p8, dt, p10, p11, p12, p13, p14, T, N, pn,
        scale, st);
})
ENTRY(dg_balance_loss, BALANCE, 15, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p3{P(3)}; Ptr p4{P(4)}; Ptr p6{P(6)};
    Ptr p7{P(7)}; Ptr st{P(14)};
    int dt = I(5); int T = I(8); int E = I(9); int k = I(10); int S = I(11); int sc = I(12);
    float coef = PyErr_Occurred() ? 0.f : (float)PyFloat_AsDouble(a[13]);
    RUN(dg_balance_loss, BALANCE, p0, p1, p2, p3, p4, dt, p6, p7, T, E, k, S, sc, coef, st);
})
ENTRY(dg_balance_loss_bwd, BALANCE_BWD, 14, {
    Ptr p0{P(0)}; Ptr p1{P(1)}; Ptr p2{P(2)}; Ptr p3{P(3)}; Ptr p5{P(5)}; Ptr p6{P(6)};
    Ptr st{P(13)};
    int dt = I(4); int T = I(7); int E = I(8); int k = I(9); int S = I(10); int sc = I(11);
    float coef = PyErr_Occurred() ? 0.f : (float)PyFloat_AsDouble(a[12]);
    RUN(dg_balance_loss_bwd, BALANCE_BWD, p0, p1, p2, p3, dt, p5, p6, T, E, k, S, sc, coef, st);
})

static const char *const kNames[15] = {"dg_route_topk", "dg_route_topk_bwd", "dg_route_layout", "dg_dispatch_fp8_1x128",
                                      "dg_combine", "dg_combine_bwd", "dg_swiglu_fp8", "dg_swiglu_fp8_bwd",
                                      "dg_fp8_1x128_to_128x128", "dg_fp8_gemm_nt_epilogue", "dg_epilogue_bwd",
                                      "dg_norm_residual",
                                      "dg_norm_residual_bwd", "dg_balance_loss", "dg_balance_loss_bwd"};

/*
 * fits(tensor, kind, need, ...): the current CUDA device's index if every
 * tensor (None: absent) has the kind's elements, is dense and contiguous, holds
 * `need` of them and lies on that device, else -1.  Kinds: 1 any one-byte
 * elements, 2 bfloat16, 4 float32, 5 int32.
 */
static PyObject *fits(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n < 3 || n % 3 != 0) return PyErr_Format(PyExc_TypeError, "fits takes triples");
    NO_THROW_BEGIN
    long device = -1;
    for (Py_ssize_t i = 0; i < n; i += 3) {
        if (a[i] == Py_None) continue;
        if (!THPVariable_Check(a[i])) return PyLong_FromLong(-1);
        const at::Tensor &t = THPVariable_Unpack(a[i]);
        const long kind = PyLong_AsLong(a[i + 1]);
        const long long need = PyErr_Occurred() ? 0 : PyLong_AsLongLong(a[i + 2]);
        if (PyErr_Occurred()) return NULL;
        if (t.layout() != at::kStrided) return PyLong_FromLong(-1);
        const at::ScalarType type = t.scalar_type();
        const bool right = kind == 1   ? t.element_size() == 1
                           : kind == 2 ? type == at::kBFloat16
                           : kind == 4 ? type == at::kFloat
                                       : type == at::kInt;
        if (!right || t.numel() < need || !t.is_contiguous() || !t.is_cuda()) return PyLong_FromLong(-1);
        if (device < 0) device = c10::impl::VirtualGuardImpl(at::kCUDA).getDevice().index();
        if (t.get_device() != device) return PyLong_FromLong(-1);
    }
    return PyLong_FromLong(device);
    NO_THROW_END
}

/* bind(name, address): the C ABI function behind a call. */
static PyObject *bind(PyObject *self, PyObject *args) {
    const char *name;
    PyObject *address;
    int i;
    (void)self;
    if (!PyArg_ParseTuple(args, "sO", &name, &address)) return NULL;
    for (i = 0; i < 15; ++i)
        if (strcmp(name, kNames[i]) == 0) {
            g_entry[i] = PyLong_AsVoidPtr(address);
            if (PyErr_Occurred()) return NULL;
            Py_RETURN_NONE;
        }
    return PyErr_Format(PyExc_KeyError, "no call named %s", name);
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))py_##f, METH_FASTCALL, NULL}
static PyMethodDef kMethods[] = {
    FAST(dg_route_topk), FAST(dg_route_topk_bwd), FAST(dg_route_layout), FAST(dg_dispatch_fp8_1x128),
    FAST(dg_combine), FAST(dg_combine_bwd), FAST(dg_swiglu_fp8), FAST(dg_swiglu_fp8_bwd),
    FAST(dg_fp8_1x128_to_128x128), FAST(dg_fp8_gemm_nt_epilogue), FAST(dg_epilogue_bwd), FAST(dg_norm_residual), FAST(dg_norm_residual_bwd),
    FAST(dg_balance_loss), FAST(dg_balance_loss_bwd),
    {"fits", (PyCFunction)(void (*)(void))fits, METH_FASTCALL, NULL}, {"bind", bind, METH_VARARGS, NULL}, {NULL, NULL, 0, NULL}};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_dgcall", "Argument marshalling for libdg.so", -1,
                                     kMethods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__dgcall(void) { return PyModule_Create(&kModule); }
