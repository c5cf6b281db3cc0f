// binding.cpp -- the operators that a decode step calls, from Python.  Such a step is
// 4 to 12 us on the device, and reading the ten tensors' types, shapes and layouts
// through Python attributes and ctypes took 9 us a call before the library's own 4.
// Read here, a pass of norm_gate_residual over one token, outputs allocated, is 18 us
// instead of 28, and lora_apply's 9 instead of 20; the call itself takes 3.
// Each function checks its tensors and calls the C ABI; it returns the library's status, or
// -1 when a tensor is not what the entry point takes: the Python wrapper then says which
// one and why.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "gemmar.h"

namespace {

decltype(&norm_gate_residual) p_norm = nullptr;
decltype(&norm_gate_residual_bwd) p_norm_bwd = nullptr;
decltype(&lora_apply) p_lora = nullptr;
decltype(&lora_apply_bwd) p_lora_bwd = nullptr;
decltype(&gemm_blockscale_act) p_act = nullptr;
decltype(&gemm_blockscale_act_bwd) p_act_bwd = nullptr;
decltype(&moe_route) p_route = nullptr;
decltype(&moe_apply) p_moe = nullptr;

constexpr at::ScalarType kF32 = at::ScalarType::Float, kBf16 = at::ScalarType::BFloat16, kI32 = at::ScalarType::Int,
                         kU8 = at::ScalarType::Byte, kE4m3 = at::ScalarType::Float8_e4m3fn;

// The arguments of one call, read in order; `ok` turns false at the first tensor that does not fit.
struct Args {
    PyObject *const *at;
    bool ok = true;

    const at::Tensor *tensor(PyObject *o)
    {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    void *pointer(PyObject *o) { return o == Py_None ? nullptr : PyLong_AsVoidPtr(o); }
    int whole(PyObject *o)
    {
        const long v = PyLong_AsLong(o);
        ok = ok && v >= INT32_MIN && v <= INT32_MAX;
        return (int)v;
    }
    bool truth(PyObject *o) { return PyObject_IsTrue(o) > 0; }
    float real(PyObject *o)
    {
        const double v = PyFloat_AsDouble(o);
        return (float)v;
    }
    // [rows, cols] with contiguous rows; the stride in elements
    template <typename T>
    T *rows(PyObject *o, int64_t R, int64_t C, at::ScalarType type, int64_t &stride)
    {
        const at::Tensor *t = tensor(o);
        if (!t || t->dim() != 2 || t->size(0) != R || t->size(1) != C || t->scalar_type() != type || !t->is_cuda() ||
            (t->stride(1) != 1 && C != 1)) {
            ok = false;
            return nullptr;
        }
        stride = R > 1 ? t->stride(0) : C;
        return static_cast<T *>(t->data_ptr());
    }
    // contiguous of that shape, or None
    template <typename T>
    T *dense(PyObject *o, at::IntArrayRef shape, at::ScalarType type, at::ScalarType other = at::ScalarType::Undefined)
    {
        if (o == Py_None)
            return nullptr;
        const at::Tensor *t = tensor(o);
        if (!t || t->sizes() != shape || (t->scalar_type() != type && t->scalar_type() != other) || !t->is_cuda() ||
            !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return static_cast<T *>(t->data_ptr());
    }
    // bf16 or fp32
    at::ScalarType real_type(PyObject *o)
    {
        const at::Tensor *t = tensor(o);
        const at::ScalarType s = t ? t->scalar_type() : kF32;
        ok = ok && t && (s == kF32 || s == kBf16);
        return s;
    }
    bool shape2(PyObject *o, int64_t &a, int64_t &b)
    {
        const at::Tensor *t = tensor(o);
        ok = ok && t && t->dim() == 2;
        if (ok) {
            a = t->size(0);
            b = t->size(1);
        }
        return ok;
    }
    // a gate: None, [N] (stride 0) or [M, N]
    const uint16_t *gate(PyObject *o, int64_t M, int64_t N, int64_t &stride)
    {
        stride = 0;
        if (o == Py_None)
            return nullptr;
        const at::Tensor *t = tensor(o);
        if (t && t->dim() == 1)
            return dense<uint16_t>(o, {N}, kBf16);
        const uint16_t *p = rows<uint16_t>(o, M, N, kBf16, stride);
        ok = ok && stride != 0;
        return p;
    }
};

int code(at::ScalarType s) { return s == kBf16 ? GEMMAR_DTYPE_BF16 : GEMMAR_DTYPE_F32; }

PyObject *refused() { return PyErr_Occurred() ? nullptr : PyLong_FromLong(-1); }

// A launch may wait for room in the stream's queue: without the interpreter's lock.
template <typename F>
PyObject *status(F call)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

bool count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want)
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    return n == want;
}

// handle, y, h, w_pre, t, w_post, gate, alpha, beta, eps, u, q, scales, rstd, stream
PyObject *norm(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count(n, 15))
        return nullptr;
    Args a{v};
    int64_t M = 0, N = 0, ys = 0, hs = 0, gs = 0;
    if (!a.shape2(v[1], M, N))
        return refused();
    const at::ScalarType yt = a.real_type(v[1]), ht = a.real_type(v[2]);
    void *y = a.rows<void>(v[1], M, N, yt, ys), *h = a.rows<void>(v[2], M, N, ht, hs);
    const float *w_pre = a.dense<float>(v[3], {N}, kF32), *w_post = a.dense<float>(v[5], {N}, kF32);
    void *t = a.dense<void>(v[4], {M, N}, ht);
    const uint16_t *gate = a.gate(v[6], M, N, gs);
    uint16_t *u = a.dense<uint16_t>(v[10], {M, N}, kBf16);
    uint8_t *q = a.dense<uint8_t>(v[11], {M, N}, kU8, kE4m3);
    float *scales = a.dense<float>(v[12], {M, N / 128}, kF32), *rstd = a.dense<float>(v[13], {M, 2}, kF32);
    const float alpha = a.real(v[7]), beta = a.real(v[8]), eps = a.real(v[9]);
    void *ctx = a.pointer(v[0]), *stream = a.pointer(v[14]);
    if (!a.ok || PyErr_Occurred())
        return refused();
    return status([&] {
        return p_norm(static_cast<gemmar_ctx *>(ctx), y, code(yt), ys, h, code(ht), hs, w_post, w_pre, gate, gs, alpha,
                      beta, eps, M, N, t, u, q, scales, rstd, stream);
    });
}

// handle, y, h, rstd, dt, dy, dh, w_post, w_pre, gate, alpha, beta, du, dw_post, dw_pre, dgate, stream
PyObject *norm_bwd(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count(n, 17))
        return nullptr;
    Args a{v};
    int64_t M = 0, N = 0, ys = 0, hs = 0, gs = 0, ts = 0, us = 0;
    if (!a.shape2(v[1], M, N))
        return refused();
    const at::ScalarType yt = a.real_type(v[1]), ht = a.real_type(v[2]);
    void *y = a.rows<void>(v[1], M, N, yt, ys), *h = a.rows<void>(v[2], M, N, ht, hs);
    const float *rstd = a.dense<float>(v[3], {M, 2}, kF32);
    const void *dt = v[4] == Py_None ? nullptr : a.rows<void>(v[4], M, N, ht, ts);
    void *dy = a.dense<void>(v[5], {M, N}, yt), *dh = a.dense<void>(v[6], {M, N}, ht);
    const float *w_post = a.dense<float>(v[7], {N}, kF32), *w_pre = a.dense<float>(v[8], {N}, kF32);
    const uint16_t *gate = a.gate(v[9], M, N, gs);
    const uint16_t *du = v[12] == Py_None ? nullptr : a.rows<uint16_t>(v[12], M, N, kBf16, us);
    float *dw_post = a.dense<float>(v[13], {N}, kF32), *dw_pre = a.dense<float>(v[14], {N}, kF32);
    void *dgate = gs == 0 ? a.dense<void>(v[15], {N}, kF32) : a.dense<void>(v[15], {M, N}, kBf16);
    const float alpha = a.real(v[10]), beta = a.real(v[11]);
    void *ctx = a.pointer(v[0]), *stream = a.pointer(v[16]);
    if (!a.ok || PyErr_Occurred())
        return refused();
    return status([&] {
        return p_norm_bwd(static_cast<gemmar_ctx *>(ctx), y, code(yt), ys, h, code(ht), hs, rstd, w_post, w_pre, gate,
                          gs, alpha, beta, M, N, dt, ts, du, us, dy, dh, dw_post, dw_pre, dgate, stream);
    });
}

// What both adapter calls begin with: x, order, offsets, A, B, scales, ranks.
struct Adapters {
    int64_t T = 0, K = 0, N = 0, R = 0, r = 0, xs = 0;
    const uint16_t *x = nullptr, *A = nullptr, *B = nullptr;
    const int32_t *order = nullptr, *offsets = nullptr, *ranks = nullptr;
    const float *scales = nullptr;

    bool read(Args &a, PyObject *const *v)
    {
        const at::Tensor *tA = a.tensor(v[3]), *tB = a.tensor(v[4]);
        if (!a.shape2(v[0], T, K) || !tA || !tB || tA->dim() != 3 || tB->dim() != 3)
            return a.ok = false;
        R = tA->size(0);
        r = tA->size(1);
        N = tB->size(2);
        x = a.rows<uint16_t>(v[0], T, K, kBf16, xs);
        order = a.dense<int32_t>(v[1], {T}, kI32);
        offsets = a.dense<int32_t>(v[2], {R + 1}, kI32);
        A = a.dense<uint16_t>(v[3], {R, r, K}, kBf16);
        B = a.dense<uint16_t>(v[4], {R, r, N}, kBf16);
        scales = a.dense<float>(v[5], {R}, kF32);
        ranks = a.dense<int32_t>(v[6], {R}, kI32);
        return a.ok = a.ok && R <= INT32_MAX && r <= INT32_MAX;
    }
};

// handle, x, order, offsets, A, B, scales, ranks, out, y, v, stream
PyObject *lora(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count(n, 12))
        return nullptr;
    Args a{v};
    Adapters d;
    int64_t ys = 0, os = 0;
    if (!d.read(a, v + 1))
        return refused();
    uint16_t *out = a.rows<uint16_t>(v[8], d.T, d.N, kBf16, os);
    const uint16_t *y = v[9] == Py_None ? nullptr : a.rows<uint16_t>(v[9], d.T, d.N, kBf16, ys);
    float *keep = a.dense<float>(v[10], {d.T, d.r}, kF32);
    void *ctx = a.pointer(v[0]), *stream = a.pointer(v[11]);
    if (!a.ok || PyErr_Occurred())
        return refused();
    return status([&] {
        return p_lora(static_cast<gemmar_ctx *>(ctx), d.x, d.xs, d.order, d.offsets, d.A, d.B, d.scales, d.ranks, d.T,
                      d.K, d.N, (int)d.R, (int)d.r, y, ys, out, os, keep, stream);
    });
}

// handle, x, order, offsets, A, B, scales, ranks, dy, v, dx, dA, dB, dx0, stream
PyObject *lora_bwd(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count(n, 15))
        return nullptr;
    Args a{v};
    Adapters d;
    int64_t ys = 0, bs = 0, ds = 0;
    if (!d.read(a, v + 1))
        return refused();
    const uint16_t *dy = a.rows<uint16_t>(v[8], d.T, d.N, kBf16, ys);
    const float *keep = a.dense<float>(v[9], {d.T, d.r}, kF32);
    uint16_t *dx = a.rows<uint16_t>(v[10], d.T, d.K, kBf16, ds);
    uint16_t *dA = a.dense<uint16_t>(v[11], {d.R, d.r, d.K}, kBf16), *dB = a.dense<uint16_t>(v[12], {d.R, d.r, d.N}, kBf16);
    const uint16_t *dx0 = v[13] == Py_None ? nullptr : a.rows<uint16_t>(v[13], d.T, d.K, kBf16, bs);
    void *ctx = a.pointer(v[0]), *stream = a.pointer(v[14]);
    if (!a.ok || PyErr_Occurred())
        return refused();
    return status([&] {
        return p_lora_bwd(static_cast<gemmar_ctx *>(ctx), d.x, d.xs, dy, ys, d.order, d.offsets, d.A, d.B, d.scales,
                          d.ranks, keep, d.T, d.K, d.N, (int)d.R, (int)d.r, dx0, bs, dx, ds, dA, dB, stream);
    });
}

// handle, A, sa, B, sb, C, act, gated, bias, residual, q, scales, z, stream
PyObject *gemm_act(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count(n, 14))
        return nullptr;
    Args a{v};
    int64_t M = 0, K = 0, P = 0, K2 = 0, rs = 0, cs = 0;
    const int act = a.whole(v[6]);
    const bool gated = a.truth(v[7]);
    if (!a.shape2(v[1], M, K) || !a.shape2(v[3], P, K2) || (gated && P % 2 != 0))
        return refused();
    const int64_t N = gated ? P / 2 : P;
    const uint8_t *A = a.dense<uint8_t>(v[1], {M, K}, kU8, kE4m3), *B = a.dense<uint8_t>(v[3], {P, K}, kU8, kE4m3);
    const float *sa = a.dense<float>(v[2], {M, K / 128}, kF32), *sb = a.dense<float>(v[4], {P / 128, K / 128}, kF32);
    at::ScalarType ct = kF32, rt = kF32;
    void *C = nullptr, *res = nullptr;
    if (v[5] != Py_None) {
        ct = a.real_type(v[5]);
        C = a.rows<void>(v[5], M, N, ct, cs);
    }
    if (v[9] != Py_None) {
        rt = a.real_type(v[9]);
        res = a.rows<void>(v[9], M, N, rt, rs);
    }
    const float *bias = a.dense<float>(v[8], {P}, kF32);
    uint8_t *q = a.dense<uint8_t>(v[10], {M, N}, kU8, kE4m3);
    float *scales = a.dense<float>(v[11], {M, N / 128}, kF32);
    uint16_t *z = a.dense<uint16_t>(v[12], {M, P}, kBf16);
    void *ctx = a.pointer(v[0]), *stream = a.pointer(v[13]);
    if (!a.ok || PyErr_Occurred())
        return refused();
    return status([&] {
        return p_act(static_cast<gemmar_ctx *>(ctx), A, sa, B, sb, act, gated, bias, res, code(rt), rs, M, N, K, C, code(ct),
                     cs, q, scales, z, stream);
    });
}

// handle, dout, z, dz, act, gated, dbias, q, scales, stream
PyObject *gemm_act_bwd(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count(n, 10))
        return nullptr;
    Args a{v};
    int64_t M = 0, N = 0, ds = 0;
    const int act = a.whole(v[4]);
    const bool gated = a.truth(v[5]);
    if (!a.shape2(v[1], M, N))
        return refused();
    const int64_t P = gated ? 2 * N : N;
    const at::ScalarType dt = a.real_type(v[1]);
    const void *dout = a.rows<void>(v[1], M, N, dt, ds);
    const uint16_t *z = a.dense<uint16_t>(v[2], {M, P}, kBf16);
    uint16_t *dz = a.dense<uint16_t>(v[3], {M, P}, kBf16);
    float *dbias = a.dense<float>(v[6], {P}, kF32), *scales = a.dense<float>(v[8], {M, P / 128}, kF32);
    uint8_t *q = a.dense<uint8_t>(v[7], {M, P}, kU8, kE4m3);
    void *ctx = a.pointer(v[0]), *stream = a.pointer(v[9]);
    if (!a.ok || PyErr_Occurred())
        return refused();
    return status([&] {
        return p_act_bwd(static_cast<gemmar_ctx *>(ctx), dout, code(dt), ds, z, act, gated, M, N, dz, dbias, q, scales,
                         stream);
    });
}

// handle, x, router, ids, weights, bias, score, renorm, factor, stream
PyObject *route(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count(n, 10))
        return nullptr;
    Args a{v};
    int64_t T = 0, H = 0, E = 0, H2 = 0, T2 = 0, k = 0, xs = 0;
    const int score = a.whole(v[6]);
    const bool renorm = a.truth(v[7]);
    if (!a.shape2(v[1], T, H) || !a.shape2(v[2], E, H2) || !a.shape2(v[3], T2, k) || E > INT32_MAX || k > INT32_MAX)
        return refused();
    const uint16_t *x = a.rows<uint16_t>(v[1], T, H, kBf16, xs);
    const at::ScalarType wt = a.real_type(v[2]);
    const void *w = a.dense<void>(v[2], {E, H}, wt);
    int32_t *ids = a.dense<int32_t>(v[3], {T, k}, kI32);
    float *weights = a.dense<float>(v[4], {T, k}, kF32);
    const float *bias = a.dense<float>(v[5], {E}, kF32);
    const float factor = a.real(v[8]);
    void *ctx = a.pointer(v[0]), *stream = a.pointer(v[9]);
    if (!a.ok || PyErr_Occurred())
        return refused();
    return status([&] {
        return p_route(static_cast<gemmar_ctx *>(ctx), x, xs, w, code(wt), bias, T, H, (int)E, (int)k, score, renorm, factor,
                       ids, weights, stream);
    });
}

// handle, q, sx, ids, weights, w13, s13, w2, s2, out, act, place, y, stream
PyObject *moe(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count(n, 14))
        return nullptr;
    Args a{v};
    int64_t T = 0, H = 0, T2 = 0, k = 0, os = 0, ys = 0, places = 0;
    const int act = a.whole(v[10]);
    const at::Tensor *t2 = a.tensor(v[7]);
    if (!a.shape2(v[1], T, H) || !a.shape2(v[3], T2, k) || !t2 || t2->dim() != 3 || k > INT32_MAX ||
        t2->size(0) > INT32_MAX)
        return refused();
    const int64_t E = t2->size(0), I = t2->size(2);
    const uint8_t *q = a.dense<uint8_t>(v[1], {T, H}, kU8, kE4m3);
    const float *sx = a.dense<float>(v[2], {T, H / 128}, kF32);
    const int32_t *ids = a.dense<int32_t>(v[3], {T, k}, kI32);
    const float *weights = a.dense<float>(v[4], {T, k}, kF32);
    const uint8_t *w13 = a.dense<uint8_t>(v[5], {E, 2 * I, H}, kU8, kE4m3), *w2 = a.dense<uint8_t>(v[7], {E, H, I}, kU8, kE4m3);
    const float *s13 = a.dense<float>(v[6], {E, 2 * I / 128, H / 128}, kF32);
    const float *s2 = a.dense<float>(v[8], {E, H / 128, I / 128}, kF32);
    uint16_t *out = a.rows<uint16_t>(v[9], T, H, kBf16, os);
    const int32_t *place = nullptr;
    if (v[11] != Py_None) {
        const at::Tensor *p = a.tensor(v[11]);
        places = p && p->dim() == 1 ? p->size(0) : 0;
        place = a.dense<int32_t>(v[11], {places}, kI32);
    }
    const uint16_t *y = v[12] == Py_None ? nullptr : a.rows<uint16_t>(v[12], T, H, kBf16, ys);
    void *ctx = a.pointer(v[0]), *stream = a.pointer(v[13]);
    if (!a.ok || PyErr_Occurred())
        return refused();
    return status([&] {
        return p_moe(static_cast<gemmar_ctx *>(ctx), q, sx, ids, weights, place, places, w13, s13, w2, s2, act, T, H, I,
                     (int)E, (int)k, y, ys, out, os, stream);
    });
}

// The addresses of the library's entry points, in this order.
PyObject *bind(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count(n, 8))
        return nullptr;
    p_act = reinterpret_cast<decltype(p_act)>(PyLong_AsVoidPtr(v[4]));
    p_act_bwd = reinterpret_cast<decltype(p_act_bwd)>(PyLong_AsVoidPtr(v[5]));
    p_route = reinterpret_cast<decltype(p_route)>(PyLong_AsVoidPtr(v[6]));
    p_moe = reinterpret_cast<decltype(p_moe)>(PyLong_AsVoidPtr(v[7]));
    p_norm = reinterpret_cast<decltype(p_norm)>(PyLong_AsVoidPtr(v[0]));
    p_norm_bwd = reinterpret_cast<decltype(p_norm_bwd)>(PyLong_AsVoidPtr(v[1]));
    p_lora = reinterpret_cast<decltype(p_lora)>(PyLong_AsVoidPtr(v[2]));
    p_lora_bwd = reinterpret_cast<decltype(p_lora_bwd)>(PyLong_AsVoidPtr(v[3]));
    if (PyErr_Occurred())
        return nullptr;
    Py_RETURN_NONE;
}

// No C++ exception may leave a function that Python calls.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *v, Py_ssize_t n)
{
    try {
        return F(self, v, n);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<norm>("norm_gate_residual"), method<norm_bwd>("norm_gate_residual_bwd"),
                           method<lora>("lora_apply"), method<lora_bwd>("lora_apply_bwd"),
                           method<gemm_act>("gemm_blockscale_act"), method<gemm_act_bwd>("gemm_blockscale_act_bwd"),
                           method<route>("moe_route"), method<moe>("moe_apply"), method<bind>("bind"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_operators", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operators()
{
    PyObject *m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "torch_version", GEMMAR_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
