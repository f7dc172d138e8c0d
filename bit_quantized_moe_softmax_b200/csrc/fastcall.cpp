// fastcall.cpp -- the Python binding's short way to the operators around the
// layer: checks of the tensors and the call in one step, for calls on the
// current device whose time is the call itself (the checks in Python take about
// as long as the launch).  A function returns True where the call was made;
// False, with nothing launched, wherever something is not as it should be or the
// library refuses the arguments (the binding then goes its long way, which says
// what it was); the library's status where the call failed behind its checks:
// something of it may have been launched, so it is not made again.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/ds4moe.h"

namespace {

enum : unsigned { kF32 = 1, kBF16 = 2, kE4M3 = 4, kInt8 = 8, kInt32 = 16, kAct = kF32 | kBF16, kQ8 = kE4M3 | kInt8 };

unsigned type_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return kF32;
        case at::kBFloat16: return kBF16;
        case at::kFloat8_e4m3fn: return kE4M3;
        case at::kChar: return kInt8;
        case at::kInt: return kInt32;
        default: return 0;
    }
}

// The tensors of one call, on one device.
struct Call {
    int dev = -1;
    bool good = true;

    const at::Tensor* first(PyObject* o, int64_t dims) {
        if (!THPVariable_Check(o)) return nullptr;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.dim() != dims) return nullptr;
        dev = t.get_device();
        return dev == c10::cuda::current_device() ? &t : nullptr;
    }
    // The data of o (None: nullptr), which has to have this shape and one of these types; its type through `type`.
    void* data(PyObject* o, std::initializer_list<int64_t> shape, unsigned types, unsigned* type = nullptr) {
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) return good = false, nullptr;
        const at::Tensor& t = THPVariable_Unpack(o);
        const unsigned k = type_of(t);
        if (!(k & types) || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous() || t.sizes() != at::IntArrayRef(shape))
            return good = false, nullptr;
        if (type) *type = k;
        return t.data_ptr();
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

int32_t act(unsigned type) { return type == kBF16 ? DS4MOE_ACT_BF16 : DS4MOE_ACT_F32; }
int32_t q8(unsigned type) { return type == kInt8 ? DS4MOE_Q8_INT8 : DS4MOE_Q8_E4M3; }
bool fits(int64_t v) { return v >= 0 && v <= INT32_MAX; }
int64_t groups_of(int64_t hidden, long group) { return group > 0 ? (hidden + group - 1) / group : 1; }

enum : int { kLongWay = 0, kDone = 1 };   // or a status, which is negative

int outcome(ds4moe_status s) {
    if (s == DS4MOE_OK) return kDone;
    return s == DS4MOE_ERR_ARG || s == DS4MOE_ERR_ALIGN || s == DS4MOE_ERR_SHAPE ? kLongWay : (int)s;
}

template <typename F>
PyObject* guarded(F&& f) {
    int r = kLongWay;
    try {
        r = f();
    } catch (...) {   // no C++ exception leaves this file (and none comes from behind a launch)
        r = kLongWay;
    }
    if (PyErr_Occurred()) PyErr_Clear();
    return r == kLongWay || r == kDone ? PyBool_FromLong(r) : PyLong_FromLong(r);
}

// (x, weight, eps, residual, sum, out, q, scale, group)
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded([&]() -> int {
        Call c;
        const at::Tensor* x = n_args == 9 ? c.first(a[0], 2) : nullptr;
        if (!x || !PyFloat_Check(a[2]) || !PyLong_Check(a[8])) return kLongWay;
        const int64_t n = x->size(0), H = x->size(1);
        const long group = PyLong_AsLong(a[8]);
        if (!fits(n) || !fits(H) || group < 0 || group > 128) return kLongWay;
        unsigned xt = 0, rt = kF32, st = 0, ot = kF32, qt = kE4M3;
        void* px = c.data(a[0], {n, H}, kAct, &xt);
        void* w = c.data(a[1], {H}, kF32);
        void* res = c.data(a[3], {n, H}, kAct, &rt);
        void* sum = c.data(a[4], {n, H}, kAct, &st);
        void* out = c.data(a[5], {n, H}, kAct, &ot);
        void* q = c.data(a[6], {n, H}, kQ8, &qt);
        void* scale = c.data(a[7], {n, groups_of(H, group)}, kF32);
        if (!c.good || (st && st != rt)) return kLongWay;
        return outcome(ds4moe_add_rmsnorm(px, act(xt), res, act(rt), (const float*)w, (float)PyFloat_AS_DOUBLE(a[2]), (int32_t)n,
                                          (int32_t)H, sum, out, act(ot), q, q8(qt), (int32_t)group, (float*)scale, c.stream()));
    });
}

// (q, scale, out, group)
PyObject* widen_rows(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded([&]() -> int {
        Call c;
        const at::Tensor* t = n_args == 4 ? c.first(a[0], 2) : nullptr;
        if (!t || !PyLong_Check(a[3])) return kLongWay;
        const int64_t n = t->size(0), H = t->size(1);
        const long group = PyLong_AsLong(a[3]);
        if (!fits(n) || !fits(H) || group < 0 || group > 128) return kLongWay;
        unsigned qt = 0, ot = 0;
        void* q = c.data(a[0], {n, H}, kQ8, &qt);
        void* scale = c.data(a[1], {n, groups_of(H, group)}, kF32);
        void* out = c.data(a[2], {n, H}, kAct, &ot);
        if (!c.good) return kLongWay;
        return outcome(ds4moe_widen_rows(q, q8(qt), (const float*)scale, (int32_t)group, (int32_t)n, (int32_t)H, out, act(ot),
                                         c.stream()));
    });
}

// (x, W, out, A, B, adapter_scale, ids): scratch from the allocator
PyObject* project(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded([&]() -> int {
        Call c;
        const at::Tensor* x = n_args == 7 ? c.first(a[0], 2) : nullptr;
        if (!x || !THPVariable_Check(a[1])) return kLongWay;
        const at::Tensor& W = THPVariable_Unpack(a[1]);
        if (W.dim() != 2) return kLongWay;
        const int64_t n = x->size(0), fin = x->size(1), fout = W.size(0);
        int64_t na = 0, rank = 0;
        if (a[3] != Py_None) {
            if (!THPVariable_Check(a[3])) return kLongWay;
            const at::Tensor& A = THPVariable_Unpack(a[3]);
            if (A.dim() != 3 || a[4] == Py_None || a[5] == Py_None || a[6] == Py_None) return kLongWay;
            na = A.size(0), rank = A.size(1);
        } else if (a[4] != Py_None || a[5] != Py_None || a[6] != Py_None) {
            return kLongWay;
        }
        if (!fits(n) || !fits(fin) || !fits(fout) || !fits(na) || !fits(rank)) return kLongWay;
        void* px = c.data(a[0], {n, fin}, kBF16);
        void* pw = c.data(a[1], {fout, fin}, kBF16);
        void* out = c.data(a[2], {n, fout}, kBF16);
        void* A = c.data(a[3], {na, rank, fin}, kBF16);
        void* B = c.data(a[4], {na, fout, rank}, kBF16);
        void* scale = c.data(a[5], {na}, kF32);
        void* ids = c.data(a[6], {n}, kInt32);
        if (!c.good) return kLongWay;
        at::Tensor work;
        size_t need = 0;
        if (na && n) {
            need = ds4moe_project_work_bytes((int32_t)n, (int32_t)fin, (int32_t)fout, (int32_t)na, (int32_t)rank);
            if (!need) return kLongWay;
            work = at::empty({(int64_t)need}, x->options().dtype(at::kByte));
        }
        return outcome(ds4moe_project(px, (int32_t)n, pw, (int32_t)fin, (int32_t)fout, A, B, (const float*)scale, (int32_t)na,
                                      (int32_t)rank, (const int32_t*)ids, out, need ? work.data_ptr() : nullptr, need, c.stream()));
    });
}

// (logits, u, token, temperature, top_k, top_p, min_p, prob, probs)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded([&]() -> int {
        Call c;
        const at::Tensor* l = n_args == 9 ? c.first(a[0], 2) : nullptr;
        if (!l) return kLongWay;
        const int64_t n = l->size(0), V = l->size(1);
        const unsigned lt = type_of(*l);
        if (!(lt & kAct) || (V > 1 && l->stride(1) != 1) || !fits(n) || !fits(V)) return kLongWay;
        void* u = c.data(a[1], {n}, kF32);
        void* token = c.data(a[2], {n}, kInt32);
        void* temp = c.data(a[3], {n}, kF32);
        void* top_k = c.data(a[4], {n}, kInt32);
        void* top_p = c.data(a[5], {n}, kF32);
        void* min_p = c.data(a[6], {n}, kF32);
        void* prob = c.data(a[7], {n}, kF32);
        void* probs = c.data(a[8], {n, V}, kF32);
        if (!c.good) return kLongWay;
        return outcome(ds4moe_sample(l->data_ptr(), act(lt), n > 1 ? l->stride(0) : V, (int32_t)n, (int32_t)V, (const float*)temp,
                                     (const int32_t*)top_k, (const float*)top_p, (const float*)min_p, (const float*)u,
                                     (int32_t*)token, (float*)prob, (float*)probs, c.stream()));
    });
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(add_rmsnorm), METHOD(widen_rows), METHOD(project), METHOD(sample), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
