// Argument marshalling of the calls that take a few microseconds (step,
// prefill, accept), natively: the checks of a tensor, its pointers, the
// outputs and the stream cost 10 us and more in Python, as much as the
// kernels themselves for a few streams.
//
// Each function takes the Python call's arguments in order and looks at them.
// Where everything is as it has to be it makes the library call and returns
// the outputs (or the library's status where that is not CANOPY_OK);
// otherwise it returns None, having done nothing, and the Python side goes
// through its own checks, which say what is wrong.  The library's entry
// points are handed over by address, so that this module links against torch
// only and the library against nothing of it.  The library works on the current
// device: the tensors' is made current for the call.  An allocation may wait for
// the GPU and a launch for room in the stream's queue, so other Python threads
// run meanwhile.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "../../include/canopy.h"

namespace {

decltype(&canopy_step) step_fn = nullptr;
decltype(&canopy_prefill) prefill_fn = nullptr;
decltype(&canopy_prefill_workspace_bytes) prefill_bytes_fn = nullptr;
decltype(&canopy_accept) accept_fn = nullptr;
PyObject *bf16_obj = nullptr, *f32_obj = nullptr;  // torch.bfloat16, torch.float32

// The tensor behind obj, if it is a contiguous CUDA tensor on device dev (any
// if dev < 0: then dev is set); else null.
const at::Tensor* plain(PyObject* obj, int& dev) {
    if (!THPVariable_Check(obj)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(obj);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous()) return nullptr;
    if (dev < 0) dev = t.get_device();
    return t.get_device() == dev ? &t : nullptr;
}

// The same, with the given type and shape.
const at::Tensor* plain(PyObject* obj, int& dev, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = plain(obj, dev);
    return t && t->scalar_type() == type && t->sizes() == at::IntArrayRef(shape) ? t : nullptr;
}

// An optional tensor: null for None; `ok` becomes false where it does not fit.
const at::Tensor* maybe(PyObject* obj, int& dev, at::ScalarType type, std::initializer_list<int64_t> shape,
                        bool& ok) {
    if (obj == Py_None) return nullptr;
    const at::Tensor* t = plain(obj, dev, type, shape);
    ok = ok && t;
    return t;
}

bool code_of(at::ScalarType type, canopy_dtype& code) {
    code = type == at::kBFloat16 ? CANOPY_BF16 : CANOPY_F32;
    return type == at::kBFloat16 || type == at::kFloat;
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev));
}

template <typename T>
T* ptr(const at::Tensor* t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

PyObject* none() { Py_RETURN_NONE; }

// The library takes sizes as int.
bool ints(std::initializer_list<int64_t> sizes) {
    for (const int64_t n : sizes)
        if (n > INT32_MAX) return false;
    return true;
}

// The output given as obj, if it fits; None stays undefined for now.
bool output(PyObject* obj, int dev, at::ScalarType type, std::initializer_list<int64_t> shape, at::Tensor& out) {
    if (obj == Py_None) return true;
    const at::Tensor* t = plain(obj, dev, type, shape);
    if (t) out = *t;
    return t != nullptr;
}

// While one of these exists other Python threads run, and the device is current.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
struct OnDevice {
    Unlocked unlocked;
    c10::cuda::OptionalCUDAGuard guard;  // (set where it has to be: it costs 0.1 us)
    explicit OnDevice(int dev) {
        if (c10::cuda::current_device() != dev) guard.set_index(at::DeviceIndex(dev));
    }
};

PyObject* pair_of(PyObject* given_a, const at::Tensor& a, PyObject* given_b, const at::Tensor& b) {
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    auto put = [&](int i, PyObject* given, const at::Tensor& t) {
        PyObject* o = given == Py_None ? THPVariable_Wrap(t) : Py_NewRef(given);
        PyTuple_SET_ITEM(r, i, o);
        return o != nullptr;
    };
    if (!put(0, given_a, a) || !put(1, given_b, b)) {
        Py_DECREF(r);
        return nullptr;
    }
    return r;
}

// C++ exceptions become the Python ones that torch raises for them (an
// allocation that fails torch.OutOfMemoryError).
template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// The output type: the given out's, else the o_dtype argument's.
bool out_type(PyObject* out, PyObject* o_dtype, at::ScalarType& type) {
    if (out != Py_None) {
        if (!THPVariable_Check(out)) return false;
        type = THPVariable_Unpack(out).scalar_type();
    } else if (o_dtype == bf16_obj) {
        type = at::kBFloat16;
    } else {
        type = at::kFloat;
        if (o_dtype != f32_obj) return false;
    }
    return true;
}

// step(q, k, v, g, beta, S, o_dtype, out, S_out, scale, err)
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 11 || !step_fn || !PyFloat_Check(a[9])) return none();
    return guarded([&]() -> PyObject* {
        int dev = -1;
        const at::Tensor *q = plain(a[0], dev), *v = plain(a[2], dev);
        canopy_dtype in, oc;
        at::ScalarType ot;
        if (!q || !v || q->dim() != 3 || v->dim() != 3 || !code_of(q->scalar_type(), in) ||
            !out_type(a[7], a[6], ot) || !code_of(ot, oc))
            return none();
        const int64_t B = q->size(0), H = q->size(1), dk = q->size(2), HV = v->size(1), dv = v->size(2);
        const at::Tensor* k = plain(a[1], dev, q->scalar_type(), {B, H, dk});
        const at::Tensor *g = plain(a[3], dev, at::kFloat, {B, HV}), *beta = plain(a[4], dev, at::kFloat, {B, HV});
        const at::Tensor* S = plain(a[5], dev, at::kFloat, {B, HV, dv, dk});
        bool ok = ints({B, H, HV, dk, dv}) && k && g && beta && S && v->size(0) == B &&
                  v->scalar_type() == q->scalar_type();
        const at::Tensor* err = maybe(a[10], dev, at::kInt, {1}, ok);
        at::Tensor out, S_out;
        if (!ok || !output(a[7], dev, ot, {B, HV, dv}, out) || !output(a[8], dev, at::kFloat, {B, HV, dv, dk}, S_out))
            return none();
        const float scale = float(PyFloat_AS_DOUBLE(a[9]));
        canopy_status st;
        {
            const OnDevice on(dev);
            if (!out.defined()) out = fresh({B, HV, dv}, ot, dev);
            if (!S_out.defined()) S_out = fresh({B, HV, dv, dk}, at::kFloat, dev);
            st = step_fn(q->data_ptr(), k->data_ptr(), v->data_ptr(), in, ptr<float>(g), ptr<float>(beta),
                         ptr<float>(S), ptr<float>(&S_out), int(B), int(H), int(HV), int(dk), int(dv), scale,
                         out.data_ptr(), oc, ptr<int32_t>(err), stream_of(dev));
        }
        if (st != CANOPY_OK) return PyLong_FromLong(st);
        return pair_of(a[7], out, a[8], S_out);
    });
}

// prefill(q, k, v, g, beta, S0, starts, ws, o_dtype, out, S_out, scale, flags)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 13 || !prefill_fn || !PyFloat_Check(a[11]) || !PyLong_Check(a[12])) return none();
    return guarded([&]() -> PyObject* {
        int dev = -1;
        const at::Tensor *q = plain(a[0], dev), *v = plain(a[2], dev), *starts = plain(a[6], dev);
        const at::Tensor* ws = plain(a[7], dev);
        canopy_dtype in, oc;
        at::ScalarType ot;
        if (!q || !v || !starts || !ws || q->dim() != 3 || v->dim() != 3 || starts->dim() != 1 ||
            starts->size(0) < 2 || starts->scalar_type() != at::kInt || ws->scalar_type() != at::kByte ||
            !code_of(q->scalar_type(), in) || !out_type(a[9], a[8], ot) || !code_of(ot, oc))
            return none();
        const int64_t N = q->size(0), H = q->size(1), dk = q->size(2), HV = v->size(1), dv = v->size(2);
        const int64_t B = starts->size(0) - 1;
        const at::Tensor* k = plain(a[1], dev, q->scalar_type(), {N, H, dk});
        const at::Tensor *g = plain(a[3], dev, at::kFloat, {N, HV}), *beta = plain(a[4], dev, at::kFloat, {N, HV});
        bool ok = ints({N, B, H, HV, dk, dv}) && k && g && beta && v->size(0) == N &&
                  v->scalar_type() == q->scalar_type();
        const at::Tensor* S0 = maybe(a[5], dev, at::kFloat, {B, HV, dv, dk}, ok);
        at::Tensor out, S_out;
        if (!ok || size_t(ws->numel()) < prefill_bytes_fn(int(N), int(B), int(HV), int(dk), int(dv)) ||
            !output(a[9], dev, ot, {N, HV, dv}, out) || !output(a[10], dev, at::kFloat, {B, HV, dv, dk}, S_out))
            return none();
        const float scale = float(PyFloat_AS_DOUBLE(a[11]));
        const unsigned flags = unsigned(PyLong_AsUnsignedLong(a[12]));
        canopy_status st;
        {
            const OnDevice on(dev);
            if (!out.defined()) out = fresh({N, HV, dv}, ot, dev);
            if (!S_out.defined()) S_out = fresh({B, HV, dv, dk}, at::kFloat, dev);
            st = prefill_fn(q->data_ptr(), k->data_ptr(), v->data_ptr(), in, ptr<float>(g), ptr<float>(beta),
                            ptr<float>(S0), ptr<int32_t>(starts), int(N), int(B), int(H), int(HV), int(dk), int(dv),
                            scale, out.data_ptr(), oc, ptr<float>(&S_out), ws->data_ptr(), flags, stream_of(dev));
        }
        if (st != CANOPY_OK) return PyLong_FromLong(st);
        return pair_of(a[9], out, a[10], S_out);
    });
}

// accept(p, tokens, parent, u, noise, q, lengths, err)
PyObject* accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 8 || !accept_fn) return none();
    return guarded([&]() -> PyObject* {
        int dev = -1;
        const at::Tensor* p = plain(a[0], dev);
        canopy_dtype type;
        if (!p || p->dim() != 3 || !code_of(p->scalar_type(), type)) return none();
        const int64_t B = p->size(0), T = p->size(1), V = p->size(2);
        const at::Tensor *tokens = plain(a[1], dev, at::kInt, {B, T}), *parent = plain(a[2], dev, at::kInt, {B, T});
        const at::Tensor *u = plain(a[3], dev, at::kFloat, {B, T}), *noise = plain(a[4], dev, at::kFloat, {B, V});
        bool ok = ints({B, T, V}) && tokens && parent && u && noise;
        const at::Tensor* q = maybe(a[5], dev, p->scalar_type(), {B, T, V}, ok);
        const at::Tensor* lengths = maybe(a[6], dev, at::kInt, {B}, ok);
        const at::Tensor* err = maybe(a[7], dev, at::kInt, {1}, ok);
        if (!ok) return none();
        at::Tensor accepted, out, counts;
        canopy_status st;
        {
            const OnDevice on(dev);
            accepted = fresh({B}, at::kInt, dev);
            out = fresh({B, T}, at::kInt, dev);
            counts = fresh({B}, at::kInt, dev);
            st = accept_fn(p->data_ptr(), ptr<void>(q), type, ptr<int32_t>(tokens), ptr<int32_t>(parent),
                           ptr<int32_t>(lengths), ptr<float>(u), ptr<float>(noise), int(T), int(B), int(V),
                           ptr<int32_t>(&accepted), ptr<int32_t>(&out), ptr<int32_t>(&counts), ptr<int32_t>(err),
                           stream_of(dev));
        }
        if (st != CANOPY_OK) return PyLong_FromLong(st);
        PyObject* r = PyTuple_New(3);
        if (!r) return nullptr;
        const at::Tensor* outs[3] = {&accepted, &out, &counts};
        for (int i = 0; i < 3; ++i) {
            PyObject* o = THPVariable_Wrap(*outs[i]);
            if (!o) {
                Py_DECREF(r);
                return nullptr;
            }
            PyTuple_SET_ITEM(r, i, o);
        }
        return r;
    });
}

// bind(step, prefill, prefill_workspace_bytes, accept, torch.bfloat16, torch.float32)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes four addresses and two dtypes");
        return nullptr;
    }
    void* f[4];
    for (int i = 0; i < 4; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (!f[i] && PyErr_Occurred()) return nullptr;
    }
    step_fn = reinterpret_cast<decltype(step_fn)>(f[0]);
    prefill_fn = reinterpret_cast<decltype(prefill_fn)>(f[1]);
    prefill_bytes_fn = reinterpret_cast<decltype(prefill_bytes_fn)>(f[2]);
    accept_fn = reinterpret_cast<decltype(accept_fn)>(f[3]);
    Py_XSETREF(bf16_obj, Py_NewRef(a[4]));
    Py_XSETREF(f32_obj, Py_NewRef(a[5]));
    return none();
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"step", fast(step), METH_FASTCALL, nullptr},
                         {"prefill", fast(prefill), METH_FASTCALL, nullptr},
                         {"accept", fast(accept), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

// built_for: the Python and torch that this file was compiled for, which the
// binding compares with those that it runs on.
PyMODINIT_FUNC PyInit__marshal() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", CANOPY_MARSHAL_TAG) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
