// Argument marshalling of the calls that take a few microseconds (step,
// prefill, accept, qk_prep, attend, cache_commit), natively: the checks of a tensor, its pointers, the
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

#include <cmath>
#include <exception>
#include <initializer_list>

#include "../../include/canopy.h"

namespace {

decltype(&canopy_step) step_fn = nullptr;
decltype(&canopy_prefill) prefill_fn = nullptr;
decltype(&canopy_prefill_workspace_bytes) prefill_bytes_fn = nullptr;
decltype(&canopy_accept) accept_fn = nullptr;
decltype(&canopy_qk_prep) qk_prep_fn = nullptr;
decltype(&canopy_attend) attend_fn = nullptr;
decltype(&canopy_attend_workspace_bytes) attend_bytes_fn = nullptr;
decltype(&canopy_cache_commit) cache_commit_fn = nullptr;
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

// A Python int that fits a C int (asked while this thread still holds the interpreter's lock).
bool int_of(PyObject* obj, int& x) {
    if (!PyLong_Check(obj)) return false;
    int over = 0;
    const long y = PyLong_AsLongAndOverflow(obj, &over);
    x = int(y);
    return !over && x == y;
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

// The rows of an attention layer's call: their leading sizes and number.
struct Rows {
    c10::SmallVector<int64_t, 4> lead;
    int64_t n = 0;
    bool fits(const at::Tensor& t, int64_t heads, int64_t d) const {
        if (t.dim() != int64_t(lead.size()) + 2 || t.size(-2) != heads || t.size(-1) != d) return false;
        for (size_t i = 0; i < lead.size(); ++i)
            if (t.size(i) != lead[i]) return false;
        return true;
    }
};
bool rows_of(const at::Tensor& q, Rows& r) {
    if (q.dim() != 3 && q.dim() != 4) return false;
    r.n = 1;
    for (int64_t i = 0; i < q.dim() - 2; ++i) {
        r.lead.push_back(q.size(i));
        r.n *= q.size(i);
    }
    return true;
}

// A CUDA tensor of rows whose heads are dense but whose tokens may lie apart.
const at::Tensor* spaced(PyObject* obj, int& dev, at::ScalarType type, const Rows& r, int64_t heads, int64_t d,
                         int64_t& ld) {
    if (!THPVariable_Check(obj)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(obj);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || t.get_device() != dev ||
        t.scalar_type() != type || !r.fits(t, heads, d))
        return nullptr;
    const bool two = r.lead.size() == 2 && r.lead[0] > 1;
    ld = r.lead.back() > 1 ? t.stride(-3) : two ? t.stride(0) : heads * d;
    if ((d > 1 && t.stride(-1) != 1) || (heads > 1 && t.stride(-2) != d) || (two && t.stride(0) != ld * r.lead.back()))
        return nullptr;
    return &t;
}

// A paged cache and whose streams it is.
struct Cache {
    const at::Tensor *k, *v, *table, *context;
    int64_t B, pages, page, most;
};
bool cache_of(PyObject* k, PyObject* v, PyObject* table, PyObject* context, int& dev, at::ScalarType type, int64_t HKV,
              int64_t d, Cache& c) {
    c.k = plain(k, dev);
    c.table = plain(table, dev);
    if (!c.k || !c.table || c.k->dim() != 4 || c.k->size(1) != HKV || c.k->size(3) != d ||
        c.k->scalar_type() != type || c.table->dim() != 2 || c.table->scalar_type() != at::kInt)
        return false;
    c.B = c.table->size(0);
    c.pages = c.k->size(0);
    c.page = c.k->size(2);
    c.most = c.table->size(1);
    c.v = plain(v, dev, type, {c.pages, HKV, c.page, d});
    c.context = plain(context, dev, at::kInt, {c.B});
    return c.v && c.context && ints({c.B, c.pages, c.page, c.most});
}
bool of_streams(const Rows& r, int64_t B, bool packed) {
    if (r.lead.size() == 2) return !packed && r.lead[0] == B;
    return packed || r.lead[0] == B;
}

at::Tensor fresh_rows(const Rows& r, int64_t heads, int64_t d, at::ScalarType type, int dev) {
    c10::SmallVector<int64_t, 4> shape = r.lead;
    shape.push_back(heads);
    shape.push_back(d);
    return fresh(shape, type, dev);
}
// A rows' output given as obj, if it fits; None stays undefined for now.
bool rows_output(PyObject* obj, int dev, at::ScalarType type, const Rows& r, int64_t heads, int64_t d,
                 at::Tensor& out) {
    if (obj == Py_None) return true;
    const at::Tensor* t = plain(obj, dev);
    if (!t || t->scalar_type() != type || !r.fits(*t, heads, d)) return false;
    out = *t;
    return true;
}

// qk_prep(q, k, v, norm, q_weight, k_weight, eps, freqs, positions, axis, pairs, q_out, k_out, k_cache, v_cache,
//         page_table, context, starts, lengths, err)
PyObject* qk_prep(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int norm = 0, pairs = 0;
    if (n != 20 || !qk_prep_fn || !int_of(a[3], norm) || !PyFloat_Check(a[6]) || !int_of(a[10], pairs)) return none();
    return guarded([&]() -> PyObject* {
        if (!THPVariable_Check(a[0]) || !THPVariable_Check(a[1])) return none();
        const at::Tensor &q0 = THPVariable_Unpack(a[0]), &k0 = THPVariable_Unpack(a[1]);
        canopy_dtype type;
        Rows r;
        if (!q0.defined() || !q0.is_cuda() || !k0.defined() || !code_of(q0.scalar_type(), type) || !rows_of(q0, r) ||
            k0.dim() != q0.dim())
            return none();
        int dev = q0.get_device();
        const at::ScalarType st = q0.scalar_type();
        const int64_t HQ = q0.size(-2), HKV = k0.size(-2), d = q0.size(-1);
        int64_t ldq = 0, ldk = 0, ldv = 0;
        const at::Tensor *q = spaced(a[0], dev, st, r, HQ, d, ldq), *k = spaced(a[1], dev, st, r, HKV, d, ldk);
        const at::Tensor* v = nullptr;
        bool ok = q && k && ints({r.n, HQ, HKV, d});
        const bool cached = a[13] != Py_None, packed = a[17] != Py_None;
        Cache c = {};
        const at::Tensor *starts = nullptr, *lengths = nullptr;
        if (cached) {
            if (!ok || !cache_of(a[13], a[14], a[15], a[16], dev, st, HKV, d, c) || !of_streams(r, c.B, packed) ||
                a[12] != Py_None || (a[18] != Py_None && r.lead.size() != 2))
                return none();
            v = spaced(a[2], dev, st, r, HKV, d, ldv);
            starts = maybe(a[17], dev, at::kInt, {c.B + 1}, ok);
            lengths = maybe(a[18], dev, at::kInt, {c.B}, ok);
            ok = ok && v;
        } else {
            for (const int i : {2, 14, 15, 16, 17, 18}) ok = ok && a[i] == Py_None;
        }
        const at::Tensor *qw = maybe(a[4], dev, at::kFloat, {d}, ok), *kw = maybe(a[5], dev, at::kFloat, {d}, ok);
        const at::Tensor *freqs = nullptr, *positions = nullptr;
        int64_t half = 0, axes = 1, axis_step = 0, row_step = 1;
        if (a[7] != Py_None) {
            freqs = plain(a[7], dev);
            ok = ok && freqs && freqs->dim() == 1 && freqs->scalar_type() == at::kFloat;
            if (ok) half = freqs->size(0);
        }
        if (ok && a[8] != Py_None) {
            if (!THPVariable_Check(a[8])) return none();
            positions = &THPVariable_Unpack(a[8]);
            if (!positions->defined() || !positions->is_cuda() || positions->layout() != at::kStrided ||
                positions->get_device() != dev || positions->scalar_type() != at::kInt)
                return none();
            const int64_t more = positions->dim() - int64_t(r.lead.size());
            if (more != 0 && more != 1) return none();
            for (size_t i = 0; i < r.lead.size(); ++i)
                if (positions->size(i + more) != r.lead[i]) return none();
            if (more == 1) {
                axes = positions->size(0);
                axis_step = positions->stride(0);
            }
            const bool two = r.lead.size() == 2 && r.lead[0] > 1;
            row_step = r.lead.back() > 1 ? positions->stride(-1) : two ? positions->stride(-2) : 1;
            if (two && positions->stride(-2) != row_step * r.lead.back()) return none();
        }
        const at::Tensor* axis = maybe(a[9], dev, at::kInt, {half}, ok);
        const at::Tensor* err = maybe(a[19], dev, at::kInt, {1}, ok);
        at::Tensor q_out, k_out;
        if (!ok || !ints({2 * half, axes}) || !rows_output(a[11], dev, st, r, HQ, d, q_out) ||
            !rows_output(a[12], dev, st, r, HKV, d, k_out))
            return none();
        canopy_status s;
        {
            const OnDevice on(dev);
            if (!q_out.defined()) q_out = fresh_rows(r, HQ, d, st, dev);
            if (!cached && !k_out.defined()) k_out = fresh_rows(r, HKV, d, st, dev);
            s = qk_prep_fn(q->data_ptr(), k->data_ptr(), ptr<void>(v), type, ldq, ldk, ldv,
                           canopy_norm(norm), ptr<float>(qw), ptr<float>(kw),
                           float(PyFloat_AS_DOUBLE(a[6])), ptr<float>(freqs), int(2 * half), ptr<int32_t>(positions),
                           int(axes), axis_step, row_step, ptr<int32_t>(axis), canopy_pairs(pairs),
                           int(r.n), int(c.B), int(HQ), int(HKV), int(d), q_out.data_ptr(),
                           cached ? nullptr : k_out.data_ptr(),
                           ptr<void>(c.k), ptr<void>(c.v), ptr<int32_t>(c.table), int(c.pages), int(c.page),
                           int(c.most), ptr<int32_t>(c.context), ptr<int32_t>(starts), ptr<int32_t>(lengths),
                           ptr<int32_t>(err), stream_of(dev));
        }
        if (s != CANOPY_OK) return PyLong_FromLong(s);
        if (!cached) return pair_of(a[11], q_out, a[12], k_out);
        PyObject* o = a[11] == Py_None ? THPVariable_Wrap(q_out) : Py_NewRef(a[11]);
        if (!o) return nullptr;
        PyObject* pair = PyTuple_Pack(2, o, Py_None);
        Py_DECREF(o);
        return pair;
    });
}

// attend(q, k_cache, v_cache, page_table, context, ws, starts, parent, lengths, window, sinks, scale, out)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int window = 0, sinks = 0;
    if (n != 13 || !attend_fn || !int_of(a[9], window) || !int_of(a[10], sinks) || window < 0 || sinks < 0 ||
        (a[11] != Py_None && !PyFloat_Check(a[11])))
        return none();
    return guarded([&]() -> PyObject* {
        int dev = -1;
        const at::Tensor *q = plain(a[0], dev), *k = plain(a[1], dev), *ws = plain(a[5], dev);
        canopy_dtype type;
        Rows r;
        if (!q || !k || !ws || k->dim() != 4 || ws->scalar_type() != at::kByte || !code_of(q->scalar_type(), type) ||
            !rows_of(*q, r))
            return none();
        const at::ScalarType st = q->scalar_type();
        const int64_t HQ = q->size(-2), HKV = k->size(1), d = q->size(-1);
        const bool packed = a[6] != Py_None;
        Cache c;
        if (!cache_of(a[1], a[2], a[3], a[4], dev, st, HKV, d, c) || !of_streams(r, c.B, packed) ||
            !ints({r.n, HQ, HKV, d}) || (r.lead.size() != 2 && (a[7] != Py_None || a[8] != Py_None)))
            return none();
        bool ok = true;
        const at::Tensor* starts = maybe(a[6], dev, at::kInt, {c.B + 1}, ok);
        const at::Tensor* parent = nullptr;
        if (a[7] != Py_None) parent = maybe(a[7], dev, at::kInt, {r.lead[0], r.lead[1]}, ok);
        const at::Tensor* lengths = maybe(a[8], dev, at::kInt, {c.B}, ok);
        at::Tensor out;
        if (!ok || !rows_output(a[12], dev, st, r, HQ, d, out) ||
            size_t(ws->numel()) < attend_bytes_fn(int(r.n), int(c.B), int(HQ), int(HKV), int(d)))
            return none();
        const float scale = a[11] == Py_None ? float(1.0 / std::sqrt(double(d))) : float(PyFloat_AS_DOUBLE(a[11]));
        canopy_status s;
        {
            const OnDevice on(dev);
            if (!out.defined()) out = fresh_rows(r, HQ, d, st, dev);
            s = attend_fn(q->data_ptr(), type, c.k->data_ptr(), c.v->data_ptr(), ptr<int32_t>(c.table), int(c.pages),
                          int(c.page), int(c.most), ptr<int32_t>(c.context), ptr<int32_t>(starts),
                          ptr<int32_t>(parent), ptr<int32_t>(lengths), int(r.n), int(c.B), int(HQ), int(HKV), int(d),
                          window, sinks, scale, out.data_ptr(), ws->data_ptr(), stream_of(dev));
        }
        if (s != CANOPY_OK) return PyLong_FromLong(s);
        return a[12] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(a[12]);
    });
}

// cache_commit(accepted, parent, k_cache, v_cache, page_table, context, lengths, err)
PyObject* cache_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 8 || !cache_commit_fn) return none();
    return guarded([&]() -> PyObject* {
        int dev = -1;
        const at::Tensor *k = plain(a[2], dev), *parent = plain(a[1], dev);
        canopy_dtype type;
        Cache c;
        if (!k || !parent || k->dim() != 4 || parent->dim() != 2 || !code_of(k->scalar_type(), type) ||
            !cache_of(a[2], a[3], a[4], a[5], dev, k->scalar_type(), k->size(1), k->size(3), c))
            return none();
        const int64_t T = parent->size(1), HKV = k->size(1), d = k->size(3);
        bool ok = ints({T, HKV, d}) && plain(a[1], dev, at::kInt, {c.B, T});
        const at::Tensor* accepted = plain(a[0], dev, at::kInt, {c.B});
        const at::Tensor* lengths = maybe(a[6], dev, at::kInt, {c.B}, ok);
        const at::Tensor* err = maybe(a[7], dev, at::kInt, {1}, ok);
        if (!ok || !accepted) return none();
        at::Tensor context;
        canopy_status s;
        {
            const OnDevice on(dev);
            context = fresh({c.B}, at::kInt, dev);
            s = cache_commit_fn(ptr<int32_t>(accepted), ptr<int32_t>(parent), ptr<int32_t>(lengths), c.k->data_ptr(),
                                c.v->data_ptr(), type, ptr<int32_t>(c.table), int(c.pages), int(c.page), int(c.most),
                                ptr<int32_t>(c.context), int(T), int(c.B), int(HKV), int(d), ptr<int32_t>(&context),
                                ptr<int32_t>(err), stream_of(dev));
        }
        if (s != CANOPY_OK) return PyLong_FromLong(s);
        return THPVariable_Wrap(context);
    });
}

// bind_attention(qk_prep, attend, attend_workspace_bytes, cache_commit)
PyObject* bind_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind_attention takes four addresses");
        return nullptr;
    }
    void* f[4];
    for (int i = 0; i < 4; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i]);
        if (!f[i] && PyErr_Occurred()) return nullptr;
    }
    qk_prep_fn = reinterpret_cast<decltype(qk_prep_fn)>(f[0]);
    attend_fn = reinterpret_cast<decltype(attend_fn)>(f[1]);
    attend_bytes_fn = reinterpret_cast<decltype(attend_bytes_fn)>(f[2]);
    cache_commit_fn = reinterpret_cast<decltype(cache_commit_fn)>(f[3]);
    return none();
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
                         {"bind_attention", fast(bind_attention), METH_FASTCALL, nullptr},
                         {"qk_prep", fast(qk_prep), METH_FASTCALL, nullptr},
                         {"attend", fast(attend), METH_FASTCALL, nullptr},
                         {"cache_commit", fast(cache_commit), METH_FASTCALL, nullptr},
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
