// binding.cpp -- the calls of a kept prompt from Python in one step each: checks of
// the tensors, results and workspace, and the library's call.
//
// The wrappers in __init__.py do the same by themselves; a call from there costs 15
// to 25 us of the host's time, most of it for reading attributes one by one and
// for results made through Python.  Here a function takes the plain case: tensors
// of the right types, shapes and device, contiguous, that device current, no
// buffer given.  Anything else, and what the library refuses, gives None: the wrapper
// then goes its own way, and what is wrong is named there.  A call that failed is
// not made again: its status is raised here.
#include <Python.h>
#include <dlfcn.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "striped.h"

namespace {

struct Library {
    decltype(&striped_kv4_store) kv4_store;
    decltype(&striped_kv4_load) kv4_load;
    decltype(&striped_attn_decode_kv4) decode;
    decltype(&striped_attn_decode_kv4_workspace_size) decode_size;
    decltype(&striped_attn_key_weight) weight;
    decltype(&striped_attn_key_weight_workspace_size) weight_size;
    decltype(&striped_kv_evict) evict;
} lib{};
PyObject *failed = nullptr;  // failed(status, name) is the exception of a call that failed

// One of the library's calls: false if it refused its arguments, or failed, which is
// then the interpreter's error.  The interpreter's lock is given up for it: a launch
// waits where the GPU's queue is full, perhaps for a host function that needs
// the lock.  (Addresses are taken before that, as arguments of this function.)
template <typename F, typename... A>
bool launched(const char *name, F call, A... args) {
    PyThreadState *state = PyEval_SaveThread();
    const int status = call(args...);
    PyEval_RestoreThread(state);
    if (status == STRIPED_ERR_CUDA) {
        PyObject *e = PyObject_CallFunction(failed, "is", status, name);
        if (e) PyErr_SetObject(reinterpret_cast<PyObject *>(Py_TYPE(e)), e);
        Py_XDECREF(e);
    }
    return status == STRIPED_OK;
}

// One call's tensors: the first one tells the device, which has to be current.
class Call {
  public:
    // A contiguous tensor on the device, of `dims` dimensions; nullptr otherwise.
    const at::Tensor *take(PyObject *o, int dims, at::ScalarType type) {
        if (!THPVariable_CheckExact(o)) return nullptr;
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.dim() != dims || t.scalar_type() != type || t.layout() != at::kStrided ||
            !t.is_contiguous())
            return nullptr;
        if (device_ < 0) {
            device_ = t.get_device();
            if (device_ != c10::cuda::current_device()) return nullptr;
        }
        return t.get_device() == device_ ? &t : nullptr;
    }
    const at::Tensor *take(PyObject *o, at::IntArrayRef shape, at::ScalarType type) {
        const at::Tensor *t = take(o, (int)shape.size(), type);
        return t && t->sizes() == shape ? t : nullptr;
    }
    at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device_));
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device_).stream(); }

  private:
    int device_ = -1;
};

// A whole number, or a number; false if it is none of these (the error is cleared).
bool whole(PyObject *o, int64_t *x) {
    if (!PyLong_Check(o)) return false;
    *x = PyLong_AsLongLong(o);
    if (*x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}
bool whole32(PyObject *o, int *x) {
    int64_t y;
    if (!whole(o, &y) || y < INT32_MIN || y > INT32_MAX) return false;
    *x = (int)y;
    return true;
}
bool scale_of(PyObject *o, int64_t D, float *x) {
    if (o == Py_None) *x = (float)(1.0 / std::sqrt((double)D));
    else if (PyFloat_Check(o)) *x = (float)PyFloat_AS_DOUBLE(o);
    else return false;
    return true;
}

template <typename... T>
PyObject *tuple_of(T... t) {
    PyObject *out = PyTuple_New(sizeof...(T));
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    const bool ok = ((PyTuple_SET_ITEM(out, i, THPVariable_Wrap(std::move(t))), PyTuple_GET_ITEM(out, i++) != nullptr) && ...);
    if (!ok) Py_CLEAR(out);
    return out;
}

// A C++ exception (no memory, say) leaves the case to the wrapper, too.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F &&f) {
    if (n == want && lib.evict) {
        try {
            if (PyObject *r = f()) return r;
            if (PyErr_Occurred()) return nullptr;
        } catch (...) {
        }
    }
    Py_RETURN_NONE;
}

PyObject *kv4_store(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 2, [&]() -> PyObject * {
        Call c;
        const at::Tensor *k = c.take(a[0], 4, at::kBFloat16);
        if (!k) return nullptr;
        const at::Tensor *v = c.take(a[1], k->sizes(), at::kBFloat16);
        const int64_t B = k->size(0), H = k->size(1), S = k->size(2), D = k->size(3);
        if (!v || D % 32 != 0) return nullptr;
        const int64_t cs[4] = {B, H, S, D / 2}, ss[4] = {B, H, S, D / 32};
        at::Tensor kc = c.make(cs, at::kByte), ks = c.make(ss, at::kBFloat16), vc = c.make(cs, at::kByte),
                   vs = c.make(ss, at::kBFloat16);
        if (!launched("striped_kv4_store", lib.kv4_store, k->data_ptr(), v->data_ptr(), kc.data_ptr(), ks.data_ptr(), vc.data_ptr(),
                     vs.data_ptr(), B, H, S, D, STRIPED_BF16, c.stream()))
            return nullptr;
        return tuple_of(kc, ks, vc, vs);
    });
}

PyObject *kv4_load(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject * {
        Call c;
        const at::Tensor *kc = c.take(a[0], 4, at::kByte);
        if (!kc) return nullptr;
        const int64_t B = kc->size(0), H = kc->size(1), S = kc->size(2), D = 2 * kc->size(3);
        const int64_t xs[4] = {B, H, S, D}, ss[4] = {B, H, S, D / 32};
        const at::Tensor *ks = c.take(a[1], ss, at::kBFloat16), *vc = c.take(a[2], kc->sizes(), at::kByte),
                         *vs = c.take(a[3], ss, at::kBFloat16);
        if (!ks || !vc || !vs) return nullptr;
        at::Tensor k = c.make(xs, at::kBFloat16), v = c.make(xs, at::kBFloat16);
        if (!launched("striped_kv4_load", lib.kv4_load, kc->data_ptr(), ks->data_ptr(), vc->data_ptr(), vs->data_ptr(), k.data_ptr(),
                     v.data_ptr(), B, H, S, D, STRIPED_BF16, c.stream()))
            return nullptr;
        return tuple_of(k, v);
    });
}

// q, k_codes, k_scales, v_codes, v_scales, k_tail, v_tail, tail_lens, N, layout, scale
PyObject *decode_kv4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject * {
        Call c;
        const at::Tensor *q = c.take(a[0], 4, at::kBFloat16), *kc = c.take(a[1], 4, at::kByte),
                         *kt = c.take(a[5], 4, at::kBFloat16);
        int N, layout;
        float scale;
        if (!q || !kc || !kt || !whole32(a[8], &N) || !whole32(a[9], &layout) || !scale_of(a[10], q->size(3), &scale))
            return nullptr;
        const int64_t B = q->size(0), H = q->size(1), T = q->size(2), D = q->size(3), Bp = kc->size(0), P = kc->size(2);
        const int64_t Hkv = kt->size(1), C = kt->size(2);
        const int64_t cs[4] = {Bp, Hkv, P, D / 2}, ss[4] = {Bp, Hkv, P, D / 32}, ts[4] = {B, Hkv, C, D}, ls[1] = {B};
        if (kc->sizes() != at::IntArrayRef(cs) || kt->sizes() != at::IntArrayRef(ts)) return nullptr;
        const at::Tensor *ks = c.take(a[2], ss, at::kBFloat16), *vc = c.take(a[3], cs, at::kByte),
                         *vs = c.take(a[4], ss, at::kBFloat16), *vt = c.take(a[6], ts, at::kBFloat16),
                         *lens = c.take(a[7], ls, at::kInt);
        if (!ks || !vc || !vs || !vt || !lens) return nullptr;
        const int64_t bytes = (int64_t)lib.decode_size(B, Bp, H, Hkv, T, P, C, D, N, layout, STRIPED_BF16);
        if (bytes <= 0) return nullptr;
        const int64_t os[4] = {B, H, T, D}, lses[3] = {B, H, T}, wss[1] = {bytes};
        at::Tensor o = c.make(os, at::kBFloat16), lse = c.make(lses, at::kFloat), ws = c.make(wss, at::kByte);
        if (!launched("striped_attn_decode_kv4", lib.decode, q->data_ptr(), kc->data_ptr(), ks->data_ptr(), vc->data_ptr(), vs->data_ptr(),
                     kt->data_ptr(), vt->data_ptr(), static_cast<const int32_t *>(lens->data_ptr()), o.data_ptr(),
                     static_cast<float *>(lse.data_ptr()), ws.data_ptr(), (size_t)bytes, B, Bp, H, Hkv, T, P, C, D, N,
                     layout, STRIPED_BF16, scale, c.stream()))
            return nullptr;
        return tuple_of(o, lse);
    });
}

// q, k, lse, N, layout, first, scale
PyObject *key_weight(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        Call c;
        const at::Tensor *q = c.take(a[0], 4, at::kBFloat16), *k = c.take(a[1], 4, at::kBFloat16);
        int N, layout;
        int64_t first;
        float scale;
        if (!q || !k || !whole32(a[3], &N) || !whole32(a[4], &layout) || !whole(a[5], &first) ||
            !scale_of(a[6], q->size(3), &scale))
            return nullptr;
        const int64_t B = q->size(0), H = q->size(1), S = q->size(2), D = q->size(3), Hkv = k->size(1);
        const int64_t ks[4] = {B, Hkv, S, D}, lses[3] = {B, H, S}, wts[3] = {B, Hkv, S};
        const at::Tensor *lse = c.take(a[2], lses, at::kFloat);
        if (!lse || k->sizes() != at::IntArrayRef(ks)) return nullptr;
        const int64_t bytes = (int64_t)lib.weight_size(B, H, Hkv, S, D, N, layout, STRIPED_BF16, first);
        if (bytes <= 0) return nullptr;
        const int64_t wss[1] = {bytes};
        at::Tensor w = c.make(wts, at::kFloat), ws = c.make(wss, at::kByte);
        if (!launched("striped_attn_key_weight", lib.weight, q->data_ptr(), k->data_ptr(), static_cast<const float *>(lse->data_ptr()),
                     static_cast<float *>(w.data_ptr()), ws.data_ptr(), (size_t)bytes, B, H, Hkv, S, D, N, layout,
                     STRIPED_BF16, first, 0, scale, c.stream()))
            return nullptr;
        return THPVariable_Wrap(std::move(w));
    });
}

// weight, keep, sinks, recent, N, layout, then the tensors
PyObject *kv_evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
    const int m = (int)n - 6;
    return guarded(n, m == 4 ? 10 : 8, [&]() -> PyObject * {
        Call c;
        const at::Tensor *w = c.take(a[0], 3, at::kFloat);
        int64_t keep, sinks, recent;
        int N, layout;
        if (!w || !whole(a[1], &keep) || !whole(a[2], &sinks) || !whole(a[3], &recent) || !whole32(a[4], &N) ||
            !whole32(a[5], &layout))
            return nullptr;
        const int64_t B = w->size(0), H = w->size(1), S = w->size(2);
        if (keep < 1 || keep > S) return nullptr;
        const void *x[4];
        void *y[4];
        int64_t row[4];
        at::Tensor out[4];
        for (int i = 0; i < m; ++i) {
            if (!THPVariable_CheckExact(a[6 + i])) return nullptr;
            const at::Tensor *t = c.take(a[6 + i], 4, THPVariable_Unpack(a[6 + i]).scalar_type());
            if (!t || t->size(0) != B || t->size(1) != H || t->size(2) != S) return nullptr;
            const int64_t os[4] = {B, H, keep, t->size(3)};
            out[i] = c.make(os, t->scalar_type());
            x[i] = t->data_ptr(), y[i] = out[i].data_ptr(), row[i] = t->size(3) * (int64_t)t->element_size();
        }
        const int64_t ks[3] = {B, H, keep};
        at::Tensor index = c.make(ks, at::kInt), weight = c.make(ks, at::kFloat);
        if (!launched("striped_kv_evict", lib.evict, x, y, row, m, static_cast<const float *>(w->data_ptr()),
                     static_cast<int32_t *>(index.data_ptr()), static_cast<float *>(weight.data_ptr()), B, H, S, keep,
                     sinks, recent, N, layout, c.stream()))
            return nullptr;
        return m == 2 ? tuple_of(out[0], out[1], index, weight) : tuple_of(out[0], out[1], out[2], out[3], index, weight);
    });
}

// The library that is loaded already, by its path, and the exception for its
// failures; True if it has all calls.
PyObject *use(PyObject *, PyObject *args) {
    const char *name;
    PyObject *exception;
    if (!PyArg_ParseTuple(args, "sO", &name, &exception)) return nullptr;
    void *h = dlopen(name, RTLD_NOW | RTLD_NOLOAD);
    if (!h) Py_RETURN_FALSE;
    Library l{};
    auto get = [&](auto &f, const char *symbol) {
        f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, symbol));
        return f != nullptr;
    };
    if (!get(l.kv4_store, "striped_kv4_store") || !get(l.kv4_load, "striped_kv4_load") ||
        !get(l.decode, "striped_attn_decode_kv4") || !get(l.decode_size, "striped_attn_decode_kv4_workspace_size") ||
        !get(l.weight, "striped_attn_key_weight") || !get(l.weight_size, "striped_attn_key_weight_workspace_size") ||
        !get(l.evict, "striped_kv_evict"))
        Py_RETURN_FALSE;
    lib = l;
    Py_INCREF(exception);
    Py_XDECREF(failed);
    failed = exception;
    Py_RETURN_TRUE;
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"use", use, METH_VARARGS, nullptr},
                         {"kv4_store", fast(kv4_store), METH_FASTCALL, nullptr},
                         {"kv4_load", fast(kv4_load), METH_FASTCALL, nullptr},
                         {"decode_kv4", fast(decode_kv4), METH_FASTCALL, nullptr},
                         {"key_weight", fast(key_weight), METH_FASTCALL, nullptr},
                         {"kv_evict", fast(kv_evict), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "striped_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_striped_binding() { return PyModule_Create(&module); }
