// token_calls.cpp - the quick way from Python to the token operators: a CPython module that
// looks at the tensors of an ordinary call (every one of the shape, type and device that the
// configuration says) and makes it, without ctypes.  Anything else it leaves alone and returns
// None: pbsa.py then says what is wrong, or makes the call itself.  A token's call is mostly
// host time: norm and rotation of one token took 7 us in Python's checks and ctypes.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "pbsa.h"

namespace {

struct Call {
    int dev;
    bool ok = true, whole = true;   // everything fits; all strided tensors are contiguous
    int64_t strides[18];
    int n_strides = 0;

    const at::Tensor* tensor(PyObject* o, at::ScalarType dt, std::initializer_list<int64_t> shape) {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor& t = THPVariable_Unpack(o);
        ok = t.layout() == at::kStrided && t.scalar_type() == dt && t.is_cuda() && t.get_device() == dev &&
             t.sizes() == at::IntArrayRef(shape.begin(), shape.size());
        return ok ? &t : nullptr;
    }
    // A contiguous tensor's memory.
    void* need(PyObject* o, at::ScalarType dt, std::initializer_list<int64_t> shape) {
        const at::Tensor* t = tensor(o, dt, shape);
        if (!t || !(ok = t->is_contiguous())) return nullptr;
        return t->data_ptr();
    }
    void* may(PyObject* o, at::ScalarType dt, std::initializer_list<int64_t> shape) {
        return o == Py_None ? nullptr : need(o, dt, shape);
    }
    // A [B, T, H, D] tensor of contiguous channels; an output's elements must be its own.
    void* heads(PyObject* o, at::ScalarType dt, int64_t B, int64_t T, int64_t H, int64_t D, bool output = false) {
        int64_t* s = strides + n_strides;
        n_strides += 3;
        s[0] = s[1] = s[2] = 0;
        if (H == 0) return nullptr;
        const at::Tensor* t = tensor(o, dt, {B, T, H, D});
        if (!t) return nullptr;
        ok = t->stride(3) == 1;
        for (int i = 0; i < 3; ++i) {
            s[i] = t->size(i) == 1 ? 0 : t->stride(i);   // of one element the stride says nothing
            ok = ok && !(output && s[i] == 0 && t->size(i) > 1);
        }
        whole = whole && t->is_contiguous();
        return ok ? t->data_ptr() : nullptr;
    }
    const int64_t* used_strides() const { return whole ? nullptr : strides; }
    void* workspace(PyObject* o, size_t& bytes) {
        bytes = 0;
        if (!ok || o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor& t = THPVariable_Unpack(o);
        ok = t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev && t.is_contiguous();
        if (!ok) return nullptr;
        bytes = t.nbytes();
        return t.data_ptr();
    }
};

at::ScalarType type_of(int dtype) {
    switch (dtype) {
        case PBSA_DTYPE_BF16: return at::kBFloat16;
        case PBSA_DTYPE_FP16: return at::kHalf;
        case PBSA_DTYPE_FP32: return at::kFloat;
        default: return at::ScalarType::Undefined;
    }
}

template <typename T>
T* as(void* p) { return static_cast<T*>(p); }

// Arguments of every call: configuration's address, device, stream, then `body`'s own.
template <typename Config, typename Body>
PyObject* make(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, Body body) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        const Config* cfg = static_cast<const Config*>(PyLong_AsVoidPtr(args[0]));
        const long dev = PyLong_AsLong(args[1]);
        void* stream = PyLong_AsVoidPtr(args[2]);
        if (PyErr_Occurred()) {   // a stream of another kind
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        Call c;
        c.dev = static_cast<int>(dev);
        int rc = 0;
        if (dev < 0 || !body(c, *cfg, stream, args + 3, rc)) Py_RETURN_NONE;
        return PyLong_FromLong(rc);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

struct Shared {   // of both directions of norm and rotation
    void *wq, *wk, *cos = nullptr, *sin = nullptr, *pos = nullptr, *status;

    Shared(Call& c, const pbsa_qk_config& g, PyObject* const* a, PyObject* st) {   // wq, wk, cos, sin, pos
        wq = c.may(a[0], at::kFloat, {g.D});
        wk = c.may(a[1], at::kFloat, {g.D});
        if (g.rot_dim > 0) {
            cos = c.need(a[2], at::kFloat, {g.table_len, g.rot_dim / 2});
            sin = c.need(a[3], at::kFloat, {g.table_len, g.rot_dim / 2});
            pos = c.need(a[4], at::kInt, {g.B, g.T, g.n_axes});
            status = c.need(st, at::kInt, {1});
        } else {
            status = c.may(st, at::kInt, {1});
        }
    }
};

PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return make<pbsa_qk_config>(args, n, 13, [](Call& c, const pbsa_qk_config& g, void* stream, PyObject* const* a, int& rc) {
        const at::ScalarType dt = type_of(g.dtype);
        void* q = c.heads(a[0], dt, g.B, g.T, g.Hq, g.D);
        void* k = c.heads(a[1], dt, g.B, g.T, g.Hkv, g.D);
        void* qo = c.heads(a[7], dt, g.B, g.T, g.Hq, g.D, true);
        void* ko = c.heads(a[8], dt, g.B, g.T, g.Hkv, g.D, true);
        const Shared s(c, g, a + 2, a[9]);
        if (!c.ok) return false;
        rc = pbsa_qk_norm_rope(&g, q, k, c.used_strides(), as<float>(s.wq), as<float>(s.wk), as<float>(s.cos),
                               as<float>(s.sin), as<int32_t>(s.pos), qo, ko, as<int32_t>(s.status), stream);
        return true;
    });
}

PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return make<pbsa_qk_config>(args, n, 18, [](Call& c, const pbsa_qk_config& g, void* stream, PyObject* const* a, int& rc) {
        const at::ScalarType dt = type_of(g.dtype), gt = type_of(g.grad_dtype);
        void* q = c.heads(a[0], dt, g.B, g.T, g.Hq, g.D);
        void* k = c.heads(a[1], dt, g.B, g.T, g.Hkv, g.D);
        void* dqo = c.heads(a[7], gt, g.B, g.T, g.Hq, g.D);
        void* dko = c.heads(a[8], gt, g.B, g.T, g.Hkv, g.D);
        void* dq = c.heads(a[9], dt, g.B, g.T, g.Hq, g.D, true);
        void* dk = c.heads(a[10], dt, g.B, g.T, g.Hkv, g.D, true);
        const Shared s(c, g, a + 2, a[14]);
        void* dwq = c.may(a[11], at::kFloat, {g.D});
        void* dwk = c.may(a[12], at::kFloat, {g.D});
        size_t bytes;
        void* ws = c.workspace(a[13], bytes);
        if (!c.ok) return false;
        rc = pbsa_qk_norm_rope_bwd(&g, q, k, c.used_strides(), as<float>(s.wq), as<float>(s.wk), as<float>(s.cos),
                                   as<float>(s.sin), as<int32_t>(s.pos), dqo, dko, dq, dk, as<float>(dwq), as<float>(dwk),
                                   ws, bytes, as<int32_t>(s.status), stream);
        return true;
    });
}

// The calls over a cache: its struct's address comes first.
const pbsa_kv4_cache* cache_of(PyObject* o) { return static_cast<const pbsa_kv4_cache*>(PyLong_AsVoidPtr(o)); }

// Size of a dimension of a tensor, -1 where there is none.
int64_t size_of(PyObject* o, int dim) {
    if (!THPVariable_Check(o)) return -1;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.dim() > dim && t.size(dim) <= INT_MAX ? t.size(dim) : -1;
}

PyObject* kv4_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return make<pbsa_kv4_config>(args, n, 10, [](Call& c, const pbsa_kv4_config& g, void* stream, PyObject* const* a, int& rc) {
        const at::ScalarType dt = type_of(g.dtype);
        const int64_t T = size_of(a[1], 1);
        void* k = c.heads(a[1], dt, g.B, T, g.Hkv, g.D);
        void* v = c.heads(a[2], dt, g.B, T, g.Hkv, g.D);
        void* pos = c.need(a[3], at::kInt, {g.B, T});
        void* rows = c.may(a[4], at::kInt, {g.B, g.Hkv, T});
        void* mass = c.may(a[5], at::kFloat, {g.B, g.Hkv, g.capacity});
        void* status = c.need(a[6], at::kInt, {1});
        if (!c.ok) return false;
        rc = pbsa_kv4_append(&g, cache_of(a[0]), k, v, c.used_strides(), static_cast<int>(T), as<int32_t>(pos),
                             as<int32_t>(rows), as<float>(mass), as<int32_t>(status), stream);
        return true;
    });
}

PyObject* kv4_read(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return make<pbsa_kv4_config>(args, n, 8, [](Call& c, const pbsa_kv4_config& g, void* stream, PyObject* const* a, int& rc) {
        const at::ScalarType dt = type_of(g.dtype);
        const int64_t m = size_of(a[2], 2);
        void* rows = c.may(a[1], at::kInt, {g.B, g.Hkv, m});
        void* k = c.need(a[2], dt, {g.B, g.Hkv, m, g.D});
        void* v = c.need(a[3], dt, {g.B, g.Hkv, m, g.D});
        void* status = c.need(a[4], at::kInt, {1});
        if (!c.ok) return false;
        rc = pbsa_kv4_read(&g, cache_of(a[0]), as<int32_t>(rows), static_cast<int>(m), k, v, as<int32_t>(status), stream);
        return true;
    });
}

PyObject* kv4_attn(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return make<pbsa_kv4_config>(args, n, 12, [](Call& c, const pbsa_kv4_config& g, void* stream, PyObject* const* a, int& rc) {
        const at::ScalarType dt = type_of(g.dtype);
        const int64_t T = size_of(a[1], 1);
        void* q = c.heads(a[1], dt, g.B, T, g.Hq, g.D);
        void* q_pos = c.may(a[2], at::kInt, {g.B, T});
        void* len = c.need(a[3], at::kInt, {g.B});
        void* out = c.need(a[4], dt, {g.B, T, g.Hq, g.D});
        void* lse = c.need(a[5], at::kFloat, {g.B, g.Hq, T});
        void* mass = c.may(a[6], at::kFloat, {g.B, g.Hkv, g.capacity});
        size_t bytes;
        void* ws = c.workspace(a[7], bytes);
        void* status = c.need(a[8], at::kInt, {1});
        if (!c.ok) return false;
        rc = pbsa_kv4_attn(&g, cache_of(a[0]), q, c.used_strides(), static_cast<int>(T), as<int32_t>(q_pos),
                           as<int32_t>(len), out, as<float>(lse), as<float>(mass), ws, bytes, as<int32_t>(status), stream);
        return true;
    });
}

PyObject* kv4_evict(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return make<pbsa_kv4_config>(args, n, 9, [](Call& c, const pbsa_kv4_config& g, void* stream, PyObject* const* a, int& rc) {
        const int64_t m = size_of(a[4], 2);
        void* pos = c.need(a[0], at::kInt, {g.B, g.Hkv, g.capacity});
        void* mass = c.need(a[1], at::kFloat, {g.B, g.Hkv, g.capacity});
        const long sink = PyLong_AsLong(a[2]);
        if (PyErr_Occurred()) {   // pbsa.py's call says what is wrong with it
            PyErr_Clear();
            return false;
        }
        void* keep = c.may(a[3], at::kInt, {g.B});
        void* rows = c.need(a[4], at::kInt, {g.B, g.Hkv, m});
        void* status = c.need(a[5], at::kInt, {1});
        if (!c.ok || sink < INT_MIN || sink > INT_MAX) return false;
        rc = pbsa_kv4_evict(&g, as<int32_t>(pos), as<float>(mass), static_cast<int>(m), static_cast<int>(sink),
                            as<int32_t>(keep), as<int32_t>(rows), as<int32_t>(status), stream);
        return true;
    });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(qk_norm_rope), FAST(qk_norm_rope_bwd), FAST(kv4_append), FAST(kv4_read),
                         FAST(kv4_attn), FAST(kv4_evict), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "token_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The torch whose tensors this reads: pbsa.py takes no other's, build.py builds again for another.
#define MARK "token_calls for torch "
const char* const mark = MARK TORCH_VERSION_BUILT;

PyMODINIT_FUNC PyInit_token_calls() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", mark + sizeof(MARK) - 1)) Py_CLEAR(m);
    return m;
}
