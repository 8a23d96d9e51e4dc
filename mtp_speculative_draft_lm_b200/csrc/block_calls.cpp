// The block cache's calls from torch tensors (the module _block): each function checks its
// tensors as api.py documents and makes one call of the C ABI, whose addresses it is given.
//
// A step of a few tokens runs for 3 to 8 us on the device, and eager callers make one of these
// calls per layer: the same checks and the call through ctypes took 9 us (append, evict) to 14
// (attention) of host time, of which the launches themselves are 3 to 6.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <sstream>
#include <stdexcept>
#include <string>

#include "mtp.h"

namespace {

using c10::ScalarType;

struct Abi {
    decltype(&mtp_block_append) append;
    decltype(&mtp_block_attn_ws_bytes) attn_ws_bytes;
    decltype(&mtp_block_attn) attn;
    decltype(&mtp_block_select_ws_bytes) select_ws_bytes;
    decltype(&mtp_block_select) select;
    decltype(&mtp_block_sparse_attn_ws_bytes) sparse_attn_ws_bytes;
    decltype(&mtp_block_sparse_attn) sparse_attn;
    decltype(&mtp_block_evict) evict;
} abi;

struct Refused : std::runtime_error {  // becomes a ValueError
    using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python error is set
struct Unlocked {  // other Python threads run while a call is made (a full launch queue makes it wait)
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// The call's arguments in order.
struct Args {
    PyObject* const* at;
    PyObject* next() { return *at++; }
    const at::Tensor* tensor() {  // None: null
        PyObject* o = next();
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) throw Refused("expected a tensor or None");
        return &THPVariable_Unpack(o);
    }
    int64_t integer() {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw Raised();
        return v;
    }
    int32_t small() {
        const int64_t v = integer();
        if (v != (int32_t)v) throw Refused("an argument does not fit 32 bits");
        return (int32_t)v;
    }
    double real() {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw Raised();
        return v;
    }
    void* stream(int64_t device) {  // None: the current one of the device
        if (*at != Py_None) return address();
        ++at;
        return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    }
    void* address() {  // None: null
        PyObject* o = next();
        if (o == Py_None) return nullptr;
        void* p = PyLong_AsVoidPtr(o);
        if (!p && PyErr_Occurred()) throw Raised();
        return p;
    }
};

// Null stays null; else the data of a contiguous tensor of this type, size and device.
void* need(const at::Tensor* t, ScalarType type, int64_t numel, int64_t device) {
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->numel() != numel || t->get_device() != device || !t->is_contiguous()) {
        std::ostringstream s;
        s << "expected a contiguous " << type << " tensor of " << numel << " elements on device " << device << ", got "
          << t->scalar_type() << " " << t->sizes() << " on " << t->device();
        throw Refused(s.str());
    }
    return t->data_ptr();
}

// Elements between the tokens of x [B, T, heads, hd], whose heads are packed.
int64_t token_stride(const at::Tensor& x) {
    if (x.dim() != 4 || x.scalar_type() != ScalarType::BFloat16 || x.stride(3) != 1 || (x.size(2) > 1 && x.stride(2) != x.size(3)))
        throw Refused("expected bf16 [B, T, heads, hd] with packed heads");
    const int64_t B = x.size(0), T = x.size(1);
    const int64_t step = T > 1 ? x.stride(1) : B > 1 ? x.stride(0) : x.size(2) * x.size(3);
    if (B > 1 && x.stride(0) != T * step) throw Refused("sequences must be T token strides apart");
    return step;
}

// What every call over a cache begins with: (descriptor, device, tokens x [B, T, heads, hd],
// block_table, seq_lens, q_lens, dev_err, stream).
struct Call {
    const mtp_block_cache* cache;
    int64_t device;
    const at::Tensor* x;
    int64_t B, T, heads, step, n_table;
    const int32_t *table, *lens, *q_lens;
    int32_t* err;
    void* stream;

    explicit Call(Args& a) {
        cache = static_cast<const mtp_block_cache*>(a.address());
        device = a.integer();
        x = a.tensor();
        const at::Tensor *t = a.tensor(), *l = a.tensor(), *q = a.tensor(), *e = a.tensor();
        if (!cache || !x || !t || !l) throw Refused("tokens, block_table and seq_lens are needed");
        if (x->get_device() != device || device < 0 || device != c10::cuda::current_device())
            throw Refused("the cache is on device " + std::to_string(device) + ", the tokens on " + std::to_string(x->get_device()) +
                          "; both must be the current one");
        stream = a.stream(device);
        step = token_stride(*x);
        B = x->size(0), T = x->size(1), heads = x->size(2);
        if (x->size(3) != cache->hd)
            throw Refused("heads of " + std::to_string(x->size(3)) + ", the cache's of " + std::to_string(cache->hd));
        if (t->dim() != 2) throw Refused("block_table must be [B, n_table]");
        if (B != (int32_t)B || T != (int32_t)T || heads != (int32_t)heads) throw Refused("a size does not fit 32 bits");
        n_table = t->size(1);
        table = static_cast<const int32_t*>(need(t, ScalarType::Int, B * n_table, device));
        lens = static_cast<const int32_t*>(need(l, ScalarType::Int, B, device));
        q_lens = static_cast<const int32_t*>(need(q, ScalarType::Int, B, device));
        err = static_cast<int32_t*>(need(e, ScalarType::Int, 1, device));
    }
    float scale(PyObject* o) const {
        if (o == Py_None) return (float)(1.0 / std::sqrt((double)cache->hd));
        Args a{&o};
        return (float)a.real();
    }
};

// A call with a workspace: the bytes it needs where ws is null or smaller (nothing is launched),
// else minus the call's status.
template <class F>
int64_t with_ws(const at::Tensor* ws, size_t bytes, int64_t device, const F& call) {
    if (!ws || ws->nbytes() < bytes) return (int64_t)(bytes ? bytes : 1);
    if (ws->get_device() != device || !ws->is_contiguous()) throw Refused("ws must be contiguous on the cache's device");
    void* at = ws->data_ptr();
    const Unlocked u;
    return -(int64_t)call(at, ws->nbytes());
}

template <class F>
PyObject* guarded(const char* name, Py_ssize_t n, Py_ssize_t want, const F& f) {
    if (n != want) return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, want);
    try {
        return PyLong_FromLongLong(f());
    } catch (const Raised&) {
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* py_stride(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("token_stride", n, 1, [&]() -> int64_t {
        const at::Tensor* x = Args{args}.tensor();
        if (!x) throw Refused("expected a tensor");
        return token_stride(*x);
    });
}

// (call, v)
PyObject* py_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("append", n, 9, [&]() -> int64_t {
        Args a{args};
        const Call c(a);
        const at::Tensor* v = a.tensor();
        if (!v || v->sizes() != c.x->sizes() || c.heads != c.cache->nkv || v->get_device() != c.device || token_stride(*v) != c.step)
            throw Refused("k and v must be the cache's heads with one token stride, on its device");
        const uint16_t *ka = static_cast<const uint16_t*>(c.x->data_ptr()), *va = static_cast<const uint16_t*>(v->data_ptr());
        const Unlocked u;
        return -(int64_t)abi.append(c.cache, ka, va, c.step, (int32_t)c.B, c.T, c.lens, c.q_lens, c.table, c.n_table, c.err, c.stream);
    });
}

// (call, scale, out, out_lse, mass, out_mass, ws)
PyObject* py_attn(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("attn", n, 14, [&]() -> int64_t {
        Args a{args};
        const Call c(a);
        const float scale = c.scale(a.next());
        void* out = need(a.tensor(), ScalarType::BFloat16, c.x->numel(), c.device);
        void* lse = need(a.tensor(), ScalarType::Float, c.B * c.T * c.heads, c.device);
        void* mass = need(a.tensor(), ScalarType::Float, c.B * c.n_table, c.device);
        void* out_mass = need(a.tensor(), ScalarType::Float, c.B * c.n_table, c.device);
        const int32_t B = (int32_t)c.B, T = (int32_t)c.T, nq = (int32_t)c.heads;
        return with_ws(a.tensor(), abi.attn_ws_bytes(c.cache, B, T, nq, c.n_table, out_mass != nullptr), c.device,
                       [&](void* ws, size_t bytes) {
                           return abi.attn(c.cache, static_cast<const uint16_t*>(c.x->data_ptr()), c.step, B, T, nq, c.lens, c.q_lens,
                                           c.table, c.n_table, scale, static_cast<uint16_t*>(out), static_cast<float*>(lse),
                                           static_cast<const float*>(mass), static_cast<float*>(out_mass), c.err, ws, bytes,
                                           c.stream);
                       });
    });
}

// (call, n_sel, n_first, n_last, out, ws)
PyObject* py_select(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("select", n, 13, [&]() -> int64_t {
        Args a{args};
        const Call c(a);
        const int32_t n_sel = a.small(), n_first = a.small(), n_last = a.small();
        void* out = need(a.tensor(), ScalarType::Int, c.B * c.T * c.cache->nkv * n_sel, c.device);
        const int32_t B = (int32_t)c.B, T = (int32_t)c.T;
        return with_ws(a.tensor(), abi.select_ws_bytes(c.cache, B, T, c.n_table), c.device, [&](void* ws, size_t bytes) {
            return abi.select(c.cache, static_cast<const uint16_t*>(c.x->data_ptr()), c.step, B, T, (int32_t)c.heads, c.lens, c.q_lens,
                              c.table, c.n_table, n_sel, n_first, n_last, static_cast<int32_t*>(out), c.err, ws, bytes,
                              c.stream);
        });
    });
}

// (call, sel, scale, out, out_lse, ws)
PyObject* py_sparse_attn(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("sparse_attn", n, 13, [&]() -> int64_t {
        Args a{args};
        const Call c(a);
        const at::Tensor* sel = a.tensor();
        if (!sel || sel->dim() != 4 || sel->size(3) != (int32_t)sel->size(3)) throw Refused("sel must be [B, T, nkv, n_sel]");
        const int32_t n_sel = (int32_t)sel->size(3), B = (int32_t)c.B, T = (int32_t)c.T, nq = (int32_t)c.heads;
        void* list = need(sel, ScalarType::Int, c.B * c.T * c.cache->nkv * n_sel, c.device);
        const float scale = c.scale(a.next());
        void* out = need(a.tensor(), ScalarType::BFloat16, c.x->numel(), c.device);
        void* lse = need(a.tensor(), ScalarType::Float, c.B * c.T * c.heads, c.device);
        return with_ws(a.tensor(), abi.sparse_attn_ws_bytes(c.cache, B, T, nq, n_sel), c.device, [&](void* ws, size_t bytes) {
            return abi.sparse_attn(c.cache, static_cast<const uint16_t*>(c.x->data_ptr()), c.step, B, T, nq, c.lens, c.q_lens, c.table,
                                   c.n_table, static_cast<const int32_t*>(list), n_sel, scale, static_cast<uint16_t*>(out),
                                   static_cast<float*>(lse), c.err, ws, bytes, c.stream);
        });
    });
}

// (block_table, seq_lens, mass, block_size, keep, n_first, n_last, out_table, out_lens, out_mass,
//  freed, n_freed, stream)
PyObject* py_evict(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("evict", n, 13, [&]() -> int64_t {
        Args a{args};
        const at::Tensor *table = a.tensor(), *lens = a.tensor(), *mass = a.tensor();
        const int32_t bs = a.small(), keep = a.small(), n_first = a.small(), n_last = a.small();
        if (!table || table->dim() != 2 || table->size(0) != (int32_t)table->size(0)) throw Refused("block_table must be [B, n_table]");
        const int64_t B = table->size(0), n_table = table->size(1), device = table->get_device();
        if (device < 0 || device != c10::cuda::current_device())
            throw Refused("block_table is on device " + std::to_string(device) + ", which must be the current one");
        auto ints = [&](const at::Tensor* t, int64_t numel) { return static_cast<int32_t*>(need(t, ScalarType::Int, numel, device)); };
        auto floats = [&](const at::Tensor* t) { return static_cast<float*>(need(t, ScalarType::Float, B * n_table, device)); };
        const int32_t* table_at = ints(table, B * n_table);
        const int32_t* lens_at = ints(lens, B);
        const float* mass_at = floats(mass);
        int32_t* out_table = ints(a.tensor(), B * n_table);
        int32_t* out_lens = ints(a.tensor(), B);
        float* out_mass = floats(a.tensor());
        int32_t* freed = ints(a.tensor(), B * n_table);
        int32_t* n_freed = ints(a.tensor(), B);
        void* stream = a.stream(device);
        const Unlocked u;
        return -(int64_t)abi.evict((int32_t)B, table_at, n_table, lens_at, mass_at, bs, keep, n_first, n_last, out_table, out_lens,
                                   out_mass, freed, n_freed, stream);
    });
}

// The addresses of the functions of Abi, in its order.
PyObject* py_init(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded("init", n, sizeof(Abi) / sizeof(void*), [&]() -> int64_t {
        Args a{args};
        void* at[sizeof(Abi) / sizeof(void*)];
        for (void*& p : at)
            if (!(p = a.address())) throw Refused("a null address");
        static_assert(sizeof(at) == sizeof(abi));
        __builtin_memcpy(&abi, at, sizeof(abi));
        return 0;
    });
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("init", py_init),     FAST("token_stride", py_stride), FAST("append", py_append),
                         FAST("attn", py_attn),     FAST("select", py_select),       FAST("sparse_attn", py_sparse_attn),
                         FAST("evict", py_evict),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
