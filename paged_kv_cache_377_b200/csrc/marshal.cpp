// marshal.cpp -- the Python side of the step's small calls (module _marshal).
//
// A speculative step makes a call of a few microseconds per layer and several
// per step; checking ten tensors in Python took longer than the kernels they
// start. Each function here checks its tensors (type, dtype, dimensions,
// contiguity, device) and their agreement, takes the current stream unless one
// is given, and makes the C call of the same name; it returns that call's code.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "pagedkv.h"

namespace {

using at::ScalarType;

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(PyObject *type, const char *fmt, const char *a, const char *b = "") {
    PyErr_Format(type, fmt, a, b);
    throw Refused();
}

// The tensors of one call: all contiguous, on the same CUDA device, which is the current one.
class Call {
  public:
    Call(PyObject *const *args, Py_ssize_t given, Py_ssize_t wanted) : args_(args) {
        if (given != wanted) {
            PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", wanted, given);
            throw Refused();
        }
    }
    const at::Tensor &tensor(const char *name, ScalarType type, int64_t dims) {
        PyObject *o = args_[at_++];
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be on a CUDA device", name);
        if (t.scalar_type() != type)
            refuse(PyExc_TypeError, "%s must be %s", name, c10::toString(type));
        if (t.dim() != dims) {
            PyErr_Format(PyExc_ValueError, "%s must have %lld dimensions (got %lld)", name, static_cast<long long>(dims),
                         static_cast<long long>(t.dim()));
            throw Refused();
        }
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
        if (device_ < 0) device_ = t.get_device();
        if (t.get_device() != device_) refuse(PyExc_ValueError, "all tensors must be on one device (%s is on another)", name);
        return t;
    }
    bool none() {  // skips an argument that is None
        if (args_[at_] != Py_None) return false;
        ++at_;
        return true;
    }
    int integer() {
        const long long v = PyLong_AsLongLong(args_[at_++]);
        if (v == -1 && PyErr_Occurred()) throw Refused();
        if (v < -0x7fffffffLL || v > 0x7fffffffLL) {
            PyErr_SetString(PyExc_ValueError, "an integer argument does not fit 32 bits");
            throw Refused();
        }
        return static_cast<int>(v);
    }
    float real() {
        const double v = PyFloat_AsDouble(args_[at_++]);
        if (v == -1.0 && PyErr_Occurred()) throw Refused();
        return static_cast<float>(v);
    }
    // The last argument: None, a torch.cuda.Stream or a handle. Also the check of the device.
    void *stream() {
        if (c10::cuda::current_device() != device_) {
            PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%d, not on the current device", static_cast<int>(device_));
            throw Refused();
        }
        PyObject *o = args_[at_++];
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream();
        PyObject *handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        if (!handle) throw Refused();
        void *p = PyLong_AsVoidPtr(handle);
        Py_DECREF(handle);
        if (PyErr_Occurred()) throw Refused();
        return p;
    }

  private:
    PyObject *const *args_;
    Py_ssize_t at_ = 0;
    int64_t device_ = -1;
};

int size(const at::Tensor &t, int64_t d) {
    const int64_t n = t.size(d);
    if (n > 0x7fffffff) {
        PyErr_SetString(PyExc_ValueError, "a tensor's dimension does not fit 32 bits");
        throw Refused();
    }
    return static_cast<int>(n);
}

int32_t *i32(const at::Tensor &t) { return static_cast<int32_t *>(t.data_ptr()); }

void agree(bool ok, const char *what) {
    if (!ok) refuse(PyExc_ValueError, "%s", what);
}

template <typename F>
PyObject *guarded(F &&call) {
    try {
        return PyLong_FromLong(call());
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

int tree(Call c, bool fp8) {
    const ScalarType pool = fp8 ? ScalarType::Byte : ScalarType::BFloat16;
    const at::Tensor &out = c.tensor("out", ScalarType::BFloat16, 3), &q = c.tensor("q", ScalarType::BFloat16, 3),
                     &k = c.tensor("k_cache", pool, 4), &v = c.tensor("v_cache", pool, 4);
    const float *scales[2] = {nullptr, nullptr};
    if (fp8) {
        const at::Tensor &ks = c.tensor("k_scale", ScalarType::Float, 1), &vs = c.tensor("v_scale", ScalarType::Float, 1);
        agree(ks.size(0) == k.size(2) && vs.size(0) == k.size(2), "k_scale and v_scale must have num_kv_heads entries");
        scales[0] = static_cast<const float *>(ks.data_ptr());
        scales[1] = static_cast<const float *>(vs.data_ptr());
    }
    const at::Tensor &bt = c.tensor("block_tables", ScalarType::Int, 2), &cl = c.tensor("context_lens", ScalarType::Int, 1),
                     &qs = c.tensor("query_start", ScalarType::Int, 1), &mask = c.tensor("tree_mask", ScalarType::Int, 2);
    const int max_query_len = c.integer();
    const float scale = c.real();
    const at::Tensor &ws = c.tensor("workspace", ScalarType::Byte, 1);
    void *stream = c.stream();
    const int S = size(bt, 0), MB = size(bt, 1), T = size(q, 0), Hq = size(q, 1), D = size(q, 2);
    const int NB = size(k, 0), bs = size(k, 1), Hkv = size(k, 2);
    agree(out.sizes() == q.sizes() && v.sizes() == k.sizes() && k.size(3) == D,
          "shape mismatch between q/out or k_cache/v_cache");
    agree(cl.size(0) == S && qs.size(0) == S + int64_t(1) && mask.size(0) == T,
          "context_lens needs num_seqs entries, query_start num_seqs + 1 and tree_mask num_tokens rows");
    if (fp8)
        return paged_attn_tree_fp8(out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), scales[0], scales[1], i32(bt),
                                   i32(cl), i32(qs), i32(mask), size(mask, 1), S, T, max_query_len, Hq, Hkv, D, bs, scale,
                                   MB, NB, ws.data_ptr(), ws.numel(), stream);
    return paged_attn_tree(out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), i32(bt), i32(cl), i32(qs), i32(mask),
                           size(mask, 1), S, T, max_query_len, Hq, Hkv, D, bs, scale, MB, NB, ws.data_ptr(), ws.numel(),
                           stream);
}

PyObject *py_tree(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&] { return tree(Call(args, n, 12), false); });
}

PyObject *py_tree_fp8(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&] { return tree(Call(args, n, 14), true); });
}

PyObject *py_mask(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 7);
        const at::Tensor &mask = c.tensor("tree_mask", ScalarType::Int, 2), &depths = c.tensor("depths", ScalarType::Int, 1),
                         &parents = c.tensor("parents", ScalarType::Int, 1),
                         &qs = c.tensor("query_start", ScalarType::Int, 1);
        const int max_query_len = c.integer();
        const at::Tensor &status = c.tensor("status", ScalarType::Int, 1);
        void *stream = c.stream();
        const int T = size(parents, 0);
        agree(mask.size(0) == T && depths.size(0) == T && qs.size(0) >= 1 && status.size(0) >= 1,
              "tree_mask and depths need a row per token, query_start num_seqs + 1 entries, status one");
        return paged_tree_mask(i32(mask), i32(depths), i32(parents), i32(qs), size(qs, 0) - 1, T, max_query_len,
                               size(mask, 1), i32(status), stream);
    });
}

PyObject *py_grow(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 12);
        const at::Tensor &bt = c.tensor("block_tables", ScalarType::Int, 2), &cl = c.tensor("context_lens", ScalarType::Int, 1),
                         &add = c.tensor("new_tokens", ScalarType::Int, 1), &free = c.tensor("free_blocks", ScalarType::Int, 1),
                         &top = c.tensor("num_free", ScalarType::Int, 1), &lens = c.tensor("new_lens", ScalarType::Int, 1),
                         &qs = c.tensor("query_start", ScalarType::Int, 1),
                         &slots = c.tensor("slot_mapping", ScalarType::Long, 1),
                         &left = c.tensor("num_free_out", ScalarType::Int, 1);
        const int bs = c.integer();
        const at::Tensor &status = c.tensor("status", ScalarType::Int, 1);
        void *stream = c.stream();
        const int S = size(bt, 0);
        agree(cl.size(0) == S && add.size(0) == S && lens.size(0) == S && qs.size(0) == S + int64_t(1) && top.size(0) == 1 &&
                  left.size(0) == 1 && status.size(0) >= 1,
              "context_lens, new_tokens and new_lens need num_seqs entries, query_start num_seqs + 1, num_free, "
              "num_free_out and status one");
        return kv_tables_grow(i32(bt), i32(cl), i32(add), i32(free), i32(top), i32(lens), i32(qs),
                              static_cast<int64_t *>(slots.data_ptr()), i32(left), S, size(slots, 0), size(bt, 1), bs,
                              size(free, 0), i32(status), stream);
    });
}

PyObject *py_trim(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 9);
        const at::Tensor &bt = c.tensor("block_tables", ScalarType::Int, 2), &cl = c.tensor("context_lens", ScalarType::Int, 1),
                         &keep = c.tensor("keep_lens", ScalarType::Int, 1), &free = c.tensor("free_blocks", ScalarType::Int, 1),
                         &top = c.tensor("num_free", ScalarType::Int, 1), &left = c.tensor("num_free_out", ScalarType::Int, 1);
        const int bs = c.integer();
        const at::Tensor &status = c.tensor("status", ScalarType::Int, 1);
        void *stream = c.stream();
        const int S = size(bt, 0);
        agree(cl.size(0) == S && keep.size(0) == S && top.size(0) == 1 && left.size(0) == 1 && status.size(0) >= 1,
              "context_lens and keep_lens need num_seqs entries, num_free, num_free_out and status one");
        return kv_tables_trim(i32(bt), i32(cl), i32(keep), i32(free), i32(top), i32(left), S, size(bt, 1), bs, size(free, 0),
                              i32(status), stream);
    });
}

PyObject *py_keep(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&] {
        Call c(args, n, 10);
        const bool codes = n > 0 && THPVariable_Check(args[0]) &&
                           THPVariable_Unpack(args[0]).scalar_type() == ScalarType::Byte;
        const ScalarType pool = codes ? ScalarType::Byte : ScalarType::BFloat16;
        const at::Tensor &k = c.tensor("k_cache", pool, 4), &v = c.tensor("v_cache", pool, 4),
                         &bt = c.tensor("block_tables", ScalarType::Int, 2), &cl = c.tensor("context_lens", ScalarType::Int, 1),
                         &qs = c.tensor("query_start", ScalarType::Int, 1), &acc = c.tensor("accepted", ScalarType::Int, 2),
                         &num = c.tensor("num_accepted", ScalarType::Int, 1);
        const int S = size(bt, 0);
        int32_t *lens = nullptr;
        if (!c.none()) {
            const at::Tensor &t = c.tensor("new_lens", ScalarType::Int, 1);
            agree(t.size(0) == S, "new_lens needs num_seqs entries");
            lens = i32(t);
        }
        const at::Tensor &status = c.tensor("status", ScalarType::Int, 1);
        void *stream = c.stream();
        agree(v.sizes() == k.sizes(), "shape mismatch between k_cache and v_cache");
        agree(cl.size(0) == S && qs.size(0) == S + int64_t(1) && acc.size(0) == S && num.size(0) == S && status.size(0) >= 1,
              "context_lens, accepted and num_accepted need num_seqs rows, query_start num_seqs + 1, status one");
        return kv_cache_keep(k.data_ptr(), v.data_ptr(), i32(bt), i32(cl), i32(qs), i32(acc), i32(num), lens, S, size(acc, 1),
                             size(k, 2), size(k, 3), codes ? 1 : 2, size(k, 1), size(bt, 1), size(k, 0), i32(status), stream);
    });
}

#define ENTRY(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {ENTRY("paged_attn_tree", py_tree), ENTRY("paged_attn_tree_fp8", py_tree_fp8),
                         ENTRY("paged_tree_mask", py_mask), ENTRY("kv_tables_grow", py_grow),
                         ENTRY("kv_tables_trim", py_trim),  ENTRY("kv_cache_keep", py_keep),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
