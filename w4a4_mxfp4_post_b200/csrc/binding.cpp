// binding.cpp -- ordinary calls of the few-token operators, straight from torch
// tensors to the C ABI.
//
// These calls are made once per layer and token, and their kernels run for a few
// microseconds: the checks, allocations and argument conversions of the Python
// binding took longer than the launch.  Each function here takes the tensors of
// a call without `out`, `workspace` and `stream`, checks them as the Python
// binding does, allocates and calls the library.  It returns the result, or the
// library's error status, or None where anything is out of the ordinary (a wrong
// type or shape, another device than the current one, a tensor of a subclass):
// then the Python binding does the call, or says what is wrong with it.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <array>
#include <cmath>

#include "kroquant.h"

namespace {

// The library's functions, by address: this file does not link to it.
decltype(&mxf4_gemv) p_gemv;
decltype(&mxf4_gemv_workspace) p_gemv_workspace;
decltype(&kq_sf_bytes) p_sf_bytes;
decltype(&mx_cache_write) p_write;
decltype(&mx_cache_read) p_read;
decltype(&mx_paged_attention) p_attention;
decltype(&mx_attention_workspace) p_attention_workspace;

// Without the interpreter's lock, as ctypes calls: a launch waits where the queue is full.
template <class F, class... A>
int unlocked(F f, A... args)
{
    PyThreadState *state = PyEval_SaveThread();
    const int rc = f(args...);
    PyEval_RestoreThread(state);
    return rc;
}

// The tensor of a Python argument; NULL if it is none (or of a subclass).
const at::Tensor *tensor(PyObject *o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

struct Device {
    int index = -1;

    bool set(const at::Tensor &t)
    {
        if (!t.is_cuda()) return false;
        index = t.get_device();
        return index == c10::cuda::current_device();
    }
    bool has(const at::Tensor *t, at::ScalarType type) const
    {
        return t && t->is_cuda() && t->get_device() == index && t->scalar_type() == type;
    }
    cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(index)).stream(); }
};

// The arrays of a cache from args[0..3]: k codes, k scales, v codes, v scales.
bool cache_of(PyObject *const *args, Device &dev, mx_cache &c)
{
    const at::Tensor *t[4];
    for (int i = 0; i < 4; ++i)
        if (!(t[i] = tensor(args[i]))) return false;
    if (!dev.set(*t[0]) || t[0]->dim() != 4) return false;
    const auto shape = t[0]->sizes();
    const std::array<int64_t, 4> scales{shape[0], shape[1], shape[2], shape[3] / 16};
    for (int i = 0; i < 4; ++i)
        if (!dev.has(t[i], at::kByte) || !t[i]->is_contiguous() || t[i]->sizes() != (i % 2 ? at::IntArrayRef(scales) : shape))
            return false;
    c.k_codes = static_cast<uint8_t *>(t[0]->data_ptr());
    c.k_scales = static_cast<uint8_t *>(t[1]->data_ptr());
    c.v_codes = static_cast<uint8_t *>(t[2]->data_ptr());
    c.v_scales = static_cast<uint8_t *>(t[3]->data_ptr());
    c.num_pages = shape[0];
    c.heads = shape[1];
    c.page_size = shape[2];
    c.head_dim = 2 * shape[3];
    return true;
}

// block_table and cu_seqlens from args[0..1], seq_lens from `lens` (NULL: none).
bool batch_of(PyObject *const *args, PyObject *lens, const Device &dev, mx_batch &b)
{
    const at::Tensor *table = tensor(args[0]), *cu = tensor(args[1]), *len = lens ? tensor(lens) : nullptr;
    if (!dev.has(table, at::kInt) || table->dim() != 2 || !(table->size(1) <= 1 || table->stride(1) == 1)) return false;
    b.batch = table->size(0);
    b.max_pages = table->size(1);
    b.table_stride = b.batch > 1 ? table->stride(0) : b.max_pages;           // (one row: not used)
    if (b.table_stride < b.max_pages) return false;                          // rows that overlap
    if (!dev.has(cu, at::kInt) || cu->dim() != 1 || cu->size(0) != b.batch + 1 || !cu->is_contiguous()) return false;
    if (lens && (!dev.has(len, at::kInt) || len->dim() != 1 || len->size(0) != b.batch || !len->is_contiguous())) return false;
    b.block_table = static_cast<const int32_t *>(table->data_ptr());
    b.cu_seqlens = static_cast<const int32_t *>(cu->data_ptr());
    b.seq_lens = len ? static_cast<const int32_t *>(len->data_ptr()) : nullptr;
    return true;
}

// [T][heads][head_dim], contiguous in the last dimension.
bool rows_ok(const at::Tensor *t, const Device &dev, at::ScalarType type, int64_t head_dim)
{
    return dev.has(t, type) && t->dim() == 3 && t->size(2) == head_dim && t->stride(2) == 1;
}

PyObject *none() { Py_RETURN_NONE; }

// gemv(x, b_codes, b_sf, f32) -> out
PyObject *gemv(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Device dev;
    if (n != 4) return none();
    const at::Tensor *x = tensor(args[0]), *codes = tensor(args[1]), *sf = tensor(args[2]);
    if (!x || !dev.set(*x) || !dev.has(x, at::kBFloat16) || !dev.has(codes, at::kByte) || !dev.has(sf, at::kByte)) return none();
    if (x->dim() != 2 || codes->dim() != 2 || sf->dim() != 1) return none();
    const int64_t M = x->size(0), K = x->size(1), N = codes->size(0);
    const int64_t need = p_gemv_workspace(M, N, K);          // -1: sizes that the call refuses
    if (need < 0 || x->stride(1) != 1 || codes->size(1) * 2 != K || sf->size(0) != p_sf_bytes(N, K) || !codes->is_contiguous() ||
        !sf->is_contiguous())
        return none();
    const bool f32 = args[3] == Py_True;
    at::Tensor out = at::empty({M, N}, x->options().dtype(f32 ? at::kFloat : at::kBFloat16).requires_grad(false));
    at::Tensor work;
    if (need > 0) work = at::empty({need}, codes->options());
    const int rc = unlocked(p_gemv, x->data_ptr(), M > 1 ? x->stride(0) : K, static_cast<const uint8_t *>(codes->data_ptr()),
                            static_cast<const uint8_t *>(sf->data_ptr()), out.data_ptr(), f32, M, N, K,
                            need > 0 ? work.data_ptr() : nullptr, need, dev.stream());
    return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// write(k, v, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, seq_lens) -> True
PyObject *write(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Device dev;
    mx_cache c;
    mx_batch b;
    if (n != 9 || !cache_of(args + 2, dev, c) || !batch_of(args + 6, args[8], dev, b)) return none();
    const at::Tensor *k = tensor(args[0]), *v = tensor(args[1]);
    if (!k || !v || (k->scalar_type() != at::kBFloat16 && k->scalar_type() != at::kFloat)) return none();
    if (!rows_ok(k, dev, k->scalar_type(), c.head_dim) || !rows_ok(v, dev, k->scalar_type(), c.head_dim) ||
        k->size(1) != c.heads || v->sizes() != k->sizes())
        return none();
    const int rc = unlocked(p_write, k->data_ptr(), k->stride(0), k->stride(1), v->data_ptr(), v->stride(0), v->stride(1),
                            k->scalar_type() == at::kFloat, &c, &b, k->size(0), dev.stream());
    if (rc) return PyLong_FromLong(rc);
    Py_RETURN_TRUE;
    END_HANDLE_TH_ERRORS
}

// read(k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, rows, starts or None, f32) -> (k, v)
PyObject *read(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Device dev;
    mx_cache c;
    mx_batch b;
    if (n != 9 || !PyLong_CheckExact(args[6]) || !cache_of(args, dev, c) || !batch_of(args + 4, nullptr, dev, b)) return none();
    const int64_t T = PyLong_AsLongLong(args[6]);
    if (T < 0) {
        PyErr_Clear();
        return none();
    }
    const at::Tensor *starts = nullptr;
    if (args[7] != Py_None) {
        starts = tensor(args[7]);
        if (!dev.has(starts, at::kInt) || starts->dim() != 1 || starts->size(0) != b.batch || !starts->is_contiguous()) return none();
    }
    const bool f32 = args[8] == Py_True;
    const auto options = THPVariable_Unpack(args[0]).options().dtype(f32 ? at::kFloat : at::kBFloat16);
    at::Tensor k = at::empty({T, c.heads, c.head_dim}, options), v = at::empty({T, c.heads, c.head_dim}, options);
    const int rc = unlocked(p_read, &c, &b, starts ? static_cast<const int32_t *>(starts->data_ptr()) : nullptr, k.data_ptr(),
                            v.data_ptr(), f32, T, dev.stream());
    if (rc) return PyLong_FromLong(rc);
    PyObject *pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(k));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(v));
    return pair;
    END_HANDLE_TH_ERRORS
}

// attention(q, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, seq_lens, max_new or None, scale or None,
//           causal) -> out
PyObject *attention(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Device dev;
    mx_cache c;
    mx_batch b;
    if (n != 11 || !cache_of(args + 1, dev, c) || !batch_of(args + 5, args[7], dev, b)) return none();
    const at::Tensor *q = tensor(args[0]);
    if (!rows_ok(q, dev, at::kBFloat16, c.head_dim)) return none();
    const int64_t T = q->size(0), hq = q->size(1);
    int64_t max_new = T;
    if (args[8] != Py_None) {
        if (!PyLong_CheckExact(args[8])) return none();
        max_new = PyLong_AsLongLong(args[8]);
        if (max_new < 0) {
            PyErr_Clear();
            return none();
        }
    }
    double scale = 0.0;
    if (args[9] != Py_None) {
        if (!PyFloat_CheckExact(args[9])) return none();
        scale = PyFloat_AS_DOUBLE(args[9]);
    } else {
        scale = std::pow(double(c.head_dim), -0.5);
    }
    const int64_t need = p_attention_workspace(T, hq, c.heads, c.head_dim, max_new);     // -1: sizes that the call refuses
    if (need < 0) return none();
    at::Tensor out = at::empty({T, hq, c.head_dim}, q->options().requires_grad(false));
    at::Tensor work = at::empty({need}, THPVariable_Unpack(args[1]).options());
    const int rc = unlocked(p_attention, q->data_ptr(), q->stride(0), q->stride(1), &c, &b, float(scale), args[10] != Py_False,
                            out.data_ptr(), T, hq, max_new, work.data_ptr(), need, dev.stream());
    return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// init(addresses of the library's functions, in the order of the pointers above)
PyObject *init(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    void *p[7];
    if (n != 7) return PyErr_Format(PyExc_TypeError, "init takes 7 addresses");
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "init: a NULL address");
    }
    p_gemv = reinterpret_cast<decltype(p_gemv)>(p[0]);
    p_gemv_workspace = reinterpret_cast<decltype(p_gemv_workspace)>(p[1]);
    p_sf_bytes = reinterpret_cast<decltype(p_sf_bytes)>(p[2]);
    p_write = reinterpret_cast<decltype(p_write)>(p[3]);
    p_read = reinterpret_cast<decltype(p_read)>(p[4]);
    p_attention = reinterpret_cast<decltype(p_attention)>(p[5]);
    p_attention_workspace = reinterpret_cast<decltype(p_attention_workspace)>(p[6]);
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init), FAST(gemv), FAST(write), FAST(read), FAST(attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kq_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kq_binding(void) { return PyModule_Create(&module); }
