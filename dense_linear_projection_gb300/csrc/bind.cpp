// Calls with PyTorch tensors: argument checks, output allocation and the C ABI
// call of the decode-step operators in one native function each.
//
// A call of this kind from Python costs more than the smallest kernels take:
// looking up shapes, types and pointers one by one and crossing ctypes took 9 to
// 14 us on the Grace host, against 2 to 5 us on the GPU.  The functions here
// compute nothing; each raises the library's ProjError for what it refuses.
// Each makes the tensors' device current for the call, where the library refuses
// a handle of another.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "proj.h"

namespace {

PyObject *proj_error = nullptr;  // dense_linear_projection_gb300.ProjError(status, what)

struct Refused {
    int status;
    const char *what;
};

[[noreturn]] void refuse(const char *what) { throw Refused{PROJ_ERR_INVALID_ARG, what}; }

void check(proj_status_t status, const char *what) {
    if (status != PROJ_OK) throw Refused{status, what};
}

// Runs f, turning what it throws into a Python exception.
template <typename F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const Refused &r) {
        if (PyErr_Occurred()) return nullptr;
        PyObject *e = proj_error ? PyObject_CallFunction(proj_error, "is", r.status, r.what) : nullptr;
        if (e) {
            PyErr_SetObject(proj_error, e);
            Py_DECREF(e);
        } else if (!PyErr_Occurred()) {
            PyErr_SetString(PyExc_RuntimeError, r.what);
        }
        return nullptr;
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// A tensor argument; nullptr for None.
const at::Tensor *tensor(PyObject *o, const char *what) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(what);
    return &THPVariable_Unpack(o);
}

const at::Tensor &needed(PyObject *o, const char *what) {
    const at::Tensor *t = tensor(o, what);
    if (!t) refuse(what);
    return *t;
}

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) refuse("an integer");
    return v;
}

bool truth(PyObject *o, const char *what) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) refuse(what);
    return v != 0;
}

void *handle(PyObject *o) {
    if (o == Py_None) refuse("closed");
    return reinterpret_cast<void *>(integer(o));
}

bool is(const at::Tensor &t, at::ScalarType type, int64_t device, int64_t dims) {
    return t.scalar_type() == type && t.is_cuda() && t.get_device() == device && t.dim() == dims;
}

void *stream_of(PyObject *o, int64_t device) {
    if (o != Py_None) return reinterpret_cast<void *>(integer(o));
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
}

// A new tensor of the memory of the stream `o` that the call runs on: what another
// stream gave back may still be in use there.
at::Tensor fresh(PyObject *o, int64_t device, at::IntArrayRef sizes, const at::TensorOptions &options) {
    if (o == Py_None) return at::empty(sizes, options);
    const int64_t h = integer(o);
    const auto index = static_cast<c10::DeviceIndex>(device);
    // 0 and the runtime's other name for it, 1, are the default stream.
    const c10::cuda::CUDAStreamGuard on(h == 0 || h == 1 ? c10::cuda::getDefaultCUDAStream(index)
                                                         : c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(h), index));
    return at::empty(sizes, options);
}

const void *data(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

PyObject *init(PyObject *, PyObject *error) {
    Py_XDECREF(proj_error);
    proj_error = Py_NewRef(error);
    Py_RETURN_NONE;
}

// q4(handle, N, K, packed bytes, fp32 output, X, packed, bias, out, stream) -> Y
PyObject *q4(PyObject *, PyObject *const *a, Py_ssize_t count) {
    return guarded([&]() -> PyObject * {
        if (count != 10) refuse("q4: ten arguments");
        void *h = handle(a[0]);
        const int64_t N = integer(a[1]), K = integer(a[2]), bytes = integer(a[3]);
        const at::ScalarType type = integer(a[4]) ? at::kFloat : at::kBFloat16;
        const at::Tensor &X = needed(a[5], "X: a tensor");
        const int64_t device = X.is_cuda() ? X.get_device() : -1;
        if (!is(X, at::kBFloat16, device, 2) || X.size(1) != K || !X.is_contiguous()) refuse("X: contiguous bf16 CUDA [M, K]");
        const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(device));
        const int64_t M = X.size(0);
        const at::Tensor &packed = needed(a[6], "packed: a tensor");
        if (!is(packed, at::kByte, device, 1) || packed.numel() != bytes || !packed.is_contiguous())
            refuse("packed: what pack() returned, on X's device");
        const at::Tensor *bias = tensor(a[7], "bias: a tensor");
        if (bias && (!is(*bias, at::kBFloat16, device, 1) || bias->size(0) != N || !bias->is_contiguous()))
            refuse("bias: contiguous bf16 [N], on X's device");
        at::Tensor made;
        const at::Tensor *out = tensor(a[8], "out: a tensor");
        if (!out) {
            made = fresh(a[9], device, {M, N}, X.options().dtype(type));
            out = &made;
        } else if (!is(*out, type, device, 2) || out->size(0) != M || out->size(1) != N || !out->is_contiguous()) {
            refuse("out: contiguous [M, N] of y_dtype, on X's device");
        }
        check(proj_q4_run(static_cast<proj_q4_handle_t>(h), M, X.data_ptr(), packed.data_ptr(), data(bias), out->data_ptr(),
                          stream_of(a[9], device)),
              "proj_q4_run");
        return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[8]);
    });
}

// The row stride of bf16 [n, heads, dim] with contiguous heads; throws for anything else.
int64_t rows(const at::Tensor &x, int64_t n, int64_t heads, int64_t dim, int64_t device, const char *what) {
    if (!is(x, at::kBFloat16, device, 3) || x.size(0) != n || x.size(1) != heads || x.size(2) != dim ||
        (dim > 1 && x.stride(2) != 1) || (heads > 1 && x.stride(1) != dim))
        refuse(what);
    return n > 1 ? x.stride(0) : heads * dim;
}

bool ints(const at::Tensor &x, int64_t device, int64_t dims) { return is(x, at::kInt, device, dims) && x.is_contiguous(); }

struct Cache {
    proj_kv_handle_t h;
    int64_t q_heads, kv_heads, dim, device;
    const at::Tensor *k, *v, *k_scale, *v_scale;
};

// The first nine arguments of append and attend.
Cache cache_of(PyObject *const *a) {
    Cache c;
    c.h = static_cast<proj_kv_handle_t>(handle(a[0]));
    c.q_heads = integer(a[1]);
    c.kv_heads = integer(a[2]);
    c.dim = integer(a[3]);
    c.k = &needed(a[4], "k_cache");
    c.v = &needed(a[5], "v_cache");
    c.k_scale = tensor(a[6], "k_scale");
    c.v_scale = tensor(a[7], "v_scale");
    c.device = c.k->get_device();
    return c;
}

// append(cache.., q, k, v, positions, page_table, seq_ids, rope, interleaved, q_out, stream) -> q_out
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t count) {
    return guarded([&]() -> PyObject * {
        if (count != 18) refuse("append: eighteen arguments");
        const Cache c = cache_of(a);
        const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.device));
        const at::Tensor *q = tensor(a[8], "q: a tensor");
        const at::Tensor &k = needed(a[9], "k: a tensor"), &v = needed(a[10], "v: a tensor");
        const char *kv_rows = "k, v: bf16 [tokens, kv_heads, head_dim] with contiguous heads and one row stride, on the cache's device";
        const int64_t tokens = k.dim() > 0 ? k.size(0) : 0;
        const int64_t kv_stride = rows(k, tokens, c.kv_heads, c.dim, c.device, kv_rows);
        if (rows(v, tokens, c.kv_heads, c.dim, c.device, kv_rows) != kv_stride) refuse(kv_rows);
        const at::Tensor &positions = needed(a[11], "positions: a tensor"), &table = needed(a[12], "page_table: a tensor");
        if (!ints(positions, c.device, 1) || positions.size(0) != tokens)
            refuse("positions: contiguous int32 [tokens], on the cache's device");
        if (!ints(table, c.device, 2)) refuse("page_table: contiguous int32 [sequences, pages], on the cache's device");
        const at::Tensor *seq = tensor(a[13], "seq_ids: a tensor"), *rope = tensor(a[14], "rope: a tensor");
        if (seq && (!ints(*seq, c.device, 1) || seq->size(0) != tokens))
            refuse("seq_ids: contiguous int32 [tokens], on the cache's device");
        if (rope && (!is(*rope, at::kFloat, c.device, 2) || !rope->is_contiguous()))
            refuse("rope: contiguous fp32 [positions, rot_dim], on the cache's device");
        const int interleaved = truth(a[15], "interleaved: a truth value");
        const at::Tensor *q_out = tensor(a[16], "q_out: a tensor");
        at::Tensor made;
        int64_t q_stride = 0, q_out_stride = 0;
        if (q) {
            q_stride = rows(*q, tokens, c.q_heads, c.dim, c.device,
                            "q: bf16 [tokens, q_heads, head_dim] with contiguous heads, on the cache's device");
            if (!q_out) {
                made = fresh(a[17], c.device, {tokens, c.q_heads, c.dim}, q->options());
                q_out = &made;
            }
            q_out_stride = rows(*q_out, tokens, c.q_heads, c.dim, c.device, "q_out: as q");
        } else if (q_out) {
            refuse("q_out: only with q");
        }
        check(proj_kv_append(c.h, tokens, data(q), q_stride, k.data_ptr(), v.data_ptr(), kv_stride,
                             static_cast<const int32_t *>(positions.data_ptr()), static_cast<const int32_t *>(data(seq)),
                             static_cast<const int32_t *>(table.data_ptr()), table.size(0), table.size(1),
                             static_cast<const float *>(data(rope)), rope ? rope->size(0) : 0,
                             rope ? static_cast<int32_t>(rope->size(1)) : 0, interleaved, static_cast<const float *>(data(c.k_scale)),
                             static_cast<const float *>(data(c.v_scale)), c.k->data_ptr(), c.v->data_ptr(),
                             q_out ? q_out->data_ptr() : nullptr, q_out_stride, stream_of(a[17], c.device)),
              "proj_kv_append");
        return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[16]);
    });
}

// attend(cache.., q, page_table, seq_lens, scale, window, out, return_lse, stream) -> out or (out, lse)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t count) {
    return guarded([&]() -> PyObject * {
        if (count != 16) refuse("attend: sixteen arguments");
        const Cache c = cache_of(a);
        const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.device));
        const at::Tensor &q = needed(a[8], "q: a tensor");
        const int64_t n = q.dim() > 0 ? q.size(0) : 0;
        const int64_t q_stride = rows(q, n, c.q_heads, c.dim, c.device,
                                      "q: bf16 [sequences, q_heads, head_dim] with contiguous heads, on the cache's device");
        const at::Tensor &table = needed(a[9], "page_table: a tensor"), &lens = needed(a[10], "seq_lens: a tensor");
        if (!ints(table, c.device, 2) || table.size(0) != n)
            refuse("page_table: contiguous int32 [sequences, pages], on the cache's device");
        if (!ints(lens, c.device, 1) || lens.size(0) != n) refuse("seq_lens: contiguous int32 [sequences], on the cache's device");
        const double scale = PyFloat_AsDouble(a[11]);
        if (scale == -1.0 && PyErr_Occurred()) refuse("scale: a number");
        const int64_t window = integer(a[12]);
        at::Tensor made, lse;
        const at::Tensor *out = tensor(a[13], "out: a tensor");
        if (!out) {
            made = fresh(a[15], c.device, {n, c.q_heads, c.dim}, q.options());
            out = &made;
        }
        const int64_t out_stride = rows(*out, n, c.q_heads, c.dim, c.device, "out: as q");
        const bool with_lse = truth(a[14], "return_lse: a truth value");
        if (with_lse) lse = fresh(a[15], c.device, {n, c.q_heads}, q.options().dtype(at::kFloat));
        check(proj_kv_attend(c.h, n, q.data_ptr(), q_stride, c.k->data_ptr(), c.v->data_ptr(),
                             static_cast<const float *>(data(c.k_scale)), static_cast<const float *>(data(c.v_scale)),
                             static_cast<const int32_t *>(table.data_ptr()), table.size(1),
                             static_cast<const int32_t *>(lens.data_ptr()), window, static_cast<float>(scale), out->data_ptr(),
                             out_stride, with_lse ? static_cast<float *>(lse.data_ptr()) : nullptr, stream_of(a[15], c.device)),
              "proj_kv_attend");
        PyObject *first = made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[13]);
        if (!with_lse || !first) return first;
        PyObject *second = THPVariable_Wrap(std::move(lse));
        if (!second) {
            Py_DECREF(first);
            return nullptr;
        }
        PyObject *both = PyTuple_Pack(2, first, second);
        Py_DECREF(first);
        Py_DECREF(second);
        return both;
    });
}

PyMethodDef methods[] = {
    {"init", init, METH_O, "init(ProjError): the exception that the calls raise"},
    {"q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(q4)), METH_FASTCALL, "a 4-bit projection"},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, "append to a paged cache"},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, "attention over a paged cache"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Native calls with PyTorch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
