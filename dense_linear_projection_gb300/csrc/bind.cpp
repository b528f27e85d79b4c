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

double number(PyObject *o, const char *what) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) refuse(what);
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

// The tensor made here, or the argument that was written.
PyObject *result(at::Tensor &made, PyObject *given) { return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(given); }

// A tuple of `count` new references, which it takes; nullptr where one of them is.
PyObject *together(PyObject **results, int count) {
    PyObject *all = PyTuple_New(count);
    bool ok = all != nullptr;
    for (int i = 0; i < count; ++i) {
        if (ok && results[i])
            PyTuple_SET_ITEM(all, i, results[i]);
        else
            Py_XDECREF(results[i]), ok = false;
    }
    if (ok) return all;
    Py_XDECREF(all);
    return nullptr;
}

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

// append(cache.., q, k, v, positions, page_table, seq_ids, rope, interleaved, q_out, stream, q_norm, k_norm, eps, rope_rows) -> q_out
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t count) {
    return guarded([&]() -> PyObject * {
        if (count != 22) refuse("append: twenty-two arguments");
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
        const at::Tensor *norms[2] = {tensor(a[18], "q_norm: a tensor"), tensor(a[19], "k_norm: a tensor")};
        const at::Tensor *rope_rows = tensor(a[21], "rope_rows: a tensor");
        const double eps = number(a[20], "eps: a number");
        for (const at::Tensor *w : norms)
            if (w && ((!is(*w, at::kBFloat16, c.device, 1) && !is(*w, at::kFloat, c.device, 1)) || w->size(0) != c.dim || !w->is_contiguous()))
                refuse("q_norm, k_norm: contiguous bf16 or fp32 [head_dim], on the cache's device");
        if (norms[0] && norms[1] && norms[0]->scalar_type() != norms[1]->scalar_type()) refuse("q_norm, k_norm: of one type");
        if (norms[0] && !q) refuse("q_norm: only with q");
        if (rope_rows && (!rope || !ints(*rope_rows, c.device, 1) || rope_rows->size(0) != tokens))
            refuse("rope_rows: contiguous int32 [tokens], on the cache's device, with a rope table");
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
        if (norms[0] || norms[1] || rope_rows) {
            const at::Tensor *w = norms[0] ? norms[0] : norms[1];
            check(proj_kv_append_normed(
                      c.h, tokens, data(q), q_stride, k.data_ptr(), v.data_ptr(), kv_stride, data(norms[0]), data(norms[1]),
                      w && w->scalar_type() == at::kFloat ? PROJ_F32 : PROJ_BF16, static_cast<float>(eps),
                      static_cast<const int32_t *>(positions.data_ptr()), static_cast<const int32_t *>(data(seq)),
                      static_cast<const int32_t *>(table.data_ptr()), table.size(0), table.size(1),
                      static_cast<const int32_t *>(data(rope_rows)), static_cast<const float *>(data(rope)), rope ? rope->size(0) : 0,
                      rope ? static_cast<int32_t>(rope->size(1)) : 0, interleaved, static_cast<const float *>(data(c.k_scale)),
                      static_cast<const float *>(data(c.v_scale)), c.k->data_ptr(), c.v->data_ptr(),
                      q_out ? q_out->data_ptr() : nullptr, q_out_stride, stream_of(a[17], c.device)),
                  "proj_kv_append_normed");
            return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[16]);
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
        const double scale = number(a[11], "scale: a number");
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
        PyObject *results[2] = {result(made, a[13]), with_lse ? THPVariable_Wrap(std::move(lse)) : nullptr};
        return with_lse ? together(results, 2) : results[0];
    });
}

// The queries, lengths and outputs that the two forms of attention below share with attend.
struct Attention {
    const at::Tensor *q, *table, *lens;
    int64_t n, q_stride, out_stride;
    float scale;
    at::Tensor made, lse;  // where they are made here
    const at::Tensor *out;
    bool with_lse;
    float *lse_ptr() { return with_lse ? static_cast<float *>(lse.data_ptr()) : nullptr; }
};
Attention attention_of(const Cache &c, PyObject *q, PyObject *table, PyObject *lens, PyObject *scale, PyObject *out, PyObject *return_lse,
                       PyObject *stream) {
    Attention x;
    x.q = &needed(q, "q: a tensor");
    x.n = x.q->dim() > 0 ? x.q->size(0) : 0;
    x.q_stride = rows(*x.q, x.n, c.q_heads, c.dim, c.device,
                      "q: bf16 [sequences, q_heads, head_dim] with contiguous heads, on the cache's device");
    x.table = &needed(table, "page_table: a tensor");
    x.lens = &needed(lens, "seq_lens: a tensor");
    if (!ints(*x.table, c.device, 2) || x.table->size(0) != x.n)
        refuse("page_table: contiguous int32 [sequences, pages], on the cache's device");
    if (!ints(*x.lens, c.device, 1) || x.lens->size(0) != x.n) refuse("seq_lens: contiguous int32 [sequences], on the cache's device");
    x.scale = static_cast<float>(number(scale, "scale: a number"));
    x.out = tensor(out, "out: a tensor");
    x.out_stride = x.out ? rows(*x.out, x.n, c.q_heads, c.dim, c.device, "out: as q") : c.q_heads * c.dim;
    x.with_lse = truth(return_lse, "return_lse: a truth value");
    if (!x.out) x.made = fresh(stream, c.device, {x.n, c.q_heads, c.dim}, x.q->options());
    if (x.with_lse) x.lse = fresh(stream, c.device, {x.n, c.q_heads}, x.q->options().dtype(at::kFloat));
    return x;
}
at::Tensor workspace_of(PyObject *stream, const Cache &c, size_t bytes, const at::Tensor &like) {
    return fresh(stream, c.device, {static_cast<int64_t>(bytes)}, like.options().dtype(at::kByte));
}

// attend_shared(cache.., q, prefix_pages, prefix_len, page_table, seq_lens, scale, out, return_lse, stream) -> out or (out, lse)
PyObject *attend_shared(PyObject *, PyObject *const *a, Py_ssize_t count) {
    return guarded([&]() -> PyObject * {
        if (count != 17) refuse("attend_shared: seventeen arguments");
        const Cache c = cache_of(a);
        const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.device));
        const at::Tensor &prefix = needed(a[9], "prefix_pages: a tensor");
        if (!ints(prefix, c.device, 1)) refuse("prefix_pages: contiguous int32 [pages], on the cache's device");
        const int64_t prefix_len = integer(a[10]);
        Attention x = attention_of(c, a[8], a[11], a[12], a[13], a[14], a[15], a[16]);
        const at::Tensor &out = x.out ? *x.out : x.made;
        size_t bytes = 0;
        check(proj_kv_shared_workspace(c.h, x.n, prefix_len, &bytes), "proj_kv_shared_workspace");
        const at::Tensor workspace = workspace_of(a[16], c, bytes, *x.q);
        check(proj_kv_attend_shared(c.h, x.n, x.q->data_ptr(), x.q_stride, c.k->data_ptr(), c.v->data_ptr(),
                                    static_cast<const float *>(data(c.k_scale)), static_cast<const float *>(data(c.v_scale)),
                                    static_cast<const int32_t *>(prefix.data_ptr()), prefix.size(0), prefix_len,
                                    static_cast<const int32_t *>(x.table->data_ptr()), x.table->size(1),
                                    static_cast<const int32_t *>(x.lens->data_ptr()), x.scale, workspace.data_ptr(), out.data_ptr(),
                                    x.out_stride, x.lse_ptr(), stream_of(a[16], c.device)),
              "proj_kv_attend_shared");
        PyObject *results[2] = {result(x.made, a[14]), x.with_lse ? THPVariable_Wrap(std::move(x.lse)) : nullptr};
        return x.with_lse ? together(results, 2) : results[0];
    });
}

// fp32 [sequences, kv_heads, tokens] with room for every token of the page table.
void scores_fit(const at::Tensor &s, const Cache &c, int64_t n, int64_t tokens, const char *what) {
    if (!is(s, at::kFloat, c.device, 3) || s.size(0) != n || s.size(1) != c.kv_heads || s.size(2) < tokens || !s.is_contiguous()) refuse(what);
}

// attend_scored(cache.., q, page_table, seq_lens, scores, scale, window, scores_out, out, return_lse, stream)
//   -> (out, scores_out) or (out, scores_out, lse)
PyObject *attend_scored(PyObject *, PyObject *const *a, Py_ssize_t count) {
    return guarded([&]() -> PyObject * {
        if (count != 18) refuse("attend_scored: eighteen arguments");
        const Cache c = cache_of(a);
        const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.device));
        Attention x = attention_of(c, a[8], a[9], a[10], a[12], a[15], a[16], a[17]);
        const at::Tensor &out = x.out ? *x.out : x.made;
        const char *shape = "scores, scores_out: contiguous fp32 [sequences, kv_heads, tokens of the page table or more], of one shape, "
                            "on the cache's device, one tensor or apart";
        const at::Tensor &scores = needed(a[11], "scores: a tensor");
        const int64_t tokens = x.table->size(1) * c.k->size(1);
        scores_fit(scores, c, x.n, tokens, shape);
        const at::Tensor *to = tensor(a[14], "scores_out: a tensor");
        if (to) {
            scores_fit(*to, c, x.n, tokens, shape);
            const char *p0 = static_cast<const char *>(scores.data_ptr()), *p1 = static_cast<const char *>(to->data_ptr());
            const int64_t bytes = scores.numel() * 4;
            if (to->size(2) != scores.size(2) || (p0 != p1 && p0 < p1 + bytes && p1 < p0 + bytes)) refuse(shape);
        }
        const int64_t window = integer(a[13]);
        size_t bytes = 0;
        check(proj_kv_scored_workspace(c.h, x.n, x.table->size(1), &bytes), "proj_kv_scored_workspace");
        const at::Tensor workspace = workspace_of(a[17], c, bytes, *x.q);
        check(proj_kv_attend_scored(c.h, x.n, x.q->data_ptr(), x.q_stride, c.k->data_ptr(), c.v->data_ptr(),
                                    static_cast<const float *>(data(c.k_scale)), static_cast<const float *>(data(c.v_scale)),
                                    static_cast<const int32_t *>(x.table->data_ptr()), x.table->size(1),
                                    static_cast<const int32_t *>(x.lens->data_ptr()), window, x.scale,
                                    static_cast<const float *>(scores.data_ptr()),
                                    static_cast<float *>(to ? to->data_ptr() : scores.data_ptr()), scores.size(2), workspace.data_ptr(),
                                    out.data_ptr(), x.out_stride, x.lse_ptr(), stream_of(a[17], c.device)),
              "proj_kv_attend_scored");
        PyObject *results[3] = {result(x.made, a[15]), Py_NewRef(to ? a[14] : a[11]),
                                x.with_lse ? THPVariable_Wrap(std::move(x.lse)) : nullptr};
        return together(results, x.with_lse ? 3 : 2);
    });
}

// evict(cache.., page_table, seq_lens, scores, to_table, keep, recent, stream) -> (lens, scores, kept)
PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t count) {
    return guarded([&]() -> PyObject * {
        if (count != 15) refuse("evict: fifteen arguments");
        const Cache c = cache_of(a);
        const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.device));
        const at::Tensor &table = needed(a[8], "page_table: a tensor"), &lens = needed(a[9], "seq_lens: a tensor");
        if (!ints(table, c.device, 2)) refuse("page_table: contiguous int32 [sequences, pages], on the cache's device");
        const int64_t n = table.size(0), page = c.k->size(1);
        if (!ints(lens, c.device, 1) || lens.size(0) != n) refuse("seq_lens: contiguous int32 [sequences], on the cache's device");
        const at::Tensor &scores = needed(a[10], "scores: a tensor"), &to = needed(a[11], "to_table: a tensor");
        scores_fit(scores, c, n, table.size(1) * page,
                   "scores: contiguous fp32 [sequences, kv_heads, tokens of the page table or more], on the cache's device");
        if (!ints(to, c.device, 2) || to.size(0) != n) refuse("to_table: contiguous int32 [sequences, pages], on the cache's device");
        const int64_t keep = integer(a[12]), recent = integer(a[13]);
        if (keep < 0 || recent < 0 || recent > keep || keep > to.size(1) * page)
            refuse("keep, recent: 0 <= recent <= keep, and no more than to_table has room for");
        at::Tensor lens_out = fresh(a[14], c.device, {n}, lens.options());
        at::Tensor scores_out = fresh(a[14], c.device, {n, c.kv_heads, to.size(1) * page}, scores.options());
        at::Tensor kept = fresh(a[14], c.device, {n, c.kv_heads, keep}, lens.options());
        check(proj_kv_evict(c.h, n, static_cast<const int32_t *>(table.data_ptr()), table.size(1),
                            static_cast<const int32_t *>(lens.data_ptr()), static_cast<const float *>(scores.data_ptr()), scores.size(2),
                            static_cast<const int32_t *>(to.data_ptr()), to.size(1), keep, recent, c.k->data_ptr(), c.v->data_ptr(),
                            static_cast<int32_t *>(lens_out.data_ptr()), static_cast<float *>(scores_out.data_ptr()),
                            static_cast<int32_t *>(kept.data_ptr()), stream_of(a[14], c.device)),
              "proj_kv_evict");
        PyObject *results[3] = {THPVariable_Wrap(std::move(lens_out)), THPVariable_Wrap(std::move(scores_out)),
                                THPVariable_Wrap(std::move(kept))};
        return together(results, 3);
    });
}

PyMethodDef methods[] = {
    {"init", init, METH_O, "init(ProjError): the exception that the calls raise"},
    {"q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(q4)), METH_FASTCALL, "a 4-bit projection"},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, "append to a paged cache"},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, "attention over a paged cache"},
    {"attend_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend_shared)), METH_FASTCALL,
     "attention over a shared prefix and a paged cache"},
    {"attend_scored", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend_scored)), METH_FASTCALL,
     "attention over a paged cache that adds up weights"},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(evict)), METH_FASTCALL, "eviction from a paged cache"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Native calls with PyTorch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
