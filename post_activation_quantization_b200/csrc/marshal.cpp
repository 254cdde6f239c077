// marshal.cpp -- argument marshalling of the paged-cache entry points for Python.
//
// A serving loop makes these calls every step on tensors of every shape, and checking fifteen tensors in Python
// takes longer than a small step takes on the GPU (15 us a call against 3 us here).  The functions below do what
// rptq.py's ctypes calls do: check type, shape, layout and device of every tensor, allocate the outputs that were
// not passed, and call the C ABI (whose addresses bind() is given).  They return the call's status; rptq.py raises.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/rptq.h"

namespace {

decltype(&rptq_kv_paged_append) f_append;
decltype(&rptq_kv_paged_dequant) f_dequant;
decltype(&rptq_kv_paged_attention_workspace_size) f_workspace;
decltype(&rptq_kv_paged_attention) f_attention;
decltype(&rptq_kv_paged_evict) f_evict;

int dtype_code(at::ScalarType t)
{
    return t == at::kFloat ? RPTQ_F32 : t == at::kHalf ? RPTQ_F16 : t == at::kBFloat16 ? RPTQ_BF16 : -1;
}

// The arguments of one call: `ok` is cleared by the first that does not fit.
struct Args {
    PyObject *const *v;
    int i = 0;
    bool ok = true;
    int dev = -1;

    PyObject *next() { return v[i++]; }
    int64_t integer()
    {
        const long long x = PyLong_AsLongLong(next());
        if (x == -1 && PyErr_Occurred()) throw python_error();
        return x;
    }
    double real()
    {
        const double x = PyFloat_AsDouble(next());
        if (x == -1.0 && PyErr_Occurred()) throw python_error();
        return x;
    }
    int narrow()
    {
        const int64_t x = integer();
        ok &= x >= INT32_MIN && x <= INT32_MAX;
        return (int)x;
    }
    // A tensor, or nullptr for None (cleared `ok` where neither).
    const at::Tensor *tensor()
    {
        PyObject *o = next();
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    template <typename T = void>
    T *dense(const at::Tensor *t, at::ScalarType type, at::IntArrayRef shape)
    {
        if (t == nullptr) return nullptr;
        ok &= t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->sizes() == shape && t->is_contiguous();
        return ok ? static_cast<T *>(t->data_ptr()) : nullptr;
    }
    // [T, heads, D] whose rows may be further apart than one row
    void *rows(const at::Tensor *t, at::ScalarType type, at::IntArrayRef shape)
    {
        if (t == nullptr) return nullptr;
        ok &= t->scalar_type() == type && t->is_cuda() && t->get_device() == dev && t->sizes() == shape &&
              (t->numel() == 0 || (t->stride(2) == 1 && (shape[1] == 1 || t->stride(1) == shape[2])));
        return ok ? t->data_ptr() : nullptr;
    }
};

// The stream of a call: the current one for None, else the given handle, which is then the current one while this lives,
// so that what is allocated for the call belongs to it.
struct Stream {
    c10::cuda::OptionalCUDAStreamGuard guard;
    rptq_stream_t handle = nullptr;
    Stream(Args &a, PyObject *o)
    {
        if (!a.ok) return;
        const auto dev = (c10::DeviceIndex)a.dev;
        if (o != Py_None) {
            void *p = PyLong_AsVoidPtr(o);
            if (p == nullptr && PyErr_Occurred()) throw python_error();
            guard.reset_stream(p == nullptr ? c10::cuda::getDefaultCUDAStream(dev)
                                            : c10::cuda::getStreamFromExternal((cudaStream_t)p, dev));
            handle = (rptq_stream_t)p;
        } else {
            handle = (rptq_stream_t)c10::cuda::getCurrentCUDAStream(dev).stream();
        }
    }
};

int64_t row_stride(const at::Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2); }

// Sizes of a pool and its page table.
struct Pool {
    int64_t n_pages = 0, H = 0, P = 0, D = 0, B = 0, max_pages = 0;
    int64_t shape[4] = {0, 0, 0, 0};
    Pool(Args &a, const at::Tensor *pages, const at::Tensor *table, int64_t bits)
    {
        a.ok &= pages != nullptr && table != nullptr && pages->dim() == 4 && table->dim() == 2 && pages->is_cuda() && bits > 0;
        if (!a.ok) return;
        a.dev = pages->get_device();
        for (int i = 0; i < 4; ++i) shape[i] = pages->size(i);
        n_pages = shape[0], H = shape[1], P = shape[2], D = shape[3] * 8 / bits;
        B = table->size(0), max_pages = table->size(1);
        a.ok &= a.dev == c10::cuda::current_device() && shape[3] * 8 % bits == 0 && H <= INT32_MAX && P <= INT32_MAX &&
                D <= INT32_MAX && B <= INT32_MAX && max_pages <= INT32_MAX;
    }
};

struct Clusters {
    const int32_t *cluster = nullptr;
    const float *scale = nullptr;
    const int32_t *zero = nullptr;
    int64_t g = 0;
    void take(Args &a, const at::Tensor *c, const at::Tensor *s, const at::Tensor *z, int64_t C)
    {
        a.ok &= c != nullptr && s != nullptr && z != nullptr;
        if (!a.ok) return;
        g = s->numel();
        cluster = a.dense<int32_t>(c, at::kInt, {C});
        scale = a.dense<float>(s, at::kFloat, {g});
        zero = a.dense<int32_t>(z, at::kInt, {g});
        a.ok &= g <= INT32_MAX;
    }
};

PyObject *status(int st) { return PyLong_FromLong(st); }
PyObject *status_and(int st, const at::Tensor &t)
{
    PyObject *r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, status(st));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(t));
    return r;
}
bool count_is(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// bind(append, dequant, workspace, attention, evict): the addresses of the C ABI's functions
PyObject *bind(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    if (!count_is(n, 5)) return nullptr;
    void *p[5];
    for (int i = 0; i < 5; ++i)
        if ((p[i] = PyLong_AsVoidPtr(v[i])) == nullptr && PyErr_Occurred()) return nullptr;
    f_append = reinterpret_cast<decltype(f_append)>(p[0]);
    f_dequant = reinterpret_cast<decltype(f_dequant)>(p[1]);
    f_workspace = reinterpret_cast<decltype(f_workspace)>(p[2]);
    f_attention = reinterpret_cast<decltype(f_attention)>(p[3]);
    f_evict = reinterpret_cast<decltype(f_evict)>(p[4]);
    Py_RETURN_NONE;
}

// append(k, v, start, lens, table, k_pages, v_pages, ck, sk, zk, cv, sv, zv, bits, weights, stream) -> status
PyObject *append(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_is(n, 16)) return nullptr;
    Args a{v};
    const at::Tensor *t[13];
    for (auto &x : t) x = a.tensor();
    const int bits = a.narrow();
    const at::Tensor *weights = a.tensor();
    const at::Tensor *x = t[0] ? t[0] : t[1], *pool = t[0] ? t[5] : t[6];
    const Pool p(a, pool, t[4], bits);
    a.ok = a.ok && x != nullptr && x->dim() == 3 && dtype_code(x->scalar_type()) >= 0;
    if (!a.ok) return status(RPTQ_ERR_INVALID_ARG);
    const int64_t T = x->size(0), C = p.H * p.D;
    const at::ScalarType ty = x->scalar_type();
    Clusters ck, cv;
    if (t[0]) ck.take(a, t[7], t[8], t[9], C);
    if (t[1]) cv.take(a, t[10], t[11], t[12], C);
    a.ok &= !(t[0] && t[1]) || (ck.g == cv.g && (T < 2 || t[0]->stride(0) == t[1]->stride(0)));
    const void *k = a.rows(t[0], ty, {T, p.H, p.D}), *w = a.rows(t[1], ty, {T, p.H, p.D});
    auto *start = a.dense<int32_t>(t[2], at::kInt, {p.B + 1}), *lens = a.dense<int32_t>(t[3], at::kInt, {p.B}),
         *table = a.dense<int32_t>(t[4], at::kInt, {p.B, p.max_pages});
    auto *kp = t[0] ? a.dense<uint8_t>(t[5], at::kByte, p.shape) : nullptr, *vp = t[1] ? a.dense<uint8_t>(t[6], at::kByte, p.shape) : nullptr;
    auto *sums = a.dense<float>(weights, at::kFloat, {p.n_pages, p.H, p.P});
    const Stream stream(a, v[15]);
    if (!a.ok) return status(RPTQ_ERR_INVALID_ARG);
    return status(f_append(k, w, dtype_code(ty), T, (int)p.H, (int)p.D, row_stride(*x), start, lens, (int)p.B, table,
                           (int)p.max_pages, p.n_pages, (int)p.P, ck.cluster, ck.scale, ck.zero, cv.cluster, cv.scale, cv.zero,
                           (int)(t[0] ? ck.g : cv.g), bits, kp, vp, sums, stream.handle));
    END_HANDLE_TH_ERRORS
}

// dequant(pages, table, start, begin, cluster, scale, zero, bits, T, out, out_dtype, stream) -> (status, out)
// T < 0: out's rows; out_dtype: its code, where out is None
PyObject *dequant(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_is(n, 12)) return nullptr;
    Args a{v};
    const at::Tensor *t[7];
    for (auto &x : t) x = a.tensor();
    const int bits = a.narrow();
    int64_t T = a.integer();
    const at::Tensor *given = a.tensor();
    const int code = a.narrow();
    const Pool p(a, t[0], t[1], bits);
    a.ok = a.ok && (given ? given->dim() == 3 && dtype_code(given->scalar_type()) >= 0 && (T < 0 || T == given->size(0))
                          : T >= 0 && code >= 0 && code <= 2);
    if (!a.ok) return status_and(RPTQ_ERR_INVALID_ARG, at::Tensor());
    const Stream stream(a, v[11]);
    at::Tensor out = given ? *given
                           : at::empty({T, p.H, p.D}, t[0]->options().dtype(code == RPTQ_F32   ? at::kFloat
                                                                           : code == RPTQ_F16 ? at::kHalf
                                                                                              : at::kBFloat16));
    T = out.size(0);
    Clusters c;
    c.take(a, t[4], t[5], t[6], p.H * p.D);
    auto *pages = a.dense<uint8_t>(t[0], at::kByte, p.shape);
    auto *start = a.dense<int32_t>(t[2], at::kInt, {p.B + 1}), *begin = a.dense<int32_t>(t[3], at::kInt, {p.B}),
         *table = a.dense<int32_t>(t[1], at::kInt, {p.B, p.max_pages});
    void *o = a.dense(&out, out.scalar_type(), {T, p.H, p.D});
    if (!a.ok) return status_and(RPTQ_ERR_INVALID_ARG, at::Tensor());
    return status_and(f_dequant(pages, (int)p.H, (int)p.D, bits, start, begin, (int)p.B, table, (int)p.max_pages, p.n_pages,
                                (int)p.P, T, c.cluster, c.scale, c.zero, (int)c.g, o, dtype_code(out.scalar_type()), stream.handle),
                      out);
    END_HANDLE_TH_ERRORS
}

// attention(q, start, lens, table, k_pages, v_pages, ck, sk, zk, cv, sv, zv, bits, max_q, max_len, scale, out, weights,
//           workspace, stream) -> (status, out)
PyObject *attention(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_is(n, 20)) return nullptr;
    Args a{v};
    const at::Tensor *t[12];
    for (auto &x : t) x = a.tensor();
    const int bits = a.narrow(), max_q = a.narrow(), max_len = a.narrow();
    const double scale = a.real();
    const at::Tensor *given = a.tensor(), *weights = a.tensor(), *space = a.tensor();
    const Pool p(a, t[4], t[3], bits);
    const at::Tensor *q = t[0];
    a.ok = a.ok && q != nullptr && q->dim() == 3 && dtype_code(q->scalar_type()) >= 0 && q->size(1) <= INT32_MAX;
    if (!a.ok) return status_and(RPTQ_ERR_INVALID_ARG, at::Tensor());
    const int64_t T = q->size(0), Hq = q->size(1);
    const at::ScalarType ty = q->scalar_type();
    const int dt = dtype_code(ty);
    Clusters ck, cv;
    ck.take(a, t[6], t[7], t[8], p.H * p.D);
    cv.take(a, t[9], t[10], t[11], p.H * p.D);
    a.ok &= ck.g == cv.g;
    void *qp = a.rows(q, ty, {T, Hq, p.D});
    auto *start = a.dense<int32_t>(t[1], at::kInt, {p.B + 1}), *lens = a.dense<int32_t>(t[2], at::kInt, {p.B}),
         *table = a.dense<int32_t>(t[3], at::kInt, {p.B, p.max_pages});
    auto *kp = a.dense<uint8_t>(t[4], at::kByte, p.shape), *vp = a.dense<uint8_t>(t[5], at::kByte, p.shape);
    auto *sums = a.dense<float>(weights, at::kFloat, {p.n_pages, p.H, p.P});
    if (!a.ok || t[5] == nullptr) return status_and(RPTQ_ERR_INVALID_ARG, at::Tensor());
    const Stream stream(a, v[19]);
    at::Tensor out = given ? *given : at::empty({T, Hq, p.D}, q->options());
    void *o = a.dense(&out, ty, {T, Hq, p.D});
    const size_t bytes = f_workspace(T, (int)Hq, (int)p.H, (int)p.D, dt, (int)p.B, max_q, max_len, weights != nullptr);
    at::Tensor own;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (space) {
        ws = a.dense(space, space->scalar_type(), space->sizes());
        ws_bytes = space->nbytes();
    } else if (bytes) {
        own = at::empty({(int64_t)bytes}, q->options().dtype(at::kByte));
        ws = own.data_ptr();
        ws_bytes = bytes;
    }
    if (!a.ok) return status_and(RPTQ_ERR_INVALID_ARG, at::Tensor());
    return status_and(f_attention(qp, dt, T, (int)Hq, (int)p.H, (int)p.D, row_stride(*q), start, lens, (int)p.B, max_q, max_len, table,
                                  (int)p.max_pages, p.n_pages, (int)p.P, kp, vp, ck.cluster, ck.scale, ck.zero, cv.cluster,
                                  cv.scale, cv.zero, (int)ck.g, bits, (float)scale, o, sums, ws, ws_bytes, stream.handle),
                      out);
    END_HANDLE_TH_ERRORS
}

// evict(k_pages, v_pages, weights, lens, table, bits, budget, recent, max_len, new_lens, kept, stream)
//   -> (status, new_lens, kept); max_len < 0: what the table has room for
PyObject *evict(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!count_is(n, 12)) return nullptr;
    Args a{v};
    const at::Tensor *t[5];
    for (auto &x : t) x = a.tensor();
    const int bits = a.narrow(), budget = a.narrow(), recent = a.narrow();
    int64_t max_len = a.integer();
    const at::Tensor *new_given = a.tensor(), *kept_given = a.tensor();
    const Pool p(a, t[0], t[4], bits);
    if (max_len < 0) max_len = p.max_pages * p.P;
    a.ok &= t[1] != nullptr && t[2] != nullptr && t[3] != nullptr && max_len <= INT32_MAX;
    const int64_t room = budget > 0 ? budget : 0;
    at::Tensor new_lens, kept;
    auto *kp = a.dense<uint8_t>(t[0], at::kByte, p.shape), *vp = a.dense<uint8_t>(t[1], at::kByte, p.shape);
    auto *sums = a.dense<float>(t[2], at::kFloat, {p.n_pages, p.H, p.P});
    auto *lens = a.dense<int32_t>(t[3], at::kInt, {p.B}), *table = a.dense<int32_t>(t[4], at::kInt, {p.B, p.max_pages});
    int st = RPTQ_ERR_INVALID_ARG;
    if (a.ok) {
        const Stream stream(a, v[11]);
        new_lens = new_given ? *new_given : at::empty({p.B}, t[3]->options());
        kept = kept_given ? *kept_given : at::empty({p.B, p.H, room}, t[3]->options());
        auto *nl = a.dense<int32_t>(&new_lens, at::kInt, {p.B}), *kt = a.dense<int32_t>(&kept, at::kInt, {p.B, p.H, room});
        if (a.ok)
            st = f_evict(kp, vp, sums, (int)p.B, (int)p.H, (int)p.D, bits, lens, table, (int)p.max_pages, p.n_pages, (int)p.P,
                         (int)max_len, budget, recent, nl, kt, stream.handle);
    }
    PyObject *r = PyTuple_New(3);
    PyTuple_SET_ITEM(r, 0, status(st));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(new_lens));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(kept));
    return r;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)())bind, METH_FASTCALL, nullptr},
                         {"append", (PyCFunction)(void (*)())append, METH_FASTCALL, nullptr},
                         {"dequant", (PyCFunction)(void (*)())dequant, METH_FASTCALL, nullptr},
                         {"attention", (PyCFunction)(void (*)())attention, METH_FASTCALL, nullptr},
                         {"evict", (PyCFunction)(void (*)())evict, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
