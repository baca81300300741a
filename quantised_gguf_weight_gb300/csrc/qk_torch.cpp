// qk_torch.cpp -- the attention operators' calls from PyTorch tensors.
//
// Argument checks, output allocation and the call into libqk, as a CPython
// extension module: a decode step's calls take a few microseconds on the GPU,
// and the same checks in Python took three times that on the host.  A tensor
// that is refused raises ValueError before anything is launched; a status
// other than QK_OK is returned as an int for the caller to raise.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qk.h"

namespace {

int code_of(const at::Tensor &t, const char *name)
{
    switch (t.scalar_type()) {
    case at::kFloat: return QK_F32;
    case at::kHalf: return QK_F16;
    case at::kBFloat16: return QK_BF16;
    default: TORCH_CHECK_VALUE(false, name, " must be float32, float16 or bfloat16, not ", t.scalar_type());
    }
}

const at::Tensor &tensor_of(PyObject *o, const char *name, int dev)
{
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a CUDA tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(t.get_device() == dev, name, " is on ", t.device(), ", the current device is cuda:", dev);
    return t;
}

// Rows of `width` elements with unit stride inside a row.
struct Rows {
    void *p = nullptr;
    int64_t n = 0, ld = 0;
    int type = 0;
};
Rows rows_of(const at::Tensor &t, int64_t width, const char *name)
{
    Rows r;
    r.type = code_of(t, name);
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(1) == width, name, " must be rows of ", width, " elements, got shape ", t.sizes());
    TORCH_CHECK_VALUE(t.stride(1) == 1 || width <= 1, name, " must have unit stride inside a row, got ", t.stride(1));
    r.n = t.size(0);
    r.ld = r.n > 1 ? t.stride(0) : width;      // a single row has no stride of its own
    TORCH_CHECK_VALUE(r.ld >= width, name, " rows are ", r.ld, " elements apart, less than their ", width);
    r.p = t.data_ptr();
    return r;
}

// A contiguous vector of at least n elements; None is null.
template <class T>
T *vector_of(PyObject *o, int64_t n, at::ScalarType type, const char *name, int dev)
{
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor_of(o, name, dev);
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", not ", t.scalar_type());
    TORCH_CHECK_VALUE(t.is_contiguous() && t.numel() >= n, name, " must be contiguous with at least ", n, " elements");
    return static_cast<T *>(t.data_ptr());
}

struct Table {
    const float *p = nullptr;
    int64_t n_pos = 0;
    int rot = 0;
    const int32_t *positions = nullptr;
};
Table table_of(PyObject *table, PyObject *positions, int64_t T, int64_t D, int dev)
{
    Table r;
    if (table == Py_None) return r;
    const at::Tensor &t = tensor_of(table, "table", dev);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat, "table must be float32, not ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == 3 && t.size(2) == 2 && t.is_contiguous() && 2 * t.size(1) <= D,
                      "table must be contiguous [n_pos][rot/2][2] with rot <= ", D, ", got ", t.sizes());
    TORCH_CHECK_VALUE(positions != Py_None, "positions are needed with a table");
    r.p = static_cast<const float *>(t.data_ptr()), r.n_pos = t.size(0), r.rot = static_cast<int>(2 * t.size(1));
    r.positions = vector_of<const int32_t>(positions, T, at::kInt, "positions", dev);
    return r;
}

qk_kv_cache_q4 cache_of(PyObject *o, int dev)
{
    const at::Tensor &t = tensor_of(o, "cache", dev);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kByte, "cache must be uint8, not ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == 4 && t.is_contiguous() && t.size(3) % 18 == 0 && t.size(1) <= INT32_MAX &&
                          t.size(2) <= INT32_MAX / 16 && t.size(3) <= INT32_MAX,
                      "cache must be a contiguous uint8 tensor [pages][kv heads][page_tokens/16][18*head_dim] (kv_cache_q4), "
                      "got shape ", t.sizes());
    qk_kv_cache_q4 c;
    c.pages = t.data_ptr(), c.n_pages = t.size(0), c.n_kv_heads = static_cast<int>(t.size(1));
    c.head_dim = static_cast<int>(t.size(3) / 18), c.page_tokens = static_cast<int>(16 * t.size(2));
    return c;
}

int64_t int_of(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

int int32_of(PyObject *o, const char *name)
{
    const int64_t v = int_of(o);
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, " is out of range: ", v);
    return static_cast<int>(v);
}

float float_of(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return static_cast<float>(v);
}

// None: the current stream of the current device; else a stream's handle.
qk_stream_t stream_of(PyObject *o)
{
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    return reinterpret_cast<qk_stream_t>(int_of(o));
}

// New memory that a call on `stream` writes.  It is that stream's, so that nothing queued on another still uses it, and
// is not given out again before what the current stream has queued by the time it is freed is done.
at::Tensor new_rows(int64_t n, int64_t width, const at::Tensor &like, at::ScalarType type, PyObject *stream)
{
    if (stream == Py_None) return at::empty({n, width}, like.options().dtype(type));
    const auto current = c10::cuda::getCurrentCUDAStream();
    const auto own = c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream_of(stream)), like.get_device());
    const c10::cuda::CUDAStreamGuard guard(own);
    const at::Tensor t = at::empty({n, width}, like.options().dtype(type));
    t.record_stream(current);
    return t;
}

// A status other than QK_OK, as an int; else the result.
PyObject *done(int status, PyObject *given, const at::Tensor &made)
{
    if (status != QK_OK) return PyLong_FromLong(status);
    if (given) return Py_NewRef(given);
    return THPVariable_Wrap(made);
}

void count_args(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "takes ", want, " arguments, got ", n); }

// norm_rope(x, n_q_heads, n_k_heads, head_dim, positions, table, q_weight, k_weight, eps, interleaved, y, stream)
PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count_args(n, 12);
    const int dev = c10::cuda::current_device();
    const int nq = int32_of(a[1], "n_q_heads"), nk = int32_of(a[2], "n_k_heads"), D = int32_of(a[3], "head_dim");
    const int64_t width = (static_cast<int64_t>(nq) + nk) * D;
    const at::Tensor &xt = tensor_of(a[0], "x", dev);
    const Rows x = rows_of(xt, width, "x");
    at::Tensor made;
    const bool given = a[10] != Py_None;
    if (!given) made = new_rows(x.n, width, xt, xt.scalar_type(), a[11]);
    const Rows y = rows_of(given ? tensor_of(a[10], "y", dev) : made, width, "y");
    TORCH_CHECK_VALUE(y.n >= x.n, "y has ", y.n, " rows, x ", x.n);
    const Table t = table_of(a[5], a[4], x.n, D, dev);
    const int status = qk_norm_rope(x.p, x.ld, x.type, nq, nk, D, vector_of<const float>(a[6], D, at::kFloat, "q_weight", dev),
                                    vector_of<const float>(a[7], D, at::kFloat, "k_weight", dev), float_of(a[8]), t.p,
                                    t.n_pos, t.rot, PyObject_IsTrue(a[9]), t.positions, x.n, y.p, y.ld, y.type,
                                    stream_of(a[11]));
    return done(status, given ? a[10] : nullptr, made);
    END_HANDLE_TH_ERRORS
}

// kv_append_q4(cache, q, k, v, positions, slots, table, q_weight, k_weight, eps, interleaved, q_out, stream)
PyObject *kv_append_q4(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count_args(n, 13);
    const int dev = c10::cuda::current_device();
    const qk_kv_cache_q4 c = cache_of(a[0], dev);
    const int64_t D = c.head_dim, width = c.n_kv_heads * D;
    const Rows k = rows_of(tensor_of(a[2], "k", dev), width, "k"), v = rows_of(tensor_of(a[3], "v", dev), width, "v");
    TORCH_CHECK_VALUE(v.type == k.type, "v and k must have one element type");
    TORCH_CHECK_VALUE(v.n == k.n, "k has ", k.n, " rows, v ", v.n);
    const int64_t *slots = vector_of<const int64_t>(a[5], k.n, at::kLong, "slots", dev);
    TORCH_CHECK_VALUE(slots || k.n == 0, "slots must be a CUDA tensor");
    const Table t = table_of(a[6], a[4], k.n, D, dev);
    Rows q, qo;
    int heads = 0;
    at::Tensor made;
    const bool has_q = a[1] != Py_None, given = has_q && a[11] != Py_None;
    if (has_q) {
        const at::Tensor &qt = tensor_of(a[1], "q", dev);
        const int64_t wq = qt.dim() == 2 ? qt.size(1) : 0;
        TORCH_CHECK_VALUE(wq > 0 && wq % D == 0 && wq / D <= INT32_MAX, "q must be rows of heads of ", D, " channels");
        q = rows_of(qt, wq, "q");
        TORCH_CHECK_VALUE(q.type == k.type, "q and k must have one element type");
        TORCH_CHECK_VALUE(q.n == k.n, "q has ", q.n, " rows, k ", k.n);
        if (!given) made = new_rows(q.n, wq, qt, qt.scalar_type(), a[12]);
        qo = rows_of(given ? tensor_of(a[11], "q_out", dev) : made, wq, "q_out");
        TORCH_CHECK_VALUE(qo.n >= q.n, "q_out has ", qo.n, " rows, q ", q.n);
        heads = static_cast<int>(wq / D);
    }
    const int status = qk_kv_append_q4(&c, q.p, q.ld, heads, k.p, k.ld, v.p, v.ld, k.type,
                                       vector_of<const float>(a[7], D, at::kFloat, "q_weight", dev),
                                       vector_of<const float>(a[8], D, at::kFloat, "k_weight", dev), float_of(a[9]), t.p,
                                       t.n_pos, t.rot, PyObject_IsTrue(a[10]), t.positions, slots, k.n, qo.p, qo.ld,
                                       qo.type, stream_of(a[12]));
    return done(status, given ? a[11] : (has_q ? nullptr : Py_None), made);
    END_HANDLE_TH_ERRORS
}

// kv_read_q4(cache, slots, type, stream) -> (k, v)
PyObject *kv_read_q4(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count_args(n, 4);
    const int dev = c10::cuda::current_device();
    const qk_kv_cache_q4 c = cache_of(a[0], dev);
    const int64_t T = tensor_of(a[1], "slots", dev).numel(), width = static_cast<int64_t>(c.n_kv_heads) * c.head_dim;
    const int64_t *slots = vector_of<const int64_t>(a[1], T, at::kLong, "slots", dev);
    const int type = int32_of(a[2], "type");
    const at::ScalarType st = type == QK_F32 ? at::kFloat : (type == QK_F16 ? at::kHalf : at::kBFloat16);
    const at::Tensor &like = THPVariable_Unpack(a[0]);
    const at::Tensor k = new_rows(T, width, like, st, a[3]), v = new_rows(T, width, like, st, a[3]);
    const int status = qk_kv_read_q4(&c, slots, T, k.data_ptr(), 0, v.data_ptr(), 0, type, stream_of(a[3]));
    if (status != QK_OK) return PyLong_FromLong(status);
    PyObject *pair = PyTuple_New(2);
    if (!pair) throw python_error();
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(k));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(v));
    return pair;
    END_HANDLE_TH_ERRORS
}

// attn_q4(cache, q, page_table, lens, q_start, max_q, max_len, scale or None, window, out, workspace, stream)
PyObject *attn_q4(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count_args(n, 12);
    const int dev = c10::cuda::current_device();
    const qk_kv_cache_q4 c = cache_of(a[0], dev);
    const int64_t D = c.head_dim;
    const at::Tensor &qt = tensor_of(a[1], "q", dev);
    const int64_t width = qt.dim() == 2 ? qt.size(1) : 0;
    TORCH_CHECK_VALUE(width > 0 && c.n_kv_heads > 0 && D > 0 && width % (D * c.n_kv_heads) == 0 && width / D <= INT32_MAX,
                      "q must be rows of a multiple of ", c.n_kv_heads, " heads of ", D, " channels");
    const Rows q = rows_of(qt, width, "q");
    const int64_t B = tensor_of(a[3], "lens", dev).numel();
    const int32_t *lens = vector_of<const int32_t>(a[3], B, at::kInt, "lens", dev);
    const at::Tensor &pt = tensor_of(a[2], "page_table", dev);
    TORCH_CHECK_VALUE(pt.scalar_type() == at::kInt, "page_table must be int32, not ", pt.scalar_type());
    TORCH_CHECK_VALUE(pt.dim() == 2 && pt.size(0) >= B, "page_table must be [", B, "][pages], got ", pt.sizes());
    const int64_t pages = pt.size(1), ld = pt.size(0) > 1 ? pt.stride(0) : pages;
    TORCH_CHECK_VALUE((pt.stride(1) == 1 || pages <= 1) && ld >= pages, "page_table must have unit stride and rows at least ",
                      pages, " apart, got ", pt.strides());
    at::Tensor made;
    const bool given = a[9] != Py_None;
    if (!given) made = new_rows(q.n, width, qt, qt.scalar_type(), a[11]);
    const Rows o = rows_of(given ? tensor_of(a[9], "out", dev) : made, width, "out");
    TORCH_CHECK_VALUE(o.n >= q.n, "out has ", o.n, " rows, q ", q.n);
    void *workspace = nullptr;
    size_t bytes = 0;
    if (a[10] != Py_None) {
        const at::Tensor &w = tensor_of(a[10], "workspace", dev);
        TORCH_CHECK_VALUE(w.is_contiguous(), "workspace must be contiguous");
        workspace = w.data_ptr(), bytes = w.nbytes();
    }
    const float scale = a[7] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : float_of(a[7]);
    const int status = qk_attn_q4(&c, q.p, q.ld, q.type, static_cast<int>(width / D), static_cast<const int32_t *>(pt.data_ptr()),
                                  ld, pages, lens, vector_of<const int32_t>(a[4], B + 1, at::kInt, "q_start", dev), B, q.n,
                                  int_of(a[5]), int_of(a[6]), scale, int_of(a[8]), o.p, o.ld, o.type, workspace, bytes,
                                  stream_of(a[11]));
    return done(status, given ? a[9] : nullptr, made);
    END_HANDLE_TH_ERRORS
}

template <class F>
PyCFunction fast(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"norm_rope", fast(norm_rope), METH_FASTCALL, nullptr},
                         {"kv_append_q4", fast(kv_append_q4), METH_FASTCALL, nullptr},
                         {"kv_read_q4", fast(kv_read_q4), METH_FASTCALL, nullptr},
                         {"attn_q4", fast(attn_q4), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "qk_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qk_torch() { return PyModule_Create(&module); }
