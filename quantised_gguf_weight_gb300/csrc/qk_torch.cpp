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

bool bool_of(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
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
                                    t.n_pos, t.rot, bool_of(a[9]), t.positions, x.n, y.p, y.ld, y.type,
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
                                       t.n_pos, t.rot, bool_of(a[10]), t.positions, slots, k.n, qo.p, qo.ld,
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

// [T][k] int32 and fp32, contiguous.
template <class V>
V *pairs_of(const at::Tensor &t, int64_t T, int64_t k, at::ScalarType type, const char *name)
{
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", not ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == T && t.size(1) == k && t.is_contiguous(), name, " must be contiguous [", T,
                      "][", k, "], got ", t.sizes());
    return static_cast<V *>(t.data_ptr());
}

// moe_route(logits, top_k, score, bias, n_groups, top_groups, group_top, renorm, scale, ids, weights, stream) -> (ids, weights)
PyObject *moe_route(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count_args(n, 12);
    const int dev = c10::cuda::current_device();
    const at::Tensor &lt = tensor_of(a[0], "logits", dev);
    const int64_t E = lt.dim() == 2 ? lt.size(1) : 0;
    TORCH_CHECK_VALUE(E > 0 && E <= INT32_MAX, "logits must be rows of the experts' logits, got shape ", lt.sizes());
    const Rows l = rows_of(lt, E, "logits");
    const int k = int32_of(a[1], "top_k");
    TORCH_CHECK_VALUE(k > 0 && k <= E, "top_k must be in 1..", E, ", got ", k);
    at::Tensor ids = a[9] == Py_None ? new_rows(l.n, k, lt, at::kInt, a[11]) : tensor_of(a[9], "ids", dev);
    at::Tensor weights = a[10] == Py_None ? new_rows(l.n, k, lt, at::kFloat, a[11]) : tensor_of(a[10], "weights", dev);
    int32_t *ip = pairs_of<int32_t>(ids, l.n, k, at::kInt, "ids");
    float *wp = pairs_of<float>(weights, l.n, k, at::kFloat, "weights");
    const int status = qk_moe_route(l.p, l.ld, l.type, l.n, static_cast<int>(E), k, int32_of(a[2], "score"),
                                    vector_of<const float>(a[3], E, at::kFloat, "bias", dev), int32_of(a[4], "n_groups"),
                                    int32_of(a[5], "top_groups"), int32_of(a[6], "group_top"), bool_of(a[7]),
                                    float_of(a[8]), ip, wp, stream_of(a[11]));
    if (status != QK_OK) return PyLong_FromLong(status);
    PyObject *pair = PyTuple_New(2);
    if (!pair) throw python_error();
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(ids));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(weights));
    return pair;
    END_HANDLE_TH_ERRORS
}

int64_t row_bytes(int format, int64_t cols)
{
    return format == QK_Q8_0 ? qk_row_bytes_q8_0(cols) : format == QK_Q4_K ? qk_row_bytes_q4_k(cols) : qk_row_bytes_q6_k(cols);
}

// Four arguments from a[0]: format, bytes, row_offset, expert_rows; `rows` rows of `cols` columns of each of E experts.
qk_expert_weights weights_of(PyObject *const *a, int64_t E, int64_t rows, int64_t cols, const char *name, int dev)
{
    qk_expert_weights w;
    w.format = int32_of(a[0], "format");
    const at::Tensor &t = tensor_of(a[1], name, dev);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    w.w = t.data_ptr();
    w.row_offset = int_of(a[2]), w.expert_rows = int_of(a[3]);
    const int64_t per = w.expert_rows == 0 ? rows : w.expert_rows, rb = row_bytes(w.format, cols);
    constexpr int64_t kMost = int64_t(1) << 40;          // no row number is beyond it: the products below cannot overflow
    TORCH_CHECK_VALUE(w.row_offset >= 0 && per >= rows && w.row_offset <= kMost && per <= INT32_MAX && E <= (1 << 20), name,
                      " has no such rows: offset ", w.row_offset, ", ", per, " an expert, of ", rows);
    const int64_t need = w.row_offset + (E - 1) * per + rows;
    TORCH_CHECK_VALUE(need <= static_cast<int64_t>(t.nbytes()) / rb, name, " holds ", t.nbytes(), " bytes, the call reads ", need,
                      " rows of ", rb);
    return w;
}

// moe_ffn(x, ids, weights, gate (4), up (4), down (4), n_experts, F, N, y, workspace, stream)
PyObject *moe_ffn(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count_args(n, 21);
    const int dev = c10::cuda::current_device();
    const at::Tensor &xt = tensor_of(a[0], "x", dev);
    const int64_t K = xt.dim() == 2 ? xt.size(1) : 0;
    TORCH_CHECK_VALUE(K > 0 && K <= INT32_MAX, "x must be rows, got shape ", xt.sizes());
    const Rows x = rows_of(xt, K, "x");
    const at::Tensor &it = tensor_of(a[1], "ids", dev), &wt = tensor_of(a[2], "weights", dev);
    const int64_t k = it.dim() == 2 ? it.size(1) : 0;
    TORCH_CHECK_VALUE(k > 0 && k <= INT32_MAX, "ids must be [tokens][top_k], got shape ", it.sizes());
    const int32_t *ids = pairs_of<int32_t>(it, x.n, k, at::kInt, "ids");
    const float *weights = pairs_of<float>(wt, x.n, k, at::kFloat, "weights");
    const int64_t E = int_of(a[15]), F = int_of(a[16]), N = int_of(a[17]) == 0 ? K : int_of(a[17]);
    TORCH_CHECK_VALUE(E > 0 && F > 0 && F <= INT32_MAX && N > 0 && N <= INT32_MAX, "n_experts, F and N must be positive, got ", E,
                      ", ", F, ", ", N);
    const qk_expert_weights gate = weights_of(a + 3, E, F, K, "gate", dev), up = weights_of(a + 7, E, F, K, "up", dev),
                            down = weights_of(a + 11, E, N, F, "down", dev);
    at::Tensor made;
    const bool given = a[18] != Py_None;
    if (!given) made = new_rows(x.n, N, xt, xt.scalar_type(), a[20]);
    const Rows y = rows_of(given ? tensor_of(a[18], "y", dev) : made, N, "y");
    TORCH_CHECK_VALUE(y.n >= x.n, "y has ", y.n, " rows, x ", x.n);
    at::Tensor scratch;
    if (a[19] == Py_None)
        scratch = new_rows(1, static_cast<int64_t>(qk_moe_ffn_workspace_bytes(x.n, static_cast<int>(k), E, K, F, N)), xt, at::kByte,
                           a[20]);
    else
        scratch = tensor_of(a[19], "workspace", dev);
    TORCH_CHECK_VALUE(scratch.is_contiguous(), "workspace must be contiguous");
    const int status = qk_moe_ffn(&gate, &up, &down, E, K, F, N, x.p, x.ld, x.type, x.n, ids, weights, static_cast<int>(k), y.p,
                                  y.ld, y.type, scratch.data_ptr(), scratch.nbytes(), stream_of(a[20]));
    return done(status, given ? a[18] : nullptr, made);
    END_HANDLE_TH_ERRORS
}

// lora(x, y, A, B, ids, scales, out, workspace, stream)
PyObject *lora(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count_args(n, 9);
    const int dev = c10::cuda::current_device();
    const at::Tensor &xt = tensor_of(a[0], "x", dev), &yt = tensor_of(a[1], "y", dev);
    const at::Tensor &At = tensor_of(a[2], "A", dev), &Bt = tensor_of(a[3], "B", dev);
    TORCH_CHECK_VALUE(At.dim() == 3 && Bt.dim() == 3 && At.is_contiguous() && Bt.is_contiguous() && At.size(0) == Bt.size(0) &&
                          At.size(1) == Bt.size(2) && At.size(0) > 0 && At.numel() > 0 && Bt.numel() > 0,
                      "A and B must be contiguous [adapters][rank][K] and [adapters][N][rank], got ", At.sizes(), " and ", Bt.sizes());
    const int w_type = code_of(At, "A");
    TORCH_CHECK_VALUE(code_of(Bt, "B") == w_type, "A and B must have one element type");
    TORCH_CHECK_VALUE(At.size(1) <= INT32_MAX, "rank is out of range: ", At.size(1));
    const Rows x = rows_of(xt, At.size(2), "x"), y = rows_of(yt, Bt.size(1), "y");
    TORCH_CHECK_VALUE(y.n == x.n, "x has ", x.n, " rows, y ", y.n);
    at::Tensor made;
    const bool given = a[6] != Py_None;
    if (!given) made = new_rows(x.n, Bt.size(1), yt, yt.scalar_type(), a[8]);
    const Rows o = rows_of(given ? tensor_of(a[6], "out", dev) : made, Bt.size(1), "out");
    TORCH_CHECK_VALUE(o.type == y.type, "out and y must have one element type");
    TORCH_CHECK_VALUE(o.n >= y.n, "out has ", o.n, " rows, y ", y.n);
    const int32_t *ids = vector_of<const int32_t>(a[4], x.n, at::kInt, "ids", dev);
    TORCH_CHECK_VALUE(ids || x.n == 0, "ids must be a CUDA tensor");
    at::Tensor scratch;
    const size_t need = qk_lora_workspace_bytes(x.n, static_cast<int>(At.size(1)));
    if (a[7] != Py_None) scratch = tensor_of(a[7], "workspace", dev);
    else if (need) scratch = new_rows(1, static_cast<int64_t>(need), xt, at::kByte, a[8]);
    TORCH_CHECK_VALUE(!scratch.defined() || scratch.is_contiguous(), "workspace must be contiguous");
    const int status = qk_lora(x.p, x.ld, x.type, x.n, At.size(2), At.data_ptr(), Bt.data_ptr(), w_type, At.size(0),
                               static_cast<int>(At.size(1)), Bt.size(1), ids,
                               vector_of<const float>(a[5], At.size(0), at::kFloat, "scales", dev), y.p, y.ld, o.p, o.ld, y.type,
                               scratch.defined() ? scratch.data_ptr() : nullptr, scratch.defined() ? scratch.nbytes() : 0,
                               stream_of(a[8]));
    return done(status, given ? a[6] : nullptr, made);
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
                         {"moe_route", fast(moe_route), METH_FASTCALL, nullptr},
                         {"moe_ffn", fast(moe_ffn), METH_FASTCALL, nullptr},
                         {"lora", fast(lora), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "qk_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qk_torch() { return PyModule_Create(&module); }
