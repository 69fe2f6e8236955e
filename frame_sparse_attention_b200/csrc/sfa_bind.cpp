// Binding of the 8-bit frame cache's calls for CPython (module _bind; the documented Python
// functions over it are in _cache.py).
//
// It only marshals: checks tensors, fills the descriptors of include/sfa.h, allocates what the
// caller has not given, and calls the library on the tensors' device.  At a single token these
// calls are 3 to 4 us of GPU time and the host sets their rate: with the same steps in Python and
// ctypes calls back to back took 10.8 to 15.1 us (norm and rotation 11.1, write 10.8, append 15.1,
// read 11.1), now 4.6, 4.4, 6.1 and 4.6.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <string>
#include <utility>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/full.h>
#include <ATen/ops/zeros.h>
#include <ATen/ops/zeros_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/headeronly/version.h>

#include "sfa.h"

namespace {

using at::IntArrayRef;
using at::Tensor;

// The interpreter runs other threads meanwhile: a launch can wait for room in the queue.
struct NoGil {
    PyThreadState *state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

// ----------------------------------------------------------------- arguments
bool given(PyObject *o) { return o != Py_None; }

const Tensor &tensor(const char *name, PyObject *o)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

int cuda_index(const Tensor &t) { return t.is_cuda() ? (int)t.get_device() : -1; }

double number(PyObject *o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

template <typename T>
T integer(const char *name, PyObject *o)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(x == (long long)(T)x, name, " is out of range: ", x);
    return (T)x;
}

bool truth(PyObject *o)
{
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x;
}

// A tuple or list of n items.
struct Items {
    PyObject *seq;
    Items(PyObject *o, Py_ssize_t n, const char *what) : seq(PySequence_Fast(o, what))
    {
        if (!seq) throw python_error();
        if (n >= 0 && PySequence_Fast_GET_SIZE(seq) != n) {
            Py_DECREF(seq);
            TORCH_CHECK_VALUE(false, what);
        }
    }
    Items(const Items &) = delete;
    ~Items() { Py_DECREF(seq); }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
    PyObject *operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

int32_t size32(int64_t n)
{
    TORCH_CHECK_VALUE(n == (int32_t)n, "a tensor of ", n, " entries along one dimension");
    return (int32_t)n;
}

IntArrayRef shape4(const char *name, const Tensor &t)
{
    TORCH_CHECK_VALUE(t.dim() == 4, name, " must be [B, H, L, d]");
    return t.sizes();
}

// Address of a bf16 tensor of this shape; its strides go to `to`.
void *rows(const char *name, const Tensor &t, int dev, IntArrayRef shape, int64_t *to)
{
    TORCH_CHECK_VALUE(t.scalar_type() == at::kBFloat16 && cuda_index(t) == dev && t.sizes() == shape, name,
                      " must be a bf16 tensor ", shape, " on device ", dev, ": ", t.scalar_type(), " ", t.sizes());
    const IntArrayRef st = t.strides();
    TORCH_CHECK_VALUE(st[3] == 1, name, " must have d contiguous");
    for (int i = 0; i < 3; ++i) to[i] = st[i];
    return t.data_ptr();
}

// int32 [B], [B, 1] or [B, H_kv]; its batch and head strides go to `to`.
const int32_t *per_head(const char *name, PyObject *o, int dev, int64_t B, int64_t H_kv, int64_t *to)
{
    const Tensor &t = tensor(name, o);
    const IntArrayRef s = t.sizes();
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && cuda_index(t) == dev && (s.size() == 1 || s.size() == 2) &&
                          s[0] == B && (s.size() == 1 || s[1] == H_kv || s[1] == 1),
                      name, " must be an int32 tensor [", B, "] or [", B, ", ", H_kv, "] on device ", dev);
    to[0] = t.strides()[0];
    to[1] = s.size() == 2 && s[1] > 1 ? t.strides()[1] : 0;
    return static_cast<const int32_t *>(t.data_ptr());
}

const int32_t *lengths(const char *name, PyObject *o, int dev, int64_t B)
{
    if (!given(o)) return nullptr;
    const Tensor &t = tensor(name, o);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && cuda_index(t) == dev && t.dim() == 1 && t.size(0) == B && t.is_contiguous(),
                      name, " must be a contiguous int32 tensor [", B, "] on device ", dev);
    return static_cast<const int32_t *>(t.data_ptr());
}

int32_t *dev_status(PyObject *o, int dev)
{
    if (!given(o)) return nullptr;
    const Tensor &t = tensor("dev_status", o);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && cuda_index(t) == dev && t.numel() >= 1,
                      "dev_status must be an int32 tensor on device ", dev);
    return static_cast<int32_t *>(t.data_ptr());
}

const float *weight(const char *name, PyObject *o, int dev, int64_t d)
{
    if (!given(o)) return nullptr;
    const Tensor &t = tensor(name, o);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && cuda_index(t) == dev && t.dim() == 1 && t.size(0) == d && t.is_contiguous(),
                      name, " must be a contiguous fp32 tensor [", d, "] on device ", dev);
    return static_cast<const float *>(t.data_ptr());
}

sfa_cache cache_desc(PyObject *cache, PyObject *table, int dev, int64_t B, int64_t H_kv, int64_t d)
{
    const Items c(cache, 4, "expected a cache of k, k_scale, v, v_scale");
    const Tensor &k = tensor("cache.k", c[0]), &ks = tensor("cache.k_scale", c[1]);
    const Tensor &v = tensor("cache.v", c[2]), &vs = tensor("cache.v_scale", c[3]), &t = tensor("table", table);
    const IntArrayRef shape = k.sizes();
    TORCH_CHECK_VALUE(shape.size() == 4 && shape[3] == d, "expected cache codes [n_pages, heads, page_len, ", d, "], have ", shape);
    const int64_t scales[4] = {shape[0], shape[1], shape[2], d / SFA_CACHE_BLOCK};
    TORCH_CHECK_VALUE(k.scalar_type() == at::kFloat8_e4m3fn && v.scalar_type() == at::kFloat8_e4m3fn &&
                          ks.scalar_type() == at::kFloat8_e8m0fnu && vs.scalar_type() == at::kFloat8_e8m0fnu &&
                          v.sizes() == shape && ks.sizes() == IntArrayRef(scales, 4) && vs.sizes() == IntArrayRef(scales, 4),
                      "expected a cache of float8_e4m3fn codes ", shape, " and float8_e8m0fnu scales ", IntArrayRef(scales, 4));
    TORCH_CHECK_VALUE(cuda_index(k) == dev && cuda_index(v) == dev && cuda_index(ks) == dev && cuda_index(vs) == dev &&
                          k.is_contiguous() && v.is_contiguous() && ks.is_contiguous() && vs.is_contiguous(),
                      "expected a contiguous cache on device ", dev);
    const IntArrayRef ts = t.sizes(), st = t.strides();
    const size_t n = ts.size();
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && cuda_index(t) == dev && (n == 2 || n == 3) && ts[0] == B &&
                          (ts[n - 1] <= 1 || st[n - 1] == 1) && (n == 2 || ts[1] == 1 || ts[1] == H_kv),
                      "table must be an int32 tensor [", B, ", N] or [", B, ", ", H_kv, ", N] on device ", dev, ", rows contiguous");
    sfa_cache desc = {};
    desc.n_pages = size32(shape[0]);
    desc.heads = size32(shape[1]);
    desc.page_len = size32(shape[2]);
    desc.d = size32(d);
    desc.k = k.data_ptr();
    desc.v = v.data_ptr();
    desc.k_scale = ks.data_ptr();
    desc.v_scale = vs.data_ptr();
    desc.table = static_cast<const int32_t *>(t.data_ptr());
    desc.table_len = size32(ts[n - 1]);
    desc.table_stride[0] = st[0];
    desc.table_stride[1] = n == 3 && ts[1] > 1 ? st[1] : 0;
    return desc;
}

// The rotation of this call; false: none.
bool rope_desc(sfa_rope &desc, PyObject *rope, PyObject *positions, PyObject *layout, int dev, int64_t B, int64_t L)
{
    if (!given(rope)) return false;
    const Items r(rope, 3, "expected a rope of inv_freq, axis_pairs, scale");
    const Items pairs(r[1], -1, "expected a tuple of axis_pairs");
    const int64_t n = pairs.size();
    TORCH_CHECK_VALUE(n > 0 && n <= SFA_ROPE_MAX_AXES, "expected 1 to ", SFA_ROPE_MAX_AXES, " position axes");
    desc = sfa_rope();
    int64_t sum = 0;
    for (int64_t i = 0; i < n; ++i) sum += desc.axis_pairs[i] = integer<int32_t>("axis_pairs", pairs[i]);
    const Tensor &f = tensor("rope.inv_freq", r[0]);
    TORCH_CHECK_VALUE(f.scalar_type() == at::kDouble && cuda_index(f) == dev && f.dim() == 1 && f.size(0) == sum && f.is_contiguous(),
                      "rope.inv_freq must be a contiguous float64 tensor [", sum, "] on device ", dev);
    const char *name = PyUnicode_Check(layout) ? PyUnicode_AsUTF8(layout) : "";
    if (!name) throw python_error();
    const bool half = std::strcmp(name, "half") == 0;
    TORCH_CHECK_VALUE(half || std::strcmp(name, "interleaved") == 0, "expected layout 'interleaved' or 'half'");
    TORCH_CHECK_VALUE(given(positions), "rope needs positions");
    const Tensor &p = tensor("positions", positions);
    const IntArrayRef s = p.sizes(), st = p.strides();
    const size_t k = s.size();
    TORCH_CHECK_VALUE(p.scalar_type() == at::kInt && cuda_index(p) == dev && (k == 2 || k == 3) && s[k - 1] == n &&
                          s[k - 2] == L && (k == 2 || s[0] == B || s[0] == 1) && (n == 1 || st[k - 1] == 1),
                      "positions must be an int32 tensor [", B, ", ", L, ", ", n, "] or [", L, ", ", n, "] on device ", dev);
    desc.inv_freq = static_cast<const double *>(f.data_ptr());
    desc.positions = static_cast<const int32_t *>(p.data_ptr());
    desc.pos_stride[0] = k == 3 && s[0] == B ? st[0] : 0;
    desc.pos_stride[1] = st[k - 2];
    desc.layout = half ? SFA_ROPE_HALF : SFA_ROPE_INTERLEAVED;
    desc.n_axes = (int32_t)n;
    desc.scale = (float)number(r[2]);
    return true;
}

// ----------------------------------------------------------------- the call
// Raises the library's error for a status other than SFA_OK.
void check(sfa_status status, const char *what)
{
    if (status == SFA_OK) return;
    PyObject *lib = PyImport_ImportModule("frame_sparse_attention_b200._lib");
    PyObject *type = lib ? PyObject_GetAttrString(lib, "SfaError") : nullptr;
    PyObject *args = type ? Py_BuildValue("(is)", (int)status, what) : nullptr;
    PyObject *error = args ? PyObject_CallObject(type, args) : nullptr;
    if (error) PyErr_SetObject(type, error);
    Py_XDECREF(error);
    Py_XDECREF(args);
    Py_XDECREF(type);
    Py_XDECREF(lib);
    throw python_error();
}

// The tensors' device is the current one until the end of the call, and with it the stream that
// the caller gives (a torch.cuda.Stream or its handle): what is allocated meanwhile belongs to
// that stream, whose order a fill and a later reuse of the memory then follow.
struct Place {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard on;
    Place(int dev, PyObject *stream)
    {
        if (dev < 0) return;  // refused by `launch`
        device.set_index((c10::DeviceIndex)dev);
        if (!given(stream)) return;
        PyObject *handle = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
        if (!handle) throw python_error();
        void *s = PyLong_AsVoidPtr(handle);
        Py_DECREF(handle);
        if (!s && PyErr_Occurred()) throw python_error();
        on.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), (c10::DeviceIndex)dev));
    }
};

// fn(stream) on the current stream.
template <typename F>
void launch(int dev, const char *what, F fn)
{
    TORCH_CHECK_VALUE(dev >= 0, what, ": expected CUDA tensors");
    const sfa_stream_t s = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    sfa_status status;
    {
        const NoGil free;
        status = fn(s);
    }
    check(status, what);
}

// An output: the caller's, or a new one like `t`.  padded: rows from a sequence's length on are not
// written, so a new one starts as zeros (in the caller's they stay as they are).
Tensor output(const char *name, PyObject *o, const Tensor &t, bool padded = false)
{
    if (given(o)) return tensor(name, o);
    const NoGil free;
    return padded ? at::zeros_like(t) : at::empty_like(t);
}

// The descriptor's eps: below 0 it stands for no norm, which a caller asks for with None.
float eps_of(PyObject *o)
{
    if (!given(o)) return -1.f;
    const double eps = number(o);
    TORCH_CHECK_VALUE(!(eps < 0.0), "expected eps >= 0, or None for no norm: ", eps);
    return (float)eps;
}

PyObject *pair(PyObject *a, PyObject *b)  // takes both references
{
    PyObject *t = a && b ? PyTuple_New(2) : nullptr;
    if (!t) {
        Py_XDECREF(a);
        Py_XDECREF(b);
        throw python_error();
    }
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    return t;
}

PyObject *none_or(bool there, const Tensor &t) { return there ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

void expect(Py_ssize_t have, Py_ssize_t want)
{
    TORCH_CHECK_TYPE(have == want, "expected ", want, " arguments, have ", have);
}

// q, k, rope, positions, q_weight, k_weight, eps, layout, q_out, k_out, stream
PyObject *qk_norm_rope(PyObject *, PyObject *const *x, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect(n, 11);
    const bool has_q = given(x[0]), has_k = given(x[1]);
    TORCH_CHECK_VALUE(has_q || has_k, "qk_norm_rope needs q or k");
    const Tensor &t = tensor("q and k", has_q ? x[0] : x[1]);
    const int dev = cuda_index(t);
    const Place place(dev, x[10]);
    const IntArrayRef s = shape4("q and k", t);
    const int64_t B = s[0], L = s[2], d = s[3];
    sfa_rows_desc desc = {};
    desc.B = size32(B);
    desc.L = size32(L);
    desc.d = size32(d);
    desc.eps = eps_of(x[6]);
    void *q = nullptr, *k = nullptr, *qo = nullptr, *ko = nullptr;
    Tensor q_out, k_out;
    if (has_q) {
        desc.H = size32(s[1]);
        q = rows("q", t, dev, s, desc.q_stride);
        q_out = output("q_out", x[8], t);
        qo = rows("q_out", q_out, dev, s, desc.q_out_stride);
    }
    if (has_k) {
        const Tensor &tk = tensor("k", x[1]);
        const int64_t H_kv = shape4("k", tk)[1], shape[4] = {B, H_kv, L, d};
        desc.H_kv = size32(H_kv);
        k = rows("k", tk, dev, shape, desc.k_stride);
        k_out = output("k_out", x[9], tk);
        ko = rows("k_out", k_out, dev, shape, desc.k_out_stride);
    }
    sfa_rope rope;
    const sfa_rope *r = rope_desc(rope, x[2], x[3], x[7], dev, B, L) ? &rope : nullptr;
    const float *qw = weight("q_weight", x[4], dev, d), *kw = weight("k_weight", x[5], dev, d);
    launch(dev, "sfa_qk_norm_rope",
           [&](sfa_stream_t stream) { return sfa_qk_norm_rope(&desc, r, q, k, qw, kw, qo, ko, stream); });
    PyObject *first = none_or(has_q, q_out);
    return pair(first, none_or(has_k, k_out));
    END_HANDLE_TH_ERRORS
}

// cache, k, v, table, start, lens, dev_status, stream
PyObject *cache_write(PyObject *, PyObject *const *x, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect(n, 8);
    const Tensor &tk = tensor("k", x[1]);
    const int dev = cuda_index(tk);
    const Place place(dev, x[7]);
    const IntArrayRef s = shape4("k", tk);
    sfa_rows_desc desc = {};
    desc.B = size32(s[0]);
    desc.H_kv = size32(s[1]);
    desc.L = size32(s[2]);
    desc.d = size32(s[3]);
    desc.eps = -1.f;
    const void *k = rows("k", tk, dev, s, desc.k_stride), *v = rows("v", tensor("v", x[2]), dev, s, desc.v_stride);
    const sfa_cache cache = cache_desc(x[0], x[3], dev, s[0], s[1], s[3]);
    const int32_t *start = per_head("start", x[4], dev, s[0], s[1], desc.start_stride), *lens = lengths("lens", x[5], dev, s[0]);
    int32_t *status = dev_status(x[6], dev);
    launch(dev, "sfa_cache_write",
           [&](sfa_stream_t stream) { return sfa_cache_write(&desc, &cache, k, v, start, lens, status, stream); });
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// cache, q, k, v, table, start, lens, rope, positions, q_weight, k_weight, eps, layout, q_out, dev_status, stream
PyObject *cache_append(PyObject *, PyObject *const *x, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect(n, 16);
    const Tensor &tq = tensor("q", x[1]), &tk = tensor("k", x[2]);
    const int dev = cuda_index(tq);
    const Place place(dev, x[15]);
    const IntArrayRef s = shape4("q", tq);
    const int64_t B = s[0], L = s[2], d = s[3], H_kv = shape4("k", tk)[1], shape[4] = {B, H_kv, L, d};
    sfa_rows_desc desc = {};
    desc.B = size32(B);
    desc.H = size32(s[1]);
    desc.H_kv = size32(H_kv);
    desc.L = size32(L);
    desc.d = size32(d);
    desc.eps = eps_of(x[11]);
    const void *q = rows("q", tq, dev, s, desc.q_stride), *k = rows("k", tk, dev, shape, desc.k_stride);
    const void *v = rows("v", tensor("v", x[3]), dev, shape, desc.v_stride);
    const Tensor q_out = output("q_out", x[13], tq, given(x[6]));
    void *qo = rows("q_out", q_out, dev, s, desc.q_out_stride);
    const sfa_cache cache = cache_desc(x[0], x[4], dev, B, H_kv, d);
    const int32_t *start = per_head("start", x[5], dev, B, H_kv, desc.start_stride), *lens = lengths("lens", x[6], dev, B);
    sfa_rope rope;
    const sfa_rope *r = rope_desc(rope, x[7], x[8], x[12], dev, B, L) ? &rope : nullptr;
    const float *qw = weight("q_weight", x[9], dev, d), *kw = weight("k_weight", x[10], dev, d);
    int32_t *status = dev_status(x[14], dev);
    launch(dev, "sfa_cache_append", [&](sfa_stream_t stream) {
        return sfa_cache_append(&desc, r, &cache, q, k, v, qw, kw, qo, start, lens, status, stream);
    });
    return THPVariable_Wrap(q_out);
    END_HANDLE_TH_ERRORS
}

// cache, table, start, L, lens, k_out, v_out, H_kv, dev_status, stream
PyObject *cache_read(PyObject *, PyObject *const *x, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect(n, 10);
    const Items c(x[0], 4, "expected a cache of k, k_scale, v, v_scale");
    const Tensor &pool = tensor("cache.k", c[0]), &t = tensor("table", x[1]);
    const int dev = cuda_index(pool);
    const Place place(dev, x[9]);
    const IntArrayRef ps = shape4("cache.k", pool);
    TORCH_CHECK_VALUE(t.dim() >= 1, "table must be [B, N] or [B, H_kv, N]");
    const int64_t B = t.size(0), d = ps[3], L = integer<int32_t>("L", x[3]);
    TORCH_CHECK_VALUE(L >= 0, "expected L >= 0");
    int64_t H_kv;
    if (given(x[7])) H_kv = integer<int32_t>("H_kv", x[7]);
    else if (given(x[5])) H_kv = shape4("k_out", tensor("k_out", x[5]))[1];
    else H_kv = std::max(ps[1], t.dim() == 3 ? t.size(1) : (int64_t)1);
    TORCH_CHECK_VALUE(H_kv >= 1, "expected H_kv >= 1");
    const int64_t shape[4] = {B, H_kv, L, d};
    // rows that are not read stay as they are: zero in an output allocated here
    auto zeros = [&]() {
        const NoGil free;
        return at::zeros(shape, pool.options().dtype(at::kBFloat16));
    };
    const Tensor k_out = given(x[5]) ? tensor("k_out", x[5]) : zeros();
    const Tensor v_out = given(x[6]) ? tensor("v_out", x[6]) : zeros();
    sfa_rows_desc desc = {};
    desc.B = size32(B);
    desc.H_kv = size32(H_kv);
    desc.L = (int32_t)L;
    desc.d = size32(d);
    desc.eps = -1.f;
    void *k = rows("k_out", k_out, dev, shape, desc.k_out_stride), *v = rows("v_out", v_out, dev, shape, desc.v_out_stride);
    const sfa_cache cache = cache_desc(x[0], x[1], dev, B, H_kv, d);
    const int32_t *start = per_head("start", x[2], dev, B, H_kv, desc.start_stride), *lens = lengths("lens", x[4], dev, B);
    int32_t *status = dev_status(x[8], dev);
    launch(dev, "sfa_cache_read",
           [&](sfa_stream_t stream) { return sfa_cache_read(&desc, &cache, start, lens, k, v, status, stream); });
    PyObject *first = THPVariable_Wrap(k_out);
    return pair(first, THPVariable_Wrap(v_out));
    END_HANDLE_TH_ERRORS
}

// Key heads as the caller, the pool, the table or the lengths have them.
int64_t key_heads(PyObject *H_kv, PyObject *cache, PyObject *table, PyObject *kv_lens)
{
    if (given(H_kv)) return integer<int32_t>("H_kv", H_kv);
    const Items c(cache, 4, "expected a cache of k, k_scale, v, v_scale");
    const Tensor &t = tensor("table", table), &lens = tensor("kv_lens", kv_lens);
    int64_t n = shape4("cache.k", tensor("cache.k", c[0]))[1];
    if (n == 1 && t.dim() == 3) n = t.size(1);
    if (n == 1 && lens.dim() == 2) n = lens.size(1);
    return n;
}

// q, cache, table, kv_lens, max_kv, H_kv
PyObject *forward_cache_workspace(PyObject *, PyObject *const *x, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect(n, 6);
    const Tensor &q = tensor("q", x[0]);
    const int dev = cuda_index(q);
    const Place place(dev, Py_None);
    const IntArrayRef s = shape4("q", q);
    const int64_t H_kv = key_heads(x[5], x[1], x[2], x[3]);
    const sfa_cache cache = cache_desc(x[1], x[2], dev, s[0], H_kv, s[3]);
    sfa_cache_attn_desc desc = {};
    desc.B = size32(s[0]);
    desc.H = size32(s[1]);
    desc.H_kv = size32(H_kv);
    desc.Lq = size32(s[2]);
    desc.d = size32(s[3]);
    desc.scale = 1.f;
    desc.max_kv = integer<int32_t>("max_kv", x[4]);
    per_head("kv_lens", x[3], dev, s[0], H_kv, desc.len_stride);
    size_t bytes = 0;
    check(sfa_forward_cache_workspace(&desc, &cache, &bytes), "sfa_forward_cache_workspace");
    return PyLong_FromSize_t(bytes);
    END_HANDLE_TH_ERRORS
}

// q, cache, table, kv_lens, causal, q_lens, max_kv, scale, out, lse, workspace, H_kv, dev_status, stream, timeout_us,
// debug_flags
PyObject *forward_cache(PyObject *, PyObject *const *x, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect(n, 16);
    const Tensor &tq = tensor("q", x[0]);
    const int dev = cuda_index(tq);
    const Place place(dev, x[13]);
    const IntArrayRef s = shape4("q", tq);
    const int64_t B = s[0], H = s[1], Lq = s[2], d = s[3], per_row[3] = {B, H, Lq};
    sfa_cache_attn_desc desc = {};
    const void *q = rows("q", tq, dev, s, desc.q_stride);
    const bool padded = given(x[5]);
    const Tensor out = output("out", x[8], tq, padded);
    void *o = rows("out", out, dev, s, desc.o_stride);
    Tensor lse;
    if (given(x[9])) {
        lse = tensor("lse", x[9]);
        TORCH_CHECK_VALUE(lse.scalar_type() == at::kFloat && cuda_index(lse) == dev && lse.sizes() == IntArrayRef(per_row, 3) &&
                              lse.is_contiguous(),
                          "lse must be a contiguous fp32 tensor ", IntArrayRef(per_row, 3), " on device ", dev);
    } else {
        const NoGil free;
        const auto fp32 = tq.options().dtype(at::kFloat);
        lse = padded ? at::full(per_row, -INFINITY, fp32) : at::empty(per_row, fp32);
    }
    const int64_t H_kv = key_heads(x[11], x[1], x[2], x[3]);
    const sfa_cache cache = cache_desc(x[1], x[2], dev, B, H_kv, d);
    desc.B = size32(B);
    desc.H = size32(H);
    desc.H_kv = size32(H_kv);
    desc.Lq = size32(Lq);
    desc.d = size32(d);
    desc.scale = (float)(given(x[7]) ? number(x[7]) : 1.0 / std::sqrt((double)d));
    desc.causal = truth(x[4]) ? 1 : 0;
    desc.max_kv = integer<int32_t>("max_kv", x[6]);
    const int32_t *lens = per_head("kv_lens", x[3], dev, B, H_kv, desc.len_stride);
    desc.timeout_us = integer<uint32_t>("timeout_us", x[14]);
    desc.debug_flags = integer<uint32_t>("debug_flags", x[15]);
    Tensor workspace;
    if (given(x[10])) {
        workspace = tensor("workspace", x[10]);
        TORCH_CHECK_VALUE(cuda_index(workspace) == dev && workspace.is_contiguous(), "workspace must be a contiguous tensor on device ",
                          dev);
    } else {
        size_t need = 0;
        check(sfa_forward_cache_workspace(&desc, &cache, &need), "sfa_forward_cache_workspace");
        if (need) {
            const NoGil free;
            workspace = at::empty({(int64_t)need}, tq.options().dtype(at::kByte));
        }
    }
    void *ws = workspace.defined() ? workspace.data_ptr() : nullptr;
    const size_t ws_bytes = workspace.defined() ? workspace.nbytes() : 0;
    const int32_t *q_lens = lengths("q_lens", x[5], dev, B);
    int32_t *status = dev_status(x[12], dev);
    float *l = static_cast<float *>(lse.data_ptr());
    launch(dev, "sfa_forward_cache", [&](sfa_stream_t stream) {
        return sfa_forward_cache(&desc, &cache, q, lens, q_lens, o, l, ws, ws_bytes, status, stream);
    });
    PyObject *first = THPVariable_Wrap(out);
    return pair(first, THPVariable_Wrap(lse));
    END_HANDLE_TH_ERRORS
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(qk_norm_rope), ENTRY(cache_write),             ENTRY(cache_append),
                         ENTRY(cache_read),   ENTRY(forward_cache_workspace), ENTRY(forward_cache),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind()
{
    PyObject *m = PyModule_Create(&module);
    if (!m) return nullptr;
    // bytes of the descriptors, as the C compiler lays them out
    const std::initializer_list<std::pair<const char *, size_t>> sizes = {{"sizeof_cache", sizeof(sfa_cache)},
                                                                         {"sizeof_rope", sizeof(sfa_rope)},
                                                                         {"sizeof_rows", sizeof(sfa_rows_desc)},
                                                                         {"sizeof_attn", sizeof(sfa_cache_attn_desc)}};
    for (const auto &s : sizes) {
        if (PyModule_AddIntConstant(m, s.first, (long)s.second) < 0) {
            Py_DECREF(m);
            return nullptr;
        }
    }
    // what _cache.py compares with the versions that it runs under
    const std::string built_for = "torch " + std::to_string(TORCH_VERSION_MAJOR) + "." + std::to_string(TORCH_VERSION_MINOR) +
                                  "." + std::to_string(TORCH_VERSION_PATCH) + ", python " +
                                  std::to_string(PY_MAJOR_VERSION) + "." + std::to_string(PY_MINOR_VERSION);
    if (PyModule_AddStringConstant(m, "built_for", built_for.c_str()) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
