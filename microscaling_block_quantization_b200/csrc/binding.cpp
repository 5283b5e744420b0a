// Marshalling of the decode-time operators, and of the dequantizer that reads
// their cache back, for Python: tensors checked,
// outputs allocated and the C ABI (include/mx.h) called in one step.  A decode
// step makes such calls back to back on small tensors, where the same checks
// written in Python took longer than the kernels.  No computation happens here.
//
// Each function returns its result, or the ABI's status code (an int) where a
// call failed; a wrong argument raises ValueError or TypeError.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "mx.h"

namespace {

struct Refused : std::exception {
    PyObject *type;
    std::string text;
    Refused(PyObject *t, std::string s) : type(t), text(std::move(s)) {}
};
[[noreturn]] void value_error(const std::string &s) { throw Refused(PyExc_ValueError, s); }
[[noreturn]] void type_error(const std::string &s) { throw Refused(PyExc_TypeError, s); }

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor *maybe(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

const at::Tensor &on_cuda(PyObject *o, const char *name)
{
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
    return t;
}
void same_device(const at::Tensor *t, c10::Device d, const char *name)
{
    if (t && t->device() != d) value_error(std::string(name) + " is on " + t->device().str() + ", expected " + d.str());
}
void *ptr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

int32_t dtype_code(at::ScalarType s, const char *name)
{
    if (s == at::kBFloat16) return MX_DT_BF16;
    if (s == at::kFloat) return MX_DT_FP32;
    type_error("unsupported dtype " + std::string(c10::toString(s)) + " of " + name + " (bf16 or fp32)");
}
// the type asked for: out_dtype, else out's, else `given`
at::ScalarType wanted(PyObject *out_dtype, const at::Tensor *out, at::ScalarType given)
{
    if (out_dtype == Py_None) return out ? out->scalar_type() : given;
    if (!THPDtype_Check(out_dtype)) type_error("out_dtype must be a torch.dtype");
    const at::ScalarType s = reinterpret_cast<THPDtype *>(out_dtype)->scalar_type;
    if (out && out->scalar_type() != s) value_error("out does not have out_dtype");
    return s;
}

int64_t integer(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    return v;
}
float real(PyObject *o, const char *name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be a number");
    }
    return (float)v;
}
template <typename T> const T *address(PyObject *o) { return reinterpret_cast<const T *>((uintptr_t)integer(o, "address")); }

// row stride of a 2-D tensor whose rows are contiguous
int64_t rows_of(const at::Tensor &t, int64_t cols, const char *name)
{
    const auto shape = t.sizes(), stride = t.strides();
    const int64_t n = shape.size() == 2 ? shape[0] : 1;
    if (cols > 1 && stride[shape.size() - 1] != 1) value_error(std::string(name) + " must have contiguous rows");
    if (shape.size() < 2 || n <= 1) return cols;
    if (stride[0] < cols) value_error("the rows of " + std::string(name) + " overlap");
    return stride[0];
}
// token stride of [T, heads * dim] or [T, heads, dim] with contiguous heads
int64_t heads_of(const at::Tensor &t, int64_t heads, int64_t dim, const char *name)
{
    const auto shape = t.sizes(), stride = t.strides();
    const bool three = shape.size() == 3 && shape[1] == heads && shape[2] == dim;
    const bool two = shape.size() == 2 && shape[1] == heads * dim;
    if (!((three && (dim <= 1 || stride[2] == 1) && (heads <= 1 || stride[1] == dim)) || (two && (heads * dim <= 1 || stride[1] == 1))))
        value_error(std::string(name) + " must be [T, " + std::to_string(heads * dim) + "] or [T, " + std::to_string(heads) + ", " +
                    std::to_string(dim) + "] with contiguous heads");
    if (shape[0] <= 1) return heads * dim;
    if (stride[0] < heads * dim) value_error("the tokens of " + std::string(name) + " overlap");
    return stride[0];
}
int64_t head_count(const at::Tensor &t, int64_t dim, const char *name)
{
    if (t.dim() != 2 && t.dim() != 3) value_error(std::string(name) + " must have two or three dimensions");
    return t.dim() == 3 ? t.size(1) : t.size(1) / dim;
}
// pointer of an optional contiguous vector
void *vector(const at::Tensor *t, int64_t n, at::ScalarType s, c10::Device d, const char *name)
{
    if (!t) return nullptr;
    if (t->scalar_type() != s || t->device() != d || t->numel() != n || !t->is_contiguous())
        value_error(std::string(name) + " must be " + std::to_string(n) + " contiguous " + c10::toString(s) + " on " + d.str());
    return t->data_ptr();
}
// a contiguous buffer of at least n bytes
void buffer(const at::Tensor *t, int64_t n, const char *name)
{
    if (t && ((int64_t)t->nbytes() < n || !t->is_contiguous()))
        value_error(std::string(name) + " must be contiguous and hold " + std::to_string(n) + " bytes");
}
void check_scale(const at::Tensor *t)
{
    if (t && (t->scalar_type() != at::kFloat || t->numel() < 1)) type_error("tensor_scale must be float32");
}
void *stream_of(c10::Device d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }

// A cache as a call finds it: its tensors are looked at every time, so that none
// that was replaced is written to.
struct Cache {
    mx_kv_cache c;
    const at::Tensor *all[6];
    int64_t heads, dim;
};
constexpr int kCacheArgs = 13;
// cfg (held by the caller's arguments), cfg address, uses tensor scales, codes, scales and tensor scale of keys, of values, pages,
// page_size, kv_heads, head_dim
const mx_config *cache_of(PyObject *const *a, Cache &r)
{
    const mx_config *cfg = address<mx_config>(a[1]);
    const bool ts = PyObject_IsTrue(a[2]);
    const int64_t pages = integer(a[9], "pages"), page_size = integer(a[10], "page_size");
    r.heads = integer(a[11], "kv_heads");
    r.dim = integer(a[12], "head_dim");
    if (page_size > INT32_MAX || r.heads > INT32_MAX || r.dim > INT32_MAX || page_size < INT32_MIN || r.heads < INT32_MIN || r.dim < INT32_MIN)
        value_error("page_size, kv_heads and head_dim must fit 32 bits");
    if (r.dim < 1) value_error("head_dim must be positive");   // (head counts are divided by it)
    for (int h = 0; h < 2; ++h) {
        const char *name = h ? "v" : "k";
        const at::Tensor &codes = tensor(a[3 + 3 * h], "codes"), &scales = tensor(a[4 + 3 * h], "scales");
        const at::Tensor *t = ts ? maybe(a[5 + 3 * h], "tensor_scale") : nullptr;
        // (sizes that the library refuses are left to it)
        if (pages >= 0 && page_size > 0 && pages <= INT32_MAX / page_size && r.heads > 0 && r.heads <= 4096 && r.dim > 0 && r.dim <= 256 &&
            cfg->block > 0) {
            const int64_t rows = pages * page_size, cols = r.heads * r.dim;
            const int bits = cfg->elem == MX_E2M3 || cfg->elem == MX_E3M2 ? 8 : 4;
            if ((int64_t)codes.nbytes() < rows * cols * bits / 8 || !codes.is_contiguous() ||
                (int64_t)scales.nbytes() < rows * (cols / cfg->block) || !scales.is_contiguous())
                value_error(std::string(name) + ": buffers too small for " + std::to_string(rows) + " rows of " + std::to_string(cols) +
                            ", or not contiguous");
        }
        if (ts && (!t || t->scalar_type() != at::kFloat || t->numel() < 1)) type_error(std::string(name) + ": a float32 tensor scale is needed");
        r.all[3 * h] = &codes;
        r.all[3 * h + 1] = &scales;
        r.all[3 * h + 2] = t;
    }
    r.c = {r.all[0]->data_ptr(), r.all[3]->data_ptr(), static_cast<uint8_t *>(r.all[1]->data_ptr()), static_cast<uint8_t *>(r.all[4]->data_ptr()),
           static_cast<const float *>(ptr(r.all[2])), static_cast<const float *>(ptr(r.all[5])), pages, (int32_t)page_size, (int32_t)r.heads,
           (int32_t)r.dim};
    return cfg;
}
void cache_on(const Cache &r, c10::Device dev)
{
    for (const at::Tensor *t : r.all) same_device(t, dev, "the cache");
}

// Other Python threads run while a call launches, which waits
// while the launch queue is full.
class Unlocked {
    PyThreadState *state = PyEval_SaveThread();

public:
    Unlocked() = default;
    Unlocked(const Unlocked &) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F> auto unlocked(F f)
{
    const Unlocked here;
    return f();
}

// x, codes, scales, tensor_scale, macro, offsets, cfg address, uses tensor scale, N, K, out_dtype, out
PyObject *gemv(PyObject *const *a)
{
    const at::Tensor *ts = PyObject_IsTrue(a[7]) ? maybe(a[3], "tensor_scale") : nullptr;
    check_scale(ts);
    const at::Tensor &x = on_cuda(a[0], "x"), &codes = tensor(a[1], "codes"), &scales = tensor(a[2], "scales");
    const at::Tensor *macro = maybe(a[4], "macro"), *offsets = maybe(a[5], "offsets");
    const mx_config *cfg = address<mx_config>(a[6]);
    const int64_t N = integer(a[8], "N"), K = integer(a[9], "K");
    const at::Tensor *out = maybe(a[11], "out");
    const c10::Device dev = x.device();
    if ((x.dim() != 1 && x.dim() != 2) || x.size(-1) != K)
        value_error("x must be [M, " + std::to_string(K) + "] or [" + std::to_string(K) + "]");
    const bool vec = x.dim() == 1;
    const int64_t M = vec ? 1 : x.size(0), ldx = rows_of(x, K, "x");
    const int32_t xd = dtype_code(x.scalar_type(), "x");
    same_device(&codes, dev, "codes");
    same_device(&scales, dev, "scales");
    same_device(macro, dev, "macro");
    same_device(offsets, dev, "offsets");
    same_device(out, dev, "out");
    same_device(ts, dev, "tensor_scale");
    if (N >= 0 && K >= 0 && cfg->block > 0 && (K == 0 || N < (INT64_C(1) << 32) / K)) {
        const int64_t blocks = N * (K / cfg->block);
        buffer(&codes, N * K / 2, "codes");
        buffer(&scales, blocks, "scales");
        buffer(macro, cfg->macro_block ? N * (K / 128) : 0, "macro");
        buffer(offsets, cfg->asymmetric ? 2 * blocks : 0, "offsets");
    }
    const at::ScalarType ys = wanted(a[10], out, x.scalar_type());
    const int32_t yd = dtype_code(ys, "the result");
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor y;
    int64_t ldy = N;
    if (out) {
        if (out->dim() != x.dim() || out->size(-1) != N || (!vec && out->size(0) != M))
            value_error(vec ? "out must be [" + std::to_string(N) + "]" : "out must be [" + std::to_string(M) + ", " + std::to_string(N) + "]");
        ldy = rows_of(*out, N, "out");
        y = *out;
    } else {
        y = vec ? at::empty({N}, x.options().dtype(ys)) : at::empty({M, N}, x.options().dtype(ys));
    }
    const int rc = unlocked([&] {
        return mx_gemv(cfg, x.data_ptr(), xd, ldx, M, codes.data_ptr(), static_cast<uint8_t *>(scales.data_ptr()),
                       static_cast<float *>(ptr(ts)), static_cast<uint8_t *>(ptr(macro)), static_cast<uint16_t *>(ptr(offsets)),
                       N, K, y.data_ptr(), yd, ldy, stream_of(dev));
    });
    return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(std::move(y));
}

// the cache (kCacheArgs), q, k, v, slots, positions, q_gain, k_gain, eps, inv_freq, interleaved, q_out, k_out
PyObject *kv_append(PyObject *const *a)
{
    Cache cache;
    const mx_config *cfg = cache_of(a, cache);
    const int64_t D = cache.dim, H = cache.heads;
    a += kCacheArgs;
    const at::Tensor *q = maybe(a[0], "q"), &k = on_cuda(a[1], "k"), &v = tensor(a[2], "v");
    const at::Tensor &slots = tensor(a[3], "slots"), *positions = maybe(a[4], "positions");
    const at::Tensor *q_gain = maybe(a[5], "q_gain"), *k_gain = maybe(a[6], "k_gain"), *freq = maybe(a[8], "inv_freq");
    const at::Tensor *q_out = maybe(a[10], "q_out");
    const bool make_k = a[11] == Py_True, no_k = a[11] == Py_False || a[11] == Py_None;
    const at::Tensor *k_out = make_k || no_k ? nullptr : &tensor(a[11], "k_out");
    const c10::Device dev = k.device();
    const at::ScalarType s = k.scalar_type();
    const int32_t dt = dtype_code(s, "k");
    if (k.dim() < 1) value_error("k must have two or three dimensions");
    const int64_t T = k.size(0), ldk = heads_of(k, H, D, "k");
    const struct { const at::Tensor *t; const char *name; } like[] = {{&v, "v"}, {q, "q"}, {q_out, "q_out"}, {k_out, "k_out"}};
    cache_on(cache, dev);
    for (const auto &l : like) {
        same_device(l.t, dev, l.name);
        if (l.t && (l.t->scalar_type() != s || l.t->dim() < 1 || l.t->size(0) != T))
            value_error(std::string(l.name) + " must have " + std::to_string(T) + " tokens of k's dtype");
    }
    const int64_t ldv = heads_of(v, H, D, "v"), Hq = q ? head_count(*q, D, "q") : 0, ldq = q ? heads_of(*q, Hq, D, "q") : 0;
    const int64_t rot = freq ? 2 * freq->numel() : 0;
    if (rot && !positions) value_error("a rotation needs positions");
    void *ps = vector(positions, T, at::kLong, dev, "positions"), *pf = vector(freq, rot / 2, at::kFloat, dev, "inv_freq");
    void *pq = vector(q_gain, D, at::kFloat, dev, "q_gain"), *pk = vector(k_gain, D, at::kFloat, dev, "k_gain");
    void *pl = vector(&slots, T, at::kLong, dev, "slots");
    const float eps = real(a[7], "eps");
    const int32_t interleaved = PyObject_IsTrue(a[9]) ? 1 : 0;
    const c10::cuda::CUDAGuard guard(dev);
    int64_t ldqo = Hq * D, ldko = H * D;
    at::Tensor qo, ko;
    if (q && q_out) {
        ldqo = heads_of(*q_out, Hq, D, "q_out");
        qo = *q_out;
    } else if (q) {
        qo = at::empty({T, Hq, D}, k.options());
    }
    if (k_out) {
        ldko = heads_of(*k_out, H, D, "k_out");
        ko = *k_out;
    } else if (make_k) {
        ko = at::empty({T, H, D}, k.options());
    }
    const int rc = unlocked([&] {
        return mx_kv_append(cfg, &cache.c, ptr(q), k.data_ptr(), v.data_ptr(), dt, ldq, ldk, ldv, T, (int32_t)Hq,
                            static_cast<float *>(pq), static_cast<float *>(pk), eps, static_cast<float *>(pf), (int32_t)rot,
                            interleaved, static_cast<int64_t *>(ps), static_cast<int64_t *>(pl),
                            qo.defined() ? qo.data_ptr() : nullptr, ldqo, ko.defined() ? ko.data_ptr() : nullptr, ldko, stream_of(dev));
    });
    if (rc) return PyLong_FromLong(rc);
    PyObject *r = PyTuple_New(2);
    if (!r) return nullptr;
    const auto put = [r](int i, at::Tensor &t) {
        PyObject *o = t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None);
        PyTuple_SET_ITEM(r, i, o);
    };
    put(0, qo);
    put(1, ko);
    return r;
}

// the cache (kCacheArgs), q, page_table, lengths, scale, window, sinks, lse, out_dtype, out, workspace
PyObject *attn_decode(PyObject *const *a)
{
    Cache cache;
    const mx_config *cfg = cache_of(a, cache);
    const int64_t D = cache.dim;
    a += kCacheArgs;
    const at::Tensor &q = on_cuda(a[0], "q"), &table = tensor(a[1], "page_table"), &lengths = tensor(a[2], "lengths");
    const float scale = real(a[3], "scale");
    const int64_t window = integer(a[4], "window"), sinks = integer(a[5], "sinks");
    const bool want_lse = PyObject_IsTrue(a[6]);
    const at::Tensor *out = maybe(a[8], "out"), *given = maybe(a[9], "workspace");
    const c10::Device dev = q.device();
    const int32_t qd = dtype_code(q.scalar_type(), "q");
    const int64_t Hq = head_count(q, D, "q"), S = q.size(0), ldq = heads_of(q, Hq, D, "q");
    cache_on(cache, dev);
    same_device(&table, dev, "page_table");
    same_device(out, dev, "out");
    same_device(given, dev, "workspace");
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != S)
        value_error("page_table must be int32 [" + std::to_string(S) + ", max_pages]");
    const int64_t pages = table.size(1);
    if ((pages > 1 && table.stride(1) != 1) || (S > 1 && table.stride(0) < pages)) value_error("page_table must have contiguous rows");
    const int64_t ldt = S > 1 ? table.stride(0) : pages;
    void *pl = vector(&lengths, S, at::kInt, dev, "lengths");
    if (given && (given->scalar_type() != at::kByte || !given->is_contiguous())) value_error("workspace must be contiguous uint8");
    if (window < INT32_MIN || window > INT32_MAX || sinks < INT32_MIN || sinks > INT32_MAX) value_error("window and sinks must fit 32 bits");
    if (out && (out->dim() < 1 || out->size(0) != S)) value_error("out must have " + std::to_string(S) + " rows");
    const at::ScalarType os = wanted(a[7], out, q.scalar_type());
    const int32_t od = dtype_code(os, "the result");
    const c10::cuda::CUDAGuard guard(dev);
    const int64_t ldo = out ? heads_of(*out, Hq, D, "out") : Hq * D;
    at::Tensor o = out ? *out : at::empty({S, Hq, D}, q.options().dtype(os));
    at::Tensor l, ws;
    if (want_lse) l = at::empty({S, Hq}, q.options().dtype(at::kFloat));
    const int64_t nbytes = mx_attn_workspace_bytes(&cache.c, S, (int32_t)Hq, pages, (int32_t)window, (int32_t)sinks);
    if (given) ws = *given;
    else if (nbytes) ws = at::empty({nbytes}, q.options().dtype(at::kByte));
    const int rc = unlocked([&] {
        return mx_attn_decode(cfg, &cache.c, q.data_ptr(), qd, ldq, S, (int32_t)Hq, static_cast<int32_t *>(table.data_ptr()), ldt, pages,
                              static_cast<int32_t *>(pl), scale, (int32_t)window, (int32_t)sinks, o.data_ptr(), od, ldo,
                              want_lse ? static_cast<float *>(l.data_ptr()) : nullptr, ws.defined() ? ws.data_ptr() : nullptr,
                              ws.defined() ? ws.numel() : 0, stream_of(dev));
    });
    if (rc) return PyLong_FromLong(rc);
    if (!want_lse) return THPVariable_Wrap(std::move(o));
    PyObject *r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(o)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(l)));
    return r;
}

// codes, scales, tensor_scale, macro, offsets, cfg address, rows, cols, out_dtype
PyObject *dequantize(PyObject *const *a)
{
    const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales");
    const at::Tensor *ts = maybe(a[2], "tensor_scale"), *macro = maybe(a[3], "macro"), *offsets = maybe(a[4], "offsets");
    const mx_config *cfg = address<mx_config>(a[5]);
    const int64_t rows = integer(a[6], "rows"), cols = integer(a[7], "cols");
    const at::ScalarType s = wanted(a[8], nullptr, at::kFloat);
    mx_sizes n;
    if (const int rc = mx_query_sizes(cfg, rows, cols, &n)) return PyLong_FromLong(rc);
    if (cfg->tensor_scale == MX_TS_NONE) ts = nullptr;
    buffer(&codes, n.codes_bytes, "codes");
    buffer(&scales, n.n_scales, "scales");
    buffer(macro, n.n_macro, "macro");
    buffer(offsets, 2 * n.n_offsets, "offsets");
    check_scale(ts);
    if (!codes.is_cuda()) value_error("codes must be a CUDA tensor");
    same_device(&scales, codes.device(), "scales");
    same_device(macro, codes.device(), "macro");
    same_device(offsets, codes.device(), "offsets");
    same_device(ts, codes.device(), "tensor_scale");
    const int32_t od = dtype_code(s, "the result");
    const c10::Device dev = codes.device();
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor out = at::empty({rows, cols}, codes.options().dtype(s));
    const int rc = unlocked([&] {
        return mx_dequantize(cfg, codes.data_ptr(), static_cast<uint8_t *>(scales.data_ptr()), static_cast<float *>(ptr(ts)),
                             static_cast<uint8_t *>(ptr(macro)), static_cast<uint16_t *>(ptr(offsets)), rows, cols, out.data_ptr(),
                             od, stream_of(dev));
    });
    return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(std::move(out));
}

template <PyObject *(*F)(PyObject *const *), int N> PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define MX_METHOD(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MX_METHOD(gemv, 12), MX_METHOD(kv_append, kCacheArgs + 12), MX_METHOD(attn_decode, kCacheArgs + 10), MX_METHOD(dequantize, 9),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "mx_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mx_binding() { return PyModule_Create(&module); }
