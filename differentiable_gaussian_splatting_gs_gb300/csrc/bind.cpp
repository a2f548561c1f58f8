// The decoder operators' calls on torch tensors: checks, allocation of what the caller leaves out, the device's
// current stream, and the C entry. A Python module of nine functions and one size, wrapped with their documentation in
// api.py. These calls are short (a layer norm of 2,000 x 256: 3 us on the GPU), and the same steps written in Python
// cost 12 us (layer norm) to 26 us (attention, backward) around the C entry's 4 to 8.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <sstream>
#include <stdexcept>
#include <string>
#include <vector>

#include "gs.h"

namespace {

struct Refusal : std::invalid_argument {
    using std::invalid_argument::invalid_argument;
};
struct Raised {};  // a Python exception is set

PyObject* g_check = nullptr;   // raises the exception of a status: check(status, where)
PyObject* g_memory = nullptr;  // torch's exception when device memory runs out

template <class... A>
[[noreturn]] void refuse(const char* where, const A&... a) {
    std::ostringstream s;
    s << where << ": ";
    (s << ... << a);
    throw Refusal(s.str());
}

std::string shape(at::IntArrayRef s) {
    std::ostringstream o;
    o << '(';
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

const char* type_name(at::ScalarType t) {
    return t == at::kFloat ? "float32" : t == at::kHalf ? "float16" : t == at::kBFloat16 ? "bfloat16" : c10::toString(t);
}

int dtype_code(const at::Tensor& t, const char* where) {
    const at::ScalarType s = t.scalar_type();
    if (!t.is_cuda() || (s != at::kFloat && s != at::kHalf && s != at::kBFloat16))
        refuse(where, "tensors must be float32, float16 or bfloat16 CUDA tensors");
    return s == at::kFloat ? GS_DTYPE_F32 : s == at::kHalf ? GS_DTYPE_F16 : GS_DTYPE_BF16;
}

const at::Tensor& tensor(PyObject* o, const char* where) {
    if (!THPVariable_Check(o)) refuse(where, "tensors are needed, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

// t's address; NULL, which stands for an argument left out, only where it has no elements.
void* address_of(const at::Tensor& t) {
    void* p = t.data_ptr();
    if (!p && t.numel() > 0) throw Refusal("a tensor without memory of its own");
    return p;
}

// An argument that may be None.
struct Given {
    const at::Tensor* t;
    Given(PyObject* o, const char* where) : t(o == Py_None ? nullptr : &tensor(o, where)) {}
    explicit operator bool() const { return t != nullptr; }
    const at::Tensor& operator*() const { return *t; }
    const at::Tensor* operator->() const { return t; }
    void* address() const { return t ? address_of(*t) : nullptr; }
};

at::Tensor alloc(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
    return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

struct Rows {
    int64_t n, stride;
};

// The rows of a tensor of like's shape, dtype and device whose last dimension is contiguous and whose other
// dimensions have one common stride.
Rows rows_of(const at::Tensor& t, const at::Tensor& like, const char* where) {
    if (!t.is_same(like) && (t.sizes() != like.sizes() || t.scalar_type() != like.scalar_type() || t.device() != like.device()))
        refuse(where, "a tensor of shape ", shape(like.sizes()), ", ", type_name(like.scalar_type()), ", ", like.device(), " is needed");
    const int64_t dims = t.dim();
    if (dims == 0) refuse(where, "the last dimension must be contiguous");
    const int64_t cols = t.size(-1);
    if (t.is_contiguous()) return {cols ? t.numel() / cols : 0, cols};
    if (cols > 1 && t.stride(-1) != 1) refuse(where, "the last dimension must be contiguous");
    int64_t stride = cols, next = -1;  // of the innermost dimension with more than one row; what the next one must have
    for (int64_t i = dims - 2; i >= 0; --i) {
        const int64_t n = t.size(i), s = t.stride(i);
        if (n == 1) continue;
        if (next < 0) stride = s;
        else if (s != next) refuse(where, "the rows must have one common stride");
        next = n * s;
    }
    return {t.numel() / cols, stride};
}

void check_vector(const Given& t, const at::Tensor& like, const char* where) {
    if (t && (t->dim() != 1 || t->size(0) != like.size(-1) || !t->is_contiguous() || t->device() != like.device() ||
              (t->scalar_type() != like.scalar_type() && t->scalar_type() != at::kFloat)))
        refuse(where, "weight and bias must be contiguous [", like.size(-1), "] tensors of x's dtype or float32");
}

void check_floats(const at::Tensor& t, at::IntArrayRef sizes, const at::Tensor& like, const char* where) {
    if (t.sizes() != sizes || t.scalar_type() != at::kFloat || !t.is_contiguous() || t.device() != like.device())
        refuse(where, "a contiguous float32 tensor of shape ", shape(sizes), " on ", like.device(), " is needed");
}

// The items of a tuple or list of n.
struct Items {
    PyObject* fast;
    Items(PyObject* o, int n, const char* where) : fast(PySequence_Fast(o, "a tuple of tensors is needed")) {
        if (!fast) throw Raised();
        if (PySequence_Fast_GET_SIZE(fast) != n) {
            Py_DECREF(fast);
            refuse(where, n, " tensors are needed");
        }
    }
    ~Items() { Py_DECREF(fast); }
    Items(const Items&) = delete;
    PyObject* operator[](int i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// The interpreter's lock is given up for as long as this lives, and taken again however the block is left (a tensor without
// memory of its own throws where its address is asked for).
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// The C entry on like's device and its current stream, without the interpreter's lock.
template <class F>
void call(const at::Tensor& like, const char* where, F&& f) {
    int status;
    {
        const c10::cuda::OptionalCUDAGuard guard(like.device());
        void* stream = c10::cuda::getCurrentCUDAStream(like.device().index()).stream();
        const Unlocked unlocked;
        status = f(stream);
    }
    if (status == GS_OK) return;
    PyObject* r = PyObject_CallFunction(g_check, "is", status, where);
    Py_XDECREF(r);
    if (r) PyErr_SetString(PyExc_RuntimeError, where);
    throw Raised();
}

// A workspace of `need` bytes: the caller's when it is large enough, or `own`. The kernels write to all of these bytes, so
// that the caller's must be one piece of the device's memory whatever its size.
void* workspace_of(const Given& given, size_t need, at::Tensor& own, const at::Tensor& like, const char* where) {
    if (given && (!given->is_contiguous() || given->device() != like.device()))
        refuse(where, "workspace must be a contiguous tensor on ", like.device());
    if (need == 0) return nullptr;
    if (given && (size_t)given->numel() * given->element_size() >= need) return given->data_ptr();
    own = alloc({(int64_t)need}, at::kByte, like);
    return own.data_ptr();
}

PyObject* wrap(const at::Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject* tuple_of(const at::Tensor* t, int n) {
    PyObject* r = PyTuple_New(n);
    if (!r) throw Raised();
    for (int i = 0; i < n; ++i) {
        PyObject* o = wrap(t[i]);
        if (!o) {
            Py_DECREF(r);
            throw Raised();
        }
        PyTuple_SET_ITEM(r, i, o);
    }
    return r;
}

// layer_norm_fwd(x, weight, bias, eps, out)
PyObject* layer_norm_fwd(PyObject* const* arg) {
    const char* me = "gs_layer_norm_fwd";
    const at::Tensor& x = tensor(arg[0], me);
    const int dtype = dtype_code(x, me);
    const Rows rows = rows_of(x, x, me);
    const Given weight(arg[1], me), bias(arg[2], me);
    check_vector(weight, x, me);
    check_vector(bias, x, me);
    if (weight && bias && weight->scalar_type() != bias->scalar_type()) refuse(me, "weight and bias must have one dtype");
    const double eps = PyFloat_AsDouble(arg[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised();
    const Given& kind = weight ? weight : bias;
    at::Tensor out[3];
    int64_t y_stride = x.size(-1);
    if (arg[4] == Py_None) {
        out[0] = alloc(x.sizes(), x.scalar_type(), x);
        out[1] = alloc({rows.n}, at::kFloat, x);
        out[2] = alloc({rows.n}, at::kFloat, x);
    } else {
        const Items given(arg[4], 3, me);
        for (int i = 0; i < 3; ++i) out[i] = tensor(given[i], me);
        y_stride = rows_of(out[0], x, me).stride;
        check_floats(out[1], {rows.n}, x, me);
        check_floats(out[2], {rows.n}, x, me);
    }
    call(x, me, [&](void* stream) {
        return gs_layer_norm_fwd(x.data_ptr(), rows.stride, rows.n, x.size(-1), dtype, weight.address(), bias.address(),
                                 kind ? dtype_code(*kind, me) : dtype, (float)eps, out[0].data_ptr(), y_stride,
                                 out[1].data_ptr<float>(), out[2].data_ptr<float>(), stream);
    });
    return tuple_of(out, 3);
}

// layer_norm_bwd(dy, x, mean, rstd, weight, out, workspace)
PyObject* layer_norm_bwd(PyObject* const* arg) {
    const char* me = "gs_layer_norm_bwd";
    const at::Tensor &dy = tensor(arg[0], me), &x = tensor(arg[1], me), &mean = tensor(arg[2], me), &rstd = tensor(arg[3], me);
    const int dtype = dtype_code(x, me);
    const Rows rows = rows_of(x, x, me);
    const int64_t cols = x.size(-1), dy_stride = rows_of(dy, x, me).stride;
    const Given weight(arg[4], me), room(arg[6], me);
    check_vector(weight, x, me);
    check_floats(mean, {rows.n}, x, me);
    check_floats(rstd, {rows.n}, x, me);
    at::Tensor out[3];
    int64_t dx_stride = cols;
    int kind = weight ? dtype_code(*weight, me) : -1;
    if (arg[5] == Py_None) {
        out[0] = alloc(x.sizes(), x.scalar_type(), x);
        if (weight) {
            out[1] = alloc({cols}, weight->scalar_type(), x);
            out[2] = alloc({cols}, weight->scalar_type(), x);
        }
    } else {
        const Items given(arg[5], 3, me);
        out[0] = tensor(given[0], me);
        dx_stride = rows_of(out[0], x, me).stride;
        for (int i = 1; i < 3; ++i) {
            const Given g(given[i], me);
            check_vector(g, x, me);
            if (!g) continue;
            out[i] = *g;
            const int code = dtype_code(*g, me);
            if (kind >= 0 && kind != code) refuse(me, "weight, dweight and dbias must have one dtype");
            kind = code;
        }
    }
    at::Tensor own;
    const size_t need = out[1].defined() || out[2].defined() ? gs_layer_norm_workspace_bytes(rows.n, cols) : 0;
    void* workspace = workspace_of(room, need, own, x, me);
    auto address = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    call(x, me, [&](void* stream) {
        return gs_layer_norm_bwd(dy.data_ptr(), dy_stride, x.data_ptr(), rows.stride, rows.n, cols, dtype, mean.data_ptr<float>(),
                                 rstd.data_ptr<float>(), weight.address(), kind < 0 ? dtype : kind, out[0].data_ptr(), dx_stride,
                                 address(out[1]), address(out[2]), workspace, need, stream);
    });
    return tuple_of(out, 3);
}

gs_heads heads_of(const at::Tensor& t, at::IntArrayRef sizes, const at::Tensor& like, const char* where) {
    if (t.sizes() != sizes || t.scalar_type() != like.scalar_type() || t.device() != like.device())
        refuse(where, "a tensor of shape ", shape(sizes), ", ", type_name(like.scalar_type()), ", on ", like.device(), " is needed, got ",
               shape(t.sizes()), ", ", type_name(t.scalar_type()), ", ", t.device());
    if (sizes[3] > 1 && t.stride(3) != 1) refuse(where, "the elements of a head must be contiguous");
    return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

struct Attention {
    gs_attention a;
    int64_t q[4], kv[4], stats[3];  // sizes of q, of k and v, and of lse
};

Attention attention_of(const at::Tensor& q, const at::Tensor& k, const Given& k_len, const Given& mask, PyObject* scale, const char* where) {
    Attention r{};
    const int code = dtype_code(q, where);
    if (q.dim() != 4 || k.dim() != 4) refuse(where, "q, k and v must be [batch, length, heads, head_dim]");
    const int64_t b = q.size(0), lq = q.size(1), h = q.size(2), d = q.size(3), lk = k.size(1), hk = k.size(2);
    if (h < 1 || hk < 1 || h % hk) refuse(where, h, " query heads must be a multiple of ", hk, " key heads");
    for (const int64_t n : {b, lq, h, d, lk, hk})
        if (n > 0x7fffffff) refuse(where, "a size passes 31 bits");
    if (k_len && (k_len->dim() != 1 || k_len->size(0) != b || k_len->scalar_type() != at::kInt || !k_len->is_contiguous() ||
                  k_len->device() != q.device()))
        refuse(where, "k_len must be a contiguous int32 [", b, "] tensor on ", q.device());
    if (mask && (mask->dim() != 2 || mask->size(0) != b || mask->size(1) != lk ||
                 (mask->scalar_type() != at::kBool && mask->scalar_type() != at::kByte) || (lk > 1 && mask->stride(1) != 1) ||
                 mask->device() != q.device()))
        refuse(where, "key_mask must be a bool or uint8 [", b, ", ", lk, "] tensor on ", q.device(), " with contiguous rows");
    double s = 0.0;
    if (scale != Py_None) {
        s = PyFloat_AsDouble(scale);
        if (s == -1.0 && PyErr_Occurred()) throw Raised();
        // (below float32's range it would become 0, which stands for the default)
        if (!((float)s > 0.f) || !std::isfinite((float)s)) refuse(where, "scale must be a positive, finite float32");
    }
    r.a.dtype = code;
    r.a.batch = (int32_t)b;
    r.a.heads = (int32_t)h;
    r.a.kv_heads = (int32_t)hk;
    r.a.head_dim = (int32_t)d;
    r.a.len_q = (int32_t)lq;
    r.a.len_k = (int32_t)lk;
    r.a.scale = (float)s;
    r.a.k_len = static_cast<const int32_t*>(k_len.address());
    r.a.key_mask = static_cast<const uint8_t*>(mask.address());
    r.a.key_mask_stride = mask ? mask->stride(0) : 0;
    const int64_t qs[] = {b, lq, h, d}, ks[] = {b, lk, hk, d}, ss[] = {b, h, lq};
    std::copy(qs, qs + 4, r.q);
    std::copy(ks, ks + 4, r.kv);
    std::copy(ss, ss + 3, r.stats);
    return r;
}

size_t attention_bytes(const Attention& r, const at::Tensor& like, int backward) {
    const c10::cuda::OptionalCUDAGuard guard(like.device());  // the size depends on the device's number of SMs
    return gs_cross_attention_workspace_bytes(&r.a, backward);
}

// cross_attention_workspace_bytes(q, k, k_len, key_mask, backward)
PyObject* attention_workspace_bytes(PyObject* const* arg) {
    const char* me = "gs_cross_attention_workspace_bytes";
    const at::Tensor &q = tensor(arg[0], me), &k = tensor(arg[1], me);
    const Given k_len(arg[2], me), mask(arg[3], me);
    return PyLong_FromSize_t(attention_bytes(attention_of(q, k, k_len, mask, Py_None, me), q, PyObject_IsTrue(arg[4]) == 1));
}

// cross_attention_fwd(q, k, v, k_len, key_mask, scale, out, workspace)
PyObject* attention_fwd(PyObject* const* arg) {
    const char* me = "gs_cross_attention_fwd";
    const at::Tensor &q = tensor(arg[0], me), &k = tensor(arg[1], me), &v = tensor(arg[2], me);
    const Given k_len(arg[3], me), mask(arg[4], me), room(arg[7], me);
    const Attention r = attention_of(q, k, k_len, mask, arg[5], me);
    const gs_heads hq = heads_of(q, r.q, q, me), hk = heads_of(k, r.kv, q, me), hv = heads_of(v, r.kv, q, me);
    at::Tensor out[2];
    if (arg[6] == Py_None) {
        out[0] = alloc(r.q, q.scalar_type(), q);
        out[1] = alloc(r.stats, at::kFloat, q);
    } else {
        const Items given(arg[6], 2, me);
        for (int i = 0; i < 2; ++i) out[i] = tensor(given[i], me);
        check_floats(out[1], r.stats, q, me);
    }
    const gs_heads ho = heads_of(out[0], r.q, q, me);
    at::Tensor own;
    const size_t need = attention_bytes(r, q, 0);
    void* workspace = workspace_of(room, need, own, q, me);
    call(q, me, [&](void* stream) {
        return gs_cross_attention_fwd(&r.a, &hq, &hk, &hv, &ho, out[1].data_ptr<float>(), workspace, need, stream);
    });
    return tuple_of(out, 2);
}

// cross_attention_bwd(dout, q, k, v, out, lse, k_len, key_mask, scale, grads, workspace)
PyObject* attention_bwd(PyObject* const* arg) {
    const char* me = "gs_cross_attention_bwd";
    const at::Tensor &dout = tensor(arg[0], me), &q = tensor(arg[1], me), &k = tensor(arg[2], me), &v = tensor(arg[3], me),
                     &out = tensor(arg[4], me), &lse = tensor(arg[5], me);
    const Given k_len(arg[6], me), mask(arg[7], me), room(arg[10], me);
    const Attention r = attention_of(q, k, k_len, mask, arg[8], me);
    const gs_heads hd = heads_of(dout, r.q, q, me), hq = heads_of(q, r.q, q, me), hk = heads_of(k, r.kv, q, me),
                   hv = heads_of(v, r.kv, q, me), ho = heads_of(out, r.q, q, me);
    check_floats(lse, r.stats, q, me);
    at::Tensor grad[3];
    if (arg[9] == Py_None) {
        for (int i = 0; i < 3; ++i) grad[i] = i ? alloc(r.kv, q.scalar_type(), q) : alloc(r.q, q.scalar_type(), q);
    } else {
        const Items given(arg[9], 3, me);
        for (int i = 0; i < 3; ++i) grad[i] = tensor(given[i], me);
    }
    const gs_heads gq = heads_of(grad[0], r.q, q, me), gk = heads_of(grad[1], r.kv, q, me), gv = heads_of(grad[2], r.kv, q, me);
    at::Tensor own;
    const size_t need = attention_bytes(r, q, 1);
    void* workspace = workspace_of(room, need, own, q, me);
    call(q, me, [&](void* stream) {
        return gs_cross_attention_bwd(&r.a, &hd, &hq, &hk, &hv, &ho, lse.data_ptr<float>(), &gq, &gk, &gv, workspace, need, stream);
    });
    return tuple_of(grad, 3);
}

constexpr int64_t kFp8Block = 128;

// Rows of t, also where they are empty.
int64_t leading(const at::Tensor& t) {
    int64_t n = 1;
    for (int64_t i = 0; i + 1 < t.dim(); ++i) n *= t.size(i);
    return n;
}

// 8-bit values for like's shape, in rows that start on 16 bytes.
at::Tensor alloc_fp8(const at::Tensor& like) {
    const int64_t dims = like.dim();
    std::vector<int64_t> strides(dims, 1);
    int64_t next = (like.size(-1) + 15) / 16 * 16;
    for (int64_t i = dims - 2; i >= 0; --i) {
        strides[i] = next;
        next *= like.size(i) > 0 ? like.size(i) : 1;
    }
    return at::detail::empty_strided_cuda(like.sizes(), strides, at::kFloat8_e4m3fn, like.device());
}

// Scales of `rows` x `cols` values: those of consecutive rows lie together.
at::Tensor alloc_scales(int64_t rows, int64_t cols, int64_t block, const at::Tensor& like) {
    const int64_t up = (rows + block - 1) / block, across = (cols + kFp8Block - 1) / kFp8Block;
    return at::detail::empty_strided_cuda({up, across}, {1, up > 0 ? up : 1}, at::kFloat, like.device());
}

// q, whose last dimension is contiguous and whose rows have one stride, with scales [rows / block, cols / 128]; block 0: 1 or
// 128, by the scales' rows.
gs_fp8 fp8_of(const at::Tensor& q, const at::Tensor& scale, int64_t block, const at::Tensor& like, const char* where) {
    if (!q.is_cuda() || q.scalar_type() != at::kFloat8_e4m3fn || q.device() != like.device())
        refuse(where, "8-bit values must be float8_e4m3fn CUDA tensors on ", like.device());
    const Rows rows = rows_of(q, q, where);
    const int64_t across = (q.size(-1) + kFp8Block - 1) / kFp8Block;
    if (scale.scalar_type() != at::kFloat || scale.dim() != 2 || scale.device() != like.device())
        refuse(where, "scales must be a float32 tensor of two dimensions on ", like.device());
    const int64_t n = leading(q);
    if (block == 0) block = scale.size(0) == n ? 1 : kFp8Block;
    if (scale.size(0) != (n + block - 1) / block || scale.size(1) != across)
        refuse(where, "scales of shape ", shape(scale.sizes()), " for values of shape ", shape(q.sizes()));
    return {q.data_ptr(), rows.stride, scale.data_ptr<float>(), scale.stride(0), scale.stride(1), (int32_t)block};
}

// rms_norm_fwd(x, weight, residual, eps, fp8, out)
PyObject* rms_norm_fwd(PyObject* const* arg) {
    const bool fp8 = PyObject_IsTrue(arg[4]) == 1;
    const char* me = fp8 ? "gs_rms_norm_fp8" : "gs_rms_norm_fwd";
    const at::Tensor& x = tensor(arg[0], me);
    const int dtype = dtype_code(x, me);
    const Rows rows = rows_of(x, x, me);
    const Given weight(arg[1], me), residual(arg[2], me);
    check_vector(weight, x, me);
    const int64_t cols = x.size(-1), r_stride = residual ? rows_of(*residual, x, me).stride : 0;
    const double eps = PyFloat_AsDouble(arg[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised();
    at::Tensor out[4];  // y or q, (scale,) h, rstd
    const int n = fp8 ? 4 : 3;
    at::Tensor &h = out[n - 2], &rstd = out[n - 1];
    int64_t h_stride = cols, y_stride = cols;
    if (arg[5] == Py_None) {
        out[0] = fp8 ? alloc_fp8(x) : alloc(x.sizes(), x.scalar_type(), x);
        if (fp8) out[1] = alloc_scales(rows.n, cols, 1, x);
        if (residual) h = alloc(x.sizes(), x.scalar_type(), x);
        rstd = alloc({rows.n}, at::kFloat, x);
    } else {
        const Items given(arg[5], n, me);
        for (int i = 0; i < n; ++i)
            if (i != n - 2 || residual) out[i] = tensor(given[i], me);
        if (!fp8) y_stride = rows_of(out[0], x, me).stride;
        else if (out[0].sizes() != x.sizes()) refuse(me, "8-bit values of shape ", shape(x.sizes()), " are needed, got ", shape(out[0].sizes()));
        if (residual) h_stride = rows_of(h, x, me).stride;
        check_floats(rstd, {rows.n}, x, me);
    }
    gs_fp8 q{};
    if (fp8) q = fp8_of(out[0], out[1], 1, x, me);
    call(x, me, [&](void* stream) {
        return gs_rms_norm_fwd(x.data_ptr(), rows.stride, residual.address(), r_stride, rows.n, cols, dtype, weight.address(),
                               weight ? dtype_code(*weight, me) : dtype, (float)eps, residual ? address_of(h) : nullptr, h_stride,
                               fp8 ? nullptr : out[0].data_ptr(), y_stride, fp8 ? &q : nullptr, rstd.data_ptr<float>(), stream);
    });
    if (!residual) h = x;
    return tuple_of(out, n);
}

// rms_norm_bwd(dy, h, rstd, weight, dh, out, workspace)
PyObject* rms_norm_bwd(PyObject* const* arg) {
    const char* me = "gs_rms_norm_bwd";
    const at::Tensor &dy = tensor(arg[0], me), &h = tensor(arg[1], me), &rstd = tensor(arg[2], me);
    const int dtype = dtype_code(h, me);
    const Rows rows = rows_of(h, h, me);
    const int64_t cols = h.size(-1), dy_stride = rows_of(dy, h, me).stride;
    const Given weight(arg[3], me), dh(arg[4], me), room(arg[6], me);
    check_vector(weight, h, me);
    check_floats(rstd, {rows.n}, h, me);
    const int64_t dh_stride = dh ? rows_of(*dh, h, me).stride : 0;
    at::Tensor out[2];
    int64_t dx_stride = cols;
    if (arg[5] == Py_None) {
        out[0] = alloc(h.sizes(), h.scalar_type(), h);
        if (weight) out[1] = alloc({cols}, weight->scalar_type(), h);
    } else {
        const Items given(arg[5], 2, me);
        out[0] = tensor(given[0], me);
        dx_stride = rows_of(out[0], h, me).stride;
        const Given g(given[1], me);
        check_vector(g, h, me);
        if (g && weight && g->scalar_type() != weight->scalar_type()) refuse(me, "weight and dweight must have one dtype");
        if (g) out[1] = *g;
    }
    const int kind = weight ? dtype_code(*weight, me) : out[1].defined() ? dtype_code(out[1], me) : dtype;
    at::Tensor own;
    const size_t need = out[1].defined() ? gs_rms_norm_workspace_bytes(rows.n, cols) : 0;
    void* workspace = workspace_of(room, need, own, h, me);
    call(h, me, [&](void* stream) {
        return gs_rms_norm_bwd(dy.data_ptr(), dy_stride, h.data_ptr(), rows.stride, dh.address(), dh_stride, rows.n, cols, dtype,
                               rstd.data_ptr<float>(), weight.address(), kind, out[0].data_ptr(), dx_stride,
                               out[1].defined() ? address_of(out[1]) : nullptr, workspace, need, stream);
    });
    return tuple_of(out, 2);
}

// quantize_fp8(x, block_rows, out)
PyObject* quantize_fp8(PyObject* const* arg) {
    const char* me = "gs_quantize_fp8";
    const at::Tensor& x = tensor(arg[0], me);
    const int dtype = dtype_code(x, me);
    const int64_t block = PyLong_AsLongLong(arg[1]);
    if (block == -1 && PyErr_Occurred()) throw Raised();
    if (block != 1 && block != kFp8Block) refuse(me, "block_rows must be 1 or 128, got ", block);
    if (x.dim() == 0) refuse(me, "the last dimension must be contiguous");
    const int64_t cols = x.size(-1);
    int64_t rows, row_stride, col_stride = 1;
    if (x.dim() == 2 && x.stride(1) != 1 && x.stride(0) == 1) {  // a transposed matrix
        rows = x.size(0);
        row_stride = 1;
        col_stride = x.stride(1);
    } else {
        row_stride = rows_of(x, x, me).stride;
        rows = leading(x);
    }
    at::Tensor out[2];
    if (arg[2] == Py_None) {
        out[0] = alloc_fp8(x);
        out[1] = alloc_scales(rows, cols, block, x);
    } else {
        const Items given(arg[2], 2, me);
        for (int i = 0; i < 2; ++i) out[i] = tensor(given[i], me);
        if (out[0].sizes() != x.sizes()) refuse(me, "8-bit values of shape ", shape(x.sizes()), " are needed, got ", shape(out[0].sizes()));
    }
    const gs_fp8 q = fp8_of(out[0], out[1], block, x, me);
    call(x, me, [&](void* stream) { return gs_quantize_fp8(x.data_ptr(), row_stride, col_stride, rows, cols, dtype, &q, stream); });
    return tuple_of(out, 2);
}

// matmul_fp8(a, a_scale, b, b_scale, dtype, out); dtype: GS_DTYPE_*, or -1: out's
PyObject* matmul_fp8(PyObject* const* arg) {
    const char* me = "gs_matmul_fp8";
    const at::Tensor &a = tensor(arg[0], me), &a_scale = tensor(arg[1], me), &b = tensor(arg[2], me), &b_scale = tensor(arg[3], me);
    if (a.dim() == 0 || b.dim() != 2 || a.size(-1) != b.size(1))
        refuse(me, "a [.., k] and b [n, k] are needed, got ", shape(a.sizes()), " and ", shape(b.sizes()));
    const gs_fp8 qa = fp8_of(a, a_scale, 1, a, me), qb = fp8_of(b, b_scale, 0, a, me);
    long code = PyLong_AsLong(arg[4]);
    if (code == -1 && PyErr_Occurred()) throw Raised();
    const int64_t n = b.size(0), k = b.size(1);
    const int64_t m = leading(a);
    int64_t stride = n;
    std::vector<int64_t> sizes(a.sizes().begin(), a.sizes().end());
    sizes.back() = n;
    at::Tensor out;
    if (arg[5] == Py_None) {
        out = alloc(sizes, code == GS_DTYPE_F32 ? at::kFloat : code == GS_DTYPE_F16 ? at::kHalf : at::kBFloat16, a);
    } else {
        out = tensor(arg[5], me);
        const int own = dtype_code(out, me);
        if ((code >= 0 && code != own) || out.sizes() != at::IntArrayRef(sizes) || out.device() != a.device())
            refuse(me, "a result of shape ", shape(sizes), " and the dtype asked for is needed on ", a.device());
        code = own;
        stride = rows_of(out, out, me).stride;
    }
    if (code < 0) code = GS_DTYPE_BF16;
    call(a, me, [&](void* stream) { return gs_matmul_fp8(&qa, &qb, m, n, k, (int32_t)code, out.data_ptr(), stride, stream); });
    return wrap(out);
}

// clip_grads(grads, max_norm, eps, out, norm, workspace); max_norm None: the norm alone
PyObject* clip_grads(PyObject* const* arg) {
    const char* me = "gs_clip_grads";
    PyObject* fast = PySequence_Fast(arg[0], "a list of tensors is needed");
    if (!fast) throw Raised();
    struct Release {
        PyObject* o;
        ~Release() { Py_XDECREF(o); }
    } grads{fast}, outs{nullptr};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
    if (n == 0 || n > 1000000) refuse(me, "1 to 1,000,000 gradients are needed, got ", n);
    const bool clip = arg[1] != Py_None;
    const double max_norm = clip ? PyFloat_AsDouble(arg[1]) : 0.0, eps = PyFloat_AsDouble(arg[2]);
    if (PyErr_Occurred()) throw Raised();
    if (arg[3] != Py_None) {
        if (!clip) refuse(me, "out without max_norm");
        if (!(outs.o = PySequence_Fast(arg[3], "a list of tensors is needed"))) throw Raised();
        if (PySequence_Fast_GET_SIZE(outs.o) != n) refuse(me, n, " outputs are needed");
    }
    std::vector<gs_gradient> list(n);
    const at::Tensor& first = tensor(PySequence_Fast_GET_ITEM(fast, 0), me);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor& g = tensor(PySequence_Fast_GET_ITEM(fast, i), me);
        list[i].dtype = dtype_code(g, me);
        if (g.device() != first.device()) refuse(me, "gradient ", i, " is not on ", first.device());
        if (!g.is_non_overlapping_and_dense()) refuse(me, "gradient ", i, " is not one piece of memory");
        list[i].grad = address_of(g);
        list[i].n = g.numel();
        list[i].out = nullptr;
        if (!outs.o) continue;
        const at::Tensor& o = tensor(PySequence_Fast_GET_ITEM(outs.o, i), me);
        if (o.scalar_type() != g.scalar_type() || o.device() != g.device() || o.sizes() != g.sizes() || (g.numel() > 1 && o.strides() != g.strides()))
            refuse(me, "output ", i, " must have the shape, strides, dtype and device of its gradient");
        list[i].out = address_of(o);
    }
    const Given given(arg[4], me), room(arg[5], me);
    at::Tensor norm;
    if (given) {
        norm = *given;
        check_floats(norm, {}, first, me);
    } else {
        norm = alloc({}, at::kFloat, first);
    }
    size_t need;
    {
        const c10::cuda::OptionalCUDAGuard guard(first.device());  // the size depends on the device's number of SMs
        need = gs_clip_workspace_bytes(list.data(), (int32_t)n);
    }
    at::Tensor own;
    void* workspace = workspace_of(room, need, own, first, me);
    call(first, me, [&](void* stream) {
        return gs_clip_grads(list.data(), (int32_t)n, clip, max_norm, eps, norm.data_ptr<float>(), workspace, need, stream);
    });
    return wrap(norm);
}

// init(check, memory_error)
PyObject* init(PyObject* const* arg) {
    Py_INCREF(arg[0]);
    Py_XSETREF(g_check, arg[0]);
    Py_INCREF(arg[1]);
    Py_XSETREF(g_memory, arg[1]);
    Py_RETURN_NONE;
}

// A Python function of N positional arguments; C++ exceptions become Python's.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments are needed, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(arg);
    } catch (const Raised&) {
    } catch (const Refusal& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_memory, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<init, 2>("init"),
                         method<layer_norm_fwd, 5>("layer_norm_fwd"),
                         method<layer_norm_bwd, 7>("layer_norm_bwd"),
                         method<attention_workspace_bytes, 5>("cross_attention_workspace_bytes"),
                         method<attention_fwd, 8>("cross_attention_fwd"),
                         method<attention_bwd, 11>("cross_attention_bwd"),
                         method<rms_norm_fwd, 6>("rms_norm_fwd"),
                         method<rms_norm_bwd, 7>("rms_norm_bwd"),
                         method<quantize_fp8, 3>("quantize_fp8"),
                         method<matmul_fp8, 6>("matmul_fp8"),
                         method<clip_grads, 6>("clip_grads"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "gs_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gs_bind() { return PyModule_Create(&module); }
