// The decoder operators' calls on torch tensors: checks, allocation of what the caller leaves out, the device's
// current stream, and the C entry. A Python module of four functions and one size, wrapped with their documentation in
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

// An argument that may be None.
struct Given {
    const at::Tensor* t;
    Given(PyObject* o, const char* where) : t(o == Py_None ? nullptr : &tensor(o, where)) {}
    explicit operator bool() const { return t != nullptr; }
    const at::Tensor& operator*() const { return *t; }
    const at::Tensor* operator->() const { return t; }
    void* address() const { return t ? t->data_ptr() : nullptr; }
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
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "gs_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gs_bind() { return PyModule_Create(&module); }
