// gdla_binding.cpp - the Python side of the paged-cache calls.
//
// gdla_cache_append and gdla_attn_decode_paged run once per layer and token, with eleven to
// thirteen tensors each; checking those attribute by attribute from Python and passing 25
// arguments through ctypes took 12 to 15 us a call, more than most of their kernels. Here the
// same checks read the tensors directly. The library's functions come in by address (bind), so
// this module has nothing of it linked in; PyTorch gives memory, the current stream and the errors' types.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "gdla.h"

namespace {

constexpr int64_t kGroup = GDLA_GROUP, kDqk = GDLA_DQK, kDv = GDLA_DV, kDr = GDLA_DR;

decltype(&gdla_cache_append) append_fn = nullptr;
decltype(&gdla_attn_decode_paged) decode_fn = nullptr;
decltype(&gdla_decode_paged_workspace_bytes) workspace_fn = nullptr;

struct Raised {};  // a Python error is set

[[noreturn]] void fail(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw Raised();
}
std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}
// A tensor of this type and shape on device `dev` (any strides).
const at::Tensor &shaped(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape,
                         int64_t dev) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, std::string(name) + ": expected " + at::toString(type) + ", got " + at::toString(t.scalar_type()));
    if (t.sizes() != at::IntArrayRef(shape))
        fail(PyExc_ValueError, std::string(name) + ": expected shape " + text(shape) + ", got " + text(t.sizes()));
    if (t.get_device() != dev)
        fail(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", k_pages on another device");
    return t;
}
void *dense(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape, int64_t dev) {
    const at::Tensor &t = shaped(o, name, type, shape, dev);
    if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
}

// bf16 rows whose last dimension is dense; the others may be views.
struct Rows {
    void *ptr;
    long long token, head;
};
Rows rows(PyObject *o, const char *name, std::initializer_list<int64_t> shape, int64_t dev) {
    const at::Tensor &t = shaped(o, name, at::kBFloat16, shape, dev);
    const int64_t n = t.dim();
    if (t.stride(n - 1) != 1) fail(PyExc_ValueError, std::string(name) + ": its last dimension must be contiguous");
    Rows r{t.data_ptr(), 0, 0};
    // one row: its stride says nothing
    if (t.size(0) != 1) r.token = t.stride(0);
    if (n == 3 && t.size(1) != 1) r.head = t.stride(1);
    if ((r.token | r.head) & 7)
        fail(PyExc_ValueError, std::string(name) + ": strides must be multiples of 8 elements, got " + text(t.strides()));
    return r;
}

struct Cache {
    int64_t dev, pages, heads, page, batch, width;
    int kind;
    void *k, *v, *table, *lens;
    float *k_scale, *v_scale;
};
Cache cache(PyObject *k_pages, PyObject *v_pages, PyObject *k_scale, PyObject *v_scale, PyObject *block_table,
            PyObject *seqlens_k) {
    const at::Tensor &k = tensor(k_pages, "k_pages"), &bt = tensor(block_table, "block_table");
    if (k.dim() != 4 || bt.dim() != 2)
        fail(PyExc_ValueError, "expected k_pages [pages, H, page_size, 192] and block_table [batch, pages per sequence]");
    Cache c{};
    c.dev = k.get_device();
    c.pages = k.size(0);
    c.heads = k.size(1);
    c.page = k.size(2);
    c.batch = bt.size(0);
    c.width = bt.size(1);
    const at::ScalarType type = k.scalar_type();
    if (type == at::kBFloat16) {
        c.kind = GDLA_CACHE_BF16;
        if (k_scale != Py_None || v_scale != Py_None) fail(PyExc_ValueError, "k_scale and v_scale belong to an e4m3 cache");
    } else if (type == at::kFloat8_e4m3fn) {
        c.kind = GDLA_CACHE_E4M3;
        c.k_scale = static_cast<float *>(dense(k_scale, "k_scale", at::kFloat, {c.pages, c.heads}, c.dev));
        c.v_scale = static_cast<float *>(dense(v_scale, "v_scale", at::kFloat, {c.pages, c.heads}, c.dev));
    } else {
        fail(PyExc_TypeError, std::string("k_pages: expected BFloat16 or Float8_e4m3fn, got ") + at::toString(type));
    }
    c.k = dense(k_pages, "k_pages", type, {c.pages, c.heads, c.page, kDqk}, c.dev);
    c.v = dense(v_pages, "v_pages", type, {c.pages, c.heads, c.page, kDv}, c.dev);
    c.table = dense(block_table, "block_table", at::kInt, {c.batch, c.width}, c.dev);
    c.lens = dense(seqlens_k, "seqlens_k", at::kInt, {c.batch}, c.dev);
    for (int64_t x : {c.pages, c.heads, c.page, c.batch, c.width})
        if (x > INT32_MAX) fail(PyExc_ValueError, "a size of the cache is 2^31 or more");
    return c;
}

int as_int(PyObject *o, const char *name) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised();
    if (x > INT32_MAX || x < INT32_MIN) fail(PyExc_ValueError, std::string(name) + " is outside 32 bits");
    return static_cast<int>(x);
}

// The launch stream: the given one (a torch.cuda.Stream), else the current one. It has to be of the tensors' device
// and that the current one, as the library launches there.
c10::cuda::CUDAStream launch_stream(PyObject *given, int64_t dev) {
    if (dev < 0) fail(PyExc_ValueError, "the tensors must be on a CUDA device");
    const int64_t now = c10::cuda::current_device();
    if (given == Py_None) {
        if (now != dev)
            fail(PyExc_ValueError, "the tensors are on cuda:" + std::to_string(dev) + " but the launch stream is on cuda:" +
                                       std::to_string(now));
        return c10::cuda::getCurrentCUDAStream();
    }
    PyObject *raw = PyObject_GetAttrString(given, "cuda_stream"), *index = PyObject_GetAttrString(given, "device_index");
    const long long ptr = raw ? PyLong_AsLongLong(raw) : -1;
    const long of = index ? PyLong_AsLong(index) : -1;
    Py_XDECREF(raw);
    Py_XDECREF(index);
    if (PyErr_Occurred()) throw Raised();
    if (of != dev || now != dev)
        fail(PyExc_ValueError, "the tensors are on cuda:" + std::to_string(dev) + " but the launch stream is on cuda:" +
                                   std::to_string(of) + " (current device cuda:" + std::to_string(now) + ")");
    return c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(ptr), static_cast<c10::DeviceIndex>(dev));
}

// Memory that a call makes itself, for kernels on stream `on`. The allocator hands out a freed block as soon as its own
// stream's order allows, so memory of the current stream may still be in use there when another stream writes it: it
// comes from the launch stream's blocks. The caller has it on the current stream, which is made known to the allocator for
// the day it is freed.
at::Tensor empty_for(const c10::cuda::CUDAStream &on, at::IntArrayRef shape, const at::TensorOptions &options) {
    const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(on.device_index());
    if (now.stream() == on.stream()) return at::empty(shape, options);
    at::Tensor t;
    {
        const c10::cuda::CUDAStreamGuard guard(on);
        t = at::empty(shape, options);
    }
    t.record_stream(now);
    return t;
}

template <class F>
PyObject *guarded(F &&f) {
    try {
        return f();
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return false;
}

// (k_nope, k_rope, v, k_pages, v_pages, block_table, cu_seqlens_new, seqlens_k, k_scale, v_scale, rotate, stream) -> status
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 12)) return nullptr;
    return guarded([&] {
        const Cache c = cache(a[3], a[4], a[8], a[9], a[5], a[7]);
        const at::Tensor &vt = tensor(a[2], "v");
        const int64_t n = vt.dim() > 0 ? vt.size(0) : -1;
        const Rows k = rows(a[0], "k_nope", {n, c.heads, kDqk - kDr}, c.dev);
        const Rows r = rows(a[1], "k_rope", {n, kDr}, c.dev);
        const Rows v = rows(a[2], "v", {n, c.heads, kDv}, c.dev);
        const int32_t *cu = static_cast<const int32_t *>(dense(a[6], "cu_seqlens_new", at::kInt, {c.batch + 1}, c.dev));
        const int rotate = PyObject_IsTrue(a[10]);
        if (rotate < 0) throw Raised();
        if (n > INT32_MAX) fail(PyExc_ValueError, "2^31 new tokens or more");
        cudaStream_t stream = launch_stream(a[11], c.dev).stream();
        gdla_status_t st;
        Py_BEGIN_ALLOW_THREADS;
        st = append_fn(k.ptr, k.token, k.head, r.ptr, r.token, v.ptr, v.token, v.head, c.k, c.v, c.k_scale, c.v_scale,
                       c.kind, static_cast<int>(c.pages), static_cast<int>(c.page), static_cast<const int32_t *>(c.table),
                       static_cast<int>(c.width), cu, static_cast<int>(n), static_cast<const int32_t *>(c.lens),
                       static_cast<int>(c.batch), static_cast<int>(c.heads), rotate, stream);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(st);
    });
}

// (q_sig, q_noise, k_pages, v_pages, block_table, seqlens_k, max_seqlen_k, lam, gate, window, sinks, k_scale, v_scale,
//  rotate, out, workspace, stream) -> out, or a status that is not 0
PyObject *attn_decode_paged(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 17)) return nullptr;
    return guarded([&]() -> PyObject * {
        const Cache c = cache(a[2], a[3], a[11], a[12], a[4], a[5]);
        const int64_t hs = kGroup * c.heads;
        const void *qs = dense(a[0], "q_sig", at::kBFloat16, {c.batch, hs, kDqk}, c.dev);
        const void *qn = dense(a[1], "q_noise", at::kBFloat16, {c.batch, c.heads, kDqk}, c.dev);
        const float *lam = static_cast<const float *>(dense(a[7], "lam", at::kFloat, {c.batch, hs}, c.dev));
        const void *gate = dense(a[8], "gate", at::kBFloat16, {c.batch, hs, kDv}, c.dev);
        const int most = as_int(a[6], "max_seqlen_k"), window = as_int(a[9], "window"), sinks = as_int(a[10], "sinks");
        const int rotate = PyObject_IsTrue(a[13]);
        if (rotate < 0) throw Raised();
        at::Tensor made, scratch;
        void *out;
        const auto on = launch_stream(a[16], c.dev);
        if (a[14] == Py_None) {
            made = empty_for(on, {c.batch, hs, kDv}, at::TensorOptions().dtype(at::kBFloat16).device(at::kCUDA, c.dev));
            out = made.data_ptr();
        } else {
            out = dense(a[14], "out", at::kBFloat16, {c.batch, hs, kDv}, c.dev);
        }
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (a[15] != Py_None) {
            const at::Tensor &w = tensor(a[15], "workspace");
            if (w.get_device() != c.dev || !w.is_contiguous())
                fail(PyExc_ValueError, "workspace must be a contiguous CUDA tensor on the device of the others");
            ws = w.data_ptr();
            ws_bytes = w.nbytes();
        } else if ((ws_bytes = workspace_fn(static_cast<int>(c.batch), static_cast<int>(c.heads), most, window, sinks)) > 0) {
            scratch = empty_for(on, {static_cast<int64_t>(ws_bytes)}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, c.dev));
            ws = scratch.data_ptr();
        }
        gdla_status_t st;
        Py_BEGIN_ALLOW_THREADS;
        st = decode_fn(qs, qn, c.k, c.v, c.k_scale, c.v_scale, c.kind, static_cast<int>(c.pages), static_cast<int>(c.page),
                       static_cast<const int32_t *>(c.table), static_cast<int>(c.width),
                       static_cast<const int32_t *>(c.lens), most, lam, gate, out, static_cast<int>(c.batch),
                       static_cast<int>(c.heads), window, sinks, rotate, ws, ws_bytes, on.stream());
        Py_END_ALLOW_THREADS;
        if (st != GDLA_OK) return PyLong_FromLong(st);
        if (made.defined()) return THPVariable_Wrap(made);
        Py_INCREF(a[14]);
        return a[14];
    });
}

// (address of gdla_cache_append, gdla_attn_decode_paged, gdla_decode_paged_workspace_bytes)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arity(n_args, 3)) return nullptr;
    append_fn = reinterpret_cast<decltype(append_fn)>(PyLong_AsVoidPtr(a[0]));
    decode_fn = reinterpret_cast<decltype(decode_fn)>(PyLong_AsVoidPtr(a[1]));
    workspace_fn = reinterpret_cast<decltype(workspace_fn)>(PyLong_AsVoidPtr(a[2]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
constexpr PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

}  // namespace

PyMODINIT_FUNC PyInit__gdla_binding(void) {
    static PyMethodDef methods[] = {method<cache_append>("cache_append"), method<attn_decode_paged>("attn_decode_paged"),
                                    method<bind>("bind"), {nullptr, nullptr, 0, nullptr}};
    static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdla_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
    return PyModule_Create(&module);
}
