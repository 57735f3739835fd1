// Python binding of the attention path's and the prompt's calls for torch tensors: a CPython module that checks
// and marshals arguments and calls the C ABI through the addresses that bind() receives (the
// library that the package has loaded).  These calls run once per layer and step, and at decode
// sizes their host time is the call's time.  Measured per call on GB300's host: 2.7 to 3.0 us, of
// which the launch is 2; with the checks in Python and ctypes it was 8.2 to 10.6 us.
#include <Python.h>

#include <algorithm>
#include <cstdint>
#include <exception>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "qgemv.h"

namespace {

decltype(&qg_cache_pages) call_cache_pages;
decltype(&qg_qk_norm_rope) call_qk_norm_rope;
decltype(&qg_cache_append) call_cache_append;
decltype(&qg_attention) call_attention;
decltype(&qg_packed_bytes) call_packed_bytes;
decltype(&qgemm) call_gemm;
decltype(&qgemm_experts) call_gemm_experts;
decltype(&qg_prompt_attention) call_prompt_attention;

struct Refused {};                       // a Python error is set

[[noreturn]] void refuse(PyObject* type, const char* name, const char* what) {
    PyErr_Format(type, "%s: %s", name, what);
    throw Refused{};
}

const at::Tensor* tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, "a tensor is needed");
    return &THPVariable_Unpack(o);
}
long long integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) refuse(PyExc_TypeError, name, "an integer is needed");
    return v;
}
int small(PyObject* o, const char* name) {
    const long long v = integer(o, name);
    if (v < -2147483647 || v > 2147483647) refuse(PyExc_ValueError, name, "out of range");
    return int(v);
}
float real(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) refuse(PyExc_TypeError, name, "a number is needed");
    return float(v);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v == 1;
}
void* address(PyObject* o) {
    void* const p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Refused{};
    return p;
}

// Kernels are launched on the current device, so a call's tensors have to be there: looked up
// at a call's first tensor (the interpreter's lock is held throughout), -1 before.
int current_device = -1;
void on_device(int device, const char* name) {
    if (current_device < 0) current_device = c10::cuda::current_device();
    if (device != current_device) refuse(PyExc_ValueError, name, "not on the current CUDA device");
}

// A contiguous CUDA tensor of one type with at least n entries (None gives null).
template <typename T> T* typed(PyObject* o, at::ScalarType type, const char* name, int64_t n = 0) {
    const at::Tensor* t = tensor(o, name);
    if (!t) return nullptr;
    if (!t->is_cuda() || t->scalar_type() != type || !t->is_contiguous() || t->numel() < n)
        refuse(PyExc_ValueError, name, "a contiguous CUDA tensor of the documented type and size is needed");
    on_device(t->device().index(), name);
    return static_cast<T*>(t->data_ptr());
}
int32_t* i32(PyObject* o, const char* name, int64_t n = 0) { return typed<int32_t>(o, at::kInt, name, n); }
float* f32(PyObject* o, const char* name, int64_t n = 0) { return typed<float>(o, at::kFloat, name, n); }

// Activations [n_tok, heads, head_dim] whose heads are contiguous (a slice of a projection's row is).
struct Heads {
    void* p = nullptr;
    int64_t stride = 0, n = 0, heads = 0, dim = 0;
};
Heads heads(PyObject* o, at::ScalarType type, const char* name) {
    const at::Tensor* t = tensor(o, name);
    Heads h;
    if (!t) return h;
    if (t->dim() != 3 || !t->is_cuda() || t->scalar_type() != type || t->stride(2) != 1 ||
        (t->size(1) > 1 && t->stride(1) != t->size(2)))
        refuse(PyExc_ValueError, name, "a CUDA [n_tok, heads, head_dim] tensor of one type, heads contiguous, is needed");
    on_device(t->device().index(), name);
    h.p = t->data_ptr();
    h.n = t->size(0);
    h.heads = t->size(1);
    h.dim = t->size(2);
    h.stride = h.n > 1 ? t->stride(0) : h.heads * h.dim;      // (of one token it means nothing)
    return h;
}
at::ScalarType act_type(PyObject* o, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!t) refuse(PyExc_TypeError, name, "a tensor is needed");
    if (t->scalar_type() != at::kFloat && t->scalar_type() != at::kBFloat16)
        refuse(PyExc_TypeError, name, "activations are float32 or bfloat16 tensors");
    return t->scalar_type();
}
qg_act act_of(at::ScalarType t) { return t == at::kFloat ? QG_ACT_F32 : QG_ACT_BF16; }

struct Table { int32_t* p; int64_t width; };
Table table(PyObject* o, int64_t n_req) {
    const at::Tensor* t = tensor(o, "table");
    if (!t || t->dim() != 2 || t->size(0) < n_req) refuse(PyExc_ValueError, "table", "a contiguous CUDA int32 [n_req, width] tensor is needed");
    return {i32(o, "table"), t->size(1)};
}
int64_t length(PyObject* o, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!t || t->dim() != 1) refuse(PyExc_ValueError, name, "a vector is needed");
    return t->size(0);
}

int64_t entries(PyObject* o, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!t) refuse(PyExc_ValueError, name, "a tensor is needed");
    return t->numel();
}

struct Rotation { const float* cs = nullptr; int64_t n_pos = 0; int rot = 0; const int32_t* pos = nullptr; };
Rotation rotation(PyObject* cos_sin, PyObject* positions, int64_t n) {
    Rotation r;
    r.pos = i32(positions, "positions", n);
    if (const at::Tensor* t = tensor(cos_sin, "cos_sin")) {
        if (t->dim() != 2) refuse(PyExc_ValueError, "cos_sin", "a contiguous CUDA float32 [n_pos, rot_dim] tensor is needed");
        r.cs = f32(cos_sin, "cos_sin");
        r.n_pos = t->size(0);
        r.rot = int(std::min<int64_t>(t->size(1), 1 << 20));
    }
    return r;
}

void* stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    if (PyLong_Check(o)) return address(o);
    PyObject* const h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Refused{};
    void* const s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Refused{};
    return s;
}
// device: of the cache's tensor, -1 for one that is given by its address.
const qg_cache& cache_at(PyObject* o, PyObject* device) {
    const qg_cache* const c = static_cast<const qg_cache*>(address(o));
    if (!c) refuse(PyExc_ValueError, "cache", "a qg_cache is needed");
    const long long d = integer(device, "cache");
    if (d >= 0) on_device(int(std::min<long long>(d, 1 << 30)), "cache");
    return *c;
}

template <typename F> PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
    if (got != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    current_device = -1;
    try {
        return PyLong_FromLong(f());
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// held, fresh, free_pages, table, seq_len, cu_new, slots, positions, page_tokens, free_begin, free_end, stream
PyObject* cache_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 12, [&] {
        const int64_t n = length(a[0], "held"), n_tok = entries(a[6], "slots"), n_free = entries(a[2], "free_pages");
        const Table t = table(a[3], n);
        return call_cache_pages(i32(a[0], "held"), i32(a[1], "fresh", n), int(std::min<int64_t>(n, 1 << 30)), small(a[8], "page_tokens"),
                              i32(a[2], "free_pages"), n_free, i32(a[9], "free_begin", 1), i32(a[10], "free_end", 1), t.p, t.width,
                              i32(a[4], "seq_len", n), i32(a[5], "cu_new", n + 1), typed<int64_t>(a[6], at::kLong, "slots"),
                              i32(a[7], "positions", n_tok), n_tok, stream_of(a[11]));
    });
}

unsigned head_flags(PyObject* norm, PyObject* unit, PyObject* inter) {
    return (truth(inter) ? QG_ROPE_INTERLEAVED : 0u) | (truth(unit) ? QG_NORM_UNIT_OFFSET : 0u) | (truth(norm) ? 0u : QG_NORM_NONE);
}

// q, k, q_out, k_out, positions, cos_sin, q_weight, k_weight, eps, norm, unit_offset, interleaved, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 13, [&] {
        const at::ScalarType type = act_type(a[0], "q");
        const Heads q = heads(a[0], type, "q"), k = heads(a[1], type, "k"), qo = heads(a[2], type, "q_out"), ko = heads(a[3], type, "k_out");
        if (q.n != k.n || q.n != qo.n || q.n != ko.n || q.dim != k.dim || q.dim != qo.dim || q.dim != ko.dim || q.heads != qo.heads ||
            k.heads != ko.heads || q.dim > 65536 || q.heads > 65536 || k.heads > 65536)
            refuse(PyExc_ValueError, "qg_qk_norm_rope", "q, k and their outputs differ in tokens, heads or head_dim");
        const Rotation r = rotation(a[5], a[4], q.n);
        return call_qk_norm_rope(act_of(type), q.p, q.stride, k.p, k.stride, q.n, int(q.heads), int(k.heads), int(q.dim),
                               f32(a[6], "q_weight", q.dim), f32(a[7], "k_weight", q.dim), real(a[8], "eps"),
                               head_flags(a[9], a[10], a[11]), r.cs, r.n_pos, r.rot, r.pos, qo.p, qo.stride, ko.p, ko.stride,
                               stream_of(a[12]));
    });
}

// cache address, k, v, slots, q, q_out, positions, cos_sin, q_weight, k_weight, eps, norm, unit_offset, interleaved,
// k_back, v_back, stream, cache device
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 18, [&] {
        const qg_cache& cache = cache_at(a[0], a[17]);
        const at::ScalarType type = act_type(a[1], "k");
        const Heads k = heads(a[1], type, "k"), v = heads(a[2], type, "v"), q = heads(a[4], type, "q"), qo = heads(a[5], type, "q_out");
        if (v.n != k.n || k.heads != cache.n_kv_heads || v.heads != k.heads || k.dim != cache.head_dim || v.dim != k.dim)
            refuse(PyExc_ValueError, "qg_cache_append", "k and v do not fit the cache's heads");
        if (q.p && (q.n != k.n || qo.n != k.n || q.dim != k.dim || qo.dim != k.dim || q.heads != qo.heads || q.heads > 65536))
            refuse(PyExc_ValueError, "qg_cache_append", "q and q_out differ from k in tokens or head_dim");
        const int64_t values = k.n * k.heads * k.dim;
        void* const kb = typed<void>(a[14], type, "k_back", values);
        void* const vb = typed<void>(a[15], type, "v_back", values);
        const Rotation r = rotation(a[7], a[6], k.n);
        return call_cache_append(&cache, act_of(type), q.p, q.stride, k.p, k.stride, v.p, v.stride, k.n, int(q.heads),
                               f32(a[8], "q_weight", k.dim), f32(a[9], "k_weight", k.dim), real(a[10], "eps"),
                               head_flags(a[11], a[12], a[13]), r.cs, r.n_pos, r.rot, r.pos,
                               typed<int64_t>(a[3], at::kLong, "slots", k.n), qo.p, qo.stride, kb, vb, stream_of(a[16]));
    });
}

// cache address, q, table, seq_len, cu_new, out, workspace, scale, max_new, window, span_mask, lse, stream, cache device
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 14, [&] {
        const qg_cache& cache = cache_at(a[0], a[13]);
        const at::ScalarType type = act_type(a[1], "q");
        const Heads q = heads(a[1], type, "q"), out = heads(a[5], type, "out");
        if (!out.p || q.n != out.n || q.heads != out.heads || q.dim != cache.head_dim || out.dim != q.dim || q.heads > 65536)
            refuse(PyExc_ValueError, "qg_attention", "q, out and the cache differ in tokens, heads or head_dim");
        const int64_t n_req = length(a[3], "seq_len");
        const Table t = table(a[2], n_req);
        const at::Tensor* const ws = tensor(a[6], "workspace");
        if (ws && (!ws->is_cuda() || !ws->is_contiguous())) refuse(PyExc_ValueError, "workspace", "a contiguous CUDA tensor is needed");
        if (ws) on_device(ws->device().index(), "workspace");
        return call_attention(&cache, act_of(type), q.p, q.stride, q.n, int(q.heads), t.p, t.width, i32(a[3], "seq_len"),
                            i32(a[4], "cu_new", n_req + 1), int(std::min<int64_t>(n_req, 1 << 30)), small(a[8], "max_new"),
                            small(a[9], "window"), reinterpret_cast<const uint32_t*>(i32(a[10], "span_mask", q.n)), real(a[7], "scale"),
                            out.p, out.stride, f32(a[11], "lse", q.n * q.heads), ws ? ws->data_ptr() : nullptr,
                            ws ? size_t(ws->nbytes()) : 0, stream_of(a[12]));
    });
}

// Rows [n, width] whose values are contiguous.
struct Rows {
    void* p = nullptr;
    int64_t stride = 0, n = 0, width = 0;
};
Rows rows(PyObject* o, at::ScalarType type, const char* name) {
    const at::Tensor* t = tensor(o, name);
    Rows r;
    if (!t) return r;
    if (t->dim() != 2 || !t->is_cuda() || t->scalar_type() != type || (t->size(1) > 1 && t->stride(1) != 1))
        refuse(PyExc_ValueError, name, "a CUDA matrix of one type, rows contiguous, is needed");
    on_device(t->device().index(), name);
    r.p = t->data_ptr();
    r.n = t->size(0);
    r.width = t->size(1);
    r.stride = r.n > 1 ? t->stride(0) : r.width;              // (of one row it means nothing)
    if (r.stride < 0) refuse(PyExc_ValueError, name, "rows go forward");
    return r;
}
// Packed weights: a contiguous CUDA tensor that holds them all, or an address.
const void* packed(PyObject* o, int fmt, int64_t n_rows, int64_t n_in) {
    if (PyLong_Check(o)) return address(o);
    const at::Tensor* t = tensor(o, "W");
    if (!t || !t->is_cuda() || !t->is_contiguous() || size_t(t->nbytes()) < call_packed_bytes(qg_fmt(fmt), n_rows, n_in))
        refuse(PyExc_ValueError, "W", "a contiguous CUDA tensor of qg_packed_bytes() bytes is needed");
    on_device(t->device().index(), "W");
    return t->data_ptr();
}
struct Space { void* p = nullptr; size_t bytes = 0; };
Space space(PyObject* o) {
    const at::Tensor* const t = tensor(o, "workspace");
    if (!t) return {};
    if (!t->is_cuda() || !t->is_contiguous()) refuse(PyExc_ValueError, "workspace", "a contiguous CUDA tensor is needed");
    on_device(t->device().index(), "workspace");
    return {t->data_ptr(), size_t(t->nbytes())};
}

// fmt, W, n_out, n_in, x, y, workspace, bias, activation, residual, stream
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 11, [&] {
        const int fmt = small(a[0], "fmt"), f = small(a[8], "activation");
        const int64_t n_out = integer(a[2], "n_out"), n_in = integer(a[3], "n_in"), width = f == QG_F_SWIGLU ? n_out / 2 : n_out;
        const at::ScalarType type = act_type(a[4], "x");
        const Rows x = rows(a[4], type, "x"), y = rows(a[5], type, "y"), r = rows(a[9], type, "residual");
        if (!y.p && x.n > 0) refuse(PyExc_ValueError, "y", "a tensor is needed");
        if (x.width != n_in || y.n != x.n || y.width != width) refuse(PyExc_ValueError, "qgemm", "x or y does not fit n_in, n_out or the tokens");
        if (a[9] != Py_None && (r.n != x.n || r.width != width)) refuse(PyExc_ValueError, "residual", "a matrix like y is needed");
        const Space ws = space(a[6]);
        return call_gemm(qg_fmt(fmt), packed(a[1], fmt, n_out, n_in), n_out, n_in, act_of(type), x.p, x.stride, x.n, f32(a[7], "bias", n_out),
                         qg_activation(f), r.p, r.stride, y.p, y.stride, ws.p, ws.bytes, stream_of(a[10]));
    });
}

// fmt, W, n_experts, n_out, n_in, x, offsets, y, workspace, rows, activation, stream
PyObject* gemm_experts(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 12, [&] {
        const int fmt = small(a[0], "fmt"), f = small(a[10], "activation"), n_experts = small(a[2], "n_experts");
        const int64_t n_out = integer(a[3], "n_out"), n_in = integer(a[4], "n_in"), width = f == QG_F_SWIGLU ? n_out / 2 : n_out;
        const at::ScalarType type = act_type(a[5], "x");
        const Rows x = rows(a[5], type, "x"), y = rows(a[7], type, "y");
        if (a[7] == Py_None) refuse(PyExc_ValueError, "y", "a tensor is needed");
        if (x.width != n_in || y.width != width) refuse(PyExc_ValueError, "qgemm_experts", "x or y does not fit n_in or n_out");
        if (n_experts < 1 || n_out < 1 || n_out > (int64_t(1) << 31)) refuse(PyExc_ValueError, "qgemm_experts", "n_experts and n_out are positive");
        const int32_t* const offsets = i32(a[6], "offsets", int64_t(n_experts) + 1);
        const int32_t* const which = i32(a[9], "rows", y.n);
        const Space ws = space(a[8]);
        return call_gemm_experts(qg_fmt(fmt), packed(a[1], fmt, int64_t(n_experts) * n_out, n_in), n_experts, n_out, n_in, act_of(type), x.p,
                                 x.stride, x.n, offsets, which, y.n, qg_activation(f), y.p, y.stride, ws.p, ws.bytes, stream_of(a[11]));
    });
}

// q, k, v, cu_seq, out, workspace, scale, longest, window, lse, stream
PyObject* prompt_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 11, [&] {
        const at::ScalarType type = act_type(a[0], "q");
        const Heads q = heads(a[0], type, "q"), k = heads(a[1], type, "k"), v = heads(a[2], type, "v"), out = heads(a[4], type, "out");
        if (a[1] == Py_None || a[2] == Py_None || a[4] == Py_None) refuse(PyExc_ValueError, "qg_prompt_attention", "k, v and out are tensors");
        if (k.n != q.n || v.n != q.n || out.n != q.n || k.dim != q.dim || v.dim != q.dim || out.dim != q.dim || v.heads != k.heads ||
            out.heads != q.heads || q.heads > 65535 || k.heads > 65535 || q.dim > 65536)
            refuse(PyExc_ValueError, "qg_prompt_attention", "q, k, v and out differ in tokens, heads or head_dim");
        const int64_t n_seq = length(a[3], "cu_seq") - 1;
        if (n_seq < 0) refuse(PyExc_ValueError, "cu_seq", "n_seq + 1 entries are needed");
        const Space ws = space(a[5]);
        return call_prompt_attention(act_of(type), q.p, q.stride, k.p, k.stride, v.p, v.stride, q.n, int(q.heads), int(k.heads), int(q.dim),
                                     i32(a[3], "cu_seq"), int(std::min<int64_t>(n_seq, 1 << 30)), small(a[7], "longest"), small(a[8], "window"),
                                     real(a[6], "scale"), out.p, out.stride, f32(a[9], "lse", q.n * q.heads), ws.p, ws.bytes, stream_of(a[10]));
    });
}

// The addresses of the calls in the loaded library.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 8, [&] {
        call_packed_bytes = reinterpret_cast<decltype(call_packed_bytes)>(address(a[4]));
        call_gemm = reinterpret_cast<decltype(call_gemm)>(address(a[5]));
        call_gemm_experts = reinterpret_cast<decltype(call_gemm_experts)>(address(a[6]));
        call_prompt_attention = reinterpret_cast<decltype(call_prompt_attention)>(address(a[7]));
        call_cache_pages = reinterpret_cast<decltype(call_cache_pages)>(address(a[0]));
        call_qk_norm_rope = reinterpret_cast<decltype(call_qk_norm_rope)>(address(a[1]));
        call_cache_append = reinterpret_cast<decltype(call_cache_append)>(address(a[2]));
        call_attention = reinterpret_cast<decltype(call_attention)>(address(a[3]));
        return 0;
    });
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"cache_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_pages)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attention)), METH_FASTCALL, nullptr},
    {"gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(gemm)), METH_FASTCALL, nullptr},
    {"gemm_experts", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(gemm_experts)), METH_FASTCALL, nullptr},
    {"prompt_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prompt_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "qg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qg_torch(void) { return PyModule_Create(&module); }
