// front.cpp -- the Python binding's short way into the serving operators.
//
// A serving loop makes these calls once a layer and token, on tensors of a few kilobytes, so what a call costs on the host
// is what it costs: 7 to 9 us when Python reads the tensors' types, shapes and strides and converts the arguments, of which
// the launch is 2 to 3. Here the same properties are read from the tensors themselves. A function takes what its namesake
// in binding.py takes, in a fixed order, checks the same conditions, makes the C call, and returns True; for
// anything that is not in order it returns False and has done nothing, and the Python way names the fault.
#include <Python.h>

#include <cstring>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "../../include/mha.h"

namespace {

// The library that binding.py has loaded.
struct Library {
    decltype(&mha_rotary) rotary;
    decltype(&mha_paged_append) paged_append;
    decltype(&mha_paged_attention) paged_attention;
    decltype(&mha_document_spans) document_spans;
    decltype(&mha_attention) attention;
    decltype(&mha_rmsnorm) rmsnorm;
} lib;

PyObject *s_native, *s_cuda_stream, *s_causal, *s_q_offset, *s_tensors;

struct NotInOrder {};

void need(bool ok) {
    if (!ok) throw NotInOrder{};
}

// One call's device and type, from its first tensor, and its tensors.
struct Call {
    c10::DeviceIndex dev = -1;
    at::ScalarType type = at::ScalarType::Undefined;

    static const at::Tensor& plain(PyObject* o) {
        need(THPVariable_CheckExact(o));
        const at::Tensor& t = THPVariable_Unpack(o);
        need(t.is_cuda() && t.layout() == at::kStrided);
        return t;
    }
    const at::Tensor& first(PyObject* o) {
        const at::Tensor& t = plain(o);
        dev = t.get_device();
        type = t.scalar_type();
        need(dev == c10::cuda::current_device());
        return t;
    }
    const at::Tensor& of(PyObject* o, at::ScalarType want) const {
        const at::Tensor& t = plain(o);
        need(t.scalar_type() == want && t.get_device() == dev);
        return t;
    }
    mha_dtype_t code() const {
        need(type == at::ScalarType::BFloat16 || type == at::ScalarType::Float);
        return type == at::ScalarType::BFloat16 ? MHA_BF16 : MHA_F32;
    }
    void* stream(PyObject* o) const {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
        PyObject* v = PyObject_GetAttr(o, s_cuda_stream);
        need(v != nullptr);
        void* s = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        need(s != nullptr || PyErr_Occurred() == nullptr);
        return s;
    }
};

int size_of(const at::Tensor& t, int i) {
    const int64_t n = t.size(i);
    need(n <= 0x7fffffff);
    return static_cast<int>(n);
}

// [B, L, H, d] with d adjacent
struct View {
    void* p = nullptr;
    mha_strides_t st{};
    const mha_strides_t* strides() const { return p != nullptr ? &st : nullptr; }
};
View view(const at::Tensor& t, int64_t B, int64_t L, int64_t H, int64_t d) {
    need(t.dim() == 4);
    const auto n = t.sizes(), s = t.strides();
    need(n[0] == B && n[1] == L && n[2] == H && n[3] == d && (s[3] == 1 || d == 1));
    return {t.mutable_data_ptr(), {s[0], s[1], s[2]}};
}

// Contiguous int32 of this shape, or None
int32_t* ints(const Call& c, PyObject* o, std::initializer_list<int64_t> shape) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = c.of(o, at::ScalarType::Int);
    need(t.sizes() == at::IntArrayRef(shape) && t.is_contiguous());
    return static_cast<int32_t*>(t.mutable_data_ptr());
}

// What a description of binding.py carries for this file, as packed bytes in its attribute _native.
template <typename T>
T native(PyObject* o) {
    PyObject* b = PyObject_GetAttr(o, s_native);
    need(b != nullptr);
    T v{};
    const bool ok = PyBytes_CheckExact(b) && PyBytes_GET_SIZE(b) == sizeof(T);
    if (ok) std::memcpy(&v, PyBytes_AS_STRING(b), sizeof(T));
    Py_DECREF(b);
    need(ok);
    return v;
}
struct RotaryNote {
    const mha_rotary_t* at;
    int64_t dev;
};
struct CacheNote {
    const mha_paged_cache_t* at;
    int64_t B, d, dtype, dev, heads;
};
struct ScoresNote {
    const mha_scores_t* at;
    int64_t h, dev;     // of the slopes; h = -1: none
};
const mha_rotary_t* rotary_of(const Call& c, PyObject* o) {
    const auto x = native<RotaryNote>(o);
    need(x.dev == c.dev);
    return x.at;
}
const mha_scores_t* scores_of(const Call& c, PyObject* o, int64_t h) {
    if (o == Py_None) return nullptr;
    const auto x = native<ScoresNote>(o);
    need(x.h < 0 || (x.h == h && x.dev == c.dev));
    return x.at;
}

// Runs `call` without the interpreter's lock (a launch may wait for room in its stream's queue).
template <typename F>
bool unlocked(F&& call) {
    mha_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = call();
    Py_END_ALLOW_THREADS
    return st == MHA_OK;
}

template <bool (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    bool done = false;
    try {
        if (n == kArgs) done = kCall(a);
    } catch (...) {    // also what torch throws for a tensor without storage
        done = false;
    }
    PyErr_Clear();
    return PyBool_FromLong(done);
}

// q, rotary, q_out, k, k_out, positions, stream
bool rotary(PyObject* const* a) {
    Call c;
    const at::Tensor& q = c.first(a[0]);
    need(q.dim() == 4);
    const int B = size_of(q, 0), T = size_of(q, 1), h = size_of(q, 2), d = size_of(q, 3);
    const View qv = view(q, B, T, h, d), qo = view(c.of(a[2], c.type), B, T, h, d);
    View kv, ko;
    int h_kv = 0;
    if (a[3] != Py_None) {
        const at::Tensor& k = c.of(a[3], c.type);
        need(k.dim() == 4);
        h_kv = size_of(k, 2);
        kv = view(k, B, T, h_kv, d);
        ko = view(c.of(a[4], c.type), B, T, h_kv, d);
    }
    const mha_rotary_t* r = rotary_of(c, a[1]);
    const int32_t* at = ints(c, a[5], {B, T});
    void* s = c.stream(a[6]);
    const mha_dtype_t dt = c.code();
    return unlocked([&] {
        return lib.rotary(dt, qv.p, qv.strides(), qo.p, qo.strides(), kv.p, kv.strides(), ko.p, ko.strides(), B, T, h, h_kv, d,
                          at, r, s);
    });
}

// k, v, start, cache, q, q_out, k_out, new_lens, rotary, stream
bool paged_append(PyObject* const* a) {
    Call c;
    const at::Tensor& k = c.first(a[0]);
    need(k.dim() == 4);
    const int B = size_of(k, 0), T = size_of(k, 1), h_kv = size_of(k, 2), d = size_of(k, 3);
    const mha_dtype_t dt = c.code();
    const auto cache = native<CacheNote>(a[3]);
    need(cache.B == B && cache.d == d && cache.dtype == dt && cache.dev == c.dev && cache.heads == h_kv);
    const View kv = view(k, B, T, h_kv, d), vv = view(c.of(a[1], c.type), B, T, h_kv, d);
    View qv, qo, ko;
    int h = 0;
    if (a[4] != Py_None) {
        const at::Tensor& q = c.of(a[4], c.type);
        need(q.dim() == 4);
        h = size_of(q, 2);
        qv = view(q, B, T, h, d);
        qo = view(c.of(a[5], c.type), B, T, h, d);
    }
    if (a[6] != Py_None) ko = view(c.of(a[6], c.type), B, T, h_kv, d);
    const int32_t *start = ints(c, a[2], {B}), *new_lens = ints(c, a[7], {B});
    const mha_rotary_t* r = a[8] != Py_None ? rotary_of(c, a[8]) : nullptr;
    void* s = c.stream(a[9]);
    return unlocked([&] {
        return lib.paged_append(dt, qv.p, qv.strides(), qo.p, qo.strides(), kv.p, kv.strides(), ko.p, ko.strides(), vv.p,
                                vv.strides(), B, T, h, h_kv, d, start, new_lens, r, cache.at, s);
    });
}

// q, kv_lens, cache, out, workspace, scores, stream
bool paged_attention(PyObject* const* a) {
    Call c;
    const at::Tensor& q = c.first(a[0]);
    const at::Tensor& out = c.of(a[3], c.type);
    need(q.dim() == 3 && out.sizes() == q.sizes() && q.stride(2) == 1 && out.stride(2) == 1);
    const int B = size_of(q, 0), h = size_of(q, 1), d = size_of(q, 2);
    const mha_dtype_t dt = c.code();
    const auto cache = native<CacheNote>(a[2]);
    need(cache.B == B && cache.d == d && cache.dtype == dt && cache.dev == c.dev);
    const at::Tensor& ws = Call::plain(a[4]);
    need(ws.get_device() == c.dev && ws.is_contiguous());
    const int32_t* lens = ints(c, a[1], {B});
    const mha_scores_t* scores = scores_of(c, a[5], h);
    const mha_strides_t qs{q.stride(0), 0, q.stride(1)}, os{out.stride(0), 0, out.stride(1)};
    void *qp = q.mutable_data_ptr(), *op = out.mutable_data_ptr(), *wp = ws.mutable_data_ptr(), *s = c.stream(a[6]);
    const size_t bytes = ws.nbytes();
    return unlocked([&] {
        return lib.paged_attention(dt, qp, &qs, op, &os, B, h, static_cast<int>(cache.heads), d, lens, scores, cache.at, wp, bytes,
                                   s);
    });
}

// doc_ids, spans, stream
bool document_spans(PyObject* const* a) {
    Call c;
    const at::Tensor& ids = c.first(a[0]);
    need(ids.dim() == 2);
    const int B = size_of(ids, 0), L = size_of(ids, 1);
    const int32_t* from = ints(c, a[0], {B, L});
    int32_t* spans = ints(c, a[1], {B, L, 2});
    void* s = c.stream(a[2]);
    return unlocked([&] { return lib.document_spans(from, B, L, spans, s); });
}

// Owns an object taken out of another.
struct Held {
    PyObject* o;
    explicit Held(PyObject* o_) : o(o_) { need(o != nullptr); }
    ~Held() { Py_DECREF(o); }
    Held(const Held&) = delete;
    Held& operator=(const Held&) = delete;
};
int int_of(PyObject* owner, PyObject* name) {
    const Held v(PyObject_GetAttr(owner, name));
    need(PyLong_Check(v.o));
    int over = 0;
    const long n = PyLong_AsLongAndOverflow(v.o, &over);
    need(over == 0 && n >= INT32_MIN && n <= INT32_MAX);
    return static_cast<int>(n);
}

// q, k, v, out, scores, mask, stream
bool attention(PyObject* const* a) {
    Call c;
    const at::Tensor& q = c.first(a[0]);
    const at::Tensor& k = c.of(a[1], c.type);
    need(q.dim() == 4 && k.dim() == 4);
    const int B = size_of(q, 0), Lq = size_of(q, 1), h = size_of(q, 2), d = size_of(q, 3);
    const int Lk = size_of(k, 1), h_kv = size_of(k, 2);
    const View qv = view(q, B, Lq, h, d), kv = view(k, B, Lk, h_kv, d), vv = view(c.of(a[2], c.type), B, Lk, h_kv, d),
               ov = view(c.of(a[3], c.type), B, Lq, h, d);
    const mha_scores_t* scores = scores_of(c, a[4], h);
    mha_span_mask_t m{};
    PyObject* mask = a[5];
    PyObject* parts = nullptr;
    if (mask != Py_None) {
        m.causal = int_of(mask, s_causal);
        m.q_offset = int_of(mask, s_q_offset);
        parts = PyObject_GetAttr(mask, s_tensors);
    }
    const Held held(parts != nullptr ? parts : mask == Py_None ? Py_NewRef(Py_None) : nullptr);
    if (parts != nullptr) {
        need(PyTuple_CheckExact(parts) && PyTuple_GET_SIZE(parts) == 3);
        m.key_valid_lens = ints(c, PyTuple_GET_ITEM(parts, 0), {B});
        m.prefix_lens = ints(c, PyTuple_GET_ITEM(parts, 1), {B});
        m.doc_spans = ints(c, PyTuple_GET_ITEM(parts, 2), {B, Lq, 2});
    }
    void* s = c.stream(a[6]);
    const mha_dtype_t dt = c.code();
    return unlocked([&] {
        return lib.attention(dt, qv.p, &qv.st, kv.p, &kv.st, vv.p, &vv.st, ov.p, &ov.st, B, Lq, Lk, h, h_kv, d, scores,
                             mask != Py_None ? &m : nullptr, s);
    });
}

// [rows, d] with adjacent rows
struct Rows {
    void* p = nullptr;
    int64_t stride = 0;
};
Rows rows_of(const at::Tensor& t, int64_t rows, int64_t d) {
    need(t.dim() == 2 && t.size(0) == rows && t.size(1) == d && (t.stride(1) == 1 || d == 1));
    return {t.mutable_data_ptr(), t.stride(0)};
}

// x, gain, eps, y, residual, sum_out, scales, stream
bool rmsnorm(PyObject* const* a) {
    Call c;
    const at::Tensor& x = c.first(a[0]);
    need(x.dim() == 2);
    const int64_t rows = x.size(0);
    const int d = size_of(x, 1);
    const Rows xv = rows_of(x, rows, d);
    Rows yv, rv, zv;
    float* scales = nullptr;
    int group = 0;
    if (a[6] == Py_None) {
        yv = rows_of(c.of(a[3], c.type), rows, d);
    } else {
        yv = rows_of(c.of(a[3], at::ScalarType::Float8_e4m3fn), rows, d);
        const at::Tensor& t = c.of(a[6], at::ScalarType::Float);
        need(t.dim() == 2 && t.size(0) == rows && t.is_contiguous());
        const int64_t groups = t.size(1);
        need(groups >= 1 && d % groups == 0);
        if (groups > 1) group = static_cast<int>(d / groups);
        scales = static_cast<float*>(t.mutable_data_ptr());
    }
    if (a[4] != Py_None) rv = rows_of(c.of(a[4], c.type), rows, d);
    if (a[5] != Py_None) {
        need(a[4] != Py_None);
        zv = rows_of(c.of(a[5], c.type), rows, d);
    }
    const void* gain = nullptr;
    if (a[1] != Py_None) {
        const at::Tensor& g = c.of(a[1], c.type);
        need(g.dim() == 1 && g.size(0) == d && g.is_contiguous());
        gain = g.mutable_data_ptr();
    }
    const double eps = PyFloat_AsDouble(a[2]);
    need(eps != -1.0 || PyErr_Occurred() == nullptr);
    void* s = c.stream(a[7]);
    const mha_dtype_t dt = c.code();
    return unlocked([&] {
        return lib.rmsnorm(dt, xv.p, xv.stride, rv.p, rv.stride, zv.p, zv.stride, gain, static_cast<float>(eps), rows, d, yv.p,
                           yv.stride, scales, group, s);
    });
}

// The addresses of the six functions, in the order of Library.
PyObject* set_library(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* at[6];
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "six addresses");
        return nullptr;
    }
    for (int i = 0; i < 6; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (at[i] == nullptr) {
            if (PyErr_Occurred() == nullptr) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    static_assert(sizeof(Library) == sizeof(at));
    std::memcpy(&lib, at, sizeof(at));
    Py_RETURN_NONE;
}

#define MHA_ENTRY(name, args) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, args>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    MHA_ENTRY(rotary, 7),
    MHA_ENTRY(paged_append, 10),
    MHA_ENTRY(paged_attention, 7),
    MHA_ENTRY(document_spans, 3),
    MHA_ENTRY(attention, 7),
    MHA_ENTRY(rmsnorm, 8),
    {"set_library", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&set_library)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front() {
    s_native = PyUnicode_InternFromString("_native");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    s_causal = PyUnicode_InternFromString("causal");
    s_q_offset = PyUnicode_InternFromString("q_offset");
    s_tensors = PyUnicode_InternFromString("tensors");
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
