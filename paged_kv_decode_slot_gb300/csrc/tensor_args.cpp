// tensor_args.cpp - the binding's work per call in C++, as a Python extension: a step makes several calls of ten tensors
// each, some for a few microseconds of GPU work, and the interpreter's attribute look-ups and foreign call take longer than
// the launch (a rotating append of 64 tokens takes 2.8 us on the GPU; its call 8.9 us of a Grace core with each argument
// checked here but the call made from Python, 3.8 us made here).  arg() and maybe() check one tensor; the functions further
// down check a whole call and make it if nothing about it is special, else they return None and binding.py's own form of the
// call names the fault (or takes what is allowed but rare: pinned host memory, calls without tokens).  Nothing here
// computes, and where it is not built binding.py does all of it.
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>

#include "pkv.h"

namespace {

PyObject *g_refuse = nullptr;  // binding._refuse(t, dtype, shape, name, dev): raises, or accepts pinned host memory

// The address of a contiguous tensor of this type and shape on CUDA device dev; null: something is not as asked, or Python's
// error is set.  Tensors without memory (fake ones) throw.
void *plain(PyObject *const *a)
{
    if (!THPVariable_Check(a[0]) || !THPDtype_Check(a[1]) || !PyTuple_Check(a[2])) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(a[0]);
    const long dev = PyLong_AsLong(a[4]);
    if (dev == -1 && PyErr_Occurred()) return nullptr;
    const auto sizes = t.sizes();
    bool same = t.scalar_type() == reinterpret_cast<THPDtype *>(a[1])->scalar_type && t.is_cuda() && t.get_device() == dev &&
                PyTuple_GET_SIZE(a[2]) == (Py_ssize_t)sizes.size() && t.is_contiguous();
    for (size_t i = 0; same && i < sizes.size(); ++i) {
        const long long s = PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], i));
        if (s == -1 && PyErr_Occurred()) return nullptr;
        same = s == sizes[i];
    }
    return same ? t.data_ptr() : nullptr;
}

// arg(t, dtype, shape, name, dev) -> that address; what is not as asked goes to the binding
PyObject *arg(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "arg(t, dtype, shape, name, dev)");
        return nullptr;
    }
    void *at = nullptr;
    try {
        at = plain(a);
    } catch (...) {  // nothing may pass the interpreter; it meets the same in the binding, and says so
    }
    if (at) return PyLong_FromVoidPtr(at);
    if (PyErr_Occurred()) return nullptr;
    if (!g_refuse) {
        PyErr_SetString(PyExc_RuntimeError, "set_refuse was not called");
        return nullptr;
    }
    return PyObject_Vectorcall(g_refuse, a, 5, nullptr);
}

// maybe(t, ...): None for None
PyObject *maybe(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (n == 5 && a[0] == Py_None) Py_RETURN_NONE;
    return arg(self, a, n);
}

PyObject *set_refuse(PyObject *, PyObject *f)
{
    Py_INCREF(f);
    Py_XSETREF(g_refuse, f);
    Py_RETURN_NONE;
}

// ---- whole calls ------------------------------------------------------------------------------------------------------
#define PKV_ENTRIES(X)                                                                                                          \
    X(pkv_rope_append)                                                                                                          \
    X(pkv_rope_append_fp8)                                                                                                      \
    X(pkv_rope_append_multi)                                                                                                    \
    X(pkv_rope_append_multi_fp8)                                                                                                \
    X(pkv_key_bounds)                                                                                                           \
    X(pkv_key_bounds_fp8)                                                                                                       \
    X(pkv_select_blocks)                                                                                                        \
    X(pkv_decode_attn_blocks)                                                                                                   \
    X(pkv_decode_attn_blocks_fp8)                                                                                               \
    X(pkv_verify_draft)
struct Library {
#define PKV_MEMBER(f) decltype(&::f) f = nullptr;
    PKV_ENTRIES(PKV_MEMBER)
#undef PKV_MEMBER
};
Library g_lib;
PyObject *g_stream_of = nullptr;  // binding._launch(stream or None, dev): the stream's address

// use_library(handle, stream_of): the entry points of the library that ctypes has loaded
PyObject *use_library(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "use_library(handle, stream_of)");
        return nullptr;
    }
    void *handle = PyLong_AsVoidPtr(a[0]);
    if (!handle && PyErr_Occurred()) return nullptr;
    Library lib;
    bool all = true;
#define PKV_FIND(f) all &= (lib.f = reinterpret_cast<decltype(lib.f)>(dlsym(handle, #f))) != nullptr;
    PKV_ENTRIES(PKV_FIND)
#undef PKV_FIND
    if (!all) {
        PyErr_SetString(PyExc_ImportError, "the library lacks an entry point");
        return nullptr;
    }
    g_lib = lib;
    Py_INCREF(a[1]);
    Py_XSETREF(g_stream_of, a[1]);
    Py_RETURN_NONE;
}

// A size that the first tensor with it sets and the others must have; {2}: a fixed one.
struct Dim {
    int64_t v = -1;
    operator int32_t() const { return (int32_t)v; }
};

// The arguments of one call, taken in turn; ok: each was what the call wants, not empty, on the current device.
struct Call {
    PyObject *const *next, *const *last;  // the last two: stream, device
    bool ok;
    long dev = -1;

    Call(PyObject *const *a, Py_ssize_t n, Py_ssize_t want) : next(a), last(n == want ? a + n - 2 : a), ok(n == want && g_stream_of)
    {
        if (ok) dev = integer(last[1]);
    }
    long integer(PyObject *o)
    {
        int over = 0;
        const long v = PyLong_Check(o) ? PyLong_AsLongAndOverflow(o, &over) : (ok = false, 0);
        if (over || v > INT32_MAX || v < INT32_MIN) ok = false;
        return v;
    }
    int32_t i32() { return ok ? (int32_t)integer(*next++) : 0; }
    float f32()
    {
        if (!ok) return 0.f;
        PyObject *o = *next++;
        ok = PyFloat_Check(o);
        return ok ? (float)PyFloat_AS_DOUBLE(o) : 0.f;
    }
    pkv_stream_t stream()  // the last argument, or the device's current one
    {
        if (!ok) return nullptr;
        PyObject *handle = PyObject_Vectorcall(g_stream_of, last, 2, nullptr);
        void *s = handle ? PyLong_AsVoidPtr(handle) : nullptr;
        Py_XDECREF(handle);
        if (!s && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return static_cast<pkv_stream_t>(s);
    }
    template <typename T = void>
    T *tensor(at::ScalarType type, std::initializer_list<Dim *> shape)
    {
        if (!ok) return nullptr;
        PyObject *o = *next++;
        ok = THPVariable_Check(o);
        if (!ok) return nullptr;
        const at::Tensor &t = THPVariable_Unpack(o);
        ok = t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.dim() == (int64_t)shape.size() &&
             t.is_contiguous() && t.numel() > 0;
        if (!ok) return nullptr;
        const auto sizes = t.sizes();
        size_t i = 0;
        for (Dim *d : shape) {
            if (d->v < 0) d->v = sizes[i];
            ok &= d->v == sizes[i] && (d->v <= INT32_MAX || shape.size() == 1);
            ++i;
        }
        T *at = static_cast<T *>(t.data_ptr());
        ok &= at != nullptr;
        return at;
    }
    template <typename T = void>
    T *maybe(at::ScalarType type, std::initializer_list<Dim *> shape)
    {
        if (ok && *next == Py_None) return ++next, nullptr;
        return tensor<T>(type, shape);
    }
    // [K], or [num_blocks, K]; the stride of a block
    const float *scale(Dim &blocks, Dim &heads, int32_t &stride)
    {
        if (!ok || !THPVariable_Check(*next)) return ok = false, nullptr;
        const bool per_block = THPVariable_Unpack(*next).dim() == 2;
        stride = per_block ? (int32_t)heads : 0;
        return per_block ? tensor<float>(at::kFloat, {&blocks, &heads}) : tensor<float>(at::kFloat, {&heads});
    }
    int32_t *flag()
    {
        Dim one{1};
        return maybe<int32_t>(at::kInt, {&one});
    }
};

template <typename F, typename... A>
PyObject *launch(const Call &c, F f, A... a)
{
    if (!c.ok) Py_RETURN_NONE;
    int status;
    Py_BEGIN_ALLOW_THREADS;  // a full launch queue makes the caller wait
    status = f(a...);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

// rope(q, k_new, v_new, positions | (block_tables, context_lens), inv_freq, [k_scale, v_scale,] k_cache, v_cache, q_out,
//      slot_mapping, interleaved, err_flag, stream, dev)
template <bool kFp8, bool kTables>
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    Call c(a, n, 13 + kTables + 2 * kFp8);
    Dim B, T, N, H, K, width, half, nb, bs;
    if (!kTables) T.v = 1;
    auto rows = [&](Dim &heads) {
        return kTables ? c.tensor<pkv_bf16>(at::kBFloat16, {&B, &T, &heads, &H}) : c.tensor<pkv_bf16>(at::kBFloat16, {&B, &heads, &H});
    };
    const pkv_bf16 *q = rows(N), *k_new = rows(K), *v_new = rows(K);
    const int32_t *positions = nullptr, *tables = nullptr, *lens = nullptr;
    if constexpr (kTables) {
        tables = c.tensor<int32_t>(at::kInt, {&B, &width});
        lens = c.tensor<int32_t>(at::kInt, {&B});
    } else {
        positions = c.tensor<int32_t>(at::kInt, {&B});
    }
    const double *inv_freq = c.tensor<double>(at::kDouble, {&half});
    const float *ks = nullptr, *vs = nullptr;
    int32_t stride = 0, v_stride = 0;
    PyObject *const *scales = c.next;
    if constexpr (kFp8) c.next += c.ok ? 2 : 0;  // their shape needs the pools'
    const at::ScalarType pool = kFp8 ? at::kByte : at::kBFloat16;
    void *kc = c.tensor(pool, {&nb, &bs, &K, &H}), *vc = c.tensor(pool, {&nb, &bs, &K, &H});
    if constexpr (kFp8) {
        PyObject *const *behind = c.next;
        c.next = scales;
        ks = c.scale(nb, K, stride);
        vs = c.scale(nb, K, v_stride);
        c.ok &= stride == v_stride;
        c.next = behind;
    }
    pkv_bf16 *out = rows(N);
    const int64_t apart = reinterpret_cast<const char *>(out) - reinterpret_cast<const char *>(q);
    if (apart != 0 && std::abs(apart) < 2 * B.v * T.v * N.v * H.v) c.ok = false;  // q_out may be q itself, but not overlap it
    int64_t *slots = kTables ? c.tensor<int64_t>(at::kLong, {&B, &T}) : c.tensor<int64_t>(at::kLong, {&B});
    const int32_t interleaved = c.i32();
    int32_t *err = c.flag();
    const pkv_stream_t stream = c.stream();
    const pkv_cache_desc d{nb, bs, K, H};
    const int32_t R = half.v <= H.v ? 2 * half : 0;  // 0 is refused
    if constexpr (kTables && kFp8)
        return launch(c, g_lib.pkv_rope_append_multi_fp8, q, k_new, v_new, tables, width, lens, inv_freq, R, interleaved, ks, vs, stride, B,
                      T, N, static_cast<uint8_t *>(kc), static_cast<uint8_t *>(vc), out, slots, d, err, stream);
    else if constexpr (kTables)
        return launch(c, g_lib.pkv_rope_append_multi, q, k_new, v_new, tables, width, lens, inv_freq, R, interleaved, B, T, N,
                      static_cast<pkv_bf16 *>(kc), static_cast<pkv_bf16 *>(vc), out, slots, d, err, stream);
    else if constexpr (kFp8)
        return launch(c, g_lib.pkv_rope_append_fp8, q, k_new, v_new, positions, inv_freq, R, interleaved, ks, vs, stride, slots, B, N,
                      static_cast<uint8_t *>(kc), static_cast<uint8_t *>(vc), out, d, err, stream);
    else
        return launch(c, g_lib.pkv_rope_append, q, k_new, v_new, positions, inv_freq, R, interleaved, slots, B, N,
                      static_cast<pkv_bf16 *>(kc), static_cast<pkv_bf16 *>(vc), out, d, err, stream);
}

// key_bounds(k_cache, [k_scale,] block_tables, context_lens, num_new, key_bounds, err_flag, stream, dev)
template <bool kFp8>
PyObject *key_bounds(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    Call c(a, n, 8 + kFp8);
    Dim nb, bs, K, H, B, width, two{2};
    void *kc = c.tensor(kFp8 ? at::kByte : at::kBFloat16, {&nb, &bs, &K, &H});
    int32_t stride = 0;
    const float *ks = kFp8 ? c.scale(nb, K, stride) : nullptr;
    const int32_t *tables = c.tensor<int32_t>(at::kInt, {&B, &width}), *lens = c.tensor<int32_t>(at::kInt, {&B});
    const int32_t num_new = c.i32();
    pkv_bf16 *bounds = c.tensor<pkv_bf16>(at::kBFloat16, {&nb, &K, &two, &H});
    int32_t *err = c.flag();
    const pkv_stream_t stream = c.stream();
    const pkv_cache_desc d{nb, bs, K, H};
    if constexpr (kFp8)
        return launch(c, g_lib.pkv_key_bounds_fp8, static_cast<const uint8_t *>(kc), ks, stride, tables, width, lens, B, num_new, bounds, d,
                      err, stream);
    else
        return launch(c, g_lib.pkv_key_bounds, static_cast<const pkv_bf16 *>(kc), tables, width, lens, B, num_new, bounds, d, err, stream);
}

// select_blocks(q, key_bounds, block_tables, context_lens, selected, workspace, first, last, err_flag, block_size, stream, dev)
PyObject *select_blocks(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    Call c(a, n, 12);
    Dim B, N, H, nb, K, two{2}, width, M, size;
    const pkv_bf16 *q = c.tensor<pkv_bf16>(at::kBFloat16, {&B, &N, &H});
    const pkv_bf16 *bounds = c.tensor<pkv_bf16>(at::kBFloat16, {&nb, &K, &two, &H});
    const int32_t *tables = c.tensor<int32_t>(at::kInt, {&B, &width}), *lens = c.tensor<int32_t>(at::kInt, {&B});
    int32_t *selected = c.tensor<int32_t>(at::kInt, {&B, &K, &M});
    void *ws = c.tensor(at::kByte, {&size});
    const int32_t first = c.i32(), last = c.i32();
    int32_t *err = c.flag();
    const int32_t block_size = c.i32();
    const pkv_stream_t stream = c.stream();
    return launch(c, g_lib.pkv_select_blocks, q, bounds, tables, width, lens, B, N, first, last, M, selected,
                  pkv_cache_desc{nb, block_size, K, H}, ws, (size_t)size.v, err, stream);
}

// decode_attn_blocks(q, k_cache, v_cache, [k_scale, v_scale,] block_tables, context_lens, selected, scale, out, lse_out,
//                    partition_blocks, max_partitions, workspace, err_flag, stream, dev)
template <bool kFp8>
PyObject *decode_attn_blocks(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    Call c(a, n, 15 + 2 * kFp8);
    Dim B, N, H, nb, bs, K, width, M, size{0};
    const pkv_bf16 *q = c.tensor<pkv_bf16>(at::kBFloat16, {&B, &N, &H});
    const at::ScalarType pool = kFp8 ? at::kByte : at::kBFloat16;
    void *kc = c.tensor(pool, {&nb, &bs, &K, &H}), *vc = c.tensor(pool, {&nb, &bs, &K, &H});
    int32_t stride = 0, v_stride = 0;
    const float *ks = kFp8 ? c.scale(nb, K, stride) : nullptr, *vs = kFp8 ? c.scale(nb, K, v_stride) : nullptr;
    c.ok &= stride == v_stride;
    const int32_t *tables = c.tensor<int32_t>(at::kInt, {&B, &width}), *lens = c.tensor<int32_t>(at::kInt, {&B});
    const int32_t *selected = c.tensor<int32_t>(at::kInt, {&B, &K, &M});
    const float scale = c.f32();
    pkv_bf16 *out = c.tensor<pkv_bf16>(at::kBFloat16, {&B, &N, &H});
    float *lse = c.maybe<float>(at::kFloat, {&B, &N});
    const int32_t partition_blocks = c.i32(), max_partitions = c.i32();
    if (c.ok && *c.next != Py_None) size.v = -1;
    void *ws = c.maybe(at::kByte, {&size});
    int32_t *err = c.flag();
    const pkv_stream_t stream = c.stream();
    const pkv_cache_desc d{nb, bs, K, H};
    if constexpr (kFp8)
        return launch(c, g_lib.pkv_decode_attn_blocks_fp8, q, static_cast<const uint8_t *>(kc), static_cast<const uint8_t *>(vc), ks, vs,
                      stride, tables, width, lens, selected, M, B, N, scale, out, lse, d, partition_blocks, max_partitions, ws,
                      (size_t)size.v, err, stream);
    else
        return launch(c, g_lib.pkv_decode_attn_blocks, q, static_cast<const pkv_bf16 *>(kc), static_cast<const pkv_bf16 *>(vc), tables,
                      width, lens, selected, M, B, N, scale, out, lse, d, partition_blocks, max_partitions, ws, (size_t)size.v, err,
                      stream);
}

// verify_draft(target_probs, draft_probs, draft_tokens, accept_u, sample_u, num_accepted, tokens_out, workspace, draft_lens,
//              context_lens, context_lens_out, vocab_size or None, err_flag, stream, dev)
PyObject *verify_draft(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    Call c(a, n, 15);
    Dim B, rows, wide, T, q_wide, size;
    const bool bf16 = c.ok && THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).scalar_type() == at::kBFloat16;
    const at::ScalarType type = bf16 ? at::kBFloat16 : at::kFloat;
    void *target = c.tensor(type, {&B, &rows, &wide});
    if (rows.v < 2) c.ok = false;  // no drafted tokens: the tensors for them are empty
    T.v = rows.v - 1;
    void *draft = c.maybe(type, {&B, &T, &q_wide});
    const int32_t *tokens = c.tensor<int32_t>(at::kInt, {&B, &T});
    const float *accept = c.tensor<float>(at::kFloat, {&B, &T}), *sample = c.tensor<float>(at::kFloat, {&B});
    int32_t *accepted = c.tensor<int32_t>(at::kInt, {&B}), *out = c.tensor<int32_t>(at::kInt, {&B, &rows});
    void *ws = c.tensor(at::kByte, {&size});
    const int32_t *lens = c.maybe<int32_t>(at::kInt, {&B}), *ctx = c.maybe<int32_t>(at::kInt, {&B});
    int32_t *ctx_out = c.maybe<int32_t>(at::kInt, {&B});
    const bool all = c.ok && *c.next == Py_None;
    c.next += all;
    const int32_t V = all ? (int32_t)wide : c.i32();
    if (!draft) q_wide.v = V;
    if (V > wide.v || V > q_wide.v) c.ok = false;
    int32_t *err = c.flag();
    const pkv_stream_t stream = c.stream();
    return launch(c, g_lib.pkv_verify_draft, target, wide.v, draft, q_wide.v, (int32_t)bf16, tokens, lens, accept, sample, B, T, V, accepted,
                  out, ctx, ctx_out, ws, (size_t)size.v, err, stream);
}

// A whole call; a tensor that throws (a fake one has no address) is not plain.
template <PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *whole(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    try {
        return f(self, a, n);
    } catch (...) {
        Py_RETURN_NONE;
    }
}

#define PKV_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PKV_METHOD("arg", arg),
    PKV_METHOD("maybe", maybe),
    PKV_METHOD("use_library", use_library),
    PKV_METHOD("rope_append", (whole<rope<false, false>>)),
    PKV_METHOD("rope_append_fp8", (whole<rope<true, false>>)),
    PKV_METHOD("rope_append_multi", (whole<rope<false, true>>)),
    PKV_METHOD("rope_append_multi_fp8", (whole<rope<true, true>>)),
    PKV_METHOD("key_bounds", whole<key_bounds<false>>),
    PKV_METHOD("key_bounds_fp8", whole<key_bounds<true>>),
    PKV_METHOD("select_blocks", whole<select_blocks>),
    PKV_METHOD("decode_attn_blocks", whole<decode_attn_blocks<false>>),
    PKV_METHOD("decode_attn_blocks_fp8", whole<decode_attn_blocks<true>>),
    PKV_METHOD("verify_draft", whole<verify_draft>),
    {"set_refuse", set_refuse, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tensor_args()
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) != 0) Py_CLEAR(m);  // the binding compares it with what runs
    return m;
}
