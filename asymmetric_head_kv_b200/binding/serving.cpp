// serving.cpp -- marshalling of the serving operators (page map, 8-bit cache write, decode and prefill) from torch
// tensors into the C ABI, as a CPython extension.
//
// A decode step's page map and cache write take the GPU 3 to 5 us each; checking nine tensors and converting seventeen
// arguments from Python took the host 10.  Here the checks read the tensors directly.  The entry points are called through
// the addresses that the package hands over after it has loaded the library (plain or checked build), so this file
// links against neither.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <string>

#include "../../include/diffqkv.h"

namespace {

decltype(&diffqkv_page_map) g_page_map = nullptr;
decltype(&diffqkv_kv8_store) g_store = nullptr;
decltype(&diffqkv_decode_paged_kv8) g_decode = nullptr;
decltype(&diffqkv_prefill_paged_kv8) g_prefill = nullptr;

struct Refused {};  // a Python exception has been set

[[noreturn]] void type_error(const char *name, const char *want) {
    PyErr_Format(PyExc_TypeError, "%s must be %s", name, want);
    throw Refused();
}
[[noreturn]] void value_error(const char *name, const char *want) {
    PyErr_Format(PyExc_ValueError, "%s must be %s", name, want);
    throw Refused();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error(name, "a tensor");
    return THPVariable_Unpack(o);
}

// The tensor's address if it is a contiguous CUDA tensor of this type and shape on device `dev`.
void *address(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type) type_error(name, c10::toString(type));
    if (!t.is_cuda()) value_error(name, "a CUDA tensor");
    if (t.get_device() != dev) value_error(name, "on the device of the other tensors");
    if (t.sizes() != shape || !t.is_contiguous()) {
        std::string want = "a contiguous tensor of shape (";
        for (const int64_t n : shape) want += std::to_string(n) + ", ";
        value_error(name, (want + ")").c_str());
    }
    return t.data_ptr();
}

int32_t *status_word(PyObject *o, int dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, "status");
    if (t.scalar_type() != at::kInt || !t.is_cuda() || t.numel() < 1 || t.get_device() != dev)
        type_error("status", "an int32 CUDA tensor with at least one element");
    return static_cast<int32_t *>(t.data_ptr());
}

// Device of the call's tensors (of the first of them), which must be the current one.
int device_of(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) value_error(name, "a CUDA tensor");
    const int dev = t.get_device();
    if (dev != c10::cuda::current_device()) value_error(name, "on the current CUDA device");
    return dev;
}

diffqkv_stream_t stream_of(PyObject *o, int dev) {
    if (o == Py_None) return reinterpret_cast<diffqkv_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
    PyObject *p = PyObject_GetAttrString(o, "cuda_stream");
    if (!p) throw Refused();
    void *s = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    if (PyErr_Occurred()) throw Refused();
    return static_cast<diffqkv_stream_t>(s);
}

int32_t int_arg(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    if (v < INT32_MIN || v > INT32_MAX) value_error(name, "a 32-bit integer");
    return static_cast<int32_t>(v);
}

int32_t size32(int64_t v, const char *name) {
    if (v > INT32_MAX) value_error(name, "smaller than 2^31 in every dimension");
    return static_cast<int32_t>(v);
}

// The 8-bit cache of k_pages, v_pages, k_scales, v_scales (consecutive arguments), and its head layout.
struct Cache {
    diffqkv_kv8_cache_t c;
    int dev;
    int32_t n_k, n_v, d_k, d_v;
};
Cache cache_of(PyObject *const *o) {
    const at::Tensor &k = tensor(o[0], "k_pages"), &v = tensor(o[1], "v_pages"), &ks = tensor(o[2], "k_scales");
    if (k.dim() != 4) value_error("k_pages", "[num_pages, page_size, n_k, d_k]");
    if (v.dim() != 4) value_error("v_pages", "[num_pages, page_size, n_v, d_v]");
    if (ks.dim() != 3) value_error("k_scales", "[num_pages, page_size // scale_block, n_k]");
    Cache r;
    r.dev = device_of(k, "k_pages");
    const int64_t pages = k.size(0), page = k.size(1), parts = ks.size(1);
    if (parts < 1 || page % parts) value_error("k_scales", "of scale blocks that divide the page");
    r.n_k = size32(k.size(2), "k_pages");
    r.d_k = size32(k.size(3), "k_pages");
    r.n_v = size32(v.size(2), "v_pages");
    r.d_v = size32(v.size(3), "v_pages");
    constexpr auto e4m3 = at::ScalarType::Float8_e4m3fn;
    r.c.k_pages = address(o[0], "k_pages", e4m3, k.sizes(), r.dev);
    r.c.v_pages = address(o[1], "v_pages", e4m3, {pages, page, r.n_v, r.d_v}, r.dev);
    r.c.k_scales = static_cast<uint8_t *>(address(o[2], "k_scales", at::kByte, {pages, parts, r.n_k}, r.dev));
    r.c.v_scales = static_cast<uint8_t *>(address(o[3], "v_scales", at::kByte, {pages, parts, r.n_v}, r.dev));
    r.c.num_pages = size32(pages, "k_pages");
    r.c.page_size = size32(page, "k_pages");
    r.c.scale_block = static_cast<int32_t>(page / parts);
    return r;
}

float scale_arg(PyObject *o, int32_t d_k) {
    if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d_k)));
    const double s = PyFloat_AsDouble(o);
    if (s == -1.0 && PyErr_Occurred()) throw Refused();
    return static_cast<float>(s);
}

// Calls an entry point (its arguments are plain values by then) without the interpreter's lock: a launch can wait for a full
// queue, and what it waits for can be a host function that wants the lock.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
    Unlocked() = default;
    Unlocked(const Unlocked &) = delete;
};
template <class F, class... A>
diffqkv_status_t unlocked(F entry, A... args) {
    const Unlocked u;
    return entry(args...);
}

// Runs a call; nothing crosses into Python as a C++ exception.
template <class F>
PyObject *guarded(const void *entry, F f) {
    if (!entry) {
        PyErr_SetString(PyExc_RuntimeError, "the library's entry points have not been bound");
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *wrong_count(const char *name) {
    PyErr_Format(PyExc_TypeError, "%s: wrong number of arguments", name);
    return nullptr;
}

// page_map(seq_lens, new_lens, block_table, free_pages, page_size, num_pages, query_start, slot_map, positions or None,
//          total_lens, pages_used, status or None, stream or None) -> status code
PyObject *page_map(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 13) return wrong_count("page_map");
    return guarded(reinterpret_cast<const void *>(g_page_map), [&] {
        const at::Tensor &seq = tensor(o[0], "seq_lens"), &table = tensor(o[2], "block_table");
        if (table.dim() != 2) value_error("block_table", "[B, max_blocks]");
        const int dev = device_of(seq, "seq_lens");
        const int64_t B = seq.numel(), mb = table.size(1), free = tensor(o[3], "free_pages").numel(),
                      cap = tensor(o[7], "slot_map").numel();
        auto i32 = [&](int i, const char *name, at::IntArrayRef shape) {
            return static_cast<int32_t *>(address(o[i], name, at::kInt, shape, dev));
        };
        return unlocked(
            g_page_map,
            size32(B, "seq_lens"), i32(0, "seq_lens", {B}), i32(1, "new_lens", {B}), i32(2, "block_table", {B, mb}),
            size32(mb, "block_table"), int_arg(o[4], "page_size"), int_arg(o[5], "num_pages"),
            i32(3, "free_pages", {free}), size32(free, "free_pages"), size32(cap, "slot_map"),
            i32(6, "query_start", {B + 1}), i32(7, "slot_map", {cap}),
            o[8] == Py_None ? nullptr : i32(8, "positions", {cap}), i32(9, "total_lens", {B}),
            i32(10, "pages_used", {1}), status_word(o[11], dev), stream_of(o[12], dev));
    });
}

// kv8_store(k_new, v_new, slot_map, k_pages, v_pages, k_scales, v_scales, status or None, stream or None)
PyObject *kv8_store(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 9) return wrong_count("kv8_store");
    return guarded(reinterpret_cast<const void *>(g_store), [&] {
        const Cache c = cache_of(o + 3);
        const int64_t T = tensor(o[2], "slot_map").numel();
        const int64_t n_q = static_cast<int64_t>(c.n_k) * c.n_v;
        const diffqkv_dims_t dims{1, size32(n_q, "k_pages"), c.n_k, c.n_v, c.d_k, c.d_v, 1.f};
        return unlocked(g_store, &dims, &c.c, address(o[0], "k_new", at::kBFloat16, {T, c.n_k, c.d_k}, c.dev),
                                       address(o[1], "v_new", at::kBFloat16, {T, c.n_v, c.d_v}, c.dev),
                                       static_cast<int32_t *>(address(o[2], "slot_map", at::kInt, {T}, c.dev)),
                                       size32(T, "slot_map"), status_word(o[7], c.dev), stream_of(o[8], c.dev));
    });
}

// decode_paged_kv8(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, scale or None, max_seq_len, out,
//                  workspace, stream or None)
PyObject *decode_paged_kv8(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 12) return wrong_count("decode_paged_kv8");
    return guarded(reinterpret_cast<const void *>(g_decode), [&] {
        const Cache c = cache_of(o + 1);
        const at::Tensor &q = tensor(o[0], "q"), &table = tensor(o[5], "block_table"), &ws = tensor(o[10], "workspace");
        if (q.dim() != 3) value_error("q", "[B, n_q, d_k]");
        if (table.dim() != 2) value_error("block_table", "[B, max_blocks]");
        const int64_t B = q.size(0), n_q = q.size(1), mb = table.size(1);
        const diffqkv_dims_t dims{size32(B, "q"), size32(n_q, "q"), c.n_k, c.n_v, c.d_k, c.d_v, scale_arg(o[7], c.d_k)};
        return unlocked(
            g_decode, &dims, &c.c, address(o[0], "q", at::kBFloat16, {B, n_q, c.d_k}, c.dev),
            static_cast<int32_t *>(address(o[5], "block_table", at::kInt, {B, mb}, c.dev)), size32(mb, "block_table"),
            static_cast<int32_t *>(address(o[6], "seq_lens", at::kInt, {B}, c.dev)), int_arg(o[8], "max_seq_len"),
            address(o[9], "out", at::kBFloat16, {B, n_q, c.d_v}, c.dev),
            address(o[10], "workspace", at::kByte, ws.sizes(), c.dev), static_cast<size_t>(ws.numel()),
            stream_of(o[11], c.dev));
    });
}

// prefill_paged_kv8(q, query_start, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, scale or None, out,
//                   workspace, stream or None)
PyObject *prefill_paged_kv8(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 12) return wrong_count("prefill_paged_kv8");
    return guarded(reinterpret_cast<const void *>(g_prefill), [&] {
        const Cache c = cache_of(o + 2);
        const at::Tensor &q = tensor(o[0], "q"), &table = tensor(o[6], "block_table"), &ws = tensor(o[10], "workspace");
        if (q.dim() != 3) value_error("q", "[tokens, n_q, d_k]");
        if (table.dim() != 2) value_error("block_table", "[B, max_blocks]");
        const int64_t T = q.size(0), n_q = q.size(1), B = table.size(0), mb = table.size(1);
        const diffqkv_dims_t dims{size32(B, "block_table"), size32(n_q, "q"), c.n_k, c.n_v, c.d_k, c.d_v,
                                  scale_arg(o[8], c.d_k)};
        return unlocked(
            g_prefill, &dims, &c.c, address(o[0], "q", at::kBFloat16, {T, n_q, c.d_k}, c.dev),
            static_cast<int32_t *>(address(o[1], "query_start", at::kInt, {B + 1}, c.dev)), size32(T, "q"),
            static_cast<int32_t *>(address(o[6], "block_table", at::kInt, {B, mb}, c.dev)), size32(mb, "block_table"),
            static_cast<int32_t *>(address(o[7], "seq_lens", at::kInt, {B}, c.dev)),
            address(o[9], "out", at::kBFloat16, {T, n_q, c.d_v}, c.dev),
            address(o[10], "workspace", at::kByte, ws.sizes(), c.dev), static_cast<size_t>(ws.numel()),
            stream_of(o[11], c.dev));
    });
}

// bind(addresses of diffqkv_page_map, diffqkv_kv8_store, diffqkv_decode_paged_kv8, diffqkv_prefill_paged_kv8)
PyObject *bind(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 4) return wrong_count("bind");
    void *p[4];
    for (int i = 0; i < 4; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(o[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
            return nullptr;
        }
    g_page_map = reinterpret_cast<decltype(g_page_map)>(p[0]);
    g_store = reinterpret_cast<decltype(g_store)>(p[1]);
    g_decode = reinterpret_cast<decltype(g_decode)>(p[2]);
    g_prefill = reinterpret_cast<decltype(g_prefill)>(p[3]);
    Py_RETURN_NONE;
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(page_map), ENTRY(kv8_store), ENTRY(decode_paged_kv8), ENTRY(prefill_paged_kv8),
                           ENTRY(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", "Marshalling of the serving operators.", -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&g_module); }
