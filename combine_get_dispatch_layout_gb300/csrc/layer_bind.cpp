// Python binding of the layer operators (include/ep_layer.h): tensors in, one
// call of the C ABI out.
//
// A decode step makes these calls for a few microseconds of GPU work each, and
// the same checks and conversions in Python and ctypes cost 6 to 16 us a call
// (12 to 26 before they were pared down), so they are made here. Every function
// takes its tensors (None where the C call takes NULL), scalars and the stream,
// raises ValueError for a tensor that the C ABI cannot check (type, shape,
// strides, device), and returns the call's status.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/ep_layer.h"

namespace {

struct Raised {};   // a Python error is set

template <typename... A>
[[noreturn]] void refuse(const char* format, A... args) {
    PyErr_Format(PyExc_ValueError, format, args...);
    throw Raised{};
}

// The library's entry points, looked up once.
struct Library {
    decltype(&ep_router_topk) router_topk = nullptr;
    decltype(&ep_router_topk_backward) router_topk_backward = nullptr;
    decltype(&ep_kv_append) kv_append = nullptr;
    decltype(&ep_paged_attention) paged_attention = nullptr;
    decltype(&ep_expert_w4) expert_w4 = nullptr;
    decltype(&ep_expert_w4_workspace) expert_w4_workspace = nullptr;
} library;

using Tensor = at::Tensor;
constexpr auto kBf16 = at::ScalarType::BFloat16, kFp16 = at::ScalarType::Half, kFp32 = at::ScalarType::Float,
               kInt64 = at::ScalarType::Long, kInt32 = at::ScalarType::Int, kByte = at::ScalarType::Byte,
               kE4m3 = at::ScalarType::Float8_e4m3fn;

const Tensor* optional_tensor(PyObject* o, const char* what) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse("%s must be a tensor, got %s", what, Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* what) {
    const Tensor* t = optional_tensor(o, what);
    if (!t) refuse("%s must be a tensor, got None", what);
    return *t;
}
// All CUDA tensors of a call lie on one GPU, the current one: it is that one's stream, cores and limits that the call uses.
void one_device(PyObject* const* args, Py_ssize_t count) {
    int first = -1;
    for (Py_ssize_t i = 0; i < count; ++i) {
        // (numbers and None first: that something is no tensor takes 0.1 us to find out otherwise)
        if (args[i] == Py_None || PyLong_Check(args[i]) || PyFloat_Check(args[i]) || !THPVariable_Check(args[i])) continue;
        const Tensor& t = THPVariable_Unpack(args[i]);
        if (!t.is_cuda()) continue;
        const int device = t.get_device();
        if (first < 0) first = device;
        if (device != first) refuse("tensors of one call on cuda:%d and on cuda:%d", first, device);
    }
    if (first < 0) return;
    const int current = c10::cuda::current_device();
    if (first != current) refuse("tensors on cuda:%d, the current device is cuda:%d", first, current);
}
void* address(const Tensor& t, const char* what) {
    if (!t.is_cuda() && t.numel() > 0 && !t.is_pinned()) refuse("%s must be a CUDA tensor or a pinned host tensor", what);
    return t.data_ptr();
}
int type_code(const Tensor& t, const char* what, bool fp32, bool e4m3) {
    switch (t.scalar_type()) {
        case kBf16: return EP_DTYPE_BF16;
        case kFp16: return EP_DTYPE_FP16;
        case kFp32:
            if (fp32) return EP_DTYPE_FP32;
            break;
        case kE4m3:
            if (e4m3) return EP_DTYPE_FP8_E4M3;
            break;
        default: break;
    }
    refuse("%s: %s is not supported", what, c10::toString(t.scalar_type()));
}
void dimensions(const Tensor& t, int64_t n, const char* what) {
    if (t.dim() != n) refuse("%s must have %d dimensions, got %d", what, static_cast<int>(n), static_cast<int>(t.dim()));
}
void expect(const Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape, const char* what) {
    if (t.scalar_type() == type && t.sizes() == at::IntArrayRef(shape.begin(), shape.size())) return;
    std::string want, got;
    for (const int64_t n : shape) want += (want.empty() ? "" : ", ") + std::to_string(n);
    for (const int64_t n : t.sizes()) got += (got.empty() ? "" : ", ") + std::to_string(n);
    refuse("%s must be %s [%s], got %s [%s]", what, c10::toString(type), want.c_str(), c10::toString(t.scalar_type()), got.c_str());
}
// Address of a contiguous tensor of this type and shape, NULL for None.
void* dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, const char* what) {
    const Tensor* t = optional_tensor(o, what);
    if (!t) return nullptr;
    expect(*t, type, shape, what);
    if (!t->is_contiguous()) refuse("%s must be contiguous", what);
    return address(*t, what);
}
// Address and row distance of a tensor whose rows are dense and apart.
struct Rows {
    void* at = nullptr;
    int64_t ld = 0;
};
Rows rows(const Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape, const char* what) {
    expect(t, type, shape, what);
    int64_t step = 1;
    for (int64_t k = t.dim() - 1; k > 0; --k) {
        if (t.stride(k) != step && t.size(k) != 1) refuse("%s: all but the first dimension must be contiguous", what);
        step *= t.size(k);
    }
    if (t.size(0) > 1 && t.stride(0) < step) refuse("%s: rows must not overlap", what);
    return {address(t, what), t.size(0) > 1 ? t.stride(0) : (step + 7) / 8 * 8};
}

int64_t whole(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
int small(PyObject* o, const char* what) {
    const int64_t v = whole(o);
    if (v < INT32_MIN || v > INT32_MAX) refuse("%s is out of range", what);
    return static_cast<int>(v);
}
int size_of(int64_t n, const char* what) {
    if (n > INT32_MAX) refuse("%s is out of range", what);
    return static_cast<int>(n);
}
int truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}
void* stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
    PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
    if (!s) throw Raised{};
    void* p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
}

// ep_cache_t of two [pages, page_size, heads, dim] tensors, in any order of the first three in memory.
ep_cache_t cache_of(const Tensor& k, const Tensor& v, float k_scale, float v_scale, int64_t heads, int64_t dim) {
    if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
        refuse("k_cache and v_cache must be [pages, page_size, kv_heads, head_dim] of one type");
    if (k.size(2) != heads || k.size(3) != dim)
        refuse("cache rows are [%lld, %lld], the call's are [%lld, %lld]", static_cast<long long>(k.size(2)),
               static_cast<long long>(k.size(3)), static_cast<long long>(heads), static_cast<long long>(dim));
    if ((k.stride(3) != 1 || v.stride(3) != 1) && dim != 1) refuse("the cache's last dimension must be contiguous");
    ep_cache_t c{};
    c.dtype = type_code(k, "cache", false, true);
    c.page_size = size_of(k.size(1), "page_size");
    c.num_pages = k.size(0);
    c.k_page_stride = k.stride(0), c.k_slot_stride = k.stride(1), c.k_head_stride = k.stride(2);
    c.v_page_stride = v.stride(0), c.v_slot_stride = v.stride(1), c.v_head_stride = v.stride(2);
    c.k_scale = k_scale, c.v_scale = v_scale;
    return c;
}

// (logits, topk_idx, topk_weights, bias, score, renormalize, scale, num_groups, topk_groups, group_top, stream)
long router_topk(PyObject* const* a) {
    const Tensor& logits = tensor(a[0], "logits");
    dimensions(logits, 2, "logits");
    const Tensor& idx = tensor(a[1], "topk_idx");
    dimensions(idx, 2, "topk_idx");
    const int64_t T = logits.size(0), E = logits.size(1), K = idx.size(1);
    ep_router_config_t c{};
    c.logits_dtype = type_code(logits, "logits", true, false);
    c.score = small(a[4], "score");
    c.renormalize = truth(a[5]);
    c.scale = real(a[6]);
    c.num_groups = small(a[7], "num_groups");
    c.topk_groups = small(a[8], "topk_groups");
    c.group_top = small(a[9], "group_top");
    const Rows l = rows(logits, logits.scalar_type(), {T, E}, "logits");
    tensor(a[2], "topk_weights");
    return library.router_topk(l.at, l.ld, static_cast<const float*>(dense(a[3], kFp32, {E}, "bias")), size_of(T, "T"),
                               size_of(E, "E"), size_of(K, "K"), &c, static_cast<int64_t*>(dense(a[1], kInt64, {T, K}, "topk_idx")),
                               static_cast<float*>(dense(a[2], kFp32, {T, K}, "topk_weights")), stream_of(a[10]));
}

// (logits, topk_idx, grad_weights, grad_logits, score, renormalize, scale, stream)
long router_topk_backward(PyObject* const* a) {
    const Tensor& logits = tensor(a[0], "logits");
    dimensions(logits, 2, "logits");
    const Tensor& idx = tensor(a[1], "topk_idx");
    dimensions(idx, 2, "topk_idx");
    const int64_t T = logits.size(0), E = logits.size(1), K = idx.size(1);
    ep_router_config_t c{};
    c.logits_dtype = type_code(logits, "logits", true, false);
    c.score = small(a[4], "score");
    c.renormalize = truth(a[5]);
    c.scale = real(a[6]);
    const Rows l = rows(logits, logits.scalar_type(), {T, E}, "logits");
    const Rows i = rows(idx, kInt64, {T, K}, "topk_idx");
    const Rows g = rows(tensor(a[3], "grad_logits"), logits.scalar_type(), {T, E}, "grad_logits");
    tensor(a[2], "grad_weights");
    return library.router_topk_backward(l.at, l.ld, static_cast<const int64_t*>(i.at), i.ld,
                                        static_cast<const float*>(dense(a[2], kFp32, {T, K}, "grad_weights")), size_of(T, "T"),
                                        size_of(E, "E"), size_of(K, "K"), &c, g.at, g.ld, stream_of(a[7]));
}

// (q, k, v, positions, slots, cos_sin, q_out, k_cache, v_cache, interleaved, k_scale, v_scale, device_error, stream)
long kv_append(PyObject* const* a) {
    const Tensor& k = tensor(a[1], "k");
    dimensions(k, 3, "k");
    const int64_t T = k.size(0), n = k.size(1), d = k.size(2);
    ep_append_config_t c{};
    c.dtype = type_code(k, "k", false, false);
    const Rows kr = rows(k, k.scalar_type(), {T, n, d}, "k"), vr = rows(tensor(a[2], "v"), k.scalar_type(), {T, n, d}, "v");
    Rows qr, qo;
    int64_t h = 0;
    if (const Tensor* q = optional_tensor(a[0], "q")) {
        dimensions(*q, 3, "q");
        h = q->size(1);
        qr = rows(*q, k.scalar_type(), {T, h, d}, "q");
        qo = rows(tensor(a[6], "q_out"), k.scalar_type(), {T, h, d}, "q_out");
    }
    int64_t most = 0, rot = 0;
    const Tensor* table = optional_tensor(a[5], "cos_sin");
    if (table) {
        dimensions(*table, 2, "cos_sin");
        most = table->size(0), rot = table->size(1);
    }
    const Tensor &kc = tensor(a[7], "k_cache"), &vc = tensor(a[8], "v_cache");
    const ep_cache_t cache = cache_of(kc, vc, real(a[10]), real(a[11]), n, d);
    c.num_heads = size_of(h, "heads");
    c.num_kv_heads = size_of(n, "kv_heads");
    c.head_dim = size_of(d, "head_dim");
    c.rotary_dim = size_of(rot, "rotary_dim");
    c.interleaved = truth(a[9]);
    c.q_ld = qr.ld, c.k_ld = kr.ld, c.v_ld = vr.ld, c.q_out_ld = qo.ld;
    c.max_position = most;
    return library.kv_append(qr.at, kr.at, vr.at, static_cast<const int64_t*>(dense(a[3], kInt64, {T}, "positions")),
                             static_cast<const int64_t*>(dense(a[4], kInt64, {T}, "slots")),
                             static_cast<const float*>(dense(a[5], kFp32, {most, rot}, "cos_sin")), size_of(T, "T"), &c, qo.at,
                             address(kc, "k_cache"), address(vc, "v_cache"), &cache,
                             static_cast<int32_t*>(dense(a[12], kInt32, {1}, "device_error")), stream_of(a[13]));
}

// (q, k_cache, v_cache, block_table, seq_lens, out, workspace, lse, scale or None, window, k_scale, v_scale, stream)
long paged_attention(PyObject* const* a) {
    const Tensor& q = tensor(a[0], "q");
    dimensions(q, 3, "q");
    const Tensor &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"), &table = tensor(a[3], "block_table");
    dimensions(kc, 4, "k_cache");
    dimensions(table, 2, "block_table");
    const int64_t B = q.size(0), h = q.size(1), d = q.size(2), n = kc.size(2), pages = table.size(1);
    ep_attention_config_t c{};
    c.dtype = type_code(q, "q", false, false);
    const Rows qr = rows(q, q.scalar_type(), {B, h, d}, "q"), o = rows(tensor(a[5], "out"), q.scalar_type(), {B, h, d}, "out");
    const Rows t = rows(table, kInt32, {B, pages}, "block_table");
    const ep_cache_t cache = cache_of(kc, vc, real(a[10]), real(a[11]), n, d);
    c.num_heads = size_of(h, "heads");
    c.num_kv_heads = size_of(n, "kv_heads");
    c.head_dim = size_of(d, "head_dim");
    c.max_pages = size_of(pages, "max_pages");
    c.q_ld = qr.ld, c.out_ld = o.ld, c.table_ld = t.ld;
    c.scale = a[8] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d))) : real(a[8]);
    c.window = small(a[9], "window");
    const Tensor& work = tensor(a[6], "workspace");
    if (!work.is_contiguous()) refuse("workspace must be contiguous");
    tensor(a[4], "seq_lens");
    return library.paged_attention(qr.at, address(kc, "k_cache"), address(vc, "v_cache"), &cache, static_cast<const int32_t*>(t.at),
                                   static_cast<const int32_t*>(dense(a[4], kInt32, {B}, "seq_lens")), size_of(B, "B"), &c, o.at,
                                   static_cast<float*>(dense(a[7], kFp32, {B, h}, "lse")), address(work, "workspace"),
                                   work.numel() * work.element_size(), stream_of(a[12]));
}

// (x, weights, scales, y, expert_offsets, expert_counts, zeros, activation, workspace, stream)
long expert_w4(PyObject* const* a) {
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weights"), &s = tensor(a[2], "scales");
    dimensions(x, 2, "x");
    dimensions(w, 3, "weights");
    dimensions(s, 3, "scales");
    const int64_t n = x.size(0), I = x.size(1), E = w.size(0), O = w.size(1), groups = s.size(1);
    if (2 * w.size(2) != I || groups < 1 || I % groups != 0)
        refuse("weights [%lld, %lld, %lld] and %lld groups do not fit rows of %lld", static_cast<long long>(E), static_cast<long long>(O),
               static_cast<long long>(w.size(2)), static_cast<long long>(groups), static_cast<long long>(I));
    ep_w4_config_t c{};
    c.dtype = type_code(x, "x", false, false);
    c.group_size = size_of(I / groups, "group_size");
    c.activation = small(a[7], "activation");
    const Rows xr = rows(x, x.scalar_type(), {n, I}, "x");
    const Rows y = rows(tensor(a[3], "y"), x.scalar_type(), {n, c.activation == EP_ACT_SWIGLU ? O / 2 : O}, "y");
    c.x_ld = xr.ld, c.y_ld = y.ld;
    Tensor own;
    void* work = nullptr;
    int64_t bytes;
    if (const Tensor* t = optional_tensor(a[8], "workspace")) {
        if (!t->is_cuda()) refuse("workspace must be a CUDA tensor");   // (tensor maps address it)
        if (!t->is_contiguous()) refuse("workspace must be contiguous");
        work = address(*t, "workspace");
        bytes = t->numel() * t->element_size();
    } else {
        if (a[9] != Py_None) refuse("a call on a stream of its own needs a workspace");
        bytes = library.expert_w4_workspace(n, size_of(I, "I"), c.group_size, c.dtype);
        if (bytes > 0) {   // (x may be pinned host memory: its options are not the workspace's)
            own = at::empty({bytes}, at::TensorOptions().dtype(kByte).device(at::kCUDA, c10::cuda::current_device()));
            work = own.data_ptr();
        }
    }
    return library.expert_w4(xr.at, n, size_of(I, "I"), static_cast<const uint8_t*>(dense(a[1], kByte, {E, O, I / 2}, "weights")),
                             dense(a[2], x.scalar_type(), {E, groups, O}, "scales"),
                             static_cast<const uint8_t*>(dense(a[6], kByte, {E, groups, O}, "zeros")),
                             static_cast<const int32_t*>(dense(a[4], kInt32, {E + 1}, "expert_offsets")),
                             static_cast<const int32_t*>(dense(a[5], kInt32, {E}, "expert_counts")), size_of(E, "E"),
                             size_of(O, "O"), &c, y.at, work, bytes, stream_of(a[9]));
}

// No exception leaves an entry point.
template <long (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
    if (count != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %d", N, static_cast<int>(count));
        return nullptr;
    }
    if (!library.expert_w4_workspace) {
        PyErr_SetString(PyExc_RuntimeError, "open() has not been called");
        return nullptr;
    }
    try {
        one_device(args, count);
        return PyLong_FromLong(F(args));
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
        return nullptr;
    }
}

template <typename F>
bool look_up(void* handle, const char* name, F* to) {
    *to = reinterpret_cast<F>(dlsym(handle, name));
    if (!*to) PyErr_Format(PyExc_RuntimeError, "%s is not in the library", name);
    return *to != nullptr;
}

// open(path): the library's entry points.
PyObject* open_library(PyObject*, PyObject* path) {
    const char* p = PyUnicode_AsUTF8(path);
    if (!p) return nullptr;
    void* handle = dlopen(p, RTLD_NOW | RTLD_LOCAL);
    if (!handle) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    Library l;
    if (!look_up(handle, "ep_router_topk", &l.router_topk) || !look_up(handle, "ep_router_topk_backward", &l.router_topk_backward) ||
        !look_up(handle, "ep_kv_append", &l.kv_append) || !look_up(handle, "ep_paged_attention", &l.paged_attention) ||
        !look_up(handle, "ep_expert_w4", &l.expert_w4) || !look_up(handle, "ep_expert_w4_workspace", &l.expert_w4_workspace))
        return nullptr;
    library = l;
    Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"open", open_library, METH_O, nullptr},
                         ENTRY(router_topk, 11),
                         ENTRY(router_topk_backward, 8),
                         ENTRY(kv_append, 14),
                         ENTRY(paged_attention, 13),
                         ENTRY(expert_w4, 10),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_bind() { return PyModule_Create(&module); }
