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

#include <algorithm>
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
    decltype(&ep_expert_fp8) expert_fp8 = nullptr;
    decltype(&ep_expert_ffn) expert_ffn = nullptr;
    decltype(&ep_expert_ffn_backward) expert_ffn_backward = nullptr;
} library;

using Tensor = at::Tensor;
constexpr auto kBf16 = at::ScalarType::BFloat16, kFp16 = at::ScalarType::Half, kFp32 = at::ScalarType::Float,
               kInt64 = at::ScalarType::Long, kInt32 = at::ScalarType::Int, kByte = at::ScalarType::Byte,
               kE4m3 = at::ScalarType::Float8_e4m3fn, kE5m2 = at::ScalarType::Float8_e5m2, kE8m0 = at::ScalarType::Float8_e8m0fnu;

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

// Refuses a tensor that tensor maps or later kernels address and that is not the GPU's.
const Tensor& on_gpu(const Tensor& t, const char* what) {
    if (!t.is_cuda() && t.numel() > 0) refuse("%s must be a CUDA tensor", what);
    return t;
}
Rows gpu_rows(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, const char* what) {
    return rows(on_gpu(tensor(o, what), what), type, shape, what);
}
Rows gpu_rows_or_none(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, const char* what) {
    return o == Py_None ? Rows{} : gpu_rows(o, type, shape, what);
}
void* gpu_dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, const char* what) {
    if (const Tensor* t = optional_tensor(o, what)) on_gpu(*t, what);
    return dense(o, type, shape, what);
}
// Scales [rows, blocks], fp32 or exponent bytes, in any order in memory.
struct Scales {
    void* at = nullptr;
    int64_t row = 0, block = 0;
    bool bytes = false;
};
Scales scales(PyObject* o, int64_t n, int64_t blocks, bool written, const char* what) {
    const Tensor& t = on_gpu(tensor(o, what), what);
    const auto type = t.scalar_type();
    const bool bytes = type == kByte || type == kE8m0;
    expect(t, bytes ? type : kFp32, {n, blocks}, what);
    Scales s{t.data_ptr(), t.stride(0), t.stride(1), bytes};
    // (of a dimension of one the stride says nothing)
    if (n <= 1) s.row = std::max<int64_t>(s.row, 1);
    if (blocks <= 1) s.block = std::max<int64_t>(s.block, 1);
    if (written && n > 0 && blocks > 0) {
        const bool by_row = (n == 1 || s.row > s.block * (blocks - 1)) && s.block >= 1;
        const bool by_block = (blocks == 1 || s.block > s.row * (n - 1)) && s.row >= 1;
        if (!by_row && !by_block) refuse("%s must not overlap", what);
    }
    return s;
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

// (x, x_scales, weights, weight_scales, y, y_scales, expert_offsets, expert_counts, activation, scale_mode, stream)
long expert_fp8(PyObject* const* a) {
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[2], "weights"), &y = tensor(a[4], "y");
    dimensions(x, 2, "x");
    dimensions(w, 3, "weights");
    const int64_t n = x.size(0), I = x.size(1), E = w.size(0), O = w.size(1), blocks = I / 128;
    ep_fp8_config_t c{};
    if (x.scalar_type() != kE4m3 && x.scalar_type() != kE5m2) refuse("x: %s is not supported", c10::toString(x.scalar_type()));
    c.x_dtype = x.scalar_type() == kE4m3 ? EP_DTYPE_FP8_E4M3 : EP_DTYPE_FP8_E5M2;
    c.y_dtype = type_code(y, "y", false, true);
    c.activation = small(a[8], "activation");
    const int64_t cols = c.activation == EP_ACT_SWIGLU ? O / 2 : O;
    const Rows xr = gpu_rows(a[0], x.scalar_type(), {n, I}, "x"), yr = gpu_rows(a[4], y.scalar_type(), {n, cols}, "y");
    c.x_ld = n > 1 ? xr.ld : (xr.ld + 15) / 16 * 16;
    c.y_ld = yr.ld;
    const Scales xs = scales(a[1], n, blocks, false, "x_scales");
    c.x_scale_mode = xs.bytes ? EP_SCALE_UE8M0 : EP_SCALE_FP32;
    c.x_scale_row = xs.row, c.x_scale_block = xs.block;
    Scales ys;
    if (c.y_dtype == EP_DTYPE_FP8_E4M3) {
        ys = scales(a[5], n, cols / 128, true, "y_scales");
        c.y_scale_mode = ys.bytes ? EP_SCALE_UE8M0 : small(a[9], "scale_mode");
        if (!ys.bytes && c.y_scale_mode == EP_SCALE_UE8M0) refuse("y_scales of exponents must be bytes");
        c.y_scale_row = ys.row, c.y_scale_block = ys.block;
    }
    tensor(a[3], "weight_scales");
    return library.expert_fp8(xr.at, xs.at, n, size_of(I, "I"), static_cast<const uint8_t*>(gpu_dense(a[2], kE4m3, {E, O, I}, "weights")),
                              static_cast<const float*>(gpu_dense(a[3], kFp32, {E, (O + 127) / 128, blocks}, "weight_scales")),
                              static_cast<const int32_t*>(dense(a[6], kInt32, {E + 1}, "expert_offsets")),
                              static_cast<const int32_t*>(dense(a[7], kInt32, {E}, "expert_counts")), size_of(E, "E"), size_of(O, "O"),
                              &c, yr.at, ys.at, stream_of(a[10]));
}

// Sizes of a gated block: x or grad_y [rows, H], a row tensor of width F (or 2F), E from the offsets' or the weights' tensor.
struct Block {
    int64_t n, H, E, F;
    at::ScalarType type;
};
Block block_of(const Tensor& x, const char* what, const Tensor& act, const char* act_what, int64_t parts, const Tensor& w, const char* w_what) {
    dimensions(x, 2, what);
    dimensions(act, 2, act_what);
    dimensions(w, 3, w_what);
    return {x.size(0), x.size(1), w.size(0), act.size(1) / parts, x.scalar_type()};
}

// (x, w_gate_up, w_down, act, y, gate_up, expert_offsets, expert_counts, stream)
long expert_ffn(PyObject* const* a) {
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w_gate_up"), &act = tensor(a[3], "act");
    const Block b = block_of(x, "x", act, "act", 1, w, "w_gate_up");
    ep_ffn_config_t c{};
    c.grad_w_dtype = c.dtype = type_code(x, "x", false, false);
    const Rows xr = gpu_rows(a[0], b.type, {b.n, b.H}, "x"), ar = gpu_rows(a[3], b.type, {b.n, b.F}, "act");
    const Rows yr = gpu_rows_or_none(a[4], b.type, {b.n, b.H}, "y"), gr = gpu_rows_or_none(a[5], b.type, {b.n, 2 * b.F}, "gate_up");
    if ((a[4] == Py_None) != (a[2] == Py_None)) refuse("w_down and y go together");
    c.x_ld = xr.ld, c.act_ld = ar.ld, c.y_ld = yr.ld, c.gate_up_ld = gr.ld;
    return library.expert_ffn(xr.at, b.n, size_of(b.H, "H"), gpu_dense(a[1], b.type, {b.E, 2 * b.F, b.H}, "w_gate_up"),
                              gpu_dense(a[2], b.type, {b.E, b.H, b.F}, "w_down"),
                              static_cast<const int32_t*>(dense(a[6], kInt32, {b.E + 1}, "expert_offsets")),
                              static_cast<const int32_t*>(dense(a[7], kInt32, {b.E}, "expert_counts")), size_of(b.E, "E"),
                              size_of(b.F, "F"), &c, gr.at, ar.at, yr.at, stream_of(a[8]));
}

// (grad_y, x, gate_up, act, w_gate_up, w_down, grad_gate_up, grad_x, grad_w_gate_up, grad_w_down, expert_offsets, expert_counts,
//  accumulate, stream)
long expert_ffn_backward(PyObject* const* a) {
    const Tensor &dy = tensor(a[0], "grad_y"), &gate_up = tensor(a[2], "gate_up"), &w = tensor(a[5], "w_down");
    const Block b = block_of(dy, "grad_y", gate_up, "gate_up", 2, w, "w_down");
    ep_ffn_config_t c{};
    c.grad_w_dtype = c.dtype = type_code(dy, "grad_y", false, false);
    const Rows yr = gpu_rows(a[0], b.type, {b.n, b.H}, "grad_y"), gr = gpu_rows(a[2], b.type, {b.n, 2 * b.F}, "gate_up");
    const Rows xr = gpu_rows_or_none(a[1], b.type, {b.n, b.H}, "x"), ar = gpu_rows_or_none(a[3], b.type, {b.n, b.F}, "act");
    const Rows dg = gpu_rows(a[6], b.type, {b.n, 2 * b.F}, "grad_gate_up"), dx = gpu_rows_or_none(a[7], b.type, {b.n, b.H}, "grad_x");
    auto grad_type = b.type;   // the weights' gradients: both of the tensors' type or both fp32
    for (const int i : {8, 9})
        if (const Tensor* t = optional_tensor(a[i], "a weight gradient"))
            if (t->scalar_type() == kFp32) grad_type = kFp32, c.grad_w_dtype = EP_DTYPE_FP32;
    c.accumulate = truth(a[12]);
    c.x_ld = xr.ld, c.act_ld = ar.ld, c.y_ld = yr.ld, c.gate_up_ld = gr.ld, c.grad_x_ld = dx.ld, c.grad_gate_up_ld = dg.ld;
    return library.expert_ffn_backward(yr.at, xr.at, gr.at, ar.at, b.n, size_of(b.H, "H"),
                                       gpu_dense(a[4], b.type, {b.E, 2 * b.F, b.H}, "w_gate_up"),
                                       gpu_dense(a[5], b.type, {b.E, b.H, b.F}, "w_down"),
                                       static_cast<const int32_t*>(dense(a[10], kInt32, {b.E + 1}, "expert_offsets")),
                                       static_cast<const int32_t*>(dense(a[11], kInt32, {b.E}, "expert_counts")), size_of(b.E, "E"),
                                       size_of(b.F, "F"), &c, dg.at, dx.at,
                                       gpu_dense(a[8], grad_type, {b.E, 2 * b.F, b.H}, "grad_w_gate_up"),
                                       gpu_dense(a[9], grad_type, {b.E, b.H, b.F}, "grad_w_down"), stream_of(a[13]));
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
        !look_up(handle, "ep_expert_w4", &l.expert_w4) || !look_up(handle, "ep_expert_w4_workspace", &l.expert_w4_workspace) ||
        !look_up(handle, "ep_expert_fp8", &l.expert_fp8) || !look_up(handle, "ep_expert_ffn", &l.expert_ffn) ||
        !look_up(handle, "ep_expert_ffn_backward", &l.expert_ffn_backward))
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
                         ENTRY(expert_fp8, 11),
                         ENTRY(expert_ffn, 9),
                         ENTRY(expert_ffn_backward, 14),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_bind() { return PyModule_Create(&module); }
