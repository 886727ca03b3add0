// serving_ext.cpp -- Python module `_serving`: the calls of a serving step
// (include/inkling_paged_attn.h) on PyTorch tensors.
//
// A decoding step makes three calls of a few microseconds each on the GPU, so what the host
// spends on a call counts. This module checks the tensors, allocates the outputs and calls
// the C entry points, whose addresses it is given when the library is loaded (bind). Work
// goes to the current stream of the tensors' device. Each function returns its result, or
// the library's status as an int where the library refused the call; wrong tensors raise
// ValueError or TypeError.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <utility>

#include "inkling_paged_attn.h"

namespace {

decltype(&inkling_kv_plan) g_plan = nullptr;
decltype(&inkling_kv_append) g_append = nullptr;
decltype(&inkling_rel_attn_decode) g_decode = nullptr;
decltype(&inkling_rel_attn_decode_workspace_size) g_decode_size = nullptr;

// The tensor that an argument holds; null for None.
const at::Tensor* tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* name) {
    const at::Tensor* t = tensor(o, name);
    TORCH_CHECK_TYPE(t, name, " must be a tensor");
    return *t;
}

void check_shape(const at::Tensor& t, const char* name, std::initializer_list<int64_t> want) {
    bool same = t.dim() == int64_t(want.size());
    int i = 0;
    for (int64_t w : want) same = same && t.size(i++) == w;
    TORCH_CHECK_VALUE(same, name, " must have shape ", c10::IntArrayRef(want), ", got ", t.sizes());
}
void check_kind(const at::Tensor& t, const char* name, at::Device device, at::ScalarType type) {
    TORCH_CHECK_VALUE(t.device() == device, name, " is on ", t.device(), ", expected ", device);
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
}
void check(const at::Tensor* t, const char* name, at::Device device, at::ScalarType type,
           std::initializer_list<int64_t> want) {
    if (!t) return;
    check_kind(*t, name, device, type);
    check_shape(*t, name, want);
    TORCH_CHECK_VALUE(t->is_contiguous(), name, " must be contiguous");
}

template <class T>
T* data(const at::Tensor* t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

void need_args(Py_ssize_t got, Py_ssize_t want) {
    TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got);
}
void need_library() { TORCH_CHECK(g_decode, "the library has not been loaded"); }

inkling_kv_cache_desc describe(const at::Tensor& k, const at::Tensor& v) {
    TORCH_CHECK_VALUE(k.dim() == 4 && k.sizes() == v.sizes() && k.scalar_type() == v.scalar_type(),
                      "k_cache and v_cache must be [num_pages, page_size, heads_kv, head_dim] of one shape and dtype");
    const bool e4m3 = k.scalar_type() == at::kFloat8_e4m3fn;
    TORCH_CHECK_VALUE(e4m3 || k.scalar_type() == at::kBFloat16, "a cache is bfloat16 or float8_e4m3fn, got ",
                      k.scalar_type());
    TORCH_CHECK_VALUE(k.strides() == v.strides() && k.stride(3) == 1,
                      "k_cache and v_cache must have the same strides, head_dim contiguous");
    TORCH_CHECK_VALUE(k.is_cuda() && k.device() == v.device(), "k_cache and v_cache must be on one CUDA device");
    return {k.size(0), k.size(1), k.size(2), k.size(3), e4m3 ? INKLING_KV_E4M3 : INKLING_KV_BF16,
            k.stride(0), k.stride(1), k.stride(2)};
}
void check_scales(const inkling_kv_cache_desc& c, at::Device device, const at::Tensor* k, const at::Tensor* v) {
    const bool e4m3 = c.dtype == INKLING_KV_E4M3;
    TORCH_CHECK_VALUE((k != nullptr) == e4m3 && (v != nullptr) == e4m3,
                      "an e4m3 cache needs its scales k_scale and v_scale, a bfloat16 cache takes none");
    check(k, "k_scale", device, at::kFloat, {c.heads_kv});
    check(v, "v_scale", device, at::kFloat, {c.heads_kv});
}

// The outputs of a call as tensors over one allocation, each at a multiple of 256 bytes: a
// fraction of the host time of as many allocations.
class Outputs {
  public:
    void add(at::ScalarType type, std::initializer_list<int64_t> sizes) {
        TORCH_INTERNAL_ASSERT(count_ < kMost && sizes.size() <= 3);
        Item& it = items_[count_++];
        it.type = type;
        it.dims = int(sizes.size());
        int64_t n = int64_t(c10::elementSize(type));
        int i = 0;
        for (int64_t s : sizes) {
            it.sizes[i++] = s;
            n *= s;
        }
        it.at = bytes_;
        bytes_ += (n + 255) / 256 * 256;
    }
    // on the current device and stream
    void allocate() {
        c10::Allocator* const allocator = c10::cuda::CUDACachingAllocator::get();
        whole_ = c10::Storage(c10::Storage::use_byte_size_t(), size_t(bytes_), allocator->allocate(size_t(bytes_)),
                              allocator, /*resizable=*/false);
    }
    at::Tensor get(int i) const {
        const Item& it = items_[i];
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
            c10::Storage(whole_), c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(it.type));
        t.unsafeGetTensorImpl()->set_storage_offset(it.at / int64_t(c10::elementSize(it.type)));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(c10::IntArrayRef(it.sizes, it.dims));
        return t;
    }

  private:
    static constexpr int kMost = 5;
    struct Item {
        at::ScalarType type;
        int dims;
        int64_t sizes[3], at;
    };
    Item items_[kMost];
    int count_ = 0;
    int64_t bytes_ = 0;
    c10::Storage whole_;
};

PyObject* status(inkling_status s) { return PyLong_FromLong(s); }

// kv_plan(old_lens, new_lens, block_table, free_pages, free_count, page_size, num_pages, max_tokens, lens, info)
PyObject* kv_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 10);
    need_library();
    const at::Tensor &old_lens = needed(a[0], "old_lens"), &new_lens = needed(a[1], "new_lens"),
                     &table = needed(a[2], "block_table"), &pages = needed(a[3], "free_pages"),
                     &count = needed(a[4], "free_count");
    const int64_t page_size = integer(a[5]), num_pages = integer(a[6]), T = integer(a[7]);
    TORCH_CHECK_VALUE(table.dim() == 2 && table.is_cuda(), "block_table must be a CUDA tensor [requests, max_pages]");
    TORCH_CHECK_VALUE(T >= 0, "max_tokens must not be negative");
    const at::Device dev = table.device();
    const int64_t N = table.size(0), M = table.size(1);
    check(&old_lens, "old_lens", dev, at::kInt, {N});
    check(&new_lens, "new_lens", dev, at::kInt, {N});
    check(&table, "block_table", dev, at::kInt, {N, M});
    check(&pages, "free_pages", dev, at::kInt, {num_pages});
    check(&count, "free_count", dev, at::kInt, {1});
    const at::Tensor *lens_out = tensor(a[8], "lens"), *info_out = tensor(a[9], "info");
    check(lens_out, "lens", dev, at::kInt, {N});
    check(info_out, "info", dev, at::kInt, {4});
    const c10::cuda::CUDAGuard guard(dev);
    Outputs outs;
    outs.add(at::kLong, {T});
    outs.add(at::kInt, {T});
    outs.add(at::kInt, {N + 1});
    if (!lens_out) outs.add(at::kInt, {N});
    if (!info_out) outs.add(at::kInt, {4});
    outs.allocate();
    const at::Tensor slots = outs.get(0), positions = outs.get(1), start = outs.get(2);
    const at::Tensor lens = lens_out ? *lens_out : outs.get(3), info = info_out ? *info_out : outs.get(lens_out ? 3 : 4);
    const inkling_kv_plan_dims dims{N, page_size, M, num_pages, T};
    const inkling_status s =
        g_plan(&dims, data<int32_t>(&old_lens), data<int32_t>(&new_lens), data<int32_t>(&table), data<int32_t>(&pages),
               data<int32_t>(&count), data<int32_t>(&lens), data<int32_t>(&start), data<int64_t>(&slots),
               data<int32_t>(&positions), data<int32_t>(&info), c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    if (s != INKLING_OK) return status(s);
    PyObject* const d = PyDict_New();
    if (!d) return nullptr;
    static PyObject* const names[] = {
        PyUnicode_InternFromString("lens"), PyUnicode_InternFromString("query_start"),
        PyUnicode_InternFromString("slots"), PyUnicode_InternFromString("positions"),
        PyUnicode_InternFromString("info")};
    const at::Tensor* const values[] = {&lens, &start, &slots, &positions, &info};
    for (int i = 0; i < 5; ++i) {
        PyObject* const v = THPVariable_Wrap(*values[i]);
        const bool set = v && names[i] && PyDict_SetItem(d, names[i], v) == 0;
        Py_XDECREF(v);
        if (!set) {
            Py_DECREF(d);
            return nullptr;
        }
    }
    return d;
    END_HANDLE_TH_ERRORS
}

// kv_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, threshold, clip_scale, tau)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 10);
    need_library();
    const at::Tensor &k = needed(a[0], "k"), &v = needed(a[1], "v"), &slots = needed(a[2], "slots"),
                     &kc = needed(a[3], "k_cache"), &vc = needed(a[4], "v_cache");
    const at::Tensor *ks = tensor(a[5], "k_scale"), *vs = tensor(a[6], "v_scale"), *clip = tensor(a[8], "clip_scale"),
                     *tau = tensor(a[9], "tau");
    const inkling_kv_cache_desc cache = describe(kc, vc);
    const at::Device dev = kc.device();
    const int64_t T = slots.numel(), H = cache.heads_kv, D = cache.head_dim;
    for (const auto& [x, name] : {std::pair{&k, "k"}, std::pair{&v, "v"}}) {
        check_kind(*x, name, dev, at::kBFloat16);
        check_shape(*x, name, {T, H, D});
        TORCH_CHECK_VALUE(T == 0 || (x->stride(2) == 1 && (H == 1 || x->stride(1) == D)), name,
                          " must have dense heads and values");
    }
    check(&slots, "slots", dev, at::kLong, {T});
    check(clip, "clip_scale", dev, at::kFloat, {H, D});
    check(tau, "tau", dev, at::kFloat, {T});
    check_scales(cache, dev, ks, vs);
    const bool clips = a[7] != Py_None;
    TORCH_CHECK_VALUE(clips || (!clip && !tau), "clip_scale and tau need a threshold");
    // the stride of a single row means nothing
    const inkling_kv_append_dims dims{T, T > 1 ? k.stride(0) : H * D, T > 1 ? v.stride(0) : H * D, clips,
                                      clips ? real(a[7]) : 0.0};
    const c10::cuda::CUDAGuard guard(dev);
    const inkling_status s =
        g_append(&cache, &dims, data<uint16_t>(&k), data<uint16_t>(&v), data<int64_t>(&slots), data<float>(ks),
                 data<float>(vs), data<float>(clip), data<float>(tau), kc.data_ptr(), vc.data_ptr(),
                 c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    if (s != INKLING_OK) return status(s);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// paged_decode(q, k_cache, v_cache, block_table, lens, profiles, sink, window, scale, k_scale, v_scale, workspace)
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 12);
    need_library();
    const at::Tensor &q = needed(a[0], "q"), &kc = needed(a[1], "k_cache"), &vc = needed(a[2], "v_cache"),
                     &table = needed(a[3], "block_table"), &lens = needed(a[4], "lens");
    const at::Tensor *prof = tensor(a[5], "profiles"), *sink = tensor(a[6], "sink"), *ks = tensor(a[9], "k_scale"),
                     *vs = tensor(a[10], "v_scale"), *ws = tensor(a[11], "workspace");
    const inkling_kv_cache_desc cache = describe(kc, vc);
    const at::Device dev = kc.device();
    TORCH_CHECK_VALUE(q.dim() == 3 && q.size(2) == cache.head_dim,
                      "q must be [requests, heads_q, head_dim] with the cache's head_dim");
    TORCH_CHECK_VALUE(table.dim() == 2, "block_table must be [requests, max_pages]");
    TORCH_CHECK_VALUE(!prof || prof->dim() == 3, "profiles must be [requests, heads_q, rel_extent]");
    const int64_t N = q.size(0), Hq = q.size(1), D = q.size(2), M = table.size(1), R = prof ? prof->size(2) : 0;
    check(&q, "q", dev, at::kBFloat16, {N, Hq, D});
    check(&table, "block_table", dev, at::kInt, {N, M});
    check(&lens, "lens", dev, at::kInt, {N});
    check(prof, "profiles", dev, at::kBFloat16, {N, Hq, R});
    check(sink, "sink", dev, at::kFloat, {N, Hq});
    check_scales(cache, dev, ks, vs);
    if (ws) check(ws, "workspace", dev, at::kByte, {ws->numel()});
    const inkling_rel_attn_decode_dims dims{N, Hq, R, integer(a[7]), M, a[8] == Py_None ? 0.0 : real(a[8])};
    const c10::cuda::CUDAGuard guard(dev);
    Outputs outs;
    outs.add(at::kFloat, {N, Hq, D});
    outs.add(at::kFloat, {N, Hq});
    // a workspace of its own, so that it can be used again when the call returns; a small one
    // (the sizes that need none) costs less beside the outputs
    Outputs own;
    const size_t size = ws ? 0 : g_decode_size(&cache, &dims);
    Outputs& home = size <= 256 ? outs : own;
    if (size != 0) home.add(at::kByte, {int64_t(size)});
    outs.allocate();
    const at::Tensor out = outs.get(0), lse = outs.get(1);
    if (size > 256) own.allocate();
    at::Tensor scratch;
    if (size != 0) scratch = home.get(size <= 256 ? 2 : 0);
    if (!ws) ws = &scratch;
    const inkling_status s = g_decode(
        &cache, &dims, data<uint16_t>(&q), kc.data_ptr(), vc.data_ptr(), data<float>(ks), data<float>(vs),
        R ? data<uint16_t>(prof) : nullptr, data<float>(sink), data<int32_t>(&table), data<int32_t>(&lens),
        data<float>(&out), data<float>(&lse), ws->defined() ? ws->data_ptr() : nullptr,
        ws->defined() ? size_t(ws->numel()) : 0, c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    if (s != INKLING_OK) return status(s);
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
    END_HANDLE_TH_ERRORS
}

// bind(inkling_kv_plan, inkling_kv_append, inkling_rel_attn_decode, inkling_rel_attn_decode_workspace_size): addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    need_args(n, 4);
    g_plan = reinterpret_cast<decltype(g_plan)>(integer(a[0]));
    g_append = reinterpret_cast<decltype(g_append)>(integer(a[1]));
    g_decode = reinterpret_cast<decltype(g_decode)>(integer(a[2]));
    g_decode_size = reinterpret_cast<decltype(g_decode_size)>(integer(a[3]));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<kv_plan>("kv_plan"), method<kv_append>("kv_append"),
                           method<paged_decode>("paged_decode"), method<bind>("bind"),
                           {nullptr, nullptr, 0, nullptr}};
// What this file was compiled for; the build looks for it in the module, the binding in built_for.
constexpr char kBuiltFor[] = "serving module for " INKLING_BUILT_FOR;

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__serving() {
    PyObject* const m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "built_for", kBuiltFor + sizeof("serving module for ") - 1) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
