// torch_ops.cpp -- the 8-bit cache's and the tree attention's calls on torch
// tensors, as a CPython extension.
//
// A decode step makes these calls once per layer, and for one sequence the
// kernels take less time than the checks of two dozen shapes and strides do in
// Python (14 us for a write, 34 us for an attention call).  Here the tensors
// are read through torch's C++ interface: checks, outputs, workspace and launch
// in one call.  The arguments' meaning is documented in kv_cache.py; the
// library behind include/lse_merge.h validates extents, alignment and overlap.
//
// Each function returns its result, raises ValueError or TypeError, or returns
// the library's error code as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/CUDAContextLight.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>

#include "lse_merge.h"

namespace {

// A Python error that is already set.
struct Raised {};

[[noreturn]] void value_error(const char* what) {
    PyErr_SetString(PyExc_ValueError, what);
    throw Raised{};
}
[[noreturn]] void type_error(const char* what) {
    PyErr_SetString(PyExc_TypeError, what);
    throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor, not %s", name, Py_TYPE(o)->tp_name);
        throw Raised{};
    }
    return THPVariable_Unpack(o);
}
// NULL for None.
const at::Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int dtype_code(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return LSE_MERGE_F32;
        case at::kHalf: return LSE_MERGE_F16;
        case at::kBFloat16: return LSE_MERGE_BF16;
        default: type_error("unsupported dtype; use float32, float16 or bfloat16");
    }
}
at::ScalarType dtype_arg(PyObject* o, at::ScalarType none) {
    if (o == Py_None) return none;
    if (!THPDtype_Check(o)) type_error("dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

const void* address(const at::Tensor& t) { return t.const_data_ptr(); }
template <typename T = void>
T* addr(const at::Tensor& t) { return static_cast<T*>(const_cast<void*>(address(t))); }

// Of a tensor that the call writes: its own storage (a lazy clone gets it now).
template <typename T = void>
T* addr_to_write(const at::Tensor& t) { return static_cast<T*>(t.mutable_data_ptr()); }
// Autograd sees that the tensor was written.
void written(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Strides of the first three dimensions.
void strides3(const at::Tensor& t, int64_t* s) {
    const auto st = t.strides();
    s[0] = st[0], s[1] = st[1], s[2] = st[2];
}

void same_device(const char* what, const c10::Device& dev, std::initializer_list<const at::Tensor*> ts) {
    if (!dev.is_cuda()) {
        PyErr_Format(PyExc_ValueError, "%s runs on CUDA tensors only (there is no CPU path)", what);
        throw Raised{};
    }
    for (const at::Tensor* t : ts)
        if (t && t->device() != dev) value_error("all tensors must be on the same CUDA device");
}

const int32_t* lengths(const at::Tensor* x, int64_t n, const char* what) {
    if (!x) return nullptr;
    if (x->scalar_type() != at::kInt || x->dim() != 1 || x->numel() != n || !x->is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be a contiguous int32 tensor of %lld elements", what, (long long)n);
        throw Raised{};
    }
    return addr<int32_t>(*x);
}

int as_int(int64_t n) {
    if (n < INT32_MIN || n > INT32_MAX) value_error("a size does not fit 32 bits");
    return (int)n;
}

void check_cache(const at::Tensor& k, const at::Tensor& v, const at::Tensor* ks, const at::Tensor* vs) {
    if (k.scalar_type() != at::kFloat8_e4m3fn || v.scalar_type() != at::kFloat8_e4m3fn)
        type_error("k_cache and v_cache must be float8_e4m3fn");
    if (k.dim() != 4 || k.sizes() != v.sizes()) value_error("k_cache and v_cache must both be [B, Hkv, L, D]");
    if (!ks || !vs) value_error("an e4m3 cache needs k_scale and v_scale");
    if (ks->scalar_type() != at::kFloat || vs->scalar_type() != at::kFloat)
        type_error("k_scale and v_scale must be float32");
    if (ks->sizes() != k.sizes().slice(0, 3) || vs->sizes() != k.sizes().slice(0, 3))
        value_error("k_scale and v_scale must be [B, Hkv, L]");
    if (k.stride(3) != 1 || v.stride(3) != 1) value_error("k_cache and v_cache must be contiguous along D");
}

int sm_count(int dev) {
    static int known[64];   // the same value, whoever writes it first (under the GIL)
    int n = dev < 64 ? known[dev] : 0;
    if (n == 0) {
        n = at::cuda::getDeviceProperties((c10::DeviceIndex)dev)->multiProcessorCount;
        if (dev < 64) known[dev] = n;
    }
    return n;
}

// The call without the GIL, on the current stream of the current device.
template <typename Args>
int launch(int (*call)(const Args*, lse_merge_stream_t), const Args& a) {
    const lse_merge_stream_t s = (lse_merge_stream_t)c10::cuda::getCurrentCUDAStream().stream();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call(&a, s);
    Py_END_ALLOW_THREADS
    return rc;
}

PyObject* pair(at::Tensor&& a, at::Tensor&& b) {
    PyObject* x = THPVariable_Wrap(std::move(a));
    PyObject* y = x ? THPVariable_Wrap(std::move(b)) : nullptr;
    PyObject* t = y ? PyTuple_New(2) : nullptr;
    if (!t) {
        Py_XDECREF(x);
        Py_XDECREF(y);
        return nullptr;
    }
    PyTuple_SET_ITEM(t, 0, x);
    PyTuple_SET_ITEM(t, 1, y);
    return t;
}

void nargs(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
    throw Raised{};
}

void cache_fields(lse_merge_kv_args& a, const at::Tensor& kc, const at::Tensor& vc, const at::Tensor& ks,
                  const at::Tensor& vs) {
    strides3(kc, &a.k_b);
    strides3(vc, &a.v_b);
    strides3(ks, &a.ks_b);
    strides3(vs, &a.vs_b);
    a.B = as_int(kc.size(0)), a.Hkv = as_int(kc.size(1)), a.L = as_int(kc.size(2)), a.D = as_int(kc.size(3));
}

// (k_cache, v_cache, k_scale, v_scale, k, v, start, count, select) -> code
PyObject* quantize(PyObject* const* o, Py_ssize_t n) {
    nargs(n, 9);
    const at::Tensor &kc = tensor(o[0], "k_cache"), &vc = tensor(o[1], "v_cache");
    const at::Tensor *ks = optional(o[2], "k_scale"), *vs = optional(o[3], "v_scale");
    check_cache(kc, vc, ks, vs);
    const at::Tensor &k = tensor(o[4], "k"), &v = tensor(o[5], "v");
    const at::Tensor *start = optional(o[6], "start"), *count = optional(o[7], "count"),
                     *select = optional(o[8], "select");
    const int64_t B = kc.size(0), Hkv = kc.size(1);
    if (k.dim() != 4 || k.sizes() != v.sizes() || k.size(0) != B || k.size(1) != Hkv || k.size(3) != kc.size(3))
        value_error("k and v must both be [B, Hkv, S, D]");
    if (k.scalar_type() != v.scalar_type()) type_error("k and v must share one dtype");
    if (k.stride(3) != 1 || v.stride(3) != 1) value_error("k and v must be contiguous along D");
    same_device("kv_quantize_", kc.device(), {&vc, ks, vs, &k, &v, start, count, select});
    const int64_t S = k.size(2);
    int64_t T = S;
    lse_merge_kv_args a{};
    if (select) {
        if (select->scalar_type() != at::kInt || select->dim() != 2 || select->size(0) != B || !select->is_contiguous())
            value_error("select must be a contiguous int32 tensor [B, T]");
        T = select->size(1);
        a.select = addr<int32_t>(*select);
    }
    a.start = lengths(start, B, "start");
    a.count = lengths(count, B, "count");
    if (!start && B) value_error("start must be given");
    if (B == 0 || Hkv == 0 || T == 0 || (S == 0 && select)) return PyLong_FromLong(LSE_MERGE_OK);
    const c10::cuda::CUDAGuard guard(kc.device());
    cache_fields(a, kc, vc, *ks, *vs);
    a.k_cache = addr_to_write(kc), a.v_cache = addr_to_write(vc);
    a.k_scale = addr_to_write<float>(*ks), a.v_scale = addr_to_write<float>(*vs);
    a.k = addr(k), a.v = addr(v);
    strides3(k, &a.kx_b);
    strides3(v, &a.vx_b);
    a.T = as_int(T), a.S = as_int(S);
    a.dtype = dtype_code(k.scalar_type());
    const int rc = launch(lse_merge_kv_quantize, a);
    if (rc == LSE_MERGE_OK)
        for (const at::Tensor* t : {&kc, &vc, ks, vs}) written(*t);
    return PyLong_FromLong(rc);
}

// (k_cache, v_cache, k_scale, v_scale, start, length, count, dtype) -> (k, v) or code
PyObject* dequantize(PyObject* const* o, Py_ssize_t n) {
    nargs(n, 8);
    const at::Tensor &kc = tensor(o[0], "k_cache"), &vc = tensor(o[1], "v_cache");
    const at::Tensor *ks = optional(o[2], "k_scale"), *vs = optional(o[3], "v_scale");
    check_cache(kc, vc, ks, vs);
    const at::Tensor *start = optional(o[4], "start"), *count = optional(o[6], "count");
    same_device("kv_dequantize", kc.device(), {&vc, ks, vs, start, count});
    const long long length = PyLong_AsLongLong(o[5]);
    if (length == -1 && PyErr_Occurred()) throw Raised{};
    if (length < 0) value_error("length must not be negative");
    const at::ScalarType dtype = dtype_arg(o[7], at::kBFloat16);
    lse_merge_kv_args a{};
    a.dtype = dtype_code(dtype);
    const int64_t B = kc.size(0), Hkv = kc.size(1), D = kc.size(3);
    a.start = lengths(start, B, "start");
    a.count = lengths(count, B, "count");
    if (!start && B) value_error("start must be given");
    const c10::cuda::CUDAGuard guard(kc.device());
    at::Tensor k = at::detail::empty_cuda({B, Hkv, length, D}, dtype, kc.device(), c10::nullopt);
    at::Tensor v = at::detail::empty_cuda({B, Hkv, length, D}, dtype, kc.device(), c10::nullopt);
    if (k.numel() != 0) {
        cache_fields(a, kc, vc, *ks, *vs);
        a.k_cache = addr(kc), a.v_cache = addr(vc);
        a.k_scale = addr<float>(*ks), a.v_scale = addr<float>(*vs);
        a.k = addr(k), a.v = addr(v);
        a.kx_b = a.vx_b = Hkv * length * D;
        a.kx_h = a.vx_h = length * D;
        a.kx_t = a.vx_t = D;
        a.T = a.S = as_int(length);
        const int rc = launch(lse_merge_kv_dequantize, a);
        if (rc != LSE_MERGE_OK) return PyLong_FromLong(rc);
    }
    return pair(std::move(k), std::move(v));
}

// (decode, q, k_cache, v_cache, k_draft, v_draft, tree, k_scale, v_scale, kv_len, draft_len, splits, scale,
//  out_dtype) -> (out, lse) or code; decode: q is [B, Hq, D] and the cache e4m3
PyObject* attention(PyObject* const* o, Py_ssize_t n) {
    nargs(n, 14);
    const bool decode = o[0] == Py_True;
    const at::Tensor &q = tensor(o[1], "q"), &k = tensor(o[2], "k_cache"), &v = tensor(o[3], "v_cache");
    const at::Tensor *kd = optional(o[4], "k_draft"), *vd = optional(o[5], "v_draft"), *tree = optional(o[6], "tree"),
                     *ks = optional(o[7], "k_scale"), *vs = optional(o[8], "v_scale"),
                     *klen = optional(o[9], "kv_len"), *dlen = optional(o[10], "draft_len");
    if (decode) {
        if (q.dim() != 3 || k.dim() != 4) value_error("q must be [B, Hq, D] and the caches [B, Hkv, L, D]");
        if (k.scalar_type() != at::kFloat8_e4m3fn) type_error("k_cache and v_cache must be float8_e4m3fn");
    } else if (q.dim() != 4 || k.dim() != 4) {
        value_error("q must be [B, T, Hq, D] and the caches [B, Hkv, L, D]");
    }
    const auto qs = q.sizes();
    const int64_t B = qs[0], T = decode ? 1 : qs[1], Hq = qs[decode ? 1 : 2], D = qs[decode ? 2 : 3];
    const int64_t Hkv = k.size(1), L = k.size(2);
    if (k.sizes() != v.sizes() || k.size(0) != B || k.size(3) != D)
        value_error("k_cache and v_cache must be [B, Hkv, L, D] with q's B and D");
    const bool fp8 = k.scalar_type() == at::kFloat8_e4m3fn;
    if (fp8)
        check_cache(k, v, ks, vs);
    else if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
        type_error("the cache must be of q's dtype, or float8_e4m3fn with scales");
    else if (ks || vs)
        value_error("k_scale and v_scale go with a float8_e4m3fn cache");
    if (q.strides().back() != 1 || k.stride(3) != 1 || v.stride(3) != 1)
        value_error("q, k_cache and v_cache must be contiguous along D");
    const c10::Device dev = q.device();
    same_device("attention", dev, {&k, &v, kd, vd, tree, ks, vs, klen, dlen});
    lse_merge_tree_args a{};
    if ((kd || vd || tree) && !(kd && vd && tree)) value_error("k_draft, v_draft and tree go together");
    if (kd) {
        if (kd->dim() != 4 || kd->size(0) != B || kd->size(1) != Hkv || kd->size(2) != T || kd->size(3) != D ||
            vd->sizes() != kd->sizes())
            value_error("k_draft and v_draft must be [B, Hkv, T, D]");
        if (kd->scalar_type() != q.scalar_type() || vd->scalar_type() != q.scalar_type())
            type_error("k_draft and v_draft must be of q's dtype");
        if (kd->stride(3) != 1 || vd->stride(3) != 1) value_error("k_draft and v_draft must be contiguous along D");
        if (tree->scalar_type() != at::kLong || tree->dim() < 1 || tree->dim() > 2 || tree->size(-1) != T ||
            (tree->dim() == 2 && tree->size(0) != B) || (T > 1 && tree->stride(-1) != 1))
            value_error("tree must be int64 [T] or [B, T], contiguous along T");
        a.k_draft = addr(*kd), a.v_draft = addr(*vd), a.tree = addr<int64_t>(*tree);
        a.tree_b = tree->dim() == 2 ? tree->stride(0) : 0;
        strides3(*kd, &a.kd_b);
        strides3(*vd, &a.vd_b);
    }
    const at::ScalarType out_dtype = dtype_arg(o[13], q.scalar_type());
    a.dtype = dtype_code(q.scalar_type());
    a.cache_dtype = fp8 ? LSE_MERGE_E4M3 : a.dtype;
    a.out_dtype = dtype_code(out_dtype);
    a.B = as_int(B), a.T = as_int(T), a.Hq = as_int(Hq), a.Hkv = as_int(Hkv), a.L = as_int(L), a.D = as_int(D);
    if (o[11] == Py_None) {
        a.R = lse_merge_tree_default_splits(a.B, a.T, a.Hq, a.Hkv, a.L, a.D, sm_count(dev.index()));
    } else {
        const long long r = PyLong_AsLongLong(o[11]);
        if (r == -1 && PyErr_Occurred()) throw Raised{};
        a.R = as_int(r);
    }
    if (o[12] == Py_None) {
        a.scale = (float)(1.0 / std::sqrt((double)D));
    } else {
        const double s = PyFloat_AsDouble(o[12]);
        if (s == -1.0 && PyErr_Occurred()) throw Raised{};
        a.scale = (float)s;
    }
    a.kv_len = lengths(klen, B, "kv_len");
    a.draft_len = lengths(dlen, B, "draft_len");
    const c10::cuda::CUDAGuard guard(dev);
    const bool empty = B == 0 || T == 0;   // no query token: nothing to launch
    int64_t need = 0;
    const int rc0 = empty ? LSE_MERGE_OK
                          : lse_merge_tree_workspace_bytes(a.B, a.T, a.Hq, a.D, a.R, kd != nullptr, &need);
    if (rc0 != LSE_MERGE_OK) return PyLong_FromLong(rc0);
    at::Tensor out = decode ? at::detail::empty_cuda({B, Hq, D}, out_dtype, dev, c10::nullopt)
                            : at::detail::empty_cuda({B, T, Hq, D}, out_dtype, dev, c10::nullopt);
    at::Tensor lse = decode ? at::detail::empty_cuda({B, Hq}, at::kFloat, dev, c10::nullopt)
                            : at::detail::empty_cuda({B, T, Hq}, at::kFloat, dev, c10::nullopt);
    if (empty) return pair(std::move(out), std::move(lse));
    // the workspace is this call's own, freed in the stream's order: calls on
    // other streams, and graphs captured from them, never share one
    c10::DataPtr ws;
    if (need) ws = c10::cuda::CUDACachingAllocator::get()->allocate((size_t)need);
    a.q = addr(q), a.k = addr(k), a.v = addr(v);
    a.k_scale = fp8 ? addr<float>(*ks) : nullptr;
    a.v_scale = fp8 ? addr<float>(*vs) : nullptr;
    a.out_o = addr(out), a.out_lse = addr<float>(lse);
    a.workspace = ws.get(), a.workspace_bytes = need;
    const auto st = q.strides();
    a.q_b = st[0], a.q_t = decode ? 0 : st[1], a.q_h = st[decode ? 1 : 2];
    strides3(k, &a.k_b);
    strides3(v, &a.v_b);
    if (fp8) {
        strides3(*ks, &a.ks_b);
        strides3(*vs, &a.vs_b);
    }
    const int rc = launch(lse_merge_tree_attention, a);
    if (rc != LSE_MERGE_OK) return PyLong_FromLong(rc);
    return pair(std::move(out), std::move(lse));
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(args, n);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name, const char* doc) {
    return {name, (PyCFunction)(void (*)(void))entry<F>, METH_FASTCALL, doc};
}

PyMethodDef methods[] = {
    method<quantize>("quantize", "(k_cache, v_cache, k_scale, v_scale, k, v, start, count, select) -> code"),
    method<dequantize>("dequantize",
                       "(k_cache, v_cache, k_scale, v_scale, start, length, count, dtype) -> (k, v) or code"),
    method<attention>("attention",
                      "(decode, q, k_cache, v_cache, k_draft, v_draft, tree, k_scale, v_scale, kv_len, draft_len, "
                      "splits, scale, out_dtype) -> (out, lse) or code"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_ops", "liblse_merge.so's calls on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops(void) { return PyModule_Create(&module); }
