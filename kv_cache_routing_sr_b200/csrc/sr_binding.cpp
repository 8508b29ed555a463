// Python side of the 8-bit cache and shared-prefix entry points: checks every
// tensor against the shapes, type and device that the call implies, allocates
// outputs that were not given, and calls the C ABI on the tensors' device and
// stream. The same checks in Python with ctypes take 8 to 16 us a call, more than
// the kernels of a short one (4 to 9 us); here they take about 1. The decoders' steps
// check theirs here too (step_fits).
//
// The entry points come as addresses (use), from whichever build of the library is
// loaded. No C++ exception leaves a function: each becomes a Python exception.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <optional>
#include <stdexcept>
#include <string>
#include <torch/csrc/autograd/python_variable.h>

#include "sinkrouter.h"

namespace {

struct Entry {
    decltype(&sr_kv_append_quant) kv_append_quant;
    decltype(&sr_kv_dequant) kv_dequant;
    decltype(&sr_rope_append_route_kv) rope_append_route_kv;
    decltype(&sr_decode_attention_quant) decode_quant;
    decltype(&sr_decode_attention_quant_partial) decode_quant_partial;
    decltype(&sr_prefix_attention) prefix;
    decltype(&sr_prefix_attention_partial) prefix_partial;
} g_entry{};

using Shape = c10::IntArrayRef;

struct ValueError : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string text(Shape s)
{
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i)
        r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        throw ValueError(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int32_t whole(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw ValueError(std::string(name) + " must be an integer");
    }
    if (v < INT32_MIN || v > INT32_MAX)
        throw ValueError(std::string(name) + " is out of range");
    return (int32_t)v;
}

int32_t dim(const at::Tensor &t, int64_t i, const char *name)
{
    if (t.size(i) > INT32_MAX)
        throw ValueError(std::string(name) + " has a dimension of more than 2^31 - 1");
    return (int32_t)t.size(i);
}

// The tensors of one call, all on one CUDA device.
struct Call {
    int device = -1;

    void on(const at::Tensor &t, const char *name)
    {
        if (!t.is_cuda())
            throw ValueError(std::string(name) + " must be a CUDA tensor");
        device = t.get_device();
    }

    void check(const at::Tensor &t, const char *name, at::ScalarType type, Shape shape, bool rows = false) const
    {
        if (!t.is_cuda())
            throw ValueError(std::string(name) + " must be a CUDA tensor");
        if (t.scalar_type() != type)
            throw ValueError(std::string(name) + " must be " + c10::toString(type) + ", got " +
                             c10::toString(t.scalar_type()));
        if (t.sizes() != shape || t.get_device() != device)
            throw ValueError(std::string(name) + " must have shape " + text(shape) + " on cuda:" + std::to_string(device) +
                             ", got " + text(t.sizes()) + " on cuda:" + std::to_string(t.get_device()));
        if (rows ? t.stride(-1) != 1 : !t.is_contiguous())
            throw ValueError(std::string(name) + (rows ? "'s last dimension must be contiguous" : " must be contiguous"));
    }

    void *ptr(PyObject *o, const char *name, at::ScalarType type, Shape shape) const
    {
        const at::Tensor &t = tensor(o, name);
        check(t, name, type, shape);
        return t.data_ptr();
    }

    void *opt(PyObject *o, const char *name, at::ScalarType type, Shape shape) const
    {
        return o == Py_None ? nullptr : ptr(o, name, type, shape);
    }

    // An output: the given tensor, or a new one, which belongs to the stream that the
    // call runs on: what earlier owners of its memory have in flight on another stream
    // would not be waited for.
    at::Tensor out(PyObject *o, const char *name, at::ScalarType type, Shape shape, PyObject *on_stream) const
    {
        if (o == Py_None) {
            std::optional<c10::cuda::CUDAStreamGuard> guard;
            if (on_stream != Py_None)
                guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream(on_stream)),
                                                               static_cast<c10::DeviceIndex>(device)));
            return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, device));
        }
        const at::Tensor &t = tensor(o, name);
        check(t, name, type, shape);
        return t;
    }

    // Handle of the given stream (an integer), or of the device's current one.
    void *stream(PyObject *o) const
    {
        if (o == Py_None)
            return c10::cuda::getCurrentCUDAStream(device).stream();
        void *s = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            throw ValueError("stream must be a CUDA stream");
        }
        return s;
    }
};

// Makes the call's device current for as long as it lives, if it is not already.
struct OnDevice {
    std::optional<c10::cuda::CUDAGuard> guard;
    explicit OnDevice(int device)
    {
        if (c10::cuda::current_device() != device)
            guard.emplace(device);
    }
};

constexpr auto kF32 = at::kFloat, kI32 = at::kInt, kBf16 = at::kBFloat16, kU8 = at::kByte;

// A cache [B, Hkv, Lmax, 128] and what it holds.
struct Cache {
    int32_t kv, B, Hkv, Lmax;
    at::ScalarType type;
    void *k, *v;
    float *scales;
};

Cache cache(Call &c, PyObject *k, PyObject *v, PyObject *scales, bool quant_only)
{
    const at::Tensor &t = tensor(k, "k_cache");
    c.on(t, "k_cache");
    Cache r;
    r.type = t.scalar_type();
    r.kv = r.type == at::kFloat8_e4m3fn ? SR_KV_E4M3 : r.type == at::kChar ? SR_KV_INT8 : SR_KV_BF16;
    if (r.kv == SR_KV_BF16 && (quant_only || r.type != kBf16))
        throw ValueError(std::string("k_cache must be float8_e4m3fn or int8") + (quant_only ? "" : " or bfloat16") +
                         ", got " + c10::toString(r.type));
    if (t.dim() != 4 || t.size(3) != 128)
        throw ValueError("k_cache must be [B, Hkv, Lmax, 128], got " + text(t.sizes()));
    if ((r.kv == SR_KV_BF16) != (scales == Py_None))
        throw ValueError(r.kv == SR_KV_BF16 ? "a bfloat16 cache has no kv_scales" : "an 8-bit cache needs kv_scales");
    r.B = dim(t, 0, "k_cache");
    r.Hkv = dim(t, 1, "k_cache");
    r.Lmax = dim(t, 2, "k_cache");
    c.check(t, "k_cache", r.type, t.sizes());
    r.k = t.data_ptr();
    r.v = c.ptr(v, "v_cache", r.type, t.sizes());
    r.scales = static_cast<float *>(c.opt(scales, "kv_scales", kF32, {r.B, r.Hkv, r.Lmax, 2}));
    return r;
}

sr_row_strides row_strides(const Call &c, const at::Tensor &t, const char *name, Shape shape)
{
    if (t.dim() != 4)
        throw ValueError(std::string(name) + " must be [B, T, Hkv, 128]");
    c.check(t, name, kBf16, shape, true);
    // the stride of a dimension of one entry is never used
    auto at = [&](int i) -> int64_t { return t.size(i) > 1 ? t.stride(i) : 0; };
    return {at(0), at(1), at(2)};
}

PyObject *status_only(sr_status st) { return PyLong_FromLong(st); }

// (k_new, v_new, start, n_new, k_cache, v_cache, kv_scales, k0, v0, device_error, stream) -> status
PyObject *kv_append_quant(PyObject *const *a)
{
    Call c;
    const Cache k = cache(c, a[4], a[5], a[6], true);
    const at::Tensor &kn = tensor(a[0], "k_new"), &vn = tensor(a[1], "v_new");
    const int64_t T = kn.dim() == 4 ? kn.size(1) : 0;
    const int64_t shape[] = {k.B, T, k.Hkv, 128}, row0[] = {k.B, k.Hkv, 128};
    const sr_row_strides ks = row_strides(c, kn, "k_new", shape), vs = row_strides(c, vn, "v_new", shape);
    const sr_dims d{k.B, k.Hkv, k.Hkv, 128, k.Lmax};
    auto *start = static_cast<int32_t *>(c.ptr(a[2], "start", kI32, {k.B}));
    auto *n = static_cast<int32_t *>(c.ptr(a[3], "n_new", kI32, {k.B}));
    void *k0 = c.opt(a[7], "k0", kBf16, row0), *v0 = c.opt(a[8], "v0", kBf16, row0);
    auto *err = static_cast<int32_t *>(c.opt(a[9], "device_error", kI32, {1}));
    if (T == 0)
        return status_only(SR_OK);
    OnDevice on(c.device);
    return status_only(g_entry.kv_append_quant(&d, k.kv, dim(kn, 1, "k_new"), kn.data_ptr(), &ks, vn.data_ptr(), &vs, start,
                                               n, k.k, k.v, k.scales, k0, v0, err, c.stream(a[10])));
}

// (k_cache, v_cache, kv_scales, start, n, k_out, v_out, device_error, stream) -> status
PyObject *kv_dequant(PyObject *const *a)
{
    Call c;
    const Cache k = cache(c, a[0], a[1], a[2], true);
    const at::Tensor &ko = tensor(a[5], "k_out");
    if (ko.dim() != 4)
        throw ValueError("k_out must be [B, Hkv, T, 128]");
    const int32_t T = dim(ko, 2, "k_out");
    const int64_t shape[] = {k.B, k.Hkv, T, 128};
    c.check(ko, "k_out", kBf16, shape);
    void *vo = c.ptr(a[6], "v_out", kBf16, shape);
    const sr_dims d{k.B, k.Hkv, k.Hkv, 128, k.Lmax};
    auto *start = static_cast<int32_t *>(c.ptr(a[3], "start", kI32, {k.B}));
    auto *n = static_cast<int32_t *>(c.ptr(a[4], "n", kI32, {k.B}));
    auto *err = static_cast<int32_t *>(c.opt(a[7], "device_error", kI32, {1}));
    if (T == 0)
        return status_only(SR_OK);
    OnDevice on(c.device);
    return status_only(g_entry.kv_dequant(&d, k.kv, T, k.k, k.v, k.scales, start, n, ko.data_ptr(), vo, err, c.stream(a[8])));
}

// (q_in, k_new, v_new, rope_cos, rope_sin, seq_lens, k_cache, v_cache, kv_scales, k0, v0, tau, pos_offset,
//  seq_lens_out, q_out, route_mask, active_list, device_error, stream) -> (status, q_out, route_mask, active_list)
PyObject *rope_append_route_kv(PyObject *const *a)
{
    Call c;
    const Cache k = cache(c, a[6], a[7], a[8], false);
    const at::Tensor &q = tensor(a[0], "q_in"), &cos = tensor(a[3], "rope_cos");
    if (q.dim() != 3 || cos.dim() != 2)
        throw ValueError("q_in must be [B, Hq, 128] and rope_cos [max_pos, 64]");
    const int32_t Hq = dim(q, 1, "q_in"), max_pos = dim(cos, 0, "rope_cos");
    const int64_t U = (int64_t)k.B * k.Hkv;
    const int64_t qs[] = {k.B, Hq, 128}, kvs[] = {k.B, k.Hkv, 128}, table[] = {max_pos, 64};
    c.check(q, "q_in", kBf16, qs);
    c.check(cos, "rope_cos", kF32, table);
    void *kn = c.ptr(a[1], "k_new", kBf16, kvs), *vn = c.ptr(a[2], "v_new", kBf16, kvs);
    auto *sin = static_cast<float *>(c.ptr(a[4], "rope_sin", kF32, table));
    auto *lens = static_cast<int32_t *>(c.ptr(a[5], "seq_lens", kI32, {k.B}));
    void *k0 = c.ptr(a[9], "k0", kBf16, kvs), *v0 = c.ptr(a[10], "v0", kBf16, kvs);
    const double tau = PyFloat_AsDouble(a[11]);
    if (tau == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw ValueError("tau must be a number");
    }
    auto *lens_out = static_cast<int32_t *>(c.opt(a[13], "seq_lens_out", kI32, {k.B}));
    auto *err = static_cast<int32_t *>(c.opt(a[17], "device_error", kI32, {1}));
    const at::Tensor qo = c.out(a[14], "q_out", kBf16, qs, a[18]), mask = c.out(a[15], "route_mask", kU8, {U}, a[18]),
                     active = c.out(a[16], "active_list", kI32, {1 + U}, a[18]);
    const sr_dims d{k.B, Hq, k.Hkv, 128, k.Lmax};
    sr_status st;
    {
        OnDevice on(c.device);
        st = g_entry.rope_append_route_kv(&d, k.kv, whole(a[12], "pos_offset"), q.data_ptr(), kn, vn,
                                          static_cast<float *>(cos.data_ptr()), sin, max_pos, lens,
                                          lens_out ? lens_out : lens, k.k, k.v, k.scales, k0, v0, (float)tau, qo.data_ptr(),
                                          static_cast<uint8_t *>(mask.data_ptr()),
                                          static_cast<int32_t *>(active.data_ptr()), err, c.stream(a[18]));
    }
    return Py_BuildValue("(iNNN)", (int)st, THPVariable_Wrap(qo), THPVariable_Wrap(mask), THPVariable_Wrap(active));
}

// (partial, q, k_cache, v_cache, kv_scales, v0, seq_lens, active_list, n_splits, out, lse, workspace pointer, bytes,
//  stream) -> (status, out, lse); lse may be None unless partial
PyObject *decode_quant(PyObject *const *a)
{
    Call c;
    const bool partial = a[0] == Py_True;
    const Cache k = cache(c, a[2], a[3], a[4], true);
    const at::Tensor &q = tensor(a[1], "q");
    if (q.dim() != 3)
        throw ValueError("q must be [B, Hq, 128]");
    const int32_t Hq = dim(q, 1, "q");
    const int64_t qs[] = {k.B, Hq, 128}, hs[] = {k.B, Hq};
    c.check(q, "q", kBf16, qs);
    void *v0 = c.ptr(a[5], "v0", kBf16, {k.B, k.Hkv, 128});
    auto *lens = static_cast<int32_t *>(c.ptr(a[6], "seq_lens", kI32, {k.B}));
    auto *active = static_cast<int32_t *>(c.ptr(a[7], "active_list", kI32, {1 + (int64_t)k.B * k.Hkv}));
    const at::Tensor out = c.out(a[9], partial ? "o_part" : "out", partial ? kF32 : kBf16, qs, a[13]);
    at::Tensor lse;
    if (partial || a[10] != Py_None)
        lse = c.out(a[10], partial ? "lse_part" : "lse", kF32, hs, a[13]);
    auto *z = lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr;
    const sr_dims d{k.B, Hq, k.Hkv, 128, k.Lmax};
    const int32_t ns = whole(a[8], "n_splits");
    void *ws = PyLong_AsVoidPtr(a[11]);
    const size_t bytes = PyLong_AsSize_t(a[12]);
    sr_status st;
    {
        OnDevice on(c.device);
        void *s = c.stream(a[13]);
        st = partial ? g_entry.decode_quant_partial(&d, k.kv, q.data_ptr(), k.k, k.v, k.scales, v0, lens, active, ns,
                                                    static_cast<float *>(out.data_ptr()), z, ws, bytes, s)
                     : g_entry.decode_quant(&d, k.kv, q.data_ptr(), k.k, k.v, k.scales, v0, lens, active, ns, out.data_ptr(),
                                            z, ws, bytes, s);
    }
    PyObject *zo = lse.defined() ? THPVariable_Wrap(lse) : (Py_INCREF(Py_None), Py_None);
    return Py_BuildValue("(iNN)", (int)st, THPVariable_Wrap(out), zo);
}

// (partial, q, k_prefix, v_prefix, prefix_len, v0, route_mask, o_suffix, lse_suffix, out, lse, workspace pointer,
//  bytes, stream) -> (status, out, lse)
PyObject *prefix(PyObject *const *a)
{
    Call c;
    const bool partial = a[0] == Py_True;
    const at::Tensor &q = tensor(a[1], "q"), &kp = tensor(a[2], "k_prefix");
    c.on(q, "q");
    if (q.dim() != 3 || kp.dim() != 3 || kp.size(2) != 128)
        throw ValueError("q must be [B, Hq, 128] and k_prefix [Hkv, max_prefix_len, 128]");
    const int32_t B = dim(q, 0, "q"), Hq = dim(q, 1, "q"), Hkv = dim(kp, 0, "k_prefix"), Lmax = dim(kp, 1, "k_prefix");
    const int64_t qs[] = {B, Hq, 128}, hs[] = {B, Hq};
    c.check(q, "q", kBf16, qs);
    c.check(kp, "k_prefix", kBf16, kp.sizes());
    void *vp = c.ptr(a[3], "v_prefix", kBf16, kp.sizes()), *v0 = c.ptr(a[5], "v0", kBf16, {B, Hkv, 128});
    auto *mask = static_cast<uint8_t *>(c.ptr(a[6], "route_mask", kU8, {(int64_t)B * Hkv}));
    auto *os = static_cast<float *>(c.opt(a[7], "o_suffix", kF32, qs));
    auto *ls = static_cast<float *>(c.opt(a[8], "lse_suffix", kF32, hs));
    const at::Tensor out = c.out(a[9], partial ? "o_part" : "out", partial ? kF32 : kBf16, qs, a[13]);
    at::Tensor lse;
    if (partial || a[10] != Py_None)
        lse = c.out(a[10], partial ? "lse_part" : "lse", kF32, hs, a[13]);
    auto *z = lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr;
    const sr_dims d{B, Hq, Hkv, 128, Lmax};
    const int32_t len = whole(a[4], "prefix_len");
    void *ws = PyLong_AsVoidPtr(a[11]);
    const size_t bytes = PyLong_AsSize_t(a[12]);
    sr_status st;
    {
        OnDevice on(c.device);
        void *s = c.stream(a[13]);
        st = partial ? g_entry.prefix_partial(&d, len, q.data_ptr(), kp.data_ptr(), vp, v0, mask,
                                              static_cast<float *>(out.data_ptr()), z, ws, bytes, s)
                     : g_entry.prefix(&d, len, q.data_ptr(), kp.data_ptr(), vp, v0, mask, os, ls, out.data_ptr(), z, ws,
                                      bytes, s);
    }
    PyObject *zo = lse.defined() ? THPVariable_Wrap(lse) : (Py_INCREF(Py_None), Py_None);
    return Py_BuildValue("(iNN)", (int)st, THPVariable_Wrap(out), zo);
}

// (out, n_kv_heads, q, k0, v0, k_prefix, v_prefix, prefix_len, k_cache, v_cache, kv_scales, seq_lens) -> None
// The checks of a decoder's step before it launches anything, against the decoder's own
// output: its other buffers have that shape whatever the tensors' is, and an appended
// token is not taken back. Without v0 only the first two, which the call on an 8-bit
// cache does not see.
PyObject *step_fits(PyObject *const *a)
{
    const at::Tensor &out = tensor(a[0], "out");
    const int64_t B = out.size(0), Hq = out.size(1), Hkv = whole(a[1], "n_kv_heads");
    auto fits = [&](PyObject *o, const char *name, at::ScalarType type, Shape shape) {
        const at::Tensor &t = tensor(o, name);
        if (t.scalar_type() != type || t.sizes() != shape || t.device() != out.device() || !t.is_contiguous())
            throw ValueError(std::string(name) + " must be contiguous " + c10::toString(type) + " of shape " + text(shape) +
                             " on " + out.device().str() + ", got " + c10::toString(t.scalar_type()) + " of " +
                             text(t.sizes()) + " on " + t.device().str());
        if (type != kI32 && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16)
            throw ValueError(std::string(name) + " must be 16-byte aligned");
    };
    fits(a[2], "q", kBf16, {B, Hq, 128});
    fits(a[3], "k0", kBf16, {B, Hkv, 128});
    if (a[4] == Py_None)
        Py_RETURN_NONE;
    fits(a[4], "v0", kBf16, {B, Hkv, 128});
    const at::Tensor &kp = tensor(a[5], "k_prefix"), &kc = tensor(a[8], "k_cache");
    const int64_t cap = kp.dim() == 3 ? kp.size(1) : 0, len = whole(a[7], "prefix_len");
    fits(a[5], "k_prefix", kBf16, {Hkv, cap, 128});
    fits(a[6], "v_prefix", kBf16, {Hkv, cap, 128});
    if (cap < 1 || len < 0 || len > cap)
        throw ValueError("prefix_len must be in [0, " + std::to_string(cap) + "] of at least one position, got " +
                         std::to_string(len));
    const at::ScalarType type = a[10] == Py_None ? kBf16 : kc.scalar_type();
    const int64_t L = kc.dim() == 4 ? kc.size(2) : 0;
    fits(a[8], "k_cache", type, {B, Hkv, L, 128});
    fits(a[9], "v_cache", type, {B, Hkv, L, 128});
    fits(a[11], "seq_lens", kI32, {B});
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N> PyObject *guarded(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        PyObject *r = F(a);
        if (PyErr_Occurred()) { // a conversion above
            Py_XDECREF(r);
            return nullptr;
        }
        return r;
    } catch (const ValueError &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// use(addresses): the entry points, in Entry's order.
PyObject *use(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void *p[7];
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "expected 7 addresses");
        return nullptr;
    }
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred())
            return nullptr;
    }
    g_entry = {reinterpret_cast<decltype(&sr_kv_append_quant)>(p[0]), reinterpret_cast<decltype(&sr_kv_dequant)>(p[1]),
               reinterpret_cast<decltype(&sr_rope_append_route_kv)>(p[2]),
               reinterpret_cast<decltype(&sr_decode_attention_quant)>(p[3]),
               reinterpret_cast<decltype(&sr_decode_attention_quant_partial)>(p[4]),
               reinterpret_cast<decltype(&sr_prefix_attention)>(p[5]),
               reinterpret_cast<decltype(&sr_prefix_attention_partial)>(p[6])};
    Py_RETURN_NONE;
}

template <typename F> PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)); }

PyMethodDef g_methods[] = {
    {"use", fast(&use), METH_FASTCALL, "set the entry points' addresses"},
    {"kv_append_quant", fast(&guarded<kv_append_quant, 11>), METH_FASTCALL, nullptr},
    {"kv_dequant", fast(&guarded<kv_dequant, 9>), METH_FASTCALL, nullptr},
    {"rope_append_route_kv", fast(&guarded<rope_append_route_kv, 19>), METH_FASTCALL, nullptr},
    {"decode_quant", fast(&guarded<decode_quant, 14>), METH_FASTCALL, nullptr},
    {"prefix", fast(&guarded<prefix, 14>), METH_FASTCALL, nullptr},
    {"step_fits", fast(&guarded<step_fits, 12>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

// The docstring names the torch that this was compiled against: the build looks for it
// in the file before Python loads it into another.
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_sr_binding", SR_BINDING_MARK, -1, g_methods};

} // namespace

PyMODINIT_FUNC PyInit__sr_binding(void) { return PyModule_Create(&g_module); }
