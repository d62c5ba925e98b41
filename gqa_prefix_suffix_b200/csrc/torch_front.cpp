// torch_front.cpp -- the torch front end of the prefix-cache operators, as a
// Python extension module: checks tensors, allocates what the caller did not
// give, and calls the C ABI on the current stream.
//
// The operators' smallest calls take 3 to 13 us on the GPU; the same checks
// and the call through ctypes took 9 to 19 us on the host, this takes 4 to 8.
// The library's entry points are handed in by address (bind), so that
// there is one loaded library whatever opened it.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "dm05_suffix_attn.h"

namespace {

struct Bad {
    std::string what;
};
struct Failed {
    int status;
    const char *what;
};

decltype(&dm05_kv8_quantize) g_quantize;
decltype(&dm05_suffix_attn_kv8) g_attn;
decltype(&dm05_suffix_attn_kv8_plan) g_plan;
decltype(&dm05_prefix_attn_mass) g_mass;
decltype(&dm05_prefix_attn_mass_kv8) g_mass_kv8;
decltype(&dm05_prefix_evict) g_evict;
decltype(&dm05_prefix_evict_kv8) g_evict_kv8;
PyObject *g_error;  // Dm05Error(status, what)

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kU8 = at::kByte,
                         kF8 = at::kFloat8_e4m3fn;

const char *type_name(at::ScalarType t)
{
    switch (t) {
    case kBf16: return "torch.bfloat16";
    case kF32: return "torch.float32";
    case kI32: return "torch.int32";
    case kU8: return "torch.uint8";
    default: return "torch.float8_e4m3fn";
    }
}

const at::Tensor &tensor(const char *name, PyObject *o)
{
    if (!THPVariable_Check(o)) throw Bad{std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}

// A dense tensor of this type and shape on CUDA device `index`.
const at::Tensor &need(const char *name, const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape, int index)
{
    if (t.scalar_type() == type && t.is_cuda() && t.get_device() == index && t.sizes() == shape && t.is_contiguous())
        return t;
    std::string s = std::string(name) + " must be a contiguous CUDA " + type_name(type) + " tensor [";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    s += "]";
    if (index >= 0) s += " on cuda:" + std::to_string(index);
    throw Bad{s};
}

void *optional(const char *name, PyObject *o, at::ScalarType type, at::IntArrayRef shape, int index)
{
    return o == Py_None ? nullptr : need(name, tensor(name, o), type, shape, index).data_ptr();
}

int64_t integer(const char *name, PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Bad{std::string(name) + " must be an integer"};
    }
    if (v > 0x7fffffffLL || v < -0x7fffffffLL) throw Bad{std::string(name) + " is out of range"};
    return v;
}

const at::Tensor &four(const char *name, PyObject *o, const char *shape)
{
    const at::Tensor &t = tensor(name, o);
    if (t.dim() != 4) throw Bad{std::string(name) + " must be " + shape};
    for (int i = 0; i < 4; ++i)
        if (t.size(i) > 0x7fffffffLL) throw Bad{std::string(name) + " is too large"};
    return t;
}

void check_block(int64_t block, const std::string &name)
{
    if (block != 16 && block != 32 && block != 64 && block != 128)
        throw Bad{name + " must be 16, 32, 64 or 128"};
}

// An 8-bit cache: the tuple (k, v, k_scale, v_scale, block).
struct Cache {
    const at::Tensor *k, *v, *ks, *vs;
    int64_t B, H, P, D, block;
};

Cache cache_of(const char *name, PyObject *o)
{
    const std::string n(name);
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) throw Bad{n + " must be a Kv8Cache"};
    Cache c{};
    c.k = &four((n + ".k").c_str(), PyTuple_GET_ITEM(o, 0), "[B,Hkv,P,D]");
    c.v = &tensor((n + ".v").c_str(), PyTuple_GET_ITEM(o, 1));
    c.ks = &tensor((n + ".k_scale").c_str(), PyTuple_GET_ITEM(o, 2));
    c.vs = &tensor((n + ".v_scale").c_str(), PyTuple_GET_ITEM(o, 3));
    c.block = integer((n + ".block").c_str(), PyTuple_GET_ITEM(o, 4));
    check_block(c.block, n + ".block");
    c.B = c.k->size(0);
    c.H = c.k->size(1);
    c.P = c.k->size(2);
    c.D = c.k->size(3);
    return c;
}

void check_cache(const char *name, const Cache &c, int index)
{
    const std::string n(name);
    const int64_t scales[3] = {c.B, c.H, (c.P + c.block - 1) / c.block};
    need((n + ".k").c_str(), *c.k, kF8, c.k->sizes(), index);
    need((n + ".v").c_str(), *c.v, kF8, c.k->sizes(), index);
    need((n + ".k_scale").c_str(), *c.ks, kF32, scales, index);
    need((n + ".v_scale").c_str(), *c.vs, kF32, scales, index);
}

// A fresh cache: zero codes, unit scales.
std::vector<at::Tensor> fresh_cache(int64_t B, int64_t H, int64_t P, int64_t D, int64_t block, const at::Device &dev)
{
    const auto codes = at::TensorOptions().dtype(kU8).device(dev), scales = at::TensorOptions().dtype(kF32).device(dev);
    const int64_t n = (P + block - 1) / block;
    return {at::zeros({B, H, P, D}, codes).view(kF8), at::zeros({B, H, P, D}, codes).view(kF8),
            at::ones({B, H, n}, scales), at::ones({B, H, n}, scales)};
}

// The tensors' device, made current, and its current stream.
struct On {
    int index;
    c10::cuda::CUDAGuard guard;
    cudaStream_t stream;
    explicit On(int i) : index(i), guard(static_cast<c10::DeviceIndex>(i)),
                         stream(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(i)).stream()) {}
};

// Device of a tensor that has to be on one.
int device_of(const char *name, const at::Tensor &t, at::ScalarType type)
{
    if (!t.is_cuda()) need(name, t, type, t.sizes(), -1);
    return t.get_device();
}

void check(int rc, const char *what)
{
    if (rc != DM05_OK) throw Failed{rc, what};
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

PyObject *tuple_of(std::initializer_list<PyObject *> items)
{
    PyObject *t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
    Py_ssize_t i = 0;
    for (PyObject *o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}

PyObject *same(PyObject *o)
{
    Py_INCREF(o);
    return o;
}

// Every entry: `n` positional arguments; Bad becomes ValueError, a status of
// the library Dm05Error.
template <class F>
PyObject *guarded(PyObject *const *a, Py_ssize_t have, Py_ssize_t n, F &&f) noexcept
{
    try {
        if (have != n) throw Bad{"wrong number of arguments"};
        if (g_error == nullptr) throw Bad{"the library is not bound"};
        return f(a);
    } catch (const Bad &e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
    } catch (const Failed &e) {
        PyObject *x = PyObject_CallFunction(g_error, "is", e.status, e.what);
        if (x != nullptr) {
            PyErr_SetObject(g_error, x);
            Py_DECREF(x);
        }
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// kv8_quantize(k, v, block, valid_len, first, out) -> (k, v, k_scale, v_scale) or None when out was given
PyObject *quantize(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded(args, n, 6, [](PyObject *const *a) -> PyObject * {
        const at::Tensor &k = four("k", a[0], "[B,Hkv,P,D]");
        const int dev = device_of("k", k, kBf16);
        const int64_t B = k.size(0), H = k.size(1), P = k.size(2), D = k.size(3), first = integer("first", a[4]);
        need("k", k, kBf16, k.sizes(), dev);
        const at::Tensor &v = need("v", tensor("v", a[1]), kBf16, k.sizes(), dev);
        void *vl = optional("valid_len", a[3], kI32, {B}, dev);
        const On on(dev);
        auto call = [&](const at::Tensor &k8, const at::Tensor &v8, const at::Tensor &ks, const at::Tensor &vs, int64_t block) {
            check(g_quantize(k.data_ptr(), v.data_ptr(), static_cast<const int32_t *>(vl), k8.data_ptr(), v8.data_ptr(),
                             static_cast<float *>(ks.data_ptr()), static_cast<float *>(vs.data_ptr()),
                             static_cast<int>(B), static_cast<int>(H), static_cast<int>(P), static_cast<int>(D),
                             static_cast<int>(block), static_cast<int>(first), on.stream),
                  "dm05_kv8_quantize");
        };
        if (a[5] != Py_None) {
            const Cache c = cache_of("out", a[5]);
            check_cache("out", c, dev);
            if (c.k->sizes() != k.sizes()) throw Bad{"out must be a cache of k's sizes"};
            call(*c.k, *c.v, *c.ks, *c.vs, c.block);
            return same(Py_None);
        }
        const int64_t block = integer("block", a[2]);
        check_block(block, "block");
        const auto c = fresh_cache(B, H, P, D, block, k.device());
        call(c[0], c[1], c[2], c[3], block);
        return tuple_of({wrap(c[0]), wrap(c[1]), wrap(c[2]), wrap(c[3])});
    });
}

// suffix_attn_kv8(q, cache, k_suffix, v_suffix, valid_len, mask, out, lse, want_lse, workspace) -> (out, lse or None)
PyObject *attn(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded(args, n, 10, [](PyObject *const *a) -> PyObject * {
        const at::Tensor &q = four("q", a[0], "[B,Hq,S,D]");
        const int dev = device_of("q", q, kBf16);
        const int64_t B = q.size(0), Hq = q.size(1), S = q.size(2), D = q.size(3);
        need("q", q, kBf16, q.sizes(), dev);
        const Cache c = cache_of("cache", a[1]);
        check_cache("cache", c, dev);
        if (c.B != B || c.D != D) throw Bad{"cache must have q's batch and head size"};
        const int64_t suffix[4] = {B, c.H, S, D}, rows[3] = {B, Hq, S};
        const at::Tensor &ks = need("k_suffix", tensor("k_suffix", a[2]), kBf16, suffix, dev);
        const at::Tensor &vs = need("v_suffix", tensor("v_suffix", a[3]), kBf16, suffix, dev);
        void *vl = optional("prefix_valid_len", a[4], kI32, {B}, dev);
        void *mask = optional("prefix_mask", a[5], kU8, {B, c.P}, dev);
        if (a[6] != Py_None) need("out", tensor("out", a[6]), kBf16, q.sizes(), dev);
        if (a[7] != Py_None) need("lse", tensor("lse", a[7]), kF32, rows, dev);
        if (a[9] != Py_None) {
            const at::Tensor &w = tensor("workspace", a[9]);
            need("workspace", w, kU8, {w.numel()}, dev);
        }
        const On on(dev);
        const int iB = static_cast<int>(B), iq = static_cast<int>(Hq), ik = static_cast<int>(c.H),
                  iP = static_cast<int>(c.P), iS = static_cast<int>(S), iD = static_cast<int>(D);
        at::Tensor out = a[6] != Py_None ? THPVariable_Unpack(a[6]) : at::empty(q.sizes(), q.options());
        at::Tensor lse;
        if (a[7] != Py_None)
            lse = THPVariable_Unpack(a[7]);
        else if (PyObject_IsTrue(a[8]))
            lse = at::empty(rows, q.options().dtype(kF32));
        at::Tensor ws;
        size_t bytes = 0;
        if (a[9] != Py_None) {
            ws = THPVariable_Unpack(a[9]);
            bytes = static_cast<size_t>(ws.numel());
        } else {
            check(g_plan(iB, iq, ik, iP, iS, iD, nullptr, nullptr, &bytes), "dm05_suffix_attn_kv8");
            if (bytes > 0) ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(kU8));
        }
        check(g_attn(q.data_ptr(), c.k->data_ptr(), c.v->data_ptr(), static_cast<const float *>(c.ks->data_ptr()),
                     static_cast<const float *>(c.vs->data_ptr()), static_cast<int>(c.block),
                     static_cast<const int32_t *>(vl), static_cast<const uint8_t *>(mask), ks.data_ptr(), vs.data_ptr(),
                     out.data_ptr(), lse.defined() ? static_cast<float *>(lse.data_ptr()) : nullptr,
                     ws.defined() ? ws.data_ptr() : nullptr, bytes, iB, iq, ik, iP, iS, iD, on.stream),
              "dm05_suffix_attn_kv8");
        return tuple_of({wrap(out), lse.defined() ? wrap(lse) : same(Py_None)});
    });
}

// prefix_attn_mass(q, k, k_scale or None, block, lse, valid_len, mask, mass_in, mass) -> mass
PyObject *mass(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded(args, n, 9, [](PyObject *const *a) -> PyObject * {
        const bool kv8 = a[2] != Py_None;
        const char *kname = kv8 ? "k8" : "k_prefix";
        const at::Tensor &q = four("q", a[0], "[B,Hq,S,D]"), &k = four(kname, a[1], "[B,Hkv,P,D]");
        const int dev = device_of("q", q, kBf16);
        const int64_t B = q.size(0), Hq = q.size(1), S = q.size(2), D = q.size(3), H = k.size(1), P = k.size(2);
        need("q", q, kBf16, q.sizes(), dev);
        need(kname, k, kv8 ? kF8 : kBf16, {B, H, P, D}, dev);
        void *ks = nullptr;
        int64_t block = 0;
        if (kv8) {
            block = integer("block", a[3]);
            check_block(block, "block");
            ks = need("k_scale", tensor("k_scale", a[2]), kF32, {B, H, (P + block - 1) / block}, dev).data_ptr();
        }
        const at::Tensor &lse = need("lse", tensor("lse", a[4]), kF32, {B, Hq, S}, dev);
        void *vl = optional("prefix_valid_len", a[5], kI32, {B}, dev);
        void *mask = optional("prefix_mask", a[6], kU8, {B, P}, dev);
        void *before = optional("mass_in", a[7], kF32, {B, H, P}, dev);
        if (a[8] != Py_None) need("mass", tensor("mass", a[8]), kF32, {B, H, P}, dev);
        const On on(dev);
        at::Tensor m = a[8] != Py_None ? THPVariable_Unpack(a[8]) : at::empty({B, H, P}, q.options().dtype(kF32));
        const int iB = static_cast<int>(B), iq = static_cast<int>(Hq), ik = static_cast<int>(H), iP = static_cast<int>(P),
                  iS = static_cast<int>(S), iD = static_cast<int>(D);
        const float *l = static_cast<const float *>(lse.data_ptr()), *in = static_cast<const float *>(before);
        float *out = static_cast<float *>(m.data_ptr());
        check(kv8 ? g_mass_kv8(q.data_ptr(), k.data_ptr(), static_cast<const float *>(ks), static_cast<int>(block),
                               static_cast<const int32_t *>(vl), static_cast<const uint8_t *>(mask), l, in, out, iB, iq,
                               ik, iP, iS, iD, on.stream)
                  : g_mass(q.data_ptr(), k.data_ptr(), static_cast<const int32_t *>(vl),
                           static_cast<const uint8_t *>(mask), l, in, out, iB, iq, ik, iP, iS, iD, on.stream),
              kv8 ? "dm05_prefix_attn_mass_kv8" : "dm05_prefix_attn_mass");
        return a[8] != Py_None ? same(a[8]) : wrap(m);
    });
}

// The eviction's tensors that both forms share.
struct Evicted {
    at::Tensor mass, pos, valid;
};

Evicted evict_outputs(PyObject *mass, PyObject *pos, PyObject *valid, int64_t B, int64_t H, int64_t bucket, int dev,
                      const at::Device &device)
{
    const int64_t shape[3] = {B, H, bucket};
    Evicted e;
    if (mass != Py_None) need("mass_out", tensor("mass_out", mass), kF32, shape, dev);
    if (pos != Py_None) need("positions", tensor("positions", pos), kI32, shape, dev);
    if (valid != Py_None) need("valid_len", tensor("valid_len", valid), kI32, {B}, dev);
    const auto opt = at::TensorOptions().device(device);
    e.mass = mass != Py_None ? THPVariable_Unpack(mass) : at::empty(shape, opt.dtype(kF32));
    e.pos = pos != Py_None ? THPVariable_Unpack(pos) : at::empty(shape, opt.dtype(kI32));
    e.valid = valid != Py_None ? THPVariable_Unpack(valid) : at::empty({B}, opt.dtype(kI32));
    return e;
}

// prefix_evict(k, v, mass, n_keep, n_first, n_last, valid_len_in, mask, bucket or None, k_out, v_out, mass_out,
//              positions, valid_len) -> (k, v, mass, positions, valid_len)
PyObject *evict(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded(args, n, 14, [](PyObject *const *a) -> PyObject * {
        const at::Tensor &k = four("k", a[0], "[B,Hkv,P,D]");
        const int dev = device_of("k", k, kBf16);
        const int64_t B = k.size(0), H = k.size(1), P = k.size(2), D = k.size(3);
        const int64_t keep = integer("n_keep", a[3]), first = integer("n_first", a[4]), last = integer("n_last", a[5]);
        if ((a[9] == Py_None) != (a[10] == Py_None)) throw Bad{"k_out and v_out must be given together"};
        int64_t bucket = keep;
        if (a[8] != Py_None)
            bucket = integer("bucket", a[8]);
        else if (a[9] != Py_None)
            bucket = four("k_out", a[9], "[B,Hkv,bucket,D]").size(2);
        need("k", k, kBf16, k.sizes(), dev);
        const at::Tensor &v = need("v", tensor("v", a[1]), kBf16, k.sizes(), dev);
        const at::Tensor &m = need("mass", tensor("mass", a[2]), kF32, {B, H, P}, dev);
        void *vl = optional("prefix_valid_len", a[6], kI32, {B}, dev);
        void *mask = optional("prefix_mask", a[7], kU8, {B, P}, dev);
        const int64_t rows = std::max<int64_t>(bucket, 0);
        if (a[9] != Py_None) {
            need("k_out", tensor("k_out", a[9]), kBf16, {B, H, rows, D}, dev);
            need("v_out", tensor("v_out", a[10]), kBf16, {B, H, rows, D}, dev);
        }
        const On on(dev);
        at::Tensor ko = a[9] != Py_None ? THPVariable_Unpack(a[9]) : at::zeros({B, H, rows, D}, k.options());
        at::Tensor vo = a[10] != Py_None ? THPVariable_Unpack(a[10]) : at::zeros({B, H, rows, D}, k.options());
        const Evicted e = evict_outputs(a[11], a[12], a[13], B, H, rows, dev, k.device());
        check(g_evict(k.data_ptr(), v.data_ptr(), static_cast<const float *>(m.data_ptr()),
                      static_cast<const int32_t *>(vl), static_cast<const uint8_t *>(mask), ko.data_ptr(), vo.data_ptr(),
                      static_cast<float *>(e.mass.data_ptr()), static_cast<int32_t *>(e.pos.data_ptr()),
                      static_cast<int32_t *>(e.valid.data_ptr()), static_cast<int>(B), static_cast<int>(H),
                      static_cast<int>(P), static_cast<int>(bucket), static_cast<int>(D), static_cast<int>(keep),
                      static_cast<int>(first), static_cast<int>(last), on.stream),
              "dm05_prefix_evict");
        return tuple_of({wrap(ko), wrap(vo), wrap(e.mass), wrap(e.pos), wrap(e.valid)});
    });
}

// prefix_evict_kv8(cache, mass, n_keep, n_first, n_last, valid_len_in, mask, bucket or None, out, mass_out, positions,
//                  valid_len) -> ((k, v, k_scale, v_scale) or None when out was given, mass, positions, valid_len)
PyObject *evict_kv8(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded(args, n, 12, [](PyObject *const *a) -> PyObject * {
        const Cache c = cache_of("cache", a[0]);
        const int dev = device_of("cache.k", *c.k, kF8);
        check_cache("cache", c, dev);
        const int64_t keep = integer("n_keep", a[2]), first = integer("n_first", a[3]), last = integer("n_last", a[4]);
        Cache o{};
        int64_t bucket = keep;
        if (a[8] != Py_None) o = cache_of("out", a[8]);
        if (a[7] != Py_None)
            bucket = integer("bucket", a[7]);
        else if (a[8] != Py_None)
            bucket = o.P;
        const int64_t rows = std::max<int64_t>(bucket, 0);
        if (a[8] != Py_None) {
            if (o.block != c.block || o.B != c.B || o.H != c.H || o.P != rows || o.D != c.D)
                throw Bad{"out must be a cache of " + std::to_string(rows) + " rows with cache's other sizes and block"};
            check_cache("out", o, dev);
        }
        const at::Tensor &m = need("mass", tensor("mass", a[1]), kF32, {c.B, c.H, c.P}, dev);
        void *vl = optional("prefix_valid_len", a[5], kI32, {c.B}, dev);
        void *mask = optional("prefix_mask", a[6], kU8, {c.B, c.P}, dev);
        const On on(dev);
        std::vector<at::Tensor> f;
        if (a[8] == Py_None) {
            f = fresh_cache(c.B, c.H, rows, c.D, c.block, c.k->device());
            o.k = &f[0];
            o.v = &f[1];
            o.ks = &f[2];
            o.vs = &f[3];
        }
        const Evicted e = evict_outputs(a[9], a[10], a[11], c.B, c.H, rows, dev, c.k->device());
        check(g_evict_kv8(c.k->data_ptr(), c.v->data_ptr(), static_cast<const float *>(c.ks->data_ptr()),
                          static_cast<const float *>(c.vs->data_ptr()), static_cast<int>(c.block),
                          static_cast<const float *>(m.data_ptr()), static_cast<const int32_t *>(vl),
                          static_cast<const uint8_t *>(mask), o.k->data_ptr(), o.v->data_ptr(),
                          static_cast<float *>(o.ks->data_ptr()), static_cast<float *>(o.vs->data_ptr()),
                          static_cast<float *>(e.mass.data_ptr()), static_cast<int32_t *>(e.pos.data_ptr()),
                          static_cast<int32_t *>(e.valid.data_ptr()), static_cast<int>(c.B), static_cast<int>(c.H),
                          static_cast<int>(c.P), static_cast<int>(bucket), static_cast<int>(c.D), static_cast<int>(keep),
                          static_cast<int>(first), static_cast<int>(last), on.stream),
              "dm05_prefix_evict_kv8");
        return tuple_of({a[8] == Py_None ? tuple_of({wrap(f[0]), wrap(f[1]), wrap(f[2]), wrap(f[3])}) : same(Py_None),
                         wrap(e.mass), wrap(e.pos), wrap(e.valid)});
    });
}

// bind(Dm05Error, addresses of the seven entry points)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 8) {
        PyErr_SetString(PyExc_ValueError, "bind takes the error class and seven addresses");
        return nullptr;
    }
    void *p[7];
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    g_quantize = reinterpret_cast<decltype(g_quantize)>(p[0]);
    g_attn = reinterpret_cast<decltype(g_attn)>(p[1]);
    g_plan = reinterpret_cast<decltype(g_plan)>(p[2]);
    g_mass = reinterpret_cast<decltype(g_mass)>(p[3]);
    g_mass_kv8 = reinterpret_cast<decltype(g_mass_kv8)>(p[4]);
    g_evict = reinterpret_cast<decltype(g_evict)>(p[5]);
    g_evict_kv8 = reinterpret_cast<decltype(g_evict_kv8)>(p[6]);
    Py_XDECREF(g_error);
    g_error = same(a[0]);
    Py_RETURN_NONE;
}

#define DM05_METHOD(name, fn) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&fn)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {DM05_METHOD("bind", bind),
                           DM05_METHOD("kv8_quantize", quantize),
                           DM05_METHOD("suffix_attn_kv8", attn),
                           DM05_METHOD("prefix_attn_mass", mass),
                           DM05_METHOD("prefix_evict", evict),
                           DM05_METHOD("prefix_evict_kv8", evict_kv8),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_front", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_front(void) { return PyModule_Create(&g_module); }
