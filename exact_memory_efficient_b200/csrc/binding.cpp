// binding.cpp -- CPython binding of the rotary and paged-cache entry points
// (include/mea_attn.h) for torch tensors: checks of shapes, types, strides and
// devices, the outputs and scratch of the allocating helpers, the stream, and the
// call of the C entry point.  Python keeps the names and documentation
// (exact_memory_efficient_b200/__init__.py).
//
// These calls are made once per layer and token in a serving loop, and a
// decode-sized kernel takes 3 to 20 us.  With the checks in Python and the call
// through ctypes the append of 16 tokens took 18 us of host time a call and the
// attention of one sequence 24; from here 6.8 and 8.8.
#include <Python.h>

#include <cmath>
#include <string>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mea_attn.h"

namespace {

PyObject* g_error = nullptr;   // MeaError

struct Refused {
    int status;
    std::string where;
};

[[noreturn]] void bad(const char* where, const std::string& what) {
    throw Refused{MEA_ERR_INVALID_ARG, std::string(where) + ": " + what};
}

void check(mea_status_t st, const char* where) {
    if (st != MEA_OK) throw Refused{(int)st, where};
}

PyObject* raise_refused(const Refused& r) {
    PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.where.c_str());
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

// Optional tensors are undefined tensors.
at::Tensor tensor(const char* where, const char* name, PyObject* o, bool optional = false) {
    if (optional && o == Py_None) return at::Tensor();
    if (!THPVariable_Check(o)) bad(where, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int integer(const char* where, const char* name, PyObject* o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        bad(where, std::string(name) + " must be a whole number");
    }
    if (x < -2147483647LL || x > 2147483647LL) bad(where, std::string(name) + " out of range");
    return (int)x;
}

float number(const char* where, const char* name, PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        bad(where, std::string(name) + " must be a number");
    }
    return (float)x;
}

bool truth(const char* where, const char* name, PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) {
        PyErr_Clear();
        bad(where, std::string(name) + " must be true or false");
    }
    return x != 0;
}

mea_dtype_t dtype_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kFloat) return MEA_DTYPE_F32;
    if (t.scalar_type() == at::kBFloat16) return MEA_DTYPE_BF16;
    throw Refused{MEA_ERR_UNSUPPORTED, std::string("dtype ") + c10::toString(t.scalar_type())};
}

// The device of the call: that of its first tensor, made current for the call.
struct Device {
    const char* where;
    c10::Device dev;
    c10::cuda::OptionalCUDAGuard guard;

    Device(const char* where_, const at::Tensor& first) : where(where_), dev(first.device()) {
        if (!first.is_cuda()) bad(where, "CUDA tensors");
        guard.set_device(dev);
    }
    // a tensor (if there is one) on the device, of a type, dense
    void dense(const char* name, const at::Tensor& t, at::ScalarType type) const {
        if (!t.defined()) return;
        if (t.device() != dev) bad(where, std::string(name) + " is not on the device of the first tensor");
        if (t.scalar_type() != type) bad(where, std::string(name) + " must be " + c10::toString(type));
        if (!t.is_contiguous()) bad(where, std::string(name) + " must be contiguous");
    }
    void here(const char* name, const at::Tensor& t) const {
        if (t.defined() && t.device() != dev) bad(where, std::string(name) + " is not on the device of the first tensor");
    }
};

// The stream of a call: None (the device's current one), a torch.cuda.Stream, or a handle.
struct Stream {
    void* handle;
    bool given;
    c10::Device dev;

    Stream(const char* where, PyObject* o, c10::Device d) : handle(nullptr), given(o != Py_None), dev(d) {
        if (!given) {
            handle = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
            return;
        }
        PyObject* h = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        if (h != nullptr) handle = PyLong_AsVoidPtr(h);
        Py_XDECREF(h);
        long index = dev.index();
        if (!PyErr_Occurred() && !PyLong_Check(o)) {
            PyObject* at = PyObject_GetAttrString(o, "device_index");
            if (at != nullptr) index = PyLong_AsLong(at);
            else PyErr_Clear();   // an object of another library with a handle only
            Py_XDECREF(at);
        }
        if (PyErr_Occurred()) {
            PyErr_Clear();
            bad(where, "stream must be a CUDA stream or its handle");
        }
        if (index != dev.index()) bad(where, "stream is not on the device of the first tensor");
    }
    // Outputs and scratch belong to the call's stream, so that the allocator does
    // not hand their memory on while the call may still run.
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        const auto options = at::TensorOptions().dtype(type).device(dev);
        if (!given) return at::empty(shape, options);
        const c10::cuda::CUDAStreamGuard g(
            c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), dev.index()));
        return at::empty(shape, options);
    }
};

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <typename T>
T* as(const at::Tensor& t) { return static_cast<T*>(ptr(t)); }

// Packed rows [T, heads, D]: heads and dims dense, any token stride (returned).
long long packed(const char* where, const char* name, const at::Tensor& t, at::ScalarType type, long long T,
                 long long heads, long long D) {
    if (t.dim() != 3 || t.scalar_type() != type || (T >= 0 && t.size(0) != T) || (heads >= 0 && t.size(1) != heads) ||
        t.size(2) != D)
        bad(where, std::string(name) + " shape/dtype mismatch");
    if ((t.size(2) > 1 && t.stride(2) != 1) || (t.size(1) > 1 && t.stride(1) != t.size(2)))
        bad(where, std::string(name) + ": heads and head dims must be dense");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

int as_int(const char* where, long long x) {
    if (x > 2147483647LL) bad(where, "size out of range");
    return (int)x;
}

// Sizes of a cache [pages, H_kv, page_size, D]; v alike, weights [pages, H_kv, page_size].
struct Cache {
    int pages, Hkv, page, D;
    Cache(const char* where, const at::Tensor& k, const at::Tensor& v, const at::Tensor& w) {
        if (k.dim() != 4) bad(where, "k_cache must be [pages, H_kv, page_size, D]");
        if (v.defined() && v.sizes() != k.sizes()) bad(where, "v_cache must be shaped like k_cache");
        if (w.defined() && w.sizes() != k.sizes().slice(0, 3)) bad(where, "weights must be [pages, H_kv, page_size]");
        pages = as_int(where, k.size(0));
        Hkv = as_int(where, k.size(1));
        page = as_int(where, k.size(2));
        D = as_int(where, k.size(3));
    }
};

struct Batch {
    int B, max_pages;
    Batch(const char* where, const at::Tensor& kv_len, const at::Tensor& table, const at::Tensor& cu_q) {
        if (kv_len.dim() != 1 || table.dim() != 2 || table.size(0) != kv_len.size(0))
            bad(where, "kv_len must be [B] and page_table [B, max_pages]");
        if (cu_q.defined() && (cu_q.dim() != 1 || cu_q.size(0) != kv_len.size(0) + 1)) bad(where, "cu_q must be [B + 1]");
        B = as_int(where, table.size(0));
        max_pages = as_int(where, table.size(1));
    }
};

size_t workspace_bytes(const Device& d, const at::Tensor& ws) {
    if (!ws.defined()) return 0;
    if (ws.device() != d.dev || !ws.is_contiguous()) bad(d.where, "workspace must be a contiguous tensor on the device");
    return ws.nbytes();
}

// The C call without the interpreter lock: a launch may wait for room in the queue.
template <typename F>
void call(const char* where, F&& f) {
    mea_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    check(st, where);
}

PyObject* none_or(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject* x = none_or(a);
    PyObject* y = none_or(b);
    PyObject* t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

// (x, y or None: allocated, positions, freq, layout, mscale, inverse, stream) -> y
PyObject* rope(PyObject* const* p) {
    const char* w = "mea_rope";
    const at::Tensor x = tensor(w, "x", p[0]);
    at::Tensor y = tensor(w, "y", p[1], true);
    const at::Tensor positions = tensor(w, "positions", p[2]), freq = tensor(w, "freq", p[3]);
    if (x.dim() != 4) bad(w, "x must be [B, H, N, D]");
    if (y.defined() && (y.sizes() != x.sizes() || y.scalar_type() != x.scalar_type())) bad(w, "y shape/dtype mismatch");
    if (freq.dim() != 1) bad(w, "freq must be [rot_dim / 2]");
    const long long B = x.size(0), N = x.size(2);
    const bool per_batch = positions.dim() == 2;
    if (!(positions.dim() == 1 && positions.size(0) == N) &&
        !(per_batch && positions.size(0) == B && positions.size(1) == N))
        bad(w, "positions must be [N] or [B, N]");
    const mea_dtype_t dt = dtype_of(x);
    const int layout = integer(w, "layout", p[4]), inverse = truth(w, "inverse", p[6]);
    const float mscale = number(w, "mscale", p[5]);
    const Device d(w, x);
    d.dense("x", x, x.scalar_type());
    d.dense("y", y, x.scalar_type());
    d.dense("positions", positions, at::kInt);
    d.dense("freq", freq, at::kDouble);
    const Stream s(w, p[7], d.dev);
    if (!y.defined()) y = s.empty(x.sizes(), x.scalar_type());
    const int b = as_int(w, B), h = as_int(w, x.size(1)), n = as_int(w, N), D = as_int(w, x.size(3)),
              rot = as_int(w, 2 * freq.size(0));
    call(w, [&] {
        return mea_rope(ptr(x), ptr(y), as<int>(positions), as<double>(freq), b, h, n, D, rot, per_batch,
                        (mea_rope_layout_t)layout, mscale, inverse, dt, s.handle);
    });
    return none_or(y);
}

// (q, q_out, allocate q_out, k, v, k_cache, v_cache, weights, cu_q, kv_len, page_table, positions, freq, layout,
//  mscale, stream) -> q_out or None
PyObject* append(PyObject* const* p) {
    const char* w = "mea_paged_append";
    const at::Tensor q = tensor(w, "q", p[0], true);
    at::Tensor q_out = tensor(w, "q_out", p[1], true);
    const bool make = p[2] == Py_True;
    const at::Tensor k = tensor(w, "k", p[3]), v = tensor(w, "v", p[4]), kc = tensor(w, "k_cache", p[5]),
                     vc = tensor(w, "v_cache", p[6]), wt = tensor(w, "weights", p[7], true),
                     cu = tensor(w, "cu_q", p[8]), kv = tensor(w, "kv_len", p[9]), tab = tensor(w, "page_table", p[10]),
                     pos = tensor(w, "positions", p[11], true), freq = tensor(w, "freq", p[12], true);
    const Cache c(w, kc, vc, wt);
    const Batch b(w, kv, tab, cu);
    const mea_dtype_t dt = dtype_of(kc);
    const at::ScalarType type = kc.scalar_type();
    const long long ks = packed(w, "k", k, type, -1, c.Hkv, c.D);
    const int T = as_int(w, k.size(0));
    const long long vs = packed(w, "v", v, type, T, c.Hkv, c.D);
    if (!make && q.defined() != q_out.defined()) bad(w, "q and q_out go together");
    long long qs = 0;
    int H = 0;
    if (q.defined()) {
        qs = packed(w, "q", q, type, T, -1, c.D);
        H = as_int(w, q.size(1));
        if (!make && q_out.sizes() != q.sizes()) bad(w, "q_out must be shaped like q");
    }
    if (pos.defined() && (pos.dim() != 1 || pos.size(0) != T)) bad(w, "positions must be [T]");
    if (freq.defined() && freq.dim() != 1) bad(w, "freq must be [rot_dim / 2]");
    const Device d(w, k);
    d.here("v", v);
    d.here("q", q);
    d.dense("k_cache", kc, type);
    d.dense("v_cache", vc, type);
    d.dense("weights", wt, at::kFloat);
    d.dense("cu_q", cu, at::kInt);
    d.dense("kv_len", kv, at::kInt);
    d.dense("page_table", tab, at::kInt);
    d.dense("positions", pos, at::kInt);
    d.dense("freq", freq, at::kDouble);
    d.dense("q_out", q_out, type);
    const int layout = integer(w, "layout", p[13]);
    const float mscale = number(w, "mscale", p[14]);
    const Stream s(w, p[15], d.dev);
    if (make && q.defined()) q_out = s.empty(q.sizes(), type);
    const int rot = freq.defined() ? as_int(w, 2 * freq.size(0)) : 0;
    call(w, [&] {
        return mea_paged_append(ptr(q), ptr(q_out), ptr(k), ptr(v), ptr(kc), ptr(vc), as<float>(wt), as<int>(cu),
                                as<int>(kv), as<int>(tab), as<int>(pos), as<double>(freq), T, b.B, H, c.Hkv, c.D, qs,
                                ks, vs, c.pages, c.page, b.max_pages, rot, (mea_rope_layout_t)layout, mscale, dt,
                                s.handle);
    });
    return none_or(q_out);
}

float scale_of(const char* w, PyObject* o, int D) {
    return o == Py_None ? (float)(1.0 / std::sqrt((double)D)) : number(w, "scale", o);
}

// (q, k_cache, v_cache, o, lse, allocate, cu_q, kv_len, page_table, max_q, max_kv, scale, workspace, stream) -> (o, lse)
PyObject* attend(PyObject* const* p) {
    const char* w = "mea_attn_paged";
    const at::Tensor q = tensor(w, "q", p[0]), kc = tensor(w, "k_cache", p[1]), vc = tensor(w, "v_cache", p[2]);
    at::Tensor o = tensor(w, "o", p[3], true), lse = tensor(w, "lse", p[4], true), ws = tensor(w, "workspace", p[12], true);
    const bool make = p[5] == Py_True;
    const at::Tensor cu = tensor(w, "cu_q", p[6]), kv = tensor(w, "kv_len", p[7]), tab = tensor(w, "page_table", p[8]);
    const int max_q = integer(w, "max_q", p[9]), max_kv = integer(w, "max_kv", p[10]);
    const Cache c(w, kc, vc, at::Tensor());
    const Batch b(w, kv, tab, cu);
    const mea_dtype_t dt = dtype_of(kc);
    const at::ScalarType type = kc.scalar_type();
    const long long qs = packed(w, "q", q, type, -1, -1, c.D);
    const int T = as_int(w, q.size(0)), H = as_int(w, q.size(1));
    if (!make) {
        if (!o.defined() || !lse.defined() || o.sizes() != q.sizes() || lse.dim() != 2 || lse.size(0) != T || lse.size(1) != H)
            bad(w, "o must be shaped like q, lse [T, H]");
    }
    const Device d(w, q);
    d.dense("k_cache", kc, type);
    d.dense("v_cache", vc, type);
    d.dense("o", o, type);
    d.dense("lse", lse, at::kFloat);
    d.dense("cu_q", cu, at::kInt);
    d.dense("kv_len", kv, at::kInt);
    d.dense("page_table", tab, at::kInt);
    const float scale = scale_of(w, p[11], c.D);
    const Stream s(w, p[13], d.dev);
    if (make) {
        size_t n = 0;
        check(mea_attn_paged_workspace_size(T, b.B, H, c.Hkv, c.D, max_q, max_kv, dt, &n), w);
        o = s.empty(q.sizes(), type);
        lse = s.empty({T, H}, at::kFloat);
        if (n > 0) ws = s.empty({(int64_t)n}, at::kByte);
    }
    const size_t bytes = workspace_bytes(d, ws);
    call(w, [&] {
        return mea_attn_paged(ptr(q), ptr(kc), ptr(vc), ptr(o), as<float>(lse), as<int>(cu), as<int>(kv), as<int>(tab),
                              T, b.B, H, c.Hkv, c.D, qs, c.pages, c.page, b.max_pages, max_q, max_kv, scale, dt,
                              ptr(ws), bytes, s.handle);
    });
    return pair(o, lse);
}

// (q, lse, k_cache, weights, allocate the workspace, cu_q, kv_len, page_table, max_q, max_kv, scale, workspace, stream)
PyObject* weigh(PyObject* const* p) {
    const char* w = "mea_attn_paged_weights";
    const at::Tensor q = tensor(w, "q", p[0]), lse = tensor(w, "lse", p[1]), kc = tensor(w, "k_cache", p[2]),
                     wt = tensor(w, "weights", p[3]);
    const bool make = p[4] == Py_True;
    const at::Tensor cu = tensor(w, "cu_q", p[5]), kv = tensor(w, "kv_len", p[6]), tab = tensor(w, "page_table", p[7]);
    const int max_q = integer(w, "max_q", p[8]), max_kv = integer(w, "max_kv", p[9]);
    at::Tensor ws = tensor(w, "workspace", p[11], true);
    const Cache c(w, kc, at::Tensor(), wt);
    const Batch b(w, kv, tab, cu);
    const mea_dtype_t dt = dtype_of(kc);
    const long long qs = packed(w, "q", q, kc.scalar_type(), -1, -1, c.D);
    const int T = as_int(w, q.size(0)), H = as_int(w, q.size(1));
    if (lse.dim() != 2 || lse.size(0) != T || lse.size(1) != H) bad(w, "lse must be [T, H]");
    const Device d(w, q);
    d.dense("k_cache", kc, kc.scalar_type());
    d.dense("weights", wt, at::kFloat);
    d.dense("lse", lse, at::kFloat);
    d.dense("cu_q", cu, at::kInt);
    d.dense("kv_len", kv, at::kInt);
    d.dense("page_table", tab, at::kInt);
    const float scale = scale_of(w, p[10], c.D);
    const Stream s(w, p[12], d.dev);
    if (make) {
        size_t n = 0;
        check(mea_attn_paged_weights_workspace_size(T, b.B, H, c.Hkv, c.D, max_q, max_kv, dt, &n), w);
        if (n > 0) ws = s.empty({(int64_t)n}, at::kByte);
    }
    const size_t bytes = workspace_bytes(d, ws);
    call(w, [&] {
        return mea_attn_paged_weights(ptr(q), as<float>(lse), ptr(kc), as<float>(wt), as<int>(cu), as<int>(kv),
                                      as<int>(tab), T, b.B, H, c.Hkv, c.D, qs, c.pages, c.page, b.max_pages, max_q,
                                      max_kv, scale, dt, ptr(ws), bytes, s.handle);
    });
    Py_RETURN_NONE;
}

// (k_cache, v_cache, weights, page_table, kv_len, dst_table, kv_len_out, keep_idx, n_keep or None: no allocation,
//  n_recent, stream) -> (keep_idx, kv_len_out)
PyObject* evict(PyObject* const* p) {
    const char* w = "mea_paged_evict";
    const at::Tensor kc = tensor(w, "k_cache", p[0]), vc = tensor(w, "v_cache", p[1]), wt = tensor(w, "weights", p[2]),
                     tab = tensor(w, "page_table", p[3]), kv = tensor(w, "kv_len", p[4]), dst = tensor(w, "dst_table", p[5]);
    at::Tensor out = tensor(w, "kv_len_out", p[6], true), idx = tensor(w, "keep_idx", p[7], true);
    const bool make = p[8] != Py_None;
    const Cache c(w, kc, vc, wt);
    const Batch b(w, kv, tab, at::Tensor());
    const mea_dtype_t dt = dtype_of(kc);
    if (dst.dim() != 2 || dst.size(0) != b.B) bad(w, "dst_table must be [B, dst_max_pages]");
    int keep;
    if (make) {
        keep = integer(w, "n_keep", p[8]);
        if (keep < 1) bad(w, "n_keep below 1");
    } else {
        if (!idx.defined() || idx.dim() != 3 || idx.size(0) != b.B || idx.size(1) != c.Hkv)
            bad(w, "keep_idx must be [B, H_kv, n_keep]");
        if (out.defined() && out.sizes() != kv.sizes()) bad(w, "kv_len_out must be [B]");
        keep = as_int(w, idx.size(2));
    }
    const int recent = integer(w, "n_recent", p[9]);
    const Device d(w, kc);
    d.dense("k_cache", kc, kc.scalar_type());
    d.dense("v_cache", vc, kc.scalar_type());
    d.dense("weights", wt, at::kFloat);
    d.dense("page_table", tab, at::kInt);
    d.dense("kv_len", kv, at::kInt);
    d.dense("dst_table", dst, at::kInt);
    d.dense("keep_idx", idx, at::kInt);
    d.dense("kv_len_out", out, at::kInt);
    const Stream s(w, p[10], d.dev);
    if (make) {
        idx = s.empty({b.B, c.Hkv, keep}, at::kInt);
        out = s.empty({b.B}, at::kInt);
    }
    const int dst_pages = as_int(w, dst.size(1));
    call(w, [&] {
        return mea_paged_evict(ptr(kc), ptr(vc), as<float>(wt), as<int>(tab), as<int>(kv), as<int>(dst), as<int>(out),
                               as<int>(idx), b.B, c.Hkv, c.D, c.pages, c.page, b.max_pages, dst_pages, keep, recent, dt,
                               s.handle);
    });
    return pair(idx, out);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& r) {
        return raise_refused(r);
    }
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_XDECREF(g_error);
    g_error = Py_NewRef(cls);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyCFunction method() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>));
}

PyMethodDef g_methods[] = {
    {"set_error", set_error, METH_O, "the exception class of refused calls"},
    {"rope", method<rope, 8>(), METH_FASTCALL, nullptr},
    {"append", method<append, 16>(), METH_FASTCALL, nullptr},
    {"attend", method<attend, 14>(), METH_FASTCALL, nullptr},
    {"weigh", method<weigh, 13>(), METH_FASTCALL, nullptr},
    {"evict", method<evict, 11>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&g_module);
    // the Python and torch that this was compiled against (build.py looks for the text in the file)
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", MEA_BINDING_FOR) != 0) Py_CLEAR(m);
    return m;
}
