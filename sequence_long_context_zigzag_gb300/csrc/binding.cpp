// binding.cpp -- the Python binding of the paged K/V cache calls: argument checks, output allocation and the
// current stream in C++, then the C ABI (include/usp.h).
//
// Serving calls these once per layer and token, where a short call's GPU work is about 15 microseconds; in
// Python the same checks and allocations took 18 to 20 (page plan, attention of a few short requests, on the
// GPU's Grace host), so they bounded it. The functions take their arguments by position; the package's
// Python functions carry the names, defaults and documentation. They return the call's tensors, or the
// ABI's status where that is not USP_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "usp.h"

namespace {

using at::Tensor;

decltype(&usp_page_plan) g_plan;
decltype(&usp_cache_append) g_append;
decltype(&usp_paged_attn) g_attn;
decltype(&usp_paged_attn_workspace_size) g_attn_workspace;

struct Refused {
    PyObject *type;
    std::string what;
};
[[noreturn]] void refuse(std::string what, PyObject *type = PyExc_ValueError) { throw Refused{type, std::move(what)}; }
void need(bool ok, const char *what) {
    if (!ok) refuse(what);
}
struct PythonError {};  // a Python error is set

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor", PyExc_TypeError);
    return THPVariable_Unpack(o);
}
int64_t integer(PyObject *o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw PythonError{};
    return x;
}
int32_t integer32(PyObject *o, const char *name) {
    const int64_t x = integer(o);
    if (x < INT32_MIN || x > INT32_MAX) refuse(std::string(name) + " is out of range");
    return (int32_t)x;
}

// the device of a call's tensors
int device_of(std::initializer_list<const Tensor *> ts) {
    const at::Device d = (*ts.begin())->device();
    if (!d.is_cuda()) refuse("expected CUDA tensors");
    for (const Tensor *t : ts)
        if (t->device() != d) refuse("expected tensors on one device, got " + d.str() + " and " + t->device().str());
    return d.index();
}
void same_device(int index, const Tensor &t) {
    if (!t.is_cuda() || t.get_device() != index)
        refuse("expected tensors on one device, got cuda:" + std::to_string(index) + " and " + t.device().str());
}
void i32(const char *name, const Tensor &t, int64_t n = -1) {
    if (t.scalar_type() != at::kInt || t.dim() != 1 || !t.is_contiguous())
        refuse(std::string(name) + " must be a contiguous 1-D int32 tensor");
    if (n >= 0 && t.numel() != n)
        refuse(std::string(name) + " must have " + std::to_string(n) + " entries, got " + std::to_string(t.numel()));
}
// the stride of the first axis in elements, 0 where the tensor is contiguous; what an entry of the first
// axis holds must be contiguous
int64_t dense_rows(const char *name, const Tensor &t) {
    if (t.is_contiguous()) return 0;
    int64_t inner = 1;
    bool ok = t.dim() >= 2;
    for (int64_t d = t.dim() - 1; ok && d > 0; --d) {
        ok = t.size(d) == 1 || t.stride(d) == inner;
        inner *= t.size(d);
    }
    if (!ok || t.stride(0) < inner) refuse(std::string(name) + ": only the first axis may be strided");
    return t.stride(0);
}
int32_t dtype_code(const Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return USP_BF16;
    if (t.scalar_type() == at::kFloat) return USP_F32;
    refuse(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " (bf16 or fp32)", PyExc_TypeError);
}
int32_t size32(const Tensor &t, int64_t d) { return (int32_t)std::min<int64_t>(t.size(d), INT32_MAX); }
usp_cache_dims cache_dims(const Tensor &k, const Tensor &v) {
    if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
        refuse("k_cache and v_cache must be (num_pages, hkv, page_size, hd), of one shape and dtype");
    usp_cache_dims d{};
    d.num_pages = k.size(0);
    d.k_page_stride = dense_rows("k_cache", k);
    d.v_page_stride = dense_rows("v_cache", v);
    d.hkv = size32(k, 1);
    d.page_size = size32(k, 2);
    d.hd = size32(k, 3);
    d.dtype = dtype_code(k);
    return d;
}
int64_t block_table(const Tensor &t, int64_t nreq) {  // its row stride
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != nreq)
        refuse("block_table must be an int32 tensor of " + std::to_string(nreq) + " rows");
    const int64_t s = dense_rows("block_table", t);
    return s ? s : t.size(1);
}
const int32_t *ints(const Tensor &t) { return static_cast<const int32_t *>(t.const_data_ptr()); }
int32_t *mutable_ints(const Tensor &t) { return static_cast<int32_t *>(t.mutable_data_ptr()); }
usp_stream_t stream_of(int index) {
    return reinterpret_cast<usp_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream());
}

// (without the dispatcher: a page plan allocates four of these; 8.0 -> 6.2 us a call)
Tensor empty(at::IntArrayRef sizes, at::ScalarType type, int index) {
    return Tensor(at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, (c10::DeviceIndex)index), std::nullopt));
}

// A call's output: the caller's tensor, returned as it came, or a new one.
struct Output {
    PyObject *given = nullptr;
    Tensor t;
    PyObject *result() {
        if (!given) return THPVariable_Wrap(std::move(t));
        Py_INCREF(given);
        return given;
    }
};
template <typename Check>
Output output(PyObject *o, const char *name, int index, at::IntArrayRef sizes, at::ScalarType type, Check check) {
    Output r;
    if (o == Py_None) {
        r.t = empty(sizes, type, index);
        return r;
    }
    r.given = o;
    r.t = tensor(o, name);
    check(r.t);
    same_device(index, r.t);
    return r;
}
PyObject *tuple(std::initializer_list<Output *> outs) {
    PyObject *r = PyTuple_New((Py_ssize_t)outs.size());
    if (!r) throw PythonError{};
    Py_ssize_t i = 0;
    for (Output *o : outs) {
        PyObject *x = o->result();
        if (!x) {
            Py_DECREF(r);
            throw PythonError{};
        }
        PyTuple_SET_ITEM(r, i++, x);
    }
    return r;
}

// ctx_lens, new_lens, free_pages, free_head, block_table, page_size, num_pages, max_tokens, slot_map, cu_new,
// kv_lens, counts
PyObject *page_plan(PyObject *const *a) {
    const Tensor &ctx = tensor(a[0], "ctx_lens"), &fresh = tensor(a[1], "new_lens"), &pages = tensor(a[2], "free_pages"),
                 &head = tensor(a[3], "free_head"), &table = tensor(a[4], "block_table");
    usp_plan_dims d{};
    const int64_t nreq = ctx.numel();
    i32("ctx_lens", ctx, nreq);
    i32("new_lens", fresh, nreq);
    i32("free_pages", pages);
    i32("free_head", head, 1);
    d.table_stride = block_table(table, nreq);
    need(nreq <= INT32_MAX, "too many requests");
    d.nreq = (int32_t)nreq;
    d.page_size = integer32(a[5], "page_size");
    d.num_pages = integer(a[6]);
    d.max_tokens = integer(a[7]);
    need(d.max_tokens >= 0, "max_tokens must not be negative");
    d.free_count = pages.numel();
    d.max_pages = size32(table, 1);
    const int index = device_of({&ctx, &fresh, &pages, &head, &table});
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    auto out = [&](PyObject *o, const char *name, int64_t n) {
        return output(o, name, index, {n}, at::kInt, [&](const Tensor &t) { i32(name, t, n); });
    };
    Output slots = out(a[8], "slot_map", d.max_tokens), cu = out(a[9], "cu_new", nreq + 1),
           kv = out(a[10], "kv_lens", nreq), counts = out(a[11], "counts", 4);
    const int rc = g_plan(ints(ctx), ints(fresh), ints(pages), ints(head), mutable_ints(table), mutable_ints(slots.t),
                          mutable_ints(cu.t), mutable_ints(kv.t), mutable_ints(counts.t), d, stream_of(index));
    if (rc) return PyLong_FromLong(rc);
    return tuple({&slots, &cu, &kv, &counts});
}

// k, v, k_cache, v_cache, slot_map
PyObject *cache_append(PyObject *const *a) {
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &kc = tensor(a[2], "k_cache"),
                 &vc = tensor(a[3], "v_cache"), &slots = tensor(a[4], "slot_map");
    const usp_cache_dims d = cache_dims(kc, vc);
    if (k.dim() != 3 || k.size(1) != d.hkv || k.size(2) != d.hd || v.sizes() != k.sizes())
        refuse("k and v must be (tokens, hkv, hd) like the cache");
    need(k.scalar_type() == kc.scalar_type() && v.scalar_type() == kc.scalar_type(), "dtype mismatch");
    i32("slot_map", slots, k.size(0));
    const int64_t ks = dense_rows("k", k), vs = dense_rows("v", v);
    const int index = device_of({&k, &v, &kc, &vc, &slots});
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    return PyLong_FromLong(g_append(k.const_data_ptr(), v.const_data_ptr(), kc.mutable_data_ptr(), vc.mutable_data_ptr(),
                                    ints(slots), k.size(0), ks, vs, d, stream_of(index)));
}

usp_paged_desc paged_desc(const Tensor &q, const Tensor &kc, const Tensor &vc, const Tensor &table, int64_t nreq,
                          PyObject *max_new) {
    usp_paged_desc d{};
    d.cache = cache_dims(kc, vc);
    if (q.dim() != 3 || q.size(2) != d.cache.hd || q.scalar_type() != kc.scalar_type())
        refuse("q must be (tokens, hq, hd), of the cache's head dim and dtype");
    need(nreq <= INT32_MAX, "too many requests");
    d.tokens = q.size(0);
    d.q_stride = dense_rows("q", q);
    d.table_stride = block_table(table, nreq);
    d.nreq = (int32_t)nreq;
    d.max_pages = size32(table, 1);
    d.hq = size32(q, 1);
    d.max_new = max_new == Py_None ? (int32_t)std::min<int64_t>(d.tokens, INT32_MAX) : integer32(max_new, "max_new");
    return d;
}

// q, k_cache, block_table, max_new
PyObject *paged_attn_workspace_size(PyObject *const *a) {
    const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &table = tensor(a[2], "block_table");
    const usp_paged_desc d = paged_desc(q, kc, kc, table, table.size(0), a[3]);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device_of({&q}));
    const size_t n = g_attn_workspace(d);
    need(n > 0, "invalid paged attention shapes");
    return PyLong_FromSize_t(n);
}

// q, k_cache, v_cache, block_table, cu_new, kv_lens, max_new, causal, scale, out, lse, workspace
PyObject *paged_attn(PyObject *const *a) {
    const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"),
                 &table = tensor(a[3], "block_table"), &cu = tensor(a[4], "cu_new"), &kv = tensor(a[5], "kv_lens");
    const int64_t nreq = kv.numel();
    i32("cu_new", cu, nreq + 1);
    i32("kv_lens", kv);
    usp_paged_desc d = paged_desc(q, kc, vc, table, nreq, a[6]);
    const int causal = PyObject_IsTrue(a[7]);
    if (causal < 0) throw PythonError{};
    d.causal = causal;
    d.scale = 0.f;
    if (a[8] != Py_None) {
        d.scale = (float)PyFloat_AsDouble(a[8]);
        if (PyErr_Occurred()) throw PythonError{};
    }
    const int index = device_of({&q, &kc, &vc, &table, &cu, &kv});
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    Output out = output(a[9], "out", index, q.sizes(), q.scalar_type(), [&](const Tensor &t) {
        need(t.sizes() == q.sizes() && t.scalar_type() == q.scalar_type(), "out must match q");
        d.out_stride = dense_rows("out", t);
    });
    const int64_t rows[2] = {q.size(0), q.size(1)};
    Output lse = output(a[10], "lse", index, rows, at::kFloat, [&](const Tensor &t) {
        need(t.sizes() == at::IntArrayRef(rows) && t.scalar_type() == at::kFloat && t.is_contiguous(),
             "lse must be contiguous fp32 (tokens, hq)");
    });
    Tensor work;
    if (a[11] == Py_None) {
        work = empty({(int64_t)g_attn_workspace(d)}, at::kByte, index);
    } else {
        work = tensor(a[11], "workspace");
        need(work.is_cuda() && work.get_device() == index && work.is_contiguous(),
             "workspace must be contiguous, on the tensors' device");
    }
    const int rc = g_attn(q.const_data_ptr(), kc.const_data_ptr(), vc.const_data_ptr(), ints(table), ints(cu), ints(kv),
                          out.t.mutable_data_ptr(), static_cast<float *>(lse.t.mutable_data_ptr()), d,
                          work.mutable_data_ptr(), work.nbytes(), stream_of(index));
    if (rc) return PyLong_FromLong(rc);
    return tuple({&out, &lse});
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        if (n != kArgs) refuse("wrong number of arguments", PyExc_TypeError);
        return F(args);
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const PythonError &) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// addresses of the library's functions
PyObject *bind(PyObject *const *a) {
    g_plan = reinterpret_cast<decltype(g_plan)>(integer(a[0]));
    g_append = reinterpret_cast<decltype(g_append)>(integer(a[1]));
    g_attn = reinterpret_cast<decltype(g_attn)>(integer(a[2]));
    g_attn_workspace = reinterpret_cast<decltype(g_attn_workspace)>(integer(a[3]));
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t kArgs> PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, kArgs>)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<bind, 4>("bind"),
                           method<page_plan, 12>("page_plan"),
                           method<cache_append, 5>("cache_append"),
                           method<paged_attn, 12>("paged_attn"),
                           method<paged_attn_workspace_size, 4>("paged_attn_workspace_size"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_usp_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__usp_binding() { return PyModule_Create(&g_module); }
