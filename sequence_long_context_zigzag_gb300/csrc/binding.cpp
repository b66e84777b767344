// binding.cpp -- the Python binding of the paged K/V cache's and the rotation's calls: argument checks, output allocation and the
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
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "usp.h"

namespace {

using at::Tensor;

decltype(&usp_page_plan) g_plan;
decltype(&usp_cache_append) g_append;
decltype(&usp_paged_attn) g_attn;
decltype(&usp_paged_attn_workspace_size) g_attn_workspace;
decltype(&usp_rope) g_rope;
decltype(&usp_rope_append) g_rope_append;
decltype(&usp_rope_append_q4) g_rope_append_q4;
decltype(&usp_paged_attn_q4) g_attn_q4;
decltype(&usp_paged_attn_q4_workspace_size) g_attn_q4_workspace;

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

// The call wrote t: a node of autograd that saved it notices. (Inference tensors count no versions.)
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
// Autograd would follow t past a call that it does not see.
void unrecorded(const char *name, const Tensor &t) {
    if (at::GradMode::is_enabled() && t.requires_grad())
        refuse(std::string(name) + " requires grad, which a rotation that is not recorded would leave wrong (UspRopeFunction is "
                                   "the differentiable form)");
}

// A call's output: the caller's tensor, returned as it came, or a new one.
struct Output {
    PyObject *given = nullptr;
    Tensor t;
    PyObject *result() {
        if (!given) return THPVariable_Wrap(std::move(t));
        if (t.defined()) written(t);
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
    written(table);
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
    const int rc = g_append(k.const_data_ptr(), v.const_data_ptr(), kc.mutable_data_ptr(), vc.mutable_data_ptr(), ints(slots),
                            k.size(0), ks, vs, d, stream_of(index));
    if (rc == USP_OK) {
        written(kc);
        written(vc);
    }
    return PyLong_FromLong(rc);
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

// ---- rotation ----
int truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw PythonError{};
    return x;
}

// the rotation's table: rows (max_pos) and rot
struct RopeTable {
    const float *data = nullptr;
    int64_t max_pos = 0;
    int32_t rot = 0;
};
RopeTable rope_table(const Tensor &t) {
    if (t.scalar_type() != at::kFloat || t.dim() != 2 || !t.is_contiguous())
        refuse("table must be a contiguous fp32 tensor (positions, rot)");
    need(t.size(1) > 0, "table must have columns");
    return {static_cast<const float *>(t.const_data_ptr()), t.size(0), size32(t, 1)};
}

// the stride of (bs, L, H, hd) over tokens in elements (0: contiguous); sequences follow one another at L times the stride
int64_t token_stride(const char *name, const Tensor &t) {
    if (t.is_contiguous()) return 0;
    const int64_t row = t.size(2) * t.size(3), st = t.stride(1);
    const bool heads = (t.size(3) == 1 || t.stride(3) == 1) && (t.size(2) == 1 || t.stride(2) == t.size(3));
    const bool seqs = t.size(0) == 1 || (t.size(1) == 1 ? t.stride(0) >= row : t.stride(0) == t.size(1) * st);
    if (!heads || !seqs || (t.size(1) > 1 && st < row)) refuse(std::string(name) + ": only the tokens' axis may be strided");
    return t.size(1) > 1 ? st : t.size(0) > 1 ? t.stride(0) : 0;
}

struct Status {  // of a call that was not USP_OK
    int rc;
};

// A rotation's arguments, checked. An undefined tensor: not given.
struct RopeCall {
    usp_rope_desc d{};
    RopeTable table;
    const int32_t *positions = nullptr, *cu = nullptr;
    int index = 0;
    RopeCall(const Tensor &q, const Tensor &k, const Tensor &t, const Tensor &pos, const Tensor &cu_seqlens, bool interleaved,
             bool inverse) {
        const bool has_k = k.defined();
        const Tensor &kk = has_k ? k : q;
        if (q.dim() != 4 || kk.dim() != 4) refuse("q and k must be (bs, L, heads, hd)");
        need(kk.size(0) == q.size(0) && kk.size(1) == q.size(1) && kk.size(3) == q.size(3) && kk.scalar_type() == q.scalar_type(),
             "q and k must agree in bs, L, hd and dtype");
        table = rope_table(t);
        d.bs = q.size(0);
        d.L = q.size(1);
        d.hq = size32(q, 2);
        d.hkv = has_k ? size32(k, 2) : 0;
        d.hd = size32(q, 3);
        d.rot = table.rot;
        d.max_pos = table.max_pos;
        d.dtype = dtype_code(q);
        d.interleaved = interleaved;
        d.inverse = inverse;
        d.q_stride = token_stride("q", q);
        if (has_k) d.k_stride = token_stride("k", k);
        index = device_of({&q, &kk, &t});
        if (pos.defined()) {
            if (pos.scalar_type() != at::kInt || pos.numel() != d.bs * d.L || !pos.is_contiguous())
                refuse("positions must be a contiguous int32 tensor, one per token");
            same_device(index, pos);
            positions = ints(pos);
        }
        if (cu_seqlens.defined()) {
            i32("cu_seqlens", cu_seqlens);
            need(cu_seqlens.numel() >= 2 && cu_seqlens.numel() <= INT32_MAX, "cu_seqlens must have an entry more than there are samples");
            same_device(index, cu_seqlens);
            d.nseq = (int32_t)(cu_seqlens.numel() - 1);
            cu = ints(cu_seqlens);
        }
    }
    int run(const Tensor &q, const Tensor &k, const Tensor &q_out, const Tensor &k_out) const {
        const bool has_k = k.defined();
        return g_rope(q.const_data_ptr(), q_out.mutable_data_ptr(), has_k ? k.const_data_ptr() : nullptr,
                      has_k ? k_out.mutable_data_ptr() : nullptr, table.data, positions, cu, d, stream_of(index));
    }
};
Tensor optional_tensor(PyObject *o, const char *name) { return o == Py_None ? Tensor() : tensor(o, name); }

// q, k or None, table, positions or None, cu_seqlens or None, interleaved, inverse, q_out, k_out
PyObject *rope(PyObject *const *a) {
    const Tensor &q = tensor(a[0], "q"), k = optional_tensor(a[1], "k");
    RopeCall call(q, k, tensor(a[2], "table"), optional_tensor(a[3], "positions"), optional_tensor(a[4], "cu_seqlens"), truth(a[5]),
                  truth(a[6]));
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)call.index);
    auto out = [&](PyObject *o, const char *name, const Tensor &like, int64_t &stride) {
        return output(o, name, call.index, like.sizes(), like.scalar_type(), [&](const Tensor &x) {
            if (x.sizes() != like.sizes() || x.scalar_type() != like.scalar_type()) refuse(std::string(name) + " must match its input");
            unrecorded(name, x);
            stride = token_stride(name, x);
        });
    };
    need(k.defined() || a[8] == Py_None, "k_out without k");
    Output qo = out(a[7], "q_out", q, call.d.q_out_stride), ko;
    if (k.defined()) ko = out(a[8], "k_out", k, call.d.k_out_stride);
    else ko.given = Py_None;
    if (const int rc = call.run(q, k, qo.t, ko.t)) return PyLong_FromLong(rc);
    return tuple({&qo, &ko});
}

// The rotation as a differentiable op: its gradient is the rotation back, itself differentiable. In C++, so that a backward
// pass needs neither the interpreter nor its lock (forward and backward of a small step took 140 us of the host's time in
// Python, twice the rest).
struct RopeFunction : torch::autograd::Function<RopeFunction> {
    using Optional = std::optional<Tensor>;
    static torch::autograd::variable_list forward(torch::autograd::AutogradContext *ctx, const Tensor &q, const Optional &opt_k,
                                                  const Tensor &table, const Optional &positions, const Optional &cu,
                                                  bool interleaved, bool inverse) {
        torch::autograd::variable_list saved{table};
        if (positions) saved.push_back(*positions);
        if (cu) saved.push_back(*cu);
        ctx->save_for_backward(std::move(saved));
        ctx->saved_data["flags"] = int64_t(positions ? POSITIONS : 0) | (interleaved ? INTERLEAVED : 0) | (inverse ? INVERSE : 0);
        return rotated(q, opt_k.value_or(Tensor()), table, positions.value_or(Tensor()), cu.value_or(Tensor()), interleaved, inverse);
    }
    enum Flags { POSITIONS = 1, INTERLEAVED = 2, INVERSE = 4 };
    static torch::autograd::variable_list rotated(const Tensor &q, const Tensor &k, const Tensor &table, const Tensor &positions,
                                                  const Tensor &cu, bool interleaved, bool inverse) {
        const RopeCall call(q, k, table, positions, cu, interleaved, inverse);
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)call.index);
        const Tensor qo = empty(q.sizes(), q.scalar_type(), call.index),
                     ko = k.defined() ? empty(k.sizes(), k.scalar_type(), call.index) : Tensor();
        if (const int rc = call.run(q, k, qo, ko)) throw Status{rc};
        return k.defined() ? torch::autograd::variable_list{qo, ko} : torch::autograd::variable_list{qo};
    }
    // a gradient as the rotation takes it; it may come expanded, or as part of another tensor at any address
    static Tensor dense(const Tensor &g) {
        const Tensor c = g.contiguous();
        return reinterpret_cast<uintptr_t>(c.const_data_ptr()) % 16 == 0 ? c : c.clone();
    }
    static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx, torch::autograd::variable_list g) {
        const auto saved = ctx->get_saved_variables();
        const bool has_k = g.size() > 1;
        try {
            const int64_t flags = ctx->saved_data["flags"].toInt();
            const bool has_pos = flags & POSITIONS, has_cu = saved.size() > 1u + has_pos;
            const bool interleaved = flags & INTERLEAVED, inverse = !(flags & INVERSE);
            const Tensor q = dense(g[0]), k = has_k ? dense(g[1]) : Tensor();
            torch::autograd::variable_list d;
            if (at::GradMode::is_enabled())  // the gradient is to be differentiated in turn
                d = apply(q, has_k ? Optional(k) : std::nullopt, saved[0], has_pos ? Optional(saved[1]) : std::nullopt,
                          has_cu ? Optional(saved.back()) : std::nullopt, interleaved, inverse);
            else
                d = rotated(q, k, saved[0], has_pos ? saved[1] : Tensor(), has_cu ? saved.back() : Tensor(), interleaved, inverse);
            return {d[0], has_k ? d[1] : Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()};
        } catch (const Refused &r) {
            TORCH_CHECK(false, r.what);
        } catch (const Status &s) {
            TORCH_CHECK(false, "usp_rope failed in a backward pass (status ", s.rc, ")");
        }
    }
};

// q, k or None, table, positions or None, cu_seqlens or None, interleaved
PyObject *rope_grad(PyObject *const *a) {
    auto given = [&](int i, const char *name) {
        return a[i] == Py_None ? RopeFunction::Optional() : RopeFunction::Optional(tensor(a[i], name));
    };
    const Tensor &table = tensor(a[2], "table");
    if (at::GradMode::is_enabled() && table.requires_grad()) refuse("the rotation has no gradient for its table, which requires grad");
    try {
        auto r = RopeFunction::apply(tensor(a[0], "q"), given(1, "k"), table, given(3, "positions"),
                                     given(4, "cu_seqlens"), (bool)truth(a[5]), false);
        Output qo, ko;
        qo.t = r[0];
        if (r.size() > 1) ko.t = r[1];
        else ko.given = Py_None;
        return tuple({&qo, &ko});
    } catch (const Status &s) {
        return PyLong_FromLong(s.rc);
    }
}

usp_q4_dims q4_dims(const Tensor &k, const Tensor &v, const Tensor &ks, const Tensor &vs) {
    if (k.dim() != 4 || v.sizes() != k.sizes() || k.scalar_type() != at::kByte || v.scalar_type() != at::kByte)
        refuse("k_cache and v_cache must be uint8 (num_pages, hkv, page_size, hd / 2)");
    if (ks.dim() != 4 || vs.sizes() != ks.sizes() || ks.scalar_type() != at::kByte || vs.scalar_type() != at::kByte ||
        ks.size(0) != k.size(0) || ks.size(1) != k.size(1) || ks.size(2) != k.size(2) || ks.size(3) * 16 != k.size(3))
        refuse("k_scales and v_scales must be uint8 (num_pages, hkv, page_size, hd / 32)");
    usp_q4_dims d{};
    d.num_pages = k.size(0);
    d.k_page_stride = dense_rows("k_cache", k);
    d.v_page_stride = dense_rows("v_cache", v);
    d.k_scale_stride = dense_rows("k_scales", ks);
    d.v_scale_stride = dense_rows("v_scales", vs);
    d.hkv = size32(k, 1);
    d.page_size = size32(k, 2);
    d.hd = (int32_t)std::min<int64_t>(2 * k.size(3), INT32_MAX);
    return d;
}
uint8_t *mutable_bytes(const Tensor &t) { return static_cast<uint8_t *>(t.mutable_data_ptr()); }
const uint8_t *bytes(const Tensor &t) { return static_cast<const uint8_t *>(t.const_data_ptr()); }

// q or None, k, v, k_cache, v_cache, k_scales or None, v_scales or None, slot_map, table or None, cu_new or None, kv_lens or
// None, positions or None, interleaved, q_out. The result: q_out (None without a q).
PyObject *rope_append(PyObject *const *a) {
    const bool has_q = a[0] != Py_None, q4 = a[5] != Py_None || a[6] != Py_None;
    const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &q = has_q ? tensor(a[0], "q") : k,
                 &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache"), &slots = tensor(a[7], "slot_map");
    const Tensor &ks = q4 ? tensor(a[5], "k_scales") : kc, &vs = q4 ? tensor(a[6], "v_scales") : kc;
    usp_cache_dims c{};
    usp_q4_dims c4{};
    if (q4) {
        c4 = q4_dims(kc, vc, ks, vs);
    } else {
        if (kc.scalar_type() == at::kByte) refuse("a 4-bit cache needs k_scales and v_scales");
        c = cache_dims(kc, vc);
        need(k.scalar_type() == kc.scalar_type(), "dtype mismatch");
    }
    const int64_t hkv = q4 ? c4.hkv : c.hkv, hd = q4 ? c4.hd : c.hd;
    if (k.dim() != 3 || k.size(1) != hkv || k.size(2) != hd || v.sizes() != k.sizes())
        refuse("k and v must be (tokens, hkv, hd) like the cache");
    if (q.dim() != 3 || q.size(0) != k.size(0) || q.size(2) != hd) refuse("q must be (tokens, hq, hd), of k's tokens and head dim");
    need(v.scalar_type() == k.scalar_type() && q.scalar_type() == k.scalar_type(), "dtype mismatch");
    usp_rope_append_desc d{};
    d.tokens = k.size(0);
    d.dtype = dtype_code(k);
    d.hq = has_q ? size32(q, 1) : 0;
    d.q_stride = has_q ? dense_rows("q", q) : 0;
    d.k_stride = dense_rows("k", k);
    d.v_stride = dense_rows("v", v);
    d.interleaved = truth(a[12]);
    i32("slot_map", slots, d.tokens);
    const int index = device_of({&k, &v, &q, &kc, &vc, &ks, &vs, &slots});
    RopeTable t;
    const int32_t *positions = nullptr, *cu = nullptr, *kv = nullptr;
    if (a[8] != Py_None) {
        const Tensor &x = tensor(a[8], "table");
        t = rope_table(x);
        same_device(index, x);
        if (a[11] != Py_None) {
            const Tensor &p = tensor(a[11], "positions");
            i32("positions", p, d.tokens);
            same_device(index, p);
            positions = ints(p);
        } else {
            const Tensor &n = tensor(a[10], "kv_lens"), &u = tensor(a[9], "cu_new");
            i32("kv_lens", n);
            i32("cu_new", u, n.numel() + 1);
            same_device(index, n);
            same_device(index, u);
            need(n.numel() <= INT32_MAX, "too many requests");
            d.nreq = (int32_t)n.numel();
            cu = ints(u);
            kv = ints(n);
        }
    }
    d.rot = t.rot;
    d.max_pos = t.max_pos;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    Output qo;
    if (has_q)
        qo = output(a[13], "q_out", index, q.sizes(), q.scalar_type(), [&](const Tensor &x) {
            need(x.sizes() == q.sizes() && x.scalar_type() == q.scalar_type(), "q_out must match q");
            unrecorded("q_out", x);
            d.q_out_stride = dense_rows("q_out", x);
        });
    const void *qp = has_q ? q.const_data_ptr() : nullptr;
    void *qop = has_q ? qo.t.mutable_data_ptr() : nullptr;
    const int rc =
        q4 ? g_rope_append_q4(qp, qop, k.const_data_ptr(), v.const_data_ptr(), kc.mutable_data_ptr(), vc.mutable_data_ptr(),
                              mutable_bytes(ks), mutable_bytes(vs), ints(slots), positions, cu, kv, t.data, d, c4, stream_of(index))
           : g_rope_append(qp, qop, k.const_data_ptr(), v.const_data_ptr(), kc.mutable_data_ptr(), vc.mutable_data_ptr(),
                           ints(slots), positions, cu, kv, t.data, d, c, stream_of(index));
    if (rc) return PyLong_FromLong(rc);
    written(kc);
    written(vc);
    if (q4) {
        written(ks);
        written(vs);
    }
    if (!has_q) Py_RETURN_NONE;
    PyObject *r = qo.result();
    if (!r) throw PythonError{};
    return r;
}

usp_paged_q4_desc paged_q4_desc(const Tensor &q, const usp_q4_dims &cache, const Tensor &table, int64_t nreq, PyObject *max_new) {
    usp_paged_q4_desc d{};
    d.cache = cache;
    if (q.dim() != 3 || q.size(2) != cache.hd) refuse("q must be (tokens, hq, hd), of the cache's head dim");
    d.dtype = dtype_code(q);
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
PyObject *paged_attn_q4_workspace_size(PyObject *const *a) {
    const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &table = tensor(a[2], "block_table");
    if (kc.dim() != 4 || kc.scalar_type() != at::kByte) refuse("k_cache must be uint8 (num_pages, hkv, page_size, hd / 2)");
    usp_q4_dims c{};
    c.num_pages = kc.size(0);
    c.hkv = size32(kc, 1);
    c.page_size = size32(kc, 2);
    c.hd = (int32_t)std::min<int64_t>(2 * kc.size(3), INT32_MAX);
    const usp_paged_q4_desc d = paged_q4_desc(q, c, table, table.size(0), a[3]);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device_of({&q}));
    const size_t n = g_attn_q4_workspace(d);
    need(n > 0, "invalid paged attention shapes");
    return PyLong_FromSize_t(n);
}

// q, k_cache, v_cache, k_scales, v_scales, block_table, cu_new, kv_lens, max_new, causal, scale, out, lse, workspace
PyObject *paged_attn_q4(PyObject *const *a) {
    const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"),
                 &ks = tensor(a[3], "k_scales"), &vs = tensor(a[4], "v_scales"), &table = tensor(a[5], "block_table"),
                 &cu = tensor(a[6], "cu_new"), &kv = tensor(a[7], "kv_lens");
    const int64_t nreq = kv.numel();
    i32("cu_new", cu, nreq + 1);
    i32("kv_lens", kv);
    usp_paged_q4_desc d = paged_q4_desc(q, q4_dims(kc, vc, ks, vs), table, nreq, a[8]);
    d.causal = truth(a[9]);
    d.scale = 0.f;
    if (a[10] != Py_None) {
        d.scale = (float)PyFloat_AsDouble(a[10]);
        if (PyErr_Occurred()) throw PythonError{};
    }
    const int index = device_of({&q, &kc, &vc, &ks, &vs, &table, &cu, &kv});
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    Output out = output(a[11], "out", index, q.sizes(), q.scalar_type(), [&](const Tensor &t) {
        need(t.sizes() == q.sizes() && t.scalar_type() == q.scalar_type(), "out must match q");
        d.out_stride = dense_rows("out", t);
    });
    const int64_t rows[2] = {q.size(0), q.size(1)};
    Output lse = output(a[12], "lse", index, rows, at::kFloat, [&](const Tensor &t) {
        need(t.sizes() == at::IntArrayRef(rows) && t.scalar_type() == at::kFloat && t.is_contiguous(),
             "lse must be contiguous fp32 (tokens, hq)");
    });
    Tensor work;
    if (a[13] == Py_None) {
        work = empty({(int64_t)g_attn_q4_workspace(d)}, at::kByte, index);
    } else {
        work = tensor(a[13], "workspace");
        need(work.is_cuda() && work.get_device() == index && work.is_contiguous(),
             "workspace must be contiguous, on the tensors' device");
    }
    const int rc = g_attn_q4(q.const_data_ptr(), kc.const_data_ptr(), vc.const_data_ptr(), bytes(ks), bytes(vs), ints(table),
                             ints(cu), ints(kv), out.t.mutable_data_ptr(), static_cast<float *>(lse.t.mutable_data_ptr()), d,
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
    g_rope = reinterpret_cast<decltype(g_rope)>(integer(a[4]));
    g_rope_append = reinterpret_cast<decltype(g_rope_append)>(integer(a[5]));
    g_rope_append_q4 = reinterpret_cast<decltype(g_rope_append_q4)>(integer(a[6]));
    g_attn_q4 = reinterpret_cast<decltype(g_attn_q4)>(integer(a[7]));
    g_attn_q4_workspace = reinterpret_cast<decltype(g_attn_q4_workspace)>(integer(a[8]));
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t kArgs> PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, kArgs>)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<bind, 9>("bind"),
                           method<page_plan, 12>("page_plan"),
                           method<cache_append, 5>("cache_append"),
                           method<paged_attn, 12>("paged_attn"),
                           method<paged_attn_workspace_size, 4>("paged_attn_workspace_size"),
                           method<rope, 9>("rope"),
                           method<rope_grad, 6>("rope_grad"),
                           method<rope_append, 14>("rope_append"),
                           method<paged_attn_q4, 14>("paged_attn_q4"),
                           method<paged_attn_q4_workspace_size, 4>("paged_attn_q4_workspace_size"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_usp_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__usp_binding() { return PyModule_Create(&g_module); }
